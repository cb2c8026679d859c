// quantize_i8.cu -- rows to 8-bit integers with one scale a row.
//
// ("Platform For AI: BladeLLM model quantization", the act-and-weight mode:
// per-token dynamic scales for activations, per-channel scales for weights,
// INT8.)  For a row x of K values
//
//   s = max |x| fp32(1 / 127),   q = clamp(rint(x / s), -127, 127),  0 where s = 0
//
// (s one product and one rounding; the rounded quotient max |x| / 127 is its
// neighbour for one row in twenty, and other codes next to a half go with it)
// with rint of the exact quotient, half to even; a row that holds an infinity
// or a NaN gets s = NaN and q = 0, so that every product with it is NaN.
//
// Bound by memory: one read of x, one write of a byte an element; in practice
// as much by instruction issue (68% of the cycles).  A row is read once and
// stays in registers (as loaded) between its maximum and its codes; only rows
// too long for that are read a second time.  Measured: 2048 x 13824 bf16 17.0
// us (5.0 TB/s), 13824 x 5120 fp16 38.5 us (5.5 TB/s).
//
// The maximum keeps NaNs (16-bit types: two values at a time in their own type)
// and is compared as an unsigned integer in the end: the bits of magnitudes
// order as they do, with infinities and then NaNs on top, so one maximum finds
// the scale and the non-finite rows.
//
// The codes are exact without a division per element.  With c = fp32(1/s)
// (or its neighbour) x c is within 127.5 * 2^-23 < 2^-16 of x/s; t = fma(x, c, 1.5 2^23)
// rounds it to an integer n (t's low byte is the code), which is the right one
// or its neighbour across a half.  The remainder e = fma(-n, s, x) is exact: for
// |x| >= s it is a multiple of s's last place below 2^24 of them, for |x| in
// [s/2, s) of half that place, below it n = 0 (or e is -s/2 .. 0).  So n is
// right where |e| < s/2, and one too small or large where |e| > s/2; where |e| =
// s/2 the even neighbour is.  That correction is a branch that a vector takes
// when it holds an |e| >= s/2.  Those would not be as rare as 127 * 2^-24:
// 16-bit values have quotients 127 a/b of small integers in a, the exact
// maximum's 127 places; one in a few hundred is a half but for the rounding of
// s.  So c is taken on the side of 1/s on which max |x| / 127 lies of s: then
// x c falls to the same side of such a half as x/s does.  (With c = fp32(1/s)
// half of the vectors of bf16 rows took the branch.)
// Rows whose scale is below 2^-100, where 1/s or s's last place leave fp32's
// normal range, take every quotient in 64 bits: of two 24-bit numbers, one that
// is no half-integer differs from one by over 2^-33 of its size.
#include <type_traits>

#include "i8.cuh"
#include "wq_internal.cuh"

namespace wq {
namespace i8 {
namespace {

// VE consecutive elements of a row as loaded: 16 bytes.
template <int TYPE>
struct Vec {
  static constexpr int VE = TYPE == kF32 ? 4 : 8;
  using Elem = typename std::conditional<TYPE == kF32, uint32_t, uint16_t>::type;

  // The largest magnitude of v and m (as bits of the type, two values of 16
  // bits side by side); a NaN stays one.
  static __device__ __forceinline__ uint32_t fold(uint32_t m, const uint4& v) {
    if constexpr (TYPE == kF32) {
      m = max(m, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu));
      return max(m, max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
    } else {
      return max2(max2(max2(v.x, v.y), max2(v.z, v.w)), m);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using T = typename std::conditional<TYPE == kF16, __half2, __nv_bfloat162>::type;
    const T r = __hmax2_nan(__habs2(*reinterpret_cast<const T*>(&a)), __habs2(*reinterpret_cast<const T*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  // The folded maximum (over lanes too) as the bits of an fp32 number.
  static __device__ __forceinline__ uint32_t to_f32_bits(uint32_t m) {
    if constexpr (TYPE == kF32) return m;
    m = max(m & 0xffffu, m >> 16);
    if constexpr (TYPE == kBF16) return m << 16;
    return __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
  }
  static __device__ __forceinline__ float value(const uint4& v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (TYPE == kF32) return __uint_as_float(w[i]);
    const uint32_t h = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
    if constexpr (TYPE == kBF16) return __uint_as_float(h << 16);
    return __half2float(__ushort_as_half(uint16_t(h)));
  }
};

// VE elements from k on, all inside the row.
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const typename Vec<TYPE>::Elem* p) {
  if constexpr (ALIGNED) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(p[2 * i]) | uint32_t(p[2 * i + 1]) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The first n < VE elements at p, zeros behind them.
template <int TYPE>
__device__ __forceinline__ uint4 load_tail(const typename Vec<TYPE>::Elem* p, int n) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Vec<TYPE>::VE; ++i)
    if (i < n) {
      if constexpr (TYPE == kF32) w[i] = p[i];
      else w[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Codes of the elements of v, one byte each, first element lowest; inv next to 1 / s, half s / 2
// (for s = 0: 0 and infinity).
template <int TYPE>
__device__ __forceinline__ void codes_of(const uint4& v, float s, float inv, float half, uint32_t (&out)[2]) {
  constexpr int VE = Vec<TYPE>::VE;
  constexpr float kMagic = 12582912.0f;   // 1.5 2^23: the unit in the last place is 1
  uint32_t b[VE];
  float e[VE], worst = 0.0f;
  const uint64_t inv2 = f32x2(inv, inv), magic2 = f32x2(kMagic, kMagic), minus2 = f32x2(-s, -s);
#pragma unroll
  for (int i = 0; i < VE; i += 2) {
    const uint64_t x = f32x2(Vec<TYPE>::value(v, i), Vec<TYPE>::value(v, i + 1));
    const uint64_t t = fma2(x, inv2, magic2);
    float t0, t1;
    unpack2(t, t0, t1);
    b[i] = __float_as_uint(t0);
    b[i + 1] = __float_as_uint(t1);
    unpack2(fma2(add2(t, f32x2(-kMagic, -kMagic)), minus2, x), e[i], e[i + 1]);
    worst = max3(worst, fabsf(e[i]), fabsf(e[i + 1]));
  }
  if (worst >= half) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      // past the half, or on it from an odd integer (the bits of magnitudes order as they do)
      const uint32_t eb = __float_as_uint(e[i]);
      if ((eb & 0x7fffffffu) + (b[i] & 1u) > __float_as_uint(half)) b[i] += uint32_t(int(eb) >> 31) | 1u;
    }
  }
#pragma unroll
  for (int i = 0; i < VE; i += 4)
    out[i / 4] = __byte_perm(__byte_perm(b[i], b[i + 1], 0x0040), __byte_perm(b[i + 2], b[i + 3], 0x0040), 0x5410);
}

// 1 / s for codes_of: fp32(1 / s), or its neighbour on the side of 1 / s where a / 127 lies of s.
__device__ __forceinline__ float inverse(float a, float s) {
  const float c = __fdiv_rn(1.0f, s);
  const float side = __fmaf_rn(-127.0f, s, a), off = __fmaf_rn(c, s, -1.0f);
  const int step = side > 0.0f && off < 0.0f ? 1 : side < 0.0f && off > 0.0f ? -1 : 0;
  return __int_as_float(__float_as_int(c) + step);
}

// 2^lw warps per row, several rows per CTA of THREADS threads.  NV > 0: each thread
// holds its NV vectors of the row in registers; NV = 0: two passes over memory.
template <int TYPE, int NV, bool ALIGNED, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_i8_kernel(const void* xv, int64_t R, int64_t K,
                                                               int64_t ldx, int8_t* __restrict__ codes, int64_t ldc,
                                                               float* __restrict__ scales, int lw) {
  using V = Vec<TYPE>;
  constexpr int VE = V::VE;
  __shared__ uint32_t smax[THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * (THREADS / 32 >> lw) + (warp >> lw);
  const bool live = r < R;
  const int tn = 32 << lw, t0 = threadIdx.x & (tn - 1);
  const auto* row = static_cast<const typename V::Elem*>(xv) + (live ? r * ldx : 0);
  const int nvec = live ? int(K) / VE : 0, rest = live ? int(K) % VE : 0;   // whole vectors, elements behind them
  pdl_start();
  pdl_wait();

  uint4 v[NV > 0 ? NV : 1], tail = make_uint4(0, 0, 0, 0);
  uint32_t m = 0;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = t0 + i * tn;
      v[i] = make_uint4(0, 0, 0, 0);
      if (j < nvec) v[i] = load_vec<TYPE, ALIGNED>(row + j * VE);
    }
    if (t0 == 0 && rest) tail = load_tail<TYPE>(row + nvec * VE, rest);
#pragma unroll
    for (int i = 0; i < NV; ++i) m = V::fold(m, v[i]);
  } else {
    if (t0 == 0 && rest) tail = load_tail<TYPE>(row + nvec * VE, rest);
#pragma unroll 4
    for (int j = t0; j < nvec; j += tn) m = V::fold(m, load_vec<TYPE, ALIGNED>(row + j * VE));
  }
  m = V::to_f32_bits(V::fold(m, tail));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lw > 0) {
    if (lane == 0) smax[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, smax[(warp >> lw << lw) + (lane & ((1 << lw) - 1))]);
  }
  if (!live) return;
  const float s = __uint_as_float(m) * (1.0f / 127.0f);
  const bool finite = m < 0x7f800000u;
  if (t0 == 0) scales[r] = finite ? s : __uint_as_float(0x7fc00000u);
  int8_t* out = codes + r * ldc;
  if (!finite || (s < 0x1p-100f && s > 0.0f)) {      // hardly ever: element by element
    for (int k = t0; k < int(K); k += tn) {
      const float x = Vec<TYPE>::value(load_tail<TYPE>(row + k, 1), 0);
      out[k] = finite ? int8_t(rint(fmin(fmax(double(x) / double(s), -127.0), 127.0))) : int8_t(0);
    }
    return;
  }
  const float inv = s > 0.0f ? inverse(__uint_as_float(m), s) : 0.0f;
  const float half = s > 0.0f ? 0.5f * s : __uint_as_float(0x7f800000u);
  auto put = [&](int j, const uint4& x) {
    uint32_t c[2];
    codes_of<TYPE>(x, s, inv, half, c);
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(out + j * VE) = make_uint2(c[0], c[1]);
    else *reinterpret_cast<uint32_t*>(out + j * VE) = c[0];
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = t0 + i * tn;
      if (j < nvec) put(j, v[i]);
    }
  } else {
#pragma unroll 2
    for (int j = t0; j < nvec; j += tn) put(j, load_vec<TYPE, ALIGNED>(row + j * VE));
  }
  if (t0 == 0 && rest) {
    uint32_t c[2];
    codes_of<TYPE>(tail, s, inv, half, c);
    for (int i = 0; i < rest; ++i) out[nvec * VE + i] = int8_t(c[i / 4] >> (8 * (i & 3)));
  }
}

template <int TYPE, bool ALIGNED>
cudaError_t launch_typed(const void* x, int64_t R, int64_t K, int64_t ldx, int8_t* codes, int64_t ldc, float* scales,
                         cudaStream_t st) {
  constexpr int VE = Vec<TYPE>::VE;
  const int64_t nvec = K / VE;
  int dev;
  const cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  const int64_t busy = 16 * sm_count(dev);     // warps
  // Warps per row: what a thread does once per row (the maxima's exchange, the
  // scale) costs as much as 20 elements, so up to eight vectors a thread; fewer
  // where the rows alone do not give every SM 16 warps.  Rows that eight warps
  // cannot hold go to CTAs of sixteen.
  int lw = 0;
  while (lw < 3 && (nvec > (256 << lw) || (nvec > (32 << lw) && (R << lw) < busy))) ++lw;
  if (nvec > 2048) lw = 4;
  const int64_t per = (nvec + (32 << lw) - 1) / (32 << lw);
  const int warps = lw == 4 ? 16 : 8;
  const int64_t grid = (R + (warps >> lw) - 1) / (warps >> lw);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* fn = lw == 4 ? (per <= 8 ? quantize_i8_kernel<TYPE, 8, ALIGNED, 512> : quantize_i8_kernel<TYPE, 0, ALIGNED, 512>)
             : per <= 1 ? quantize_i8_kernel<TYPE, 1, ALIGNED, 256>
             : per <= 2 ? quantize_i8_kernel<TYPE, 2, ALIGNED, 256>
             : per <= 4 ? quantize_i8_kernel<TYPE, 4, ALIGNED, 256>
                        : quantize_i8_kernel<TYPE, 8, ALIGNED, 256>;
  return cudaLaunchKernelEx(&cfg, fn, x, R, K, ldx, codes, ldc, scales, lw);
}

template <int TYPE>
cudaError_t launch_aligned(const void* x, int64_t R, int64_t K, int64_t ldx, int8_t* codes, int64_t ldc,
                           float* scales, cudaStream_t st) {
  const int64_t row_bytes = ldx * int64_t(type_bytes(TYPE));
  if ((reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (R == 1 || row_bytes % 16 == 0))
    return launch_typed<TYPE, true>(x, R, K, ldx, codes, ldc, scales, st);
  return launch_typed<TYPE, false>(x, R, K, ldx, codes, ldc, scales, st);
}

}  // namespace

cudaError_t launch_quantize(const void* x, int type, int64_t R, int64_t K, int64_t ldx, int8_t* codes,
                            int64_t ldc, float* scales, cudaStream_t st) {
  if (type == kBF16) return launch_aligned<kBF16>(x, R, K, ldx, codes, ldc, scales, st);
  if (type == kF16) return launch_aligned<kF16>(x, R, K, ldx, codes, ldc, scales, st);
  return launch_aligned<kF32>(x, R, K, ldx, codes, ldc, scales, st);
}

}  // namespace i8
}  // namespace wq
