// quantize_i8.cu -- rows to 8-bit integers with one scale a row.
//
// ("Platform For AI: BladeLLM model quantization", the act-and-weight mode:
// per-token dynamic scales for activations, per-channel scales for weights,
// INT8.)  For a row x of K values
//
//   s = max |x| fp32(1 / 127),   q = clamp(rint(x / s), -127, 127),  0 where s = 0
//
// with rint of the exact quotient, half to even; a row that holds an infinity
// or a NaN gets s = NaN and q = 0, so that every product with it is NaN.
//
// Bound by memory: one read of x, one write of a byte an element.  A row is
// read once and stays in registers (as loaded) between its maximum and its
// codes; only rows too long for that are read a second time.
//
// The maximum is taken over the magnitude bits as unsigned integers: they
// order as the values do, with infinities and then NaNs on top, so one integer
// maximum finds the scale and the non-finite rows, two 16-bit values at a time.
//
// The codes are exact without a division per element.  With c = fp32(1/s) the
// product x c is within 127.5 * 2^-24 < 2^-17 of x/s; t = fma(x, c, 1.5 2^23)
// rounds it to an integer n (t's low byte is the code), which is the right one
// or its neighbour across a half.  The remainder e = fma(-n, s, x) is exact: for
// |x| >= s it is a multiple of s's last place below 2^24 of them, for |x| in
// [s/2, s) of half that place, below it n = 0 (or e is -s/2 .. 0).  So n is
// right where |e| < s/2, and one too small or large where |e| > s/2; where |e| =
// s/2 the even neighbour is.  That correction is a branch that a vector takes
// when it holds an |e| >= s/2.  Those are not as rare as 127 * 2^-24: 16-bit
// values have quotients 127 a/b of small integers, one in a few hundred of
// which lies within an fp32 rounding of a half, so the branch has to be cheap
// (a 64-bit division there took 2048 x 13824 bf16 from 20 to 63 us).
// Scales below 2^-100, where 1/s or s's last place leave fp32's normal range,
// take every quotient in 64 bits: of two 24-bit numbers, one that is no
// half-integer differs from one by over 2^-33 of its size.
#include <type_traits>

#include "i8.cuh"
#include "wq_internal.cuh"

namespace wq {
namespace i8 {
namespace {

constexpr int kThreads = 256;

// VE consecutive elements of a row as loaded: 16 bytes.
template <int TYPE>
struct Vec {
  static constexpr int VE = TYPE == kF32 ? 4 : 8;
  using Elem = typename std::conditional<TYPE == kF32, uint32_t, uint16_t>::type;

  // The magnitude bits' maximum as fp32 bits, folded into m (in the type's own bits).
  static __device__ __forceinline__ uint32_t fold(uint32_t m, const uint4& v) {
    if constexpr (TYPE == kF32) {
      m = max(m, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu));
      return max(m, max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
    } else {
      m = __vmaxu2(m, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
      return __vmaxu2(m, __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    }
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
  if constexpr (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(p + i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(__ldg(p + 2 * i)) | uint32_t(__ldg(p + 2 * i + 1)) << 16;
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
      if constexpr (TYPE == kF32) w[i] = __ldg(p + i);
      else w[i >> 1] |= uint32_t(__ldg(p + i)) << (16 * (i & 1));
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

__device__ __noinline__ uint32_t code_by_division(float x, float s) {
  return uint32_t(int(rint(fmin(fmax(double(x) / double(s), -127.0), 127.0))));
}

// Codes of the elements of v, one byte each, first element lowest; inv: fp32(1 / s), or 0 for scales under 2^-100.
template <int TYPE>
__device__ __forceinline__ void codes_of(const uint4& v, float s, float inv, uint32_t (&out)[2]) {
  constexpr int VE = Vec<TYPE>::VE;
  constexpr float kMagic = 12582912.0f;   // 1.5 2^23: the unit in the last place is 1
  uint32_t b[VE];
  if (inv != 0.0f) {
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
      worst = fmaxf(worst, fmaxf(fabsf(e[i]), fabsf(e[i + 1])));
    }
    const float half = 0.5f * s;
    if (worst >= half) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        // past the half, or on it from an odd integer (the bits of magnitudes order as they do)
        const uint32_t eb = __float_as_uint(e[i]);
        if ((eb & 0x7fffffffu) + (b[i] & 1u) > __float_as_uint(half)) b[i] += uint32_t(int(eb) >> 31) | 1u;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) b[i] = code_by_division(Vec<TYPE>::value(v, i), s);
  }
#pragma unroll
  for (int i = 0; i < VE; i += 4)
    out[i / 4] = __byte_perm(__byte_perm(b[i], b[i + 1], 0x0040), __byte_perm(b[i + 2], b[i + 3], 0x0040), 0x5410);
}

// `wpr` warps per row, kThreads / 32 / wpr rows per CTA.  NV > 0: each thread
// holds its NV vectors of the row in registers; NV = 0: two passes over memory.
template <int TYPE, int NV, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) quantize_i8_kernel(const void* __restrict__ xv, int64_t R, int64_t K,
                                                               int64_t ldx, int8_t* __restrict__ codes, int64_t ldc,
                                                               float* __restrict__ scales, int wpr) {
  using V = Vec<TYPE>;
  constexpr int VE = V::VE;
  __shared__ uint32_t smax[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * (kThreads / 32 / wpr) + warp / wpr;
  const bool live = r < R;
  const int t0 = (warp % wpr) * 32 + lane, tn = 32 * wpr;
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
  if (wpr > 1) {
    if (lane == 0) smax[warp] = m;
    __syncthreads();
    const int w0 = warp / wpr * wpr;
    m = 0;
    for (int w = 0; w < wpr; ++w) m = max(m, smax[w0 + w]);
  }
  if (!live) return;
  const float s = __uint_as_float(m) * (1.0f / 127.0f);
  const bool finite = m < 0x7f800000u;
  if (t0 == 0) scales[r] = finite ? s : __uint_as_float(0x7fc00000u);
  const bool zero = !finite || s == 0.0f;
  const float inv = s >= 0x1p-100f && finite ? __fdiv_rn(1.0f, s) : 0.0f;
  int8_t* out = codes + r * ldc;
  auto put = [&](int j, const uint4& x) {
    uint32_t c[2] = {0u, 0u};
    if (!zero) codes_of<TYPE>(x, s, inv, c);
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
    uint32_t c[2] = {0u, 0u};
    if (!zero) codes_of<TYPE>(tail, s, inv, c);
    for (int i = 0; i < rest; ++i) out[nvec * VE + i] = int8_t(c[i / 4] >> (8 * (i & 3)));
  }
}

template <int TYPE, bool ALIGNED>
cudaError_t launch_typed(const void* x, int64_t R, int64_t K, int64_t ldx, int8_t* codes, int64_t ldc, float* scales,
                         cudaStream_t st) {
  constexpr int VE = Vec<TYPE>::VE;
  const int64_t nvec = K / VE;
  // warps per row: two vectors a thread and more before the next warp joins
  // in, and all eight when there are few rows
  int wpr = 1;
  while (wpr < 8 && (nvec > 64 * wpr || (R < 1024 && nvec > 32 * wpr))) wpr *= 2;
  const int64_t per = (nvec + 32 * wpr - 1) / (32 * wpr);
  const int64_t grid = (R + 8 / wpr - 1) / (8 / wpr);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* fn = per <= 1   ? quantize_i8_kernel<TYPE, 1, ALIGNED>
             : per <= 2 ? quantize_i8_kernel<TYPE, 2, ALIGNED>
             : per <= 4 ? quantize_i8_kernel<TYPE, 4, ALIGNED>
             : per <= 8 ? quantize_i8_kernel<TYPE, 8, ALIGNED>
                        : quantize_i8_kernel<TYPE, 0, ALIGNED>;
  return cudaLaunchKernelEx(&cfg, fn, x, R, K, ldx, codes, ldc, scales, wpr);
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
