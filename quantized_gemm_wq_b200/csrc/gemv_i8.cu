// gemv_i8.cu -- 8-bit integer linears for few tokens, on warp-level MMAs.
//
// With a handful of tokens the product is bound by the read of the weights, a
// byte each.  The weight rows are the M side of mma.sync.m16n8k32 (s8 x s8 ->
// s32), the tokens its N side, so up to 8 tokens cost one MMA per 512 weights.
// A sum over k may be taken in any order, so both operands are loaded 16 bytes
// a lane from the same places of their rows and the MMA's k index is renamed:
// lane (g, t) holds bytes 16 t .. 16 t + 15 of a 64-byte half chunk of rows g
// and g + 8 and of token g, which are the A and B fragments of two MMAs.
// Weights go straight from memory to registers; nothing is staged.
//
// One CTA computes 16 output rows (of both projections in a gated call) for
// all tokens; its warps take the 128-byte chunks of K in turn (whole lines of
// L2), the next chunks' loads in flight while the present ones are multiplied,
// and their int32 sums meet in shared memory.  Measured, 1 token: 4096 -> 4096
// 4.3 us, 4096 -> 11008 9.7 us (4.7 TB/s), gated 15.7 us (5.8 TB/s), 12288 ->
// 49152 85 us (7.1 TB/s, part of the 604 MB still in L2).
#include "i8.cuh"
#include "wq_internal.cuh"

namespace wq {
namespace i8 {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kTokens = kGemvTokens;    // the MMA's columns

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Weights are read once: past L1.  Not as read-only data (.nc): this kernel may
// start before the one ahead, which may write what is read here, has ended.
__device__ __forceinline__ uint4 ld_stream(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_tokens(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// The first `valid` (< 16) bytes at p, zeros behind them.
__device__ __forceinline__ uint4 ld_part(const int8_t* p, int valid) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < valid) w[i >> 2] |= uint32_t(uint8_t(p[i])) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 128-byte chunk of 16 rows (of each of RT matrices) and of the tokens.
template <int RT>
struct Chunk {
  uint4 a[2][RT][2], x[2];
};

// U: chunks a warp loads at a time.
template <bool GATED, int U>
__global__ void __launch_bounds__(32 * kMaxWarps) gemv_i8_kernel(const Linear L) {
  constexpr int RT = GATED ? 2 : 1;    // tiles of 16 rows: the gate's and the up projection's
  __shared__ int red[kMaxWarps][RT][kTokens][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  pdl_start();

  const int8_t* wp[RT][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t n = min(n0 + g + 8 * h, L.N - 1);   // rows past the last read it again; nothing is stored for them
    wp[0][h] = L.w0 + n * L.ldw + 16 * t;
    if constexpr (GATED) wp[1][h] = L.w1 + n * L.ldw + 16 * t;
  }
  const bool xlive = g < L.M;
  const int8_t* xp = L.x + (xlive ? g : 0) * L.ldx + 16 * t;
  int acc[RT][4] = {};
  auto load = [&](Chunk<RT> (&c)[U], int at) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = (at + u * warps) * 128 + 64 * i;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) c[u].a[i][r][h] = ld_stream(wp[r][h] + k);
        c[u].x[i] = xlive ? ld_tokens(xp + k) : make_uint4(0, 0, 0, 0);
      }
  };
  auto feed = [&](const uint4 (&a)[RT][2], const uint4& x) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      mma_s8(acc[r], a[r][0].x, a[r][1].x, a[r][0].y, a[r][1].y, x.x, x.y);
      mma_s8(acc[r], a[r][0].z, a[r][1].z, a[r][0].w, a[r][1].w, x.z, x.w);
    }
  };
  auto feed_all = [&](const Chunk<RT> (&c)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      feed(c[u].a[0], c[u].x[0]);
      feed(c[u].a[1], c[u].x[1]);
    }
  };
  const int chunks = int(L.K / 128), step = U * warps;
  int c = warp;
  // The first chunks of the weights on their way to L2 while the kernel ahead
  // finishes: only L2, which sees whatever that kernel may yet write to them.
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (t == 0 && c + u * warps < chunks) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) prefetch_l2(wp[r][h] + (c + u * warps) * 128);
    }
  pdl_wait();

  if (c + (U - 1) * warps < chunks) {
    Chunk<RT> p[U], q[U];
    load(p, c);
    for (;;) {
      c += step;
      bool more = c + (U - 1) * warps < chunks;
      if (more) load(q, c);
      feed_all(p);
      if (!more) break;
      c += step;
      more = c + (U - 1) * warps < chunks;
      if (more) load(p, c);
      feed_all(q);
      if (!more) break;
    }
  }
  for (; c * 128 < L.K; c += warps)      // fewer than U chunks left; the last one may be short
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = c * 128 + 64 * i;
      const int valid = int(min(int64_t(16), L.K - k - 16 * t));
      uint4 a[RT][2], x = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[r][h] = valid >= 16 ? ld_stream(wp[r][h] + k) : ld_part(wp[r][h] + k, valid);
      if (xlive) x = valid >= 16 ? ld_tokens(xp + k) : ld_part(xp + k, valid);
      feed(a, x);
    }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][r][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[r][i];
  __syncthreads();
  if (threadIdx.x < kTokens * 16) {
    const int m = threadIdx.x >> 4, row = threadIdx.x & 15;
    const int64_t n = n0 + row;
    if (n < L.N && m < L.M) {
      int s[RT] = {};
      for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r] += red[w][r][m][row];
      const float sx = L.xs[m];
      float v = scaled(s[0], sx, L.s0[n]);
      if constexpr (GATED) v = apply_act(v, L.type == kF32 ? L.act + kFull : L.act) * scaled(s[1], sx, L.s1[n]);
      store_one(L.y, m * L.ldy + n, v, L.type);
    }
  }
}

template <bool GATED, int U>
cudaError_t launch_as(const Linear& L, cudaStream_t st) {
  const int64_t tiles = (L.N + 15) / 16;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  int dev;
  const cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  // Eight warps a CTA; sixteen where there are fewer tiles than SMs (1024 rows,
  // K = 8192: 4.2 against 5.6 us; 11008 rows, K = 4096: 14.0 against 10.1).
  const int warps = tiles < sm_count(dev) ? 16 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles));
  cfg.blockDim = dim3(unsigned(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemv_i8_kernel<GATED, U>, L);
}

}  // namespace

cudaError_t launch_gemv(const Linear& L, cudaStream_t st) {
  return L.act != kNone ? launch_as<true, 1>(L, st) : launch_as<false, 2>(L, st);
}

}  // namespace i8
}  // namespace wq
