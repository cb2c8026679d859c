// gemm_i8.cu -- 8-bit integer linears on the Blackwell tensor cores
// (tcgen05.mma kind::i8, s8 x s8 -> s32, accumulators in tensor memory).
//
// Both operands are K-major bytes, so TMA brings them straight into the
// 128-byte swizzled layout the MMA reads: 128 bytes of K a row and stage, four
// MMAs of K = 32 each.  Bytes past K and rows past the matrices read as zero.
// int32 sums are exact, so a split of K needs no order.
//
// split kernel (up to 128 tokens, and more where there are few outputs): bound
//   by the read of the weights.  Up to 128 weight rows (gated: half of them the gate's, half the
//   same ones of the up projection) are the MMA's M side, as many as give every
//   SM its share, the tokens, padded to a multiple of 32, its N side: every
//   weight byte is read once.  K is split over a cluster
//   when the tiles alone leave SMs idle: rank r owns the tokens r, r + ks, ...;
//   every rank writes its int32 sums of them into the owner's shared memory,
//   and after one cluster barrier the owner adds what it holds.
//   Measured: 16 tokens 12288 -> 49152 94 us (6.4 TB/s), 64 tokens 4096 -> 11008
//   11.4 us (4.1 TB/s: 3 us to the first data, 7.5 of stream, 1 of epilogue),
//   gated 18.0 us (5.0 TB/s).
// pair kernel (larger batches): bound by the tensor cores.  Two SMs work on one
//   tile of 256 tokens x BN weight rows (cta_group::2): each loads its 128
//   tokens and half of the weight rows (gated: one SM the gate's, the other
//   the up projection's), so a byte of shared memory feeds twice the MMAs.
//   Persistent, two accumulators: a tile's epilogue runs beside the next
//   tile's MMAs.  Measured: 2048 tokens 13824 -> 5120 92 us (3159 TOP/s), gated
//   5120 -> 13824 171 us (3384 TOP/s); a stage of 128 bytes of K takes 513..530
//   cycles at 256 columns, 512 of them the tensor pipe's.
//
// Every wait is bounded (bounded_wait.cuh): an expired wait raises this file's
// device flag, the kernel drains its copies and MMAs, frees its tensor memory
// and returns.
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "i8.cuh"
#include "wq_internal.cuh"
#include "wq_ptx.cuh"

namespace wq {

__device__ unsigned int g_gemm_i8_timeout;

namespace i8 {
namespace {

using namespace ptx;

constexpr int kBK = 128;                         // bytes of K per stage: one swizzle row
constexpr uint32_t kTile = 128 * kBK;            // a 128-row operand tile
constexpr uint32_t kSmemMax = 227 * 1024;

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart, sm_100 descriptor version 1.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | uint64_t(16u >> 4) << 16 | uint64_t(1024u >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}
// kind::i8: s32 accumulator, s8 A and B, both K-major.
__host__ __device__ constexpr uint32_t i8_idesc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
__device__ __forceinline__ uint32_t mapa(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A pair's copy into this CTA's shared memory that completes on the barrier at
// cluster address `bar` (the leader's).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// Relaxed: it tells of tensor-memory reads, which have ended before it, and of
// no memory; a release would wait for the warp's stores of the tile.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Counts `bytes` as landed on the barrier's present phase.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* m, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(m), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// The waits of both kernels, for the test hook: a slot that may be filled again, a
// slot that is full, a final accumulator, an accumulator that has been read.
enum Wait { kWaitEmpty, kWaitFull, kWaitDone, kWaitAccEmpty };
#ifdef WQ_TEST_HOOKS
// Test builds: the wait that gives up at once, {which, its cluster, the CTA's rank
// in it, how many such waits before it}; none where the first is negative.
__device__ int g_give_up[4] = {-1, 0, 0, 0};
// The other waits have 20 ms, so that this one is what ends the kernel.
__device__ __noinline__ bool hooked_wait(uint64_t* b, uint32_t parity, volatile uint32_t* abort, int which, int at) {
  uint32_t cluster, rank;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const bool told = which == g_give_up[0] && int(cluster) == g_give_up[1] && int(rank) == g_give_up[2] && at == g_give_up[3];
  const uint64_t t0 = global_ns();
  while (!told) {
    if (mbar_try_wait(b, parity)) return true;
    if (*abort) return false;
    if (global_ns() - t0 > 20000000ull) break;
  }
  *abort = 1u;
  atomicExch(&g_gemm_i8_timeout, 1u);
  return false;
}
#endif
__device__ __forceinline__ bool wait_for(uint64_t* b, uint32_t parity, volatile uint32_t* abort, Wait which, int at) {
#ifdef WQ_TEST_HOOKS
  if (g_give_up[0] >= 0) return hooked_wait(b, parity, abort, which, at);
#endif
  return mbar_try_wait(b, parity) || mbar_wait(b, parity, abort, &g_gemm_i8_timeout);
}
// Position in a ring of `stages` slots: the slot and its round's parity, kept by
// counting.  (The MMA thread has 512 cycles per stage: a division by the ring's
// size, two descriptors built from scratch and the like took it past 800.)
struct Slot {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
};
// 32 consecutive tensor-memory columns of this warp's 32 lanes, not waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 16 columns; wait16 is where their values begin to exist.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four neighbouring outputs of a row at element i; `vec`: rows start where a
// store of four may.  Outputs from `n` on (of the four) are past the row.
__device__ __forceinline__ void store_four(void* y, int64_t i, const float (&v)[4], int n, int type, bool vec) {
  if (vec && n >= 4) {
    if (type == kF32)
      *reinterpret_cast<float4*>(static_cast<float*>(y) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) =
          type == kBF16 ? make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]))
                        : make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) store_one(y, i + j, v[j], type);
  }
}

// ------------------------------------------------------------ split kernel

struct alignas(64) SplitArgs {
  CUtensorMap tx, t0, t1;
  Linear L;
  int rows;      // weight rows of a tile, a multiple of 16, at least kSplitRowsMin; the MMA's rows behind them are idle
  int mt;        // tokens of a tile: a multiple of 32, at most kSplitTokens
  int stages;
  int vec;       // rows of y start where a store of four outputs may
};

constexpr int kSplitThreads = 256;
constexpr int kSplitTokens = 128;
constexpr int kSplitMax = 8;            // CTAs of a cluster along K
constexpr int kMaxStages = 12;
constexpr int kSplitRowsMin = 64;
// Stages hold a tile's own rows, no room for the MMA's others: more of them fit
// (128 tokens 4096 -> 11008 13.6 -> 13.1 us, gated 64 tokens 18.7 -> 18.0).  For
// the idle rows the MMA reads on into what follows, this far at most.
constexpr uint32_t kSplitSlack = (128 - kSplitRowsMin) * kBK;

// Tensor memory is allocated without a limit on the wait, and a cluster or a
// dependent kernel may wait for a CTA that waits for it: so CTAs that share an SM
// by their shared memory have to fit its 512 columns.  Two of this kernel do (at
// most 128 columns and at least 75 KB each), beside each other or a CTA of the
// weight-only kernels that run two an SM (256 columns, 100 KB); beside the kernels
// that take all 512 (the pair kernel, 197 KB, and the prefill GEMM) none has room.

template <int ACT>
__global__ void __launch_bounds__(kSplitThreads, 2) gemm_i8_split_kernel(const __grid_constant__ SplitArgs p) {
  constexpr bool GATED = ACT != kNone;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_slot, abort_word;
  __shared__ float xscale[kSplitTokens], wscale[128];
  volatile uint32_t* abort = &abort_word;
  const Linear& L = p.L;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = p.stages, mt = p.mt;
  const uint32_t wtile = uint32_t(p.rows) * kBK, stage = wtile + uint32_t(mt) * kBK;
  const int ks = gridDim.y, kr = blockIdx.y;
  const int kb_all = int((L.K + kBK - 1) / kBK);
  const int kb0 = int(int64_t(kb_all) * kr / ks), nkb = int(int64_t(kb_all) * (kr + 1) / ks) - kb0;
  const int out_n = GATED ? p.rows / 2 : p.rows;  // outputs per token of a tile
  const int64_t n0 = int64_t(blockIdx.x) * out_n, m0 = int64_t(blockIdx.z) * mt;
  const uint32_t cols = mt <= 32 ? 32 : mt <= 64 ? 64 : 128;

  pdl_start();
  if (threadIdx.x == 0) {
    prefetch_map(&p.t0);
    prefetch_map(&p.tx);
    if constexpr (GATED) prefetch_map(&p.t1);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    *abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (ks > 1) cluster_arrive();        // waited for before the first write to a peer: it runs by then
  // The first weight tiles on their way to L2 while the kernel ahead finishes:
  // only L2, which sees whatever that kernel may yet write to them.
  if (warp == 0 && elect_one())
    for (int i = 0; i < min(S, nkb); ++i) {
      prefetch_tile(&p.t0, (kb0 + i) * kBK, int(n0));
      if constexpr (GATED) prefetch_tile(&p.t1, (kb0 + i) * kBK, int(n0));
    }
  __syncwarp();
  pdl_wait();

  // Warps 0 and 1 stay whole, so that what they compute for the one issuing
  // lane lives in uniform registers, where the TMA and MMA instructions read it.
  int issued = 0;                      // stages that warp 0 has asked for
  if (warp == 0) {
    Slot at;
    for (int i = 0; i < nkb; ++i, at.next(S)) {
      if (i >= S && !__all_sync(0xffffffffu, wait_for(&empty[at.s], at.parity ^ 1u, abort, kWaitEmpty, i))) break;
      uint8_t* w = ring + at.s * stage;
      const int k = (kb0 + i) * kBK;
      if (elect_one()) {
        mbar_expect_tx(&full[at.s], uint32_t(p.rows + mt) * kBK);
        tma_load_2d(w, &p.t0, &full[at.s], k, int(n0));
        if constexpr (GATED) tma_load_2d(w + out_n * kBK, &p.t1, &full[at.s], k, int(n0));
        tma_load_2d(w + wtile, &p.tx, &full[at.s], k, int(m0));
      }
      ++issued;
    }
  } else if (warp == 1) {
    const uint32_t idesc = i8_idesc(128, mt);
    const uint64_t ring_desc = sw128_desc(smem_u32(ring));
    Slot at;
    for (int i = 0; i < nkb; ++i, at.next(S)) {
      if (!__all_sync(0xffffffffu, wait_for(&full[at.s], at.parity, abort, kWaitFull, i))) break;
      tc_fence_after();
      const uint64_t a = ring_desc + uint32_t(at.s) * (stage >> 4), b = a + (wtile >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)
          umma_i8<1>(tmem, a + 2 * kk, b + 2 * kk, idesc, (i > 0 || kk > 0) ? 1u : 0u);
        commit_one(&empty[at.s]);
      }
    }
    if (elect_one()) commit_one(&done);   // always: the teardown waits on it before freeing tensor memory
  }
  __syncwarp();
  // the tile's scales, while the first operands are on their way
  const int mend = int(min(int64_t(mt), L.M - m0));     // tokens of this tile
  const int row = 32 * (warp & 3) + lane;               // this lane's weight row, of tokens 32 (warp / 4) .. + 31 of 64
  const int col = GATED && row >= out_n ? row - out_n : row;
  const bool up = GATED && row >= out_n;
  const int64_t n = n0 + col;
  const float sw = row < p.rows && n < L.N ? (up ? L.s1[n] : L.s0[n]) : 0.0f;
  if (threadIdx.x < mend) xscale[threadIdx.x] = L.xs[m0 + threadIdx.x];
  if (warp < 4) wscale[row] = sw;
  bool ok = wait_for(&done, 0, abort, kWaitDone, 0);
  ok = __all_sync(0xffffffffu, ok);   // tcgen05.ld needs the whole warp
  const uint32_t tcol = tmem + (uint32_t(32 * (warp & 3)) << 16);

  if (!GATED && ks == 1) {
    // Unsplit: straight from tensor memory, neighbouring lanes to neighbouring
    // outputs.  (Through shared memory, four outputs a thread, 128 tokens of 80
    // rows took 3.8 us for this.)
    __syncthreads();                    // xscale; behind it every wait has ended
    if (!*abort) {                      // else the sums may lack a part of K, though `done` came
      tc_fence_after();
      auto store = [&](auto type) {
        for (int c = 32 * (warp >> 2); c < mend; c += 64) {
          uint32_t r[32];
          tmem_ld32(tcol + uint32_t(c), r);
          tmem_wait_ld();
          if (row < out_n && n < L.N) {
            int64_t at = (m0 + c) * L.ldy + n;
#pragma unroll
            for (int i = 0; i < 32; ++i, at += L.ldy)
              if (c + i < mend) store_one(L.y, at, scaled(int(r[i]), xscale[c + i], sw), decltype(type)::value);
          }
        }
      };
      if (L.type == kBF16) store(std::integral_constant<int, kBF16>());
      else if (L.type == kF16) store(std::integral_constant<int, kF16>());
      else store(std::integral_constant<int, kF32>());
    }
  } else {
    // The int32 sums as [rank][own token][128 rows]: gated with one rank, in the
    // idle ring (every MMA has read its operands and every copy has landed);
    // with more, behind the ring of each token's owner: token t belongs to rank
    // t % ks (ks divides 32).
    int* part = reinterpret_cast<int*>(ks > 1 ? ring + S * stage + kSplitSlack : ring);
    const int own = mt / ks, lk = 31 - __clz(ks);
    if (ks > 1) cluster_wait();
    if (ok) {
      tc_fence_after();
      const uint32_t at = smem_u32(part) + uint32_t(kr * own * 128 + row) * 4;
      for (int c = 32 * (warp >> 2); c < mt; c += 64) {
        uint32_t r[32];
        tmem_ld32(tcol + uint32_t(c), r);
        tmem_wait_ld();
        if (ks == 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i) part[(c + i) * 128 + row] = int(r[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            st_cluster(mapa(at + (uint32_t(c + i) >> lk) * 512, uint32_t(i & (ks - 1))), r[i]);
        }
      }
    }
    __syncthreads();                    // every wait has ended
    if (ks > 1) {
      // a rank that gave up has not sent (all of) its sums: nobody stores the tile
      if (*abort && threadIdx.x < uint32_t(ks)) st_cluster(mapa(smem_u32(&abort_word), threadIdx.x), 1u);
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
    // A thread takes four neighbouring outputs of a token; token t of this rank
    // is token kr + ks t of the tile.
    const int groups = out_n / 4, token0 = threadIdx.x / groups, tokens = kSplitThreads / groups;
    const int j = threadIdx.x - token0 * groups;
    const int left = token0 < tokens ? int(min(int64_t(4), L.N - n0 - 4 * j)) : 0;   // of them inside the row
    if (!*abort && left > 0) {
      float s0[4], s1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s0[i] = wscale[4 * j + i];
        s1[i] = GATED ? wscale[out_n + 4 * j + i] : 0.0f;
      }
      for (int t = token0; kr + ks * t < mend; t += tokens) {
        int a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < kSplitMax; ++r)
          if (r < ks) {
            const int4 v = *reinterpret_cast<const int4*>(part + (r * own + t) * 128 + 4 * j);
            a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
            if constexpr (GATED) {
              const int4 u = *reinterpret_cast<const int4*>(part + (r * own + t) * 128 + out_n + 4 * j);
              b[0] += u.x; b[1] += u.y; b[2] += u.z; b[3] += u.w;
            }
          }
        const int m = kr + ks * t;
        const float sx = xscale[m];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = scaled(a[e], sx, s0[e]);
          if constexpr (GATED) v[e] = apply_act(v[e], ACT) * scaled(b[e], sx, s1[e]);
        }
        store_four(L.y, (m0 + m) * L.ldy + n0 + 4 * j, v, left, L.type, p.vec);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // Given up: the copies in flight land before shared memory goes away, the
  // MMAs issued end before tensor memory does.
  if (*abort && lane == 0) {
    if (warp == 0)
      for (int i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_drain(&full[i % S], (i / S) & 1, &g_gemm_i8_timeout);
    if (warp == 1) mbar_drain(&done, 0, &g_gemm_i8_timeout);
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
}

// ------------------------------------------------------------ pair kernel

struct alignas(64) PairArgs {
  CUtensorMap tx, t0, t1;
  Linear L;
  int bn;            // MMA columns of a tile: a multiple of 32 (gated: 64), at most 256
  int tiles_m, tiles_n;
  int stages;
  int vec;           // rows of y start on 16-byte boundaries
};

constexpr int kPairThreads = 320;       // producer, MMA, eight epilogue warps
constexpr int kPairRing = 6 * 2 * int(kTile);   // six stages of the largest tile, more of smaller ones
constexpr int kPairStages = 9;
constexpr int kGroupM = 16;             // token tiles that neighbouring tiles walk through first

// A warp's 32 rows of 64 output bytes, from its staging buffer to columns n ..
// of rows m .. of y: rows of 64 bytes by 16-byte stores where y's rows allow
// them, else by elements, neighbouring lanes to neighbouring addresses.
// (Stored straight from the lanes that hold a row each, a store touches 32
// rows: 1.1 us per 32 columns, and 32-fold traffic where rows are unaligned.)
constexpr int kOutRow = 80;
__device__ __forceinline__ void flush_rows(const uint8_t* out, const Linear& L, int64_t m, int64_t n, int lane, int vec) {
  __syncwarp();
  const int eb = L.type == kF32 ? 4 : 2, cols = 64 / eb;
  uint8_t* y = static_cast<uint8_t*>(L.y);
  if (vec && n + cols <= L.N) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + lane / 4, at = (lane & 3) * 16;
      if (m + row < L.M)
        *reinterpret_cast<uint4*>(y + ((m + row) * L.ldy + n) * eb + at) =
            *reinterpret_cast<const uint4*>(out + row * kOutRow + at);
    }
  } else {
    const int col = lane & (cols - 1), per = 32 / cols, first = lane / cols;
    if (n + col < L.N) {
      const int rows = int(min(int64_t(32), L.M - m));
      const uint8_t* src = out + first * kOutRow + col * eb;
      uint8_t* dst = y + ((m + first) * L.ldy + n + col) * eb;
      const int64_t hop = per * L.ldy * eb;
      if (eb == 4) {
#pragma unroll 8
        for (int row = first; row < rows; row += 2, src += 2 * kOutRow, dst += hop)
          *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
      } else {
#pragma unroll 8
        for (int row = 0; row < rows; ++row, src += kOutRow, dst += hop)
          *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
      }
    }
  }
  __syncwarp();
}

// Tile t -> (token tile, weight tile): groups of kGroupM token tiles, token
// tiles fastest inside a group, so that the tiles in flight share operands.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per = kGroupM * tiles_n, g = t / per, first = g * kGroupM;
  const int rows = min(kGroupM, tiles_m - first), r = t - g * per;
  tm = first + r % rows;
  tn = r / rows;
}

// What is left to wait for when a CTA of the pair has given up: both call this.  The
// copies in flight have to land before shared memory goes away.  All of them complete
// on the leader's barriers, which count both CTAs' bytes, and one of the two may have
// asked for stages that the other has not come to: at most the ring's last S, as a
// slot is asked for again only behind the MMAs that read it.  The leader puts the
// missing half of these on their barriers and waits for them; then both go.
// (Its own function: inline it cost every call 0.1 us at the kernel's end.)
__device__ __noinline__ void pair_gave_up(uint64_t* full, uint64_t* done, uint32_t* peer_issued, int64_t issued, int S,
                                          uint32_t stage, uint32_t rank) {
  if (threadIdx.x == 0) {               // of the producer warp
    const uint32_t at = mapa(smem_u32(peer_issued), rank ^ 1u);
    st_cluster(at, uint32_t(issued));
    st_cluster(at + 4, uint32_t(issued >> 32));
  }
  __syncwarp();
  cluster_sync();
  if (threadIdx.x == 0 && rank == 0) {
    const volatile uint32_t* got = peer_issued;
    const int64_t theirs = int64_t(uint64_t(got[1]) << 32 | got[0]), last = issued > theirs ? issued : theirs;
    for (int64_t j = last > S ? last - S : 0; j < last; ++j) {
      uint64_t* bar = &full[j % S];
      if (j >= issued) mbar_expect_tx(bar, stage);            // the peer's copies alone
      if (j >= theirs) mbar_complete_tx(bar, stage);          // this CTA's alone
      mbar_drain(bar, uint32_t(j / S) & 1u, &g_gemm_i8_timeout);
    }
  }
  if (threadIdx.x == 32) mbar_drain(done, 0, &g_gemm_i8_timeout);
  __syncwarp();
  cluster_sync();
}

template <int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_i8_pair_kernel(const __grid_constant__ PairArgs p) {
  constexpr bool GATED = ACT != kNone;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kPairStages];      // leader's: both CTAs' copies landed
  __shared__ uint64_t empty[kPairStages];     // MMAs done with the slot (commit to both)
  __shared__ uint64_t acc_full[2];            // accumulator final (commit to both)
  __shared__ uint64_t acc_empty[2];           // leader's: both CTAs' epilogue warps have read it
  __shared__ uint64_t done;                   // all MMAs done (commit to both)
  __shared__ uint32_t tmem_slot, abort_word;
  __shared__ uint32_t peer_abort, peer_issued[2];     // the other CTA has given up; the stages it had asked for
  // per epilogue warp: the tile's weight scales; 32 rows of 64 output bytes, 16 bytes apart
  __shared__ __align__(16) float wscale_all[8][256];
  __shared__ __align__(16) uint8_t out_all[8][32 * kOutRow];
  volatile uint32_t* abort = &abort_word;
  const Linear& L = p.L;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int bn = p.bn, S = p.stages;
  const uint32_t stage = kTile + uint32_t(bn / 2) * kBK;
  const int nkb = int((L.K + kBK - 1) / kBK);
  const int tiles = p.tiles_m * p.tiles_n, step = gridDim.x / 2;
  const int out_n = GATED ? bn / 2 : bn;      // outputs per token of a tile

  pdl_start();
  if (threadIdx.x == 0) {
    prefetch_map(&p.tx);
    prefetch_map(GATED && rank == 1 ? &p.t1 : &p.t0);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);
    }
    mbar_init(&done, 1);
    *abort = 0u;
    peer_abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();       // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  pdl_wait();

  // Warps 0 and 1 stay whole, so that what they compute for the one issuing
  // lane lives in uniform registers, where the TMA and MMA instructions read it
  // (with a lone lane the MMA warp needed over 600 cycles a stage of 512).
  int64_t issued = 0;                  // stages that warp 0 has asked for
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    Slot at;
    const uint32_t full0 = mapa(smem_u32(&full[0]), 0);      // the leader's barriers
    const CUtensorMap* tw = GATED && rank == 1 ? &p.t1 : &p.t0;
    for (int t = blockIdx.x / 2; t < tiles && ok; t += step) {
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int mrow = tm * 256 + int(rank) * 128;
      const int nrow = GATED ? tn * out_n : tn * bn + int(rank) * (bn / 2);
      for (int kb = 0; kb < nkb; ++kb, ++issued, at.next(S)) {
        if (issued >= S)
          ok = __all_sync(0xffffffffu, wait_for(&empty[at.s], at.parity ^ 1u, abort, kWaitEmpty, int(issued)));
        if (!ok) break;
        uint8_t* a = ring + at.s * stage;
        const uint32_t bar = full0 + uint32_t(at.s) * 8;
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(&full[at.s], 2 * stage);
          tma_load_pair(a, &p.tx, bar, kb * kBK, mrow);
          tma_load_pair(a + kTile, tw, bar, kb * kBK, nrow);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA (leader)
    if (rank == 0) {
      const uint32_t idesc = i8_idesc(256, bn);
      const uint64_t ring_desc = sw128_desc(smem_u32(ring));
      bool ok = true;
      int n = 0;
      Slot at;
      for (int t = blockIdx.x / 2; t < tiles && ok; t += step, ++n) {
        const int a = n & 1;
        if (n >= 2)
          ok = __all_sync(0xffffffffu, wait_for(&acc_empty[a], ((n >> 1) - 1) & 1, abort, kWaitAccEmpty, n));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(a) * 256;
        for (int kb = 0; kb < nkb; ++kb, at.next(S)) {
          ok = __all_sync(0xffffffffu, wait_for(&full[at.s], at.parity, abort, kWaitFull, n * nkb + kb));
          if (!ok) break;
          tc_fence_after();
          const uint64_t sa = ring_desc + uint32_t(at.s) * (stage >> 4), sb = sa + (kTile >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)
              umma_i8<2>(d, sa + 2 * kk, sb + 2 * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
            commit_pair(&empty[at.s]);
          }
        }
        if (ok && elect_one()) commit_pair(&acc_full[a]);
      }
      if (elect_one()) commit_pair(&done);   // always: both CTAs wait on it before they free tensor memory
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp w reads tensor-memory lanes 32 (w % 4) .. (rows of this CTA's 128
    // tokens), and of the 32-column blocks of outputs every other one, in two
    // halves: while one is worked on the next is on its way to registers.
    const int q = warp & 3, half = (warp - 2) >> 2;
    float* wscale = wscale_all[warp - 2];
    uint8_t* out = out_all[warp - 2];
    const int eb = L.type == kF32 ? 4 : 2;
    bool ok = true;
    int n = 0;
    // this lane's scales of a tile: of columns lane, lane + 32, ... (gated: the
    // gate's, then the up projection's) and of its token
    float ws[8], sx;
    auto load_scales = [&](int t) {
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t m = int64_t(tm) * 256 + rank * 128 + 32 * q + lane, n0 = int64_t(tn) * out_n;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        const bool up = GATED && c >= out_n;
        const int64_t nn = n0 + (up ? c - out_n : c);
        ws[i] = c < bn && nn < L.N ? (up ? L.s1[nn] : L.s0[nn]) : 0.0f;
      }
      sx = m < L.M ? L.xs[m] : 0.0f;
    };
    load_scales(blockIdx.x / 2);
    for (int t = blockIdx.x / 2; t < tiles && ok; t += step, ++n) {
      int tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      const int a = n & 1;
      const int64_t m = int64_t(tm) * 256 + rank * 128 + 32 * q;      // the warp's first token
      const int64_t n0 = int64_t(tn) * out_n;
      // each warp keeps the columns' scales for itself, as no warp may wait for
      // one that has given up; the next tile's are fetched meanwhile
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) wscale[lane + 32 * i] = ws[i];
      __syncwarp();
      const float s = sx;
      if (t + step < tiles) load_scales(t + step);
      ok = wait_for(&acc_full[a], (n >> 1) & 1, abort, kWaitDone, n);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + (uint32_t(32 * q) << 16) + uint32_t(a) * 256;
      // 16 columns from c on, of this lane's token, into the staging row
      auto work = [&](const uint32_t (&r)[16], const uint32_t (&u)[16], int c) {
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 s0 = *reinterpret_cast<const float4*>(wscale + c + j + i);
            v[i] = scaled(int(r[j + i]), s, s0.x);
            v[i + 1] = scaled(int(r[j + i + 1]), s, s0.y);
            v[i + 2] = scaled(int(r[j + i + 2]), s, s0.z);
            v[i + 3] = scaled(int(r[j + i + 3]), s, s0.w);
            if constexpr (GATED) {
              const float4 s1 = *reinterpret_cast<const float4*>(wscale + out_n + c + j + i);
              v[i] = apply_act(v[i], ACT) * scaled(int(u[j + i]), s, s1.x);
              v[i + 1] = apply_act(v[i + 1], ACT) * scaled(int(u[j + i + 1]), s, s1.y);
              v[i + 2] = apply_act(v[i + 2], ACT) * scaled(int(u[j + i + 2]), s, s1.z);
              v[i + 3] = apply_act(v[i + 3], ACT) * scaled(int(u[j + i + 3]), s, s1.w);
            }
          }
          uint4* o = reinterpret_cast<uint4*>(out + lane * kOutRow + (((c + j) * eb) & 63));
          if (L.type == kF32) {
            o[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            o[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
          } else {
            o[0] = L.type == kBF16 ? make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                pack_bf16(v[6], v[7]))
                                   : make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]),
                                                pack_f16(v[6], v[7]));
          }
        }
      };
      auto load = [&](uint32_t (&r)[16], uint32_t (&u)[16], int c) {
        tmem_ld16(base + uint32_t(c), r);
        if constexpr (GATED) tmem_ld16(base + uint32_t(out_n + c), u);
      };
      auto landed = [&](uint32_t (&r)[16], uint32_t (&u)[16]) {
        wait16(r);
        if constexpr (GATED) wait16(u);
      };
      auto all_read = [&]() {               // this warp's columns are in registers: the MMAs may have the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(mapa(smem_u32(&acc_empty[a]), 0));
      };
      int c = 32 * half;
      if (c >= out_n) {
        all_read();
      } else {
        uint32_t r0[16], u0[16], r1[16], u1[16];
        load(r0, u0, c);
#pragma unroll 1
        for (; c < out_n; c += 64) {
          landed(r0, u0);
          load(r1, u1, c + 16);
          work(r0, u0, c);
          if (L.type == kF32) flush_rows(out, L, m, n0 + c, lane, p.vec);
          landed(r1, u1);
          if (c + 64 < out_n) load(r0, u0, c + 64);
          else all_read();
          work(r1, u1, c + 16);
          flush_rows(out, L, m, n0 + (L.type == kF32 ? c + 16 : c), lane, p.vec);
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 0) st_cluster(mapa(smem_u32(&peer_abort), rank ^ 1u), 1u);
  if (warp == 1 && lane == 0) mbar_drain(&done, 0, &g_gemm_i8_timeout);
  __syncwarp();
  cluster_sync();           // no arrival or copy of the pair is left in flight, unless one of the two has given up
  if ((*abort | *static_cast<volatile uint32_t*>(&peer_abort)) != 0u)      // the same in both
    pair_gave_up(full, &done, peer_issued, issued, S, stage, rank);
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------ host

// Largest dynamic shared memory, once per kernel and device.
template <typename F>
cudaError_t allow_smem(F* fn, uint32_t bytes, std::atomic<bool>* set, int dev) {
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, int(cudaSharedmemCarveoutMaxShared));
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
}

bool make_map(CUtensorMap* map, const int8_t* base, int64_t K, int64_t rows, int64_t ld, int box_rows) {
  return make_tensor_map_2d(map, TmaType::kU8, base, uint64_t(K), uint64_t(rows), uint64_t(ld), kBK,
                            uint32_t(box_rows), 128);
}

template <int ACT>
cudaError_t allow_split(int dev) {
  static std::atomic<bool> set[64];
  return allow_smem(gemm_i8_split_kernel<ACT>, kSmemMax - 4096, set, dev);
}

// How many clusters of ks CTAs of the split kernel, one CTA an SM, run at once:
// fewer than the SMs divided by ks, as a cluster stays within one group of SMs
// (16 clusters of 8 took two rounds: 13.1 us against 8.5 over 4).
template <int ACT>
int clusters_at_once(int dev, int ks) {
  static std::atomic<int> cached[64][kSplitMax + 1];
  int n = cached[dev][ks].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, unsigned(ks));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = kSmemMax - 4096;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = unsigned(ks);
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (allow_split<ACT>(dev) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, gemm_i8_split_kernel<ACT>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 1;
    }
    cached[dev][ks].store(n, std::memory_order_relaxed);
  }
  return n;
}

struct SplitPlan {
  int mt, rows, ks;
  int64_t tiles_n, tiles_m;
  int64_t load;      // what one SM has to read, in stages of one row (about 0.6 ns each)
};

// Rows of a tile and split of K: the least that one SM has to read: for each of
// its tiles the rows of weights and the tokens, over its share of K.  A split
// adds an exchange, as much as 250 of these for each doubling, and its clusters
// have to be on the SMs at once, one CTA an SM; smaller tiles have to read a
// good deal less to be worth it, and were not for clusters of 4 and 8.  (64
// tokens, 4096 x 4096: 9.5 us unsplit, 8.7 / 7.8 / 8.1 over 2 / 4 / 8 CTAs;
// 11008 x 4096: 11.8 us in 86 tiles of 128 rows, 11.4 in 115 of 96, 14.1 in 172
// halves of 128; 16 tokens, 1024 x 8192 over 8 CTAs: 5.5 with 128 rows, 5.9 with 80.)
template <int ACT>
SplitPlan split_plan(const Linear& L, int dev) {
  constexpr bool GATED = ACT != kNone;
  SplitPlan p = {};
  const int nsm = sm_count(dev);
  const int64_t kb = (L.K + kBK - 1) / kBK;
  p.mt = L.M > kSplitTokens ? kSplitTokens : int((L.M + 31) / 32 * 32);
  p.tiles_m = (L.M + p.mt - 1) / p.mt;
  p.load = INT64_MAX;
  for (int c = 1; c <= kSplitMax && (c == 1 || kb >= 2 * c); c *= 2)
    for (int rows = 128; rows >= (c <= 2 ? kSplitRowsMin : 128); rows -= 16) {
      const int out_n = GATED ? rows / 2 : rows;
      const int64_t tn = (L.N + out_n - 1) / out_n, t = tn * p.tiles_m;
      if (c > 1 && t > clusters_at_once<ACT>(dev, c)) break;
      const int64_t load = (c > 1 ? 1 : (t + nsm - 1) / nsm) * (rows + p.mt) * ((kb + c - 1) / c) +
                           250 * (c >= 8 ? 3 : c / 2);
      if (load < (rows < 128 ? p.load - p.load / 8 : p.load)) {
        p.load = load;
        p.ks = c;
        p.rows = rows;
        p.tiles_n = tn;
      }
    }
  return p;
}

template <int ACT>
cudaError_t split(const Linear& L, cudaStream_t st) {
  constexpr bool GATED = ACT != kNone;
  int dev;
  cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  if ((e = allow_split<ACT>(dev)) != cudaSuccess) return e;
  const int nsm = sm_count(dev);
  const SplitPlan plan = split_plan<ACT>(L, dev);
  const int ks = plan.ks;
  if (plan.tiles_n > 0x7fffffff || plan.tiles_m > 65535) return cudaErrorInvalidValue;
  SplitArgs p;
  p.L = L;
  p.mt = plan.mt;
  p.rows = plan.rows;
  const int eb = type_bytes(L.type);
  p.vec = reinterpret_cast<uintptr_t>(L.y) % (4 * eb) == 0 && (L.ldy * eb) % (4 * eb) == 0;
  const uint32_t stage = uint32_t(p.rows + p.mt) * kBK;
  const int out_n = GATED ? p.rows / 2 : p.rows;
  if (!make_map(&p.tx, L.x, L.K, L.M, L.ldx, p.mt) || !make_map(&p.t0, L.w0, L.K, L.N, L.ldw, out_n) ||
      (GATED && !make_map(&p.t1, L.w1, L.K, L.N, L.ldw, out_n)))
    return cudaErrorInvalidValue;
  const uint32_t parked = ks > 1 ? uint32_t(p.mt) * 512 : 0;
  // two CTAs an SM where there are more than SMs, else one with a deeper ring
  const uint32_t budget = (plan.tiles_n * plan.tiles_m * ks > nsm ? kSmemMax / 2 : kSmemMax) - 4096;
  p.stages = int((budget - 1024 - kSplitSlack - parked) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(plan.tiles_n), unsigned(ks), unsigned(plan.tiles_m));
  cfg.blockDim = dim3(kSplitThreads, 1, 1);
  cfg.dynamicSmemBytes = p.stages * stage + kSplitSlack + parked + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = unsigned(ks);
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_i8_split_kernel<ACT>, p);
}

// Columns of a pair's tile: the fewest that one pair works through, counting a
// tile's own cost as 32 of them.
template <bool GATED>
int pair_columns(const Linear& L, int pairs) {
  const int64_t tm = (L.M + 255) / 256;
  int64_t best = INT64_MAX;
  int columns = 256;
  for (int bn = 256; bn >= 64; bn -= GATED ? 64 : 32) {
    const int out_n = GATED ? bn / 2 : bn;
    const int64_t t = (tm * ((L.N + out_n - 1) / out_n) + pairs - 1) / pairs * (bn + 32);
    if (t < best) {
      best = t;
      columns = bn;
    }
  }
  return columns;
}

// More than 128 tokens: the pair kernel, but for few outputs and long sums, which
// leave most pairs without a tile.  Both costs in the split plan's units: a
// pair's stage takes its read or its MMAs (1.75 a column), its tile 2800 (gated
// 4300) more than a split tile, which has an epilogue of its own of 14 a token.
// The split kernel has to be well ahead: measured, split / pair, 256 tokens,
// 1024 x 8192 9.9 / 13.2 us, gated 1024 x 4096 8.4 / 8.9; 160 tokens, 256 x 4096
// 5.9 / 8.3; 146, 68 x 7554 7.3 / 16.9; but 512 tokens, 1024 x 4096 8.3 / 8.6,
// 160, 4096 x 4096 11.0 / 9.5.
template <int ACT>
bool prefer_split(const Linear& L, int dev) {
  constexpr bool GATED = ACT != kNone;
  const int pairs = sm_count(dev) / 2, bn = pair_columns<GATED>(L, pairs), out_n = GATED ? bn / 2 : bn;
  const int64_t kb = (L.K + kBK - 1) / kBK;
  const int64_t rounds = ((L.M + 255) / 256 * ((L.N + out_n - 1) / out_n) + pairs - 1) / pairs;
  const int64_t stage = 128 + bn / 2 > bn * 7 / 4 ? 128 + bn / 2 : bn * 7 / 4;
  if (rounds > 1) return false;
  const SplitPlan s = split_plan<ACT>(L, dev);
  return 2 * (s.load + 14 * s.mt) < kb * stage + (GATED ? 4300 : 2800);
}

template <int ACT>
cudaError_t pair(const Linear& L, cudaStream_t st) {
  constexpr bool GATED = ACT != kNone;
  int dev;
  cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> set[64];
  if ((e = allow_smem(gemm_i8_pair_kernel<ACT>, kPairRing + 1024, set, dev)) != cudaSuccess) return e;
  const int pairs = sm_count(dev) / 2;
  PairArgs p;
  p.L = L;
  const int64_t tm = (L.M + 255) / 256;
  p.bn = pair_columns<GATED>(L, pairs);
  const int out_n = GATED ? p.bn / 2 : p.bn;
  const int64_t tn = (L.N + out_n - 1) / out_n;
  if (tm * tn > 0x7fffffff) return cudaErrorInvalidValue;
  p.tiles_m = int(tm);
  p.tiles_n = int(tn);
  if (!make_map(&p.tx, L.x, L.K, L.M, L.ldx, 128) || !make_map(&p.t0, L.w0, L.K, L.N, L.ldw, p.bn / 2) ||
      (GATED && !make_map(&p.t1, L.w1, L.K, L.N, L.ldw, p.bn / 2)))
    return cudaErrorInvalidValue;
  const int eb = type_bytes(L.type);
  p.vec = reinterpret_cast<uintptr_t>(L.y) % 16 == 0 && (L.ldy * eb) % 16 == 0;
  const uint32_t stage = kTile + uint32_t(p.bn / 2) * kBK;
  p.stages = kPairRing / int(stage);
  if (p.stages > kPairStages) p.stages = kPairStages;
  const int64_t ctas = 2 * (tm * tn < pairs ? tm * tn : pairs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = p.stages * stage + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_i8_pair_kernel<ACT>, p);
}

template <int ACT>
cudaError_t launch_as(const Linear& L, cudaStream_t st) {
  if (L.M <= kSplitTokens) return split<ACT>(L, st);
  int dev;
  const cudaError_t e = current_device(&dev);
  if (e != cudaSuccess) return e;
  return prefer_split<ACT>(L, dev) ? split<ACT>(L, st) : pair<ACT>(L, st);
}

}  // namespace

cudaError_t current_device(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  return *dev >= 0 && *dev < 64 ? cudaSuccess : cudaErrorInvalidDevice;
}

int sm_count(int dev) {
  static std::atomic<int> cached[64];
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) n = 2;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaError_t launch_linear(const Linear& L, cudaStream_t st) {
  if (L.M <= kGemvTokens) return launch_gemv(L, st);
  if (L.act == kNone) return launch_as<kNone>(L, st);
  switch (L.type == kF32 ? L.act + kFull : L.act) {
    case kSilu: return launch_as<kSilu>(L, st);
    case kGelu: return launch_as<kGelu>(L, st);
    case kGeluTanh: return launch_as<kGeluTanh>(L, st);
    case kSilu + kFull: return launch_as<kSilu + kFull>(L, st);
    case kGelu + kFull: return launch_as<kGelu + kFull>(L, st);
    default: return launch_as<kGeluTanh + kFull>(L, st);
  }
}

bool gemm_read_and_clear_timeout(cudaError_t* err) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_gemm_i8_timeout, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_gemm_i8_timeout, &zero, sizeof(zero));
  *err = e;
  return v != 0;
}

}  // namespace i8
}  // namespace wq

#ifdef WQ_TEST_HOOKS
// Test builds only: which wait of the 8-bit kernels gives up (see g_give_up); 0 on success.
extern "C" int wq_test_give_up_i8(int which, int cluster, int rank, int at) {
  const int told[4] = {which, cluster, rank, at};
  return cudaMemcpyToSymbol(wq::i8::g_give_up, told, sizeof(told)) == cudaSuccess ? 0 : 7;
}
#endif
