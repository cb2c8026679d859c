// i8.cuh -- what the kernels of the 8-bit integer linears share: the argument
// block, the activations, the output conversion.
//
//   y[m, n] = s_x[m] s_w[n] sum_k q_x[m, k] q_w[n, k]
//   h[m, n] = act(g[m, n]) u[m, n],  g and u as y with the gate's and the up
//             projection's weights
//
// The sum is exact in int32 (the C ABI refuses K whose sums could pass 2^31),
// so neither the order of the terms nor a split of K over warps, CTAs or
// clusters changes a result: y is bit for bit the same from every kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace wq {
namespace i8 {

enum Type { kBF16 = 0, kF16 = 1, kF32 = 2 };                  // wq_type
enum Act { kSilu = 0, kGelu = 1, kGeluTanh = 2, kNone = -1 };  // wq_act; kNone: no gate
constexpr int kFull = 4;   // added to an activation: the form for an fp32 result

inline int type_bytes(int t) { return t == kF32 ? 4 : 2; }

// One product, or the two of a gated call: w0 / s0 the weights (the gate's),
// w1 / s1 the up projection's.  Row strides in elements.
struct Linear {
  const int8_t* x;
  const float* xs;
  const int8_t* w0;
  const float* s0;
  const int8_t* w1;
  const float* s1;
  void* y;
  int64_t M, N, K, ldx, ldw, ldy;
  int type;   // of y
  int act;    // kNone: y is the product
};

// erfc(z) / exp(-z^2) / t, t = 1 / (1 + 0.48 z), the form of Hastings's
// approximations: a polynomial of degree 8 in t, fitted here (least squares over
// Chebyshev nodes, reweighted to even the relative error out, the coefficients
// rounded to fp32 one by one and the others fitted again).  Off by at most 3.7e-8
// of its value for z in 0 .. 10.2, where exp(-z^2) ends in fp32.
__device__ __forceinline__ float erfc_tail(float t) {
  float p = -0.05119941011071205f;
  p = __fmaf_rn(p, t, 0.27519741654396057f);
  p = __fmaf_rn(p, t, -0.541874349117279f);
  p = __fmaf_rn(p, t, 0.4027293622493744f);
  p = __fmaf_rn(p, t, -0.0878278985619545f);
  p = __fmaf_rn(p, t, 0.2302476018667221f);
  p = __fmaf_rn(p, t, 0.23021966218948364f);
  p = __fmaf_rn(p, t, 0.27173522114753723f);
  return __fmaf_rn(p, t, 0.27077242732048035f);
}

// The hardware's 2^x (2 steps) and 1 / x (1 step).
__device__ __forceinline__ float hw_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float hw_reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The activations keep their relative accuracy for g << 0 (forms with 1 + erf or
// 1 + tanh would lose it there) until they leave fp32's normal range; their
// errors are stated at wq_gated_i8 (wq.h).
// FULL, for an fp32 result: CUDA's expf.  Else the hardware's 2^x of a rounded
// argument, whose error grows with it by 1.2 steps a unit: at its far end a
// fiftieth of the half step that bf16's rounding may take, a seventh of fp16's, and
// a gated tile's epilogue waits for these instructions (1228 x 1216 -> 12096 to
// bf16: silu 33.1 us, with expf 35.1; gelu 37.0 and 38.6).
// Every rounding is spelled out: of plain products and sums the compiler may
// contract others in each kernel, and a token's bits would depend on its batch.

// g sigmoid(v) by e = exp(-|v|) <= 1: g / (1 + e) above zero, g e / (1 + e)
// below, so that nothing overflows.  Below -64 the sum is 1, and e is taken 64
// further up (2^64, e^64), clear of the subnormals; the last product undoes it.
template <bool FULL>
__device__ __forceinline__ float gate_of(float g, float v) {
  const bool far = v < -64.0f;
  float e;
  if constexpr (FULL) e = expf(__fsub_rn(far ? 64.0f : 0.0f, fabsf(v)));     // exact for 32 <= |v| <= 128
  else e = hw_exp2(__fmaf_rn(fabsf(v), -1.4426950408889634f, far ? 64.0f : 0.0f));
  const float q = hw_reciprocal(__fadd_rn(1.0f, e)), down = FULL ? 1.6038108905486378e-28f : 0x1p-64f;   // exp(-64)
  return __fmul_rn(v > 0.0f ? g : __fmul_rn(g, e), far ? down : q);
}

template <bool FULL>
__device__ __forceinline__ float act_of(float g, int act) {
  if (act == kSilu) return gate_of<FULL>(g, g);
  if (act == kGelu) {
    const float t = hw_reciprocal(__fmaf_rn(fabsf(g), 0.33941125496954283f, 1.0f));   // 0.48 |g| / sqrt 2
    const float x = __fmul_rn(-0.5f, __fmul_rn(g, g)), e = FULL ? expf(x) : __expf(x);
    const float half = __fmul_rn(0.5f, __fmul_rn(__fmul_rn(e, t), erfc_tail(t)));     // erfc(|g| / sqrt 2) / 2
    return __fmul_rn(g, g > 0.0f ? __fsub_rn(1.0f, half) : half);
  }
  // 0.5 g (1 + tanh(t / 2)) = g sigmoid(t), t = 2 sqrt(2/pi) (g + 0.044715 g^3) = g (c + 0.044715 c g^2)
  return gate_of<FULL>(g, __fmul_rn(g, __fmaf_rn(0.07135481627260025f, __fmul_rn(g, g), 1.5957691216057308f)));
}
// act: an Act, with kFull added for an fp32 result.
__device__ __forceinline__ float apply_act(float g, int act) {
  return act >= kFull ? act_of<true>(g, act - kFull) : act_of<false>(g, act);
}

// acc s_x s_w, scaled in that order: s_x s_w alone could leave fp32's range
// where the result does not.  acc above 2^24 is rounded to fp32 (half a step,
// 2^-24), as each of the two products is.
__device__ __forceinline__ float scaled(int acc, float sx, float sw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
}

__device__ __forceinline__ void store_one(void* y, int64_t i, float v, int type) {
  if (type == kBF16)
    static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
  else if (type == kF16)
    static_cast<__half*>(y)[i] = __float2half_rn(v);
  else
    static_cast<float*>(y)[i] = v;
}

// Programmatic dependent launch: the next kernel of the stream may set itself
// up from here on; this one touches no memory of its own before the kernels
// ahead of it are complete.  (So nothing is loaded as read-only data, .nc or
// __ldg, in these kernels: what they read may be written after they start.)
__device__ __forceinline__ void pdl_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The current device (of up to 64), and its SMs.
cudaError_t current_device(int* dev);
int sm_count(int dev);

cudaError_t launch_quantize(const void* x, int type, int64_t R, int64_t K, int64_t ldx, int8_t* codes,
                            int64_t ldc, float* scales, cudaStream_t st);
// Up to kGemvTokens tokens.
constexpr int kGemvTokens = 8;
cudaError_t launch_gemv(const Linear& L, cudaStream_t st);
bool gemm_read_and_clear_timeout(cudaError_t* err);

// The kernel of one call (arguments already checked by the C ABI).
cudaError_t launch_linear(const Linear& L, cudaStream_t st);

}  // namespace i8
}  // namespace wq
