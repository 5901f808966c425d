// select.cuh -- the choice of experts: what its forward (select_fwd.cuh), its backward (select.cu) and
// the router (router.cu) share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace mmmoe {

constexpr float SUM_EPS = 1e-20f;
constexpr uint32_t FULL = 0xffffffffu;

// How a launch splits a row over its W lanes: lpg lanes a group, c experts a lane.  bounded: k or more
// distinct keys take part among the lanes' two (W = 8) or the largest of each `set` of lanes (a power of
// two within a group).
struct SelArgs {
  int T, E, k, G, keep, gs, lpg, c, set;  // G = 1 where no group is dropped
  bool bounded;
  bool sigmoid, top2, renorm, vec;
  float scale;
};

// The sigmoid within 10 2^-24 of itself for l >= -87; below it falls to 0 (the division's result is 0 for
// divisors above 2^126).
__device__ __forceinline__ float sigmoid32(float l) { return __fdividef(1.f, 1.f + expf(-l)); }

// The largest of a row's logits (a NaN is passed over), in whose place e^(l - m) is finite.  Where all are
// -inf it is 0: their sum is then 0, for scores of 0, and a NaN among them makes it NaN.
template <typename F>
__device__ __forceinline__ F finite_max(F m) {
  return m == -INFINITY ? F(0) : m;
}

// Reductions over W lanes.
template <int W>
__device__ __forceinline__ float max_of(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
template <int W>
__device__ __forceinline__ float min_of(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
template <int W, typename V>
__device__ __forceinline__ V sum_of(V v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

bool select_ok(const mm_moe_select* s);
// Whether the backward's gradient lies apart from the logits and the auxiliary gradient, of which other
// CTAs still read rows when it is written.
bool select_bwd_apart(const mm_moe_select* s, const void* logits, const float* aux,
                      const void* dlogits);
cudaError_t launch_select_fwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const float* bias, int32_t* idx, float* w);
cudaError_t launch_select_bwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out);
// of one type of logits, each in a translation unit of its own (they compile side by side)
cudaError_t launch_select_fwd_f32(const Ctx& c, const SelArgs& a, const void* logits,
                                  const float* bias, int32_t* idx, float* w);
cudaError_t launch_select_fwd_bf16(const Ctx& c, const SelArgs& a, const void* logits,
                                   const float* bias, int32_t* idx, float* w);
cudaError_t launch_select_fwd_f16(const Ctx& c, const SelArgs& a, const void* logits,
                                  const float* bias, int32_t* idx, float* w);

}  // namespace mmmoe
