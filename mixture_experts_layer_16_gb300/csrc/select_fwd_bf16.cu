// select_fwd_bf16.cu -- the choice of experts from bf16 logits.
#include "select_fwd.cuh"

namespace mmmoe {

cudaError_t launch_select_fwd_bf16(const Ctx& c, const SelArgs& a, const void* logits,
                                 const float* bias, int32_t* idx, float* w) {
  return launch_select_fwd_of(c, a, static_cast<const __nv_bfloat16*>(logits), bias, idx, w);
}

}  // namespace mmmoe
