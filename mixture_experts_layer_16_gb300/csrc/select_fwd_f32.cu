// select_fwd_f32.cu -- the choice of experts from fp32 logits.
#include "select_fwd.cuh"

namespace mmmoe {

cudaError_t launch_select_fwd_f32(const Ctx& c, const SelArgs& a, const void* logits,
                                 const float* bias, int32_t* idx, float* w) {
  return launch_select_fwd_of(c, a, static_cast<const float*>(logits), bias, idx, w);
}

}  // namespace mmmoe
