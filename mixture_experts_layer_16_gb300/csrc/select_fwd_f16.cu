// select_fwd_f16.cu -- the choice of experts from fp16 logits.
#include "select_fwd.cuh"

namespace mmmoe {

cudaError_t launch_select_fwd_f16(const Ctx& c, const SelArgs& a, const void* logits,
                                 const float* bias, int32_t* idx, float* w) {
  return launch_select_fwd_of(c, a, static_cast<const __half*>(logits), bias, idx, w);
}

}  // namespace mmmoe
