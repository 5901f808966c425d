// select.cuh -- the choice of experts (select.cu) as the router (router.cu) launches it.
#pragma once
#include <cstdint>

#include "internal.h"

namespace mmmoe {

bool select_ok(const mm_moe_select* s);
cudaError_t launch_select_fwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const float* bias, int32_t* idx, float* w);
cudaError_t launch_select_bwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out);

}  // namespace mmmoe
