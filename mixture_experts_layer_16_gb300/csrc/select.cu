// select.cu -- the choice of experts from a router's logits, and its backward.
//
//   s = softmax(l) over all experts, or sigmoid(l) each;   key = s + bias  (l itself without a bias,
//   which orders alike);  of G groups of consecutive experts the best `topk_groups` by their largest
//   key or by the sum of their two largest;  of these the k largest keys, descending, equal ones (of
//   experts and of groups) by the lower index;  w_j = scale s_j, renormalised: scale s_j / (sum_i s_i
//   + 1e-20) for the sigmoid, scale softmax over the chosen logits for the softmax.
//   Backward with g = dw (the choice held fixed), A = sum_j g_j q_j:
//     sigmoid  ds_j = scale g_j, renormalised scale (g_j - A) / N with q = s / N, N = sum s + 1e-20;
//              dl_j = ds_j s_j (1 - s_j)
//     softmax  renormalised: dl_j = scale q_j (g_j - A), q the softmax over the chosen; else, with
//              A = sum_j g_j s_j, dl_e = scale s_e (g_e - A), g_e = 0 beside the chosen: dense
//
// The forward's kernel is in select_fwd.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ops.cuh"
#include "select.cuh"

namespace mmmoe {

constexpr int SEL_THREADS = 256;  // of the backward's CTAs (8 to 32 lanes a token)

// ----------------------------------------------------------------------- backward
// U consecutive elements: 16-byte accesses for U > 1
template <int U, typename T>
__device__ __forceinline__ void load_u(const T* p, float (&f)[U]) {
  if constexpr (U == 1) {
    f[0] = to_f32(__ldg(p));
  } else {
#pragma unroll
    for (int i = 0; i < U; i += VN<T>) {
      float t[VN<T>];
      unpack(__ldg(reinterpret_cast<const uint4*>(p + i)), t, p);
#pragma unroll
      for (int j = 0; j < VN<T>; ++j) f[i + j] = t[j];
    }
  }
}

// W lanes take a token (k of them its chosen experts), in units of U elements, 32 elements a lane at
// most.  The logit gradient's row is first filled: with zeros or the auxiliary gradient, or with the
// dense softmax's -scale s_e A beside it (the row then stays in registers between its three uses);
// the chosen experts' own values go over it.  U: elements of 16 bytes of the gradient (1: rows on no
// 16-byte boundary).
template <typename T, typename O, int U, int W, bool DENSE>
__global__ void __launch_bounds__(SEL_THREADS) select_bwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ dtopk_w, const float* __restrict__ aux, const SelArgs a,
    O* __restrict__ dlogits) {
  constexpr int NU = 32 / U;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (W - 1), sub = (threadIdx.x & 31) / W;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (SEL_THREADS / W) + threadIdx.x / W;
  const bool live = t < a.T;  // (a warp's tokens go through it together)
  const int64_t first = live ? t * a.E : 0;
  const T* const row = logits + first;
  O* const out = dlogits + first;
  const float* const ax = aux != nullptr ? aux + first : nullptr;
  const bool slot = live && lane < a.k;
  const int e = slot ? __ldg(topk_idx + t * a.k + lane) : -1;
  const float g = slot ? __ldg(dtopk_w + t * a.k + lane) : 0.f;
  const auto put = [&](int i, const float (&f)[U]) {
    if constexpr (U == 1)
      out[i] = from_f32<O>(f[0]);
    else
      *reinterpret_cast<uint4*>(out + i) = pack(f, out);
  };
  if constexpr (!DENSE) {
    if (live)
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int i = (u * W + lane) * U;
        if (i >= a.E) break;
        float f[U] = {};
        if (ax != nullptr) load_u<U>(ax + i, f);
        put(i, f);
      }
  }
  const bool mine = e >= 0 && e < a.E;  // (an index outside is dropped)
  const float l = mine ? to_f32(__ldg(row + e)) : -INFINITY;
  float d;  // of the lane's chosen logit
  [[maybe_unused]] float m = -INFINITY, rz = 0.f, A = 0.f;
  if constexpr (DENSE) {
    float v[NU][U];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = (u * W + lane) * U;
      if (i < a.E) {
        load_u<U>(row + i, v[u]);
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) v[u][j] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) m = fmaxf(m, v[u][j]);
    }
    m = finite_max(max_of<W>(m));
    float z = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int j = 0; j < U; ++j) {
        v[u][j] = expf(v[u][j] - m);
        z += v[u][j];
      }
    z = sum_of<W>(z);
    rz = z == 0.f ? 0.f : 1.f / z;
    const float s = mine ? expf(l - m) * rz : 0.f;
    A = sum_of<W>(mine ? g * s : 0.f);
    d = s * g;  // (beside -s A, which every expert has)
    const float c = -a.scale * A * rz;
    if (live)
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int i = (u * W + lane) * U;
        if (i >= a.E) break;
        float f[U] = {};
        if (ax != nullptr) load_u<U>(ax + i, f);
#pragma unroll
        for (int j = 0; j < U; ++j) f[j] = fmaf(c, v[u][j], f[j]);
        put(i, f);
      }
  } else if (a.sigmoid) {
    const float s = mine ? sigmoid32(l) : 0.f;
    float ds = g;
    if (a.renorm) {
      const float n = sum_of<W>(s) + SUM_EPS, q = s / n;  // (of one expert alone 1: no gradient)
      ds = (g - sum_of<W>(mine ? g * q : 0.f)) / n;
    }
    d = mine ? a.scale * ds * s * sigmoid32(-l) : 0.f;
  } else {
    const float big = max_of<W>(l);
    const float ex = mine && !(l == -INFINITY) ? expf(l - big) : 0.f;  // (of a NaN a NaN)
    const float sum = sum_of<W>(ex);
    const float q = sum == 0.f ? 0.f : ex / sum;
    d = a.scale * q * (g - sum_of<W>(mine ? g * q : 0.f));
  }
  // the chosen experts' values, an expert that is there twice by its first lane
  const int none = -1 - static_cast<int>(threadIdx.x & 31);
  const uint32_t same = __match_any_sync(FULL, mine ? sub << 16 | e : none);
  float sum = d;
  if (__any_sync(FULL, mine && (same & (same - 1)) != 0)) {
    sum = 0.f;
    for (int j = 0; j < W; ++j) {
      const float v = __shfl_sync(FULL, d, sub * W + j);
      if (same >> (sub * W + j) & 1u) sum += v;
    }
  }
  __syncwarp();
  if (mine && __ffs(same) - 1 == sub * W + lane) {
    float f = sum;
    if constexpr (DENSE) {
      f = a.scale * (sum - expf(l - m) * rz * A);
    }
    if (ax != nullptr) f += __ldg(ax + e);
    out[e] = from_f32<O>(f);
  }
}

// ------------------------------------------------------------------------ host side
static bool al(const void* p, uintptr_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

bool select_ok(const mm_moe_select* s) {
  if (s == nullptr || s->T < 1 || s->T >= (int64_t{1} << 31) || s->E < 1 || s->E > 1024 ||
      s->k < 1 || s->k > 32 || !dtype_ok(s->dtype) || !dtype_ok(s->grad_dtype) ||
      (s->grad_dtype != s->dtype && s->grad_dtype != MM_MOE_DT_BF16) ||
      s->score < MM_MOE_SCORE_SOFTMAX || s->score > MM_MOE_SCORE_SIGMOID ||
      s->group_score < MM_MOE_GROUP_MAX || s->group_score > MM_MOE_GROUP_TOP2 ||
      s->renormalise < 0 || s->renormalise > 1 || !std::isfinite(s->scale))
    return false;
  if (s->groups < 1 || s->groups > 32 || s->E % s->groups != 0 || s->topk_groups < 1 ||
      s->topk_groups > s->groups)
    return false;
  return s->k <= s->E / s->groups * s->topk_groups;
}

bool select_bwd_apart(const mm_moe_select* s, const void* logits, const float* aux,
                      const void* dlogits) {
  const size_t n = static_cast<size_t>(s->T * s->E);
  const uintptr_t out = reinterpret_cast<uintptr_t>(dlogits);
  const uintptr_t end = out + n * dtype_bytes(s->grad_dtype);
  const auto apart = [&](const void* p, size_t bytes) {
    const uintptr_t in = reinterpret_cast<uintptr_t>(p);
    return p == nullptr || out >= in + bytes || in >= end;
  };
  return apart(logits, n * dtype_bytes(s->dtype)) && apart(aux, n * 4);
}

static SelArgs make_args(const mm_moe_select* s) {
  SelArgs a{};
  a.T = static_cast<int>(s->T);
  a.E = static_cast<int>(s->E);
  a.k = static_cast<int>(s->k);
  a.G = s->topk_groups < s->groups ? s->groups : 1;
  a.keep = a.G > 1 ? s->topk_groups : 1;
  a.gs = a.E / a.G;
  a.sigmoid = s->score == MM_MOE_SCORE_SIGMOID;
  a.top2 = s->group_score == MM_MOE_GROUP_TOP2;
  a.renorm = s->renormalise != 0;
  a.scale = s->scale;
  return a;
}

cudaError_t launch_select_fwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const float* bias, int32_t* idx, float* w) {
  const SelArgs a = make_args(s);
  prof_begin(c, K_SELECT_FWD);
  const cudaError_t e = s->dtype == MM_MOE_DT_F32 ? launch_select_fwd_f32(c, a, logits, bias, idx, w)
                        : s->dtype == MM_MOE_DT_F16
                            ? launch_select_fwd_f16(c, a, logits, bias, idx, w)
                            : launch_select_fwd_bf16(c, a, logits, bias, idx, w);
  prof_end(c, K_SELECT_FWD);
  return e;
}

template <typename T, typename O, int U, int W>
static cudaError_t launch_bwd(const Ctx& c, const SelArgs& a, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out) {
  constexpr int TOKENS = SEL_THREADS / W;
  auto* kern = !a.sigmoid && !a.renorm ? select_bwd_kernel<T, O, U, W, true>
                                       : select_bwd_kernel<T, O, U, W, false>;
  return launch_k(c.stream, kern,
                  dim3(static_cast<unsigned>((static_cast<int64_t>(a.T) + TOKENS - 1) / TOKENS)),
                  dim3(SEL_THREADS), 0, static_cast<const T*>(logits), idx, dw, aux, a,
                  static_cast<O*>(out));
}

// As few lanes a token as its chosen experts and its row leave.
template <typename T, typename O>
static cudaError_t launch_bwd_of(const Ctx& c, const SelArgs& a, const void* logits,
                                 const int32_t* idx, const float* dw, const float* aux, void* out) {
  constexpr int U = VN<O>;
  const bool vec = a.E % U == 0 && a.E * sizeof(T) % 16 == 0 && al(logits, 16) && al(out, 16) &&
                   (aux == nullptr || al(aux, 16));
  if (!vec) return launch_bwd<T, O, 1, 32>(c, a, logits, idx, dw, aux, out);
  const int lanes = std::max(a.k, (a.E + 31) / 32);
  if (lanes <= 8) return launch_bwd<T, O, U, 8>(c, a, logits, idx, dw, aux, out);
  if (lanes <= 16) return launch_bwd<T, O, U, 16>(c, a, logits, idx, dw, aux, out);
  return launch_bwd<T, O, U, 32>(c, a, logits, idx, dw, aux, out);
}

cudaError_t launch_select_bwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out) {
  const SelArgs a = make_args(s);
  prof_begin(c, K_SELECT_BWD);
  const cudaError_t e = with_dtype(s->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    if (s->grad_dtype == s->dtype) return launch_bwd_of<T, T>(c, a, logits, idx, dw, aux, out);
    return launch_bwd_of<T, __nv_bfloat16>(c, a, logits, idx, dw, aux, out);
  });
  prof_end(c, K_SELECT_BWD);
  return e;
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_select_forward(const mm_moe_select* select,
                                                          const void* logits, const float* bias,
                                                          int32_t* topk_idx, float* topk_w,
                                                          void* stream) {
  if (!select_ok(select) || !al(logits, dtype_bytes(select->dtype)) ||
      (bias != nullptr && !al(bias, 4)) || !al(topk_idx, 4) || !al(topk_w, 4))
    return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  return op_status(launch_select_fwd(c, select, logits, bias, topk_idx, topk_w));
}

extern "C" MM_MOE_API mm_moe_status mm_moe_select_backward(
    const mm_moe_select* select, const void* logits, const int32_t* topk_idx,
    const float* dtopk_w, const float* dlogits_aux, void* dlogits, void* stream) {
  if (!select_ok(select) || !al(logits, dtype_bytes(select->dtype)) || !al(topk_idx, 4) ||
      !al(dtopk_w, 4) || (dlogits_aux != nullptr && !al(dlogits_aux, 4)) ||
      !al(dlogits, dtype_bytes(select->grad_dtype)))
    return MM_MOE_EINVAL;
  if (!select_bwd_apart(select, logits, dlogits_aux, dlogits)) return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  return op_status(
      launch_select_bwd(c, select, logits, topk_idx, dtopk_w, dlogits_aux, dlogits));
}
