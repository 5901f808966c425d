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
// A warp takes a token.  Its lanes hold the row in registers, each lane consecutive experts of one
// group, as keys that compare as integers; the lowest bits are given to the place within the
// lane, so a lane's keys are sorted by minima and maxima alone (a Batcher network), and
// each of the k rounds takes the largest of the lanes' heads (one warp reduction).
//
// The order is that of the keys in 64 bits.  The fp32 keys decide where they lie further apart
// than their errors and the bits given away; a token with a closer pair (some 0.1% of tokens for
// logits of unit variance) is chosen again, from fp64 keys or, without a bias, from the logits as
// they are.  So the indices do not depend on how a kernel rounds.
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

constexpr int SEL_THREADS = 256;  // a warp a token
constexpr float SUM_EPS = 1e-20f;
constexpr uint32_t FULL = 0xffffffffu;

// How a launch splits a row over a warp: lpg lanes a group, c experts a lane.
struct SelArgs {
  int T, E, k, G, keep, gs, lpg, c;  // G = 1 where no group is dropped
  bool sigmoid, top2, renorm, vec;
  float scale;
};

// fp32 as an integer that compares alike (no -0, no NaN), and back
__device__ __forceinline__ uint32_t order(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) - 1u | 0x80000000u));
}
__device__ __forceinline__ float low_nan(float f) { return f != f ? -INFINITY : f; }
__device__ __forceinline__ float sigmoid32(float l) { return __fdividef(1.f, 1.f + expf(-l)); }

template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = max(a, b);
            v[i + j + k] = min(a, b);
          }
}

template <int N>
constexpr int bits_of = N <= 1 ? 0 : 1 + bits_of<N / 2>;
template <>
constexpr int bits_of<1> = 0;

// The lane's experts' logits, -inf where it has none.
template <typename T, int PL>
__device__ __forceinline__ void load_row(const T* row, int e0, int cnt, bool vec, float (&l)[PL]) {
  constexpr int BYTES = PL * static_cast<int>(sizeof(T));
  if (vec && BYTES % 4 == 0) {  // (whole lanes: cnt is PL or 0)
    uint32_t w[BYTES / 4 > 0 ? BYTES / 4 : 1];
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = 0;
    if (cnt > 0) {
      const T* p = row + e0;
      if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
          w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
      } else if constexpr (BYTES == 8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = q.x, w[1] = q.y;
      } else if constexpr (BYTES == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
    }
    const T* h = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = cnt > 0 ? to_f32(h[i]) : -INFINITY;
    return;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) l[i] = i < cnt ? to_f32(row[e0 + i]) : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// ------------------------------------------------------------- the choice in 64 bits
// (b, i) in front of (a, j)
__device__ __forceinline__ bool ahead(double a, int i, double b, int j) {
  return a > b || (a == b && i < j);
}

// The expert of round `lane` from keys in 64 bits; the arguments of the kernel's token.
template <typename T, int PL>
__device__ __noinline__ int choose64(const T* __restrict__ row, const float* __restrict__ bias,
                                     const SelArgs a, int e0, int cnt) {
  const int lane = threadIdx.x & 31;
  const auto low = [](double v) { return v != v ? -INFINITY : v; };
  double key[PL];
  const bool scores = bias != nullptr || (a.G > 1 && a.top2);
  double m = -INFINITY, z = 0.0;
  if (scores && !a.sigmoid) {
    for (int i = 0; i < cnt; ++i) m = fmax(m, static_cast<double>(to_f32(row[e0 + i])));
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(FULL, m, o));
    for (int i = 0; i < cnt; ++i) z += exp(static_cast<double>(to_f32(row[e0 + i])) - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
  }
  const auto score = [&](double l) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-l)) : m == -INFINITY ? 0.0 : exp(l - m) / z;
  };
  double t0 = -INFINITY, t1 = -INFINITY;  // the lane's two largest, as the groups count them
  for (int i = 0; i < cnt; ++i) {
    const double l = to_f32(row[e0 + i]);
    key[i] = low(bias != nullptr ? score(l) + static_cast<double>(bias[e0 + i]) : l);
    const double v = bias == nullptr && a.G > 1 && a.top2 ? low(score(l)) : key[i];
    t1 = fmax(t1, fmin(t0, v));
    t0 = fmax(t0, v);
  }
  bool kept = true;
  if (a.G > 1) {
    for (int o = 1; o < a.lpg; o <<= 1) {
      const double o0 = __shfl_xor_sync(FULL, t0, o), o1 = __shfl_xor_sync(FULL, t1, o);
      t1 = fmax(fmin(t0, o0), fmax(t1, o1));
      t0 = fmax(t0, o0);
    }
    const double g = a.top2 && a.gs > 1 ? t0 + t1 : t0;
    const int mine = lane / a.lpg;
    int rank = 0;
    for (int o = 0; o < a.G; ++o) rank += ahead(__shfl_sync(FULL, g, o * a.lpg), o, g, mine);
    kept = mine < a.G && rank < a.keep;
  }
  unsigned long long taken = 0;
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double b = -INFINITY;
    int e = 0x7fffffff;
    if (kept)
      for (int i = 0; i < cnt; ++i)
        if (!(taken >> i & 1u) && ahead(key[i], e0 + i, b, e)) b = key[i], e = e0 + i;
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(FULL, b, o);
      const int oe = __shfl_xor_sync(FULL, e, o);
      if (ahead(ob, oe, b, e)) b = ob, e = oe;
    }
    if (e >= e0 && e < e0 + cnt) taken |= 1ull << (e - e0);
    if (lane == j) mine = e;
  }
  return mine;
}

// PL: experts a lane holds (at least c); D: how many of its keys can matter (more than k, or all).
template <typename T, int PL, int D, bool BIAS>
__global__ void __launch_bounds__(SEL_THREADS) select_fwd_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const SelArgs a,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr int TAG = bits_of<PL>;
  constexpr uint32_t TAGS = (1u << TAG) - 1u;
  // the tag displaces bits that a 16-bit logit leaves empty
  constexpr bool EXACT = !BIAS && sizeof(T) == 2;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (SEL_THREADS / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;  // whole warps leave together
  const T* const row = logits + t * a.E;
  const int group = lane / a.lpg, within = lane % a.lpg;
  const int e0 = group * a.gs + within * a.c;
  const int cnt = group < a.G ? max(0, min(a.c, a.gs - within * a.c)) : 0;
  float l[PL];
  load_row<T, PL>(row, e0, cnt, a.vec, l);
  float m = -INFINITY, rz = 0.f;  // the row's largest logit and 1 / sum exp(l - m)
  if (!a.sigmoid && (BIAS || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) z += expf(l[i] - m);
    rz = m == -INFINITY ? 0.f : 1.f / warp_sum(z);
  }
  const auto score = [&](float v) {
    return a.sigmoid ? sigmoid32(v) : m == -INFINITY ? 0.f : expf(v - m) * rz;
  };
  uint32_t v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    float key = l[i];
    if constexpr (BIAS) {
      if (a.sigmoid)
        key = sigmoid32(key);
      else
        key = m == -INFINITY ? 0.f : expf(key - m) * rz;
      key += i < cnt ? __ldg(bias + e0 + i) : 0.f;
    }
    v[i] = i < cnt ? (order(low_nan(key)) & ~TAGS) | (PL - 1 - i) : 0u;
  }
  sort_desc<PL>(v);

  bool again = false;  // two keys are closer than they are known
  if (a.G > 1) {
    uint32_t t0 = v[0], t1 = PL > 1 ? v[1 < PL ? 1 : 0] : 0u;
    for (int o = 1; o < a.lpg; o <<= 1) {
      const uint32_t o0 = __shfl_xor_sync(FULL, t0, o), o1 = __shfl_xor_sync(FULL, t1, o);
      t1 = max(min(t0, o0), max(t1, o1));
      t0 = max(t0, o0);
    }
    // (what the tag's bits were is lost, and with them what made -inf no NaN)
    float s0 = low_nan(unorder(t0 & ~TAGS)), s1 = low_nan(unorder(t1 & ~TAGS));
    float lost = 1.f;  // by how much a score's relative error exceeds its key's
    if (!BIAS && a.top2) {  // scores of logits (the softmax's common factor does not matter)
      const float far = fmaxf(s0 == -INFINITY ? 0.f : fabsf(s0), s1 == -INFINITY ? 0.f : fabsf(s1));
      lost += __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(far)));
      const float big = a.sigmoid ? 0.f : warp_max(s0);
      s0 = a.sigmoid ? sigmoid32(s0) : big == -INFINITY ? 0.f : expf(s0 - big);
      s1 = a.sigmoid ? sigmoid32(s1) : big == -INFINITY ? 0.f : expf(s1 - big);
    }
    const bool two = a.top2 && a.gs > 1, real = group < a.G;
    const float gs = two ? s0 + s1 : s0;
    const uint32_t u = order(low_nan(gs));
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
      const uint32_t w = __shfl_sync(FULL, u, o * a.lpg);
      rank += w > u || (w == u && o < group);
    }
    const bool kept = real && rank < a.keep;
    const float least = unorder(__reduce_min_sync(FULL, kept ? u : FULL));
    const float best = unorder(__reduce_max_sync(FULL, real && !kept ? u : 0u));
    if (!(EXACT && !a.top2)) {
      // a sum's error: its scores', the bits given away and one rounding, of the largest there is
      float size = (s0 == -INFINITY ? 0.f : fabsf(s0)) + (two && s1 != -INFINITY ? fabsf(s1) : 0.f);
      size = __uint_as_float(__reduce_max_sync(FULL, real ? __float_as_uint(size) : 0u));
      if (BIAS) size += 2.f * (a.sigmoid ? 1.f : rz);
      again = !(least - best > size * lost * ((2 * PL + 32) * 0x1p-24f + 2.f * TAGS * 0x1p-23f));
    }
#pragma unroll
    for (int i = 0; i < D; ++i) v[i] = kept ? v[i] : 0u;
  }

  uint32_t my_v = 0, last_v = 0;
  int my_lane = 0;
  for (int j = 0; j <= a.k; ++j) {
    // (without the tags: of equal keys the first lane's, and in it the first)
    const uint32_t top = __reduce_max_sync(FULL, v[0] & ~TAGS);
    last_v = top;
    if (j == a.k) break;
    const int w = __ffs(__ballot_sync(FULL, (v[0] & ~TAGS) == top)) - 1;
    const uint32_t tagged = __shfl_sync(FULL, v[0], w);
    if (lane == j) my_v = tagged, my_lane = w;
    const bool pop = lane == w;
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) v[i] = pop ? v[i + 1] : v[i];
    v[D - 1] = pop ? 0u : v[D - 1];
  }
  int e = my_lane / a.lpg * a.gs + my_lane % a.lpg * a.c + (PL - 1 - static_cast<int>(my_v & TAGS));
  const bool mine = lane < a.k;
  e = mine ? e : 0;
  float lj = to_f32(row[e]);
  float sj = BIAS || a.sigmoid || !a.renorm ? score(lj) : 0.f;
  {
    float key = lj;
    if constexpr (BIAS) key = sj + __ldg(bias + e);
    key = low_nan(key);
    float next = __shfl_down_sync(FULL, key, 1), snext = __shfl_down_sync(FULL, sj, 1);
    const int enext = __shfl_down_sync(FULL, e, 1);
    bool bad = false;
    if constexpr (BIAS) {
      const float per = ((a.sigmoid ? 16 : PL + 16) * 0x1p-24f);
      if (lane == a.k - 1) {  // against everything left: no larger than this
        next = last_v == 0u ? -INFINITY : unorder(last_v | TAGS);
        snext = a.sigmoid ? 1.f : rz;
      }
      const float tol = per * (sj + snext) + 0x1p-22f * (fabsf(key) + fabsf(next));
      bad = !(key - next > tol) && !(lane == a.k - 1 && last_v == 0u);
    } else {
      if (lane < a.k - 1)
        bad = !(key > next || (key == next && e < enext));
      else
        bad = !EXACT && last_v != 0u && last_v == (my_v & ~TAGS);
    }
    again = again || __any_sync(FULL, mine && bad);
  }
  if (again) {
    e = choose64<T, PL>(row, BIAS ? bias : nullptr, a, e0, cnt);
    e = mine ? e : 0;
    lj = to_f32(row[e]);
    if (BIAS || a.sigmoid || !a.renorm) sj = score(lj);
  }
  float w;
  if (!a.renorm) {
    w = sj * a.scale;
  } else if (a.sigmoid) {
    w = a.scale * (sj / (warp_sum(mine ? sj : 0.f) + SUM_EPS));
  } else {  // the softmax over the chosen
    const float big = warp_max(mine ? lj : -INFINITY);
    const float ex = mine && big != -INFINITY ? expf(lj - big) : 0.f;
    const float sum = warp_sum(ex);
    w = sum == 0.f ? 0.f : a.scale * (ex / sum);
  }
  if (mine) {
    topk_idx[t * a.k + lane] = e;
    topk_w[t * a.k + lane] = w;
  }
}

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

// The logit gradient's row: `rest` at every expert (0, or the dense softmax's -s_e A) and the chosen
// experts' own values over it, the auxiliary gradient added to both.  U: elements of 16 bytes of the
// gradient (1: rows on no 16-byte boundary).
template <typename T, typename O, int U, bool DENSE>
__global__ void __launch_bounds__(SEL_THREADS) select_bwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ dtopk_w, const float* __restrict__ aux, const SelArgs a,
    O* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (SEL_THREADS / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const T* const row = logits + t * a.E;
  O* const out = dlogits + t * a.E;
  const float* const ax = aux != nullptr ? aux + t * a.E : nullptr;
  const int e = lane < a.k ? __ldg(topk_idx + t * a.k + lane) : -1;
  const float g = lane < a.k ? __ldg(dtopk_w + t * a.k + lane) : 0.f;
  const bool mine = e >= 0 && e < a.E;  // (an index outside is dropped)
  const float l = mine ? to_f32(row[e]) : -INFINITY;
  float d;  // of the lane's chosen logit
  [[maybe_unused]] float m = -INFINITY, rz = 0.f, A = 0.f;
  if constexpr (DENSE) {
    for (int i = lane * U; i < a.E; i += 32 * U) {
      float f[U];
      load_u<U>(row + i, f);
#pragma unroll
      for (int j = 0; j < U; ++j) m = fmaxf(m, f[j]);
    }
    m = warp_max(m);
    float z = 0.f;
    for (int i = lane * U; i < a.E; i += 32 * U) {
      float f[U];
      load_u<U>(row + i, f);
#pragma unroll
      for (int j = 0; j < U; ++j) z += expf(f[j] - m);
    }
    rz = m == -INFINITY ? 0.f : 1.f / warp_sum(z);
    const float s = mine && m != -INFINITY ? expf(l - m) * rz : 0.f;
    A = warp_sum(mine ? g * s : 0.f);
    d = s * g;  // (beside -s A, which every expert has)
  } else if (a.sigmoid) {
    const float s = mine ? sigmoid32(l) : 0.f;
    float ds = g;
    if (a.renorm) {
      const float n = warp_sum(s) + SUM_EPS;
      ds = (g - warp_sum(mine ? g * s : 0.f) / n) / n;
    }
    d = mine ? a.scale * ds * s * sigmoid32(-l) : 0.f;
  } else {
    const float big = warp_max(l);
    const float ex = mine && big != -INFINITY ? expf(l - big) : 0.f;
    const float sum = warp_sum(ex);
    const float q = sum == 0.f ? 0.f : ex / sum;
    d = a.scale * q * (g - warp_sum(mine ? g * q : 0.f));
  }
  for (int i = lane * U; i < a.E; i += 32 * U) {
    float f[U] = {}, x[U] = {};
    if constexpr (DENSE) load_u<U>(row + i, f);
    if (ax != nullptr) load_u<U>(ax + i, x);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if constexpr (DENSE) f[j] = m == -INFINITY ? 0.f : -a.scale * A * (expf(f[j] - m) * rz);
      f[j] += x[j];
    }
    if constexpr (U == 1)
      out[i] = from_f32<O>(f[0]);
    else
      *reinterpret_cast<uint4*>(out + i) = pack(f, out);
  }
  // the chosen experts' values, an expert that is there twice by its first lane
  const uint32_t same = __match_any_sync(FULL, mine ? e : -1 - lane);
  float sum = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const float v = __shfl_sync(FULL, d, j);
    if (same >> j & 1u) sum += v;
  }
  __syncwarp();
  if (mine && __ffs(same) - 1 == lane) {
    float f = sum;
    if constexpr (DENSE) {
      const float s = m == -INFINITY ? 0.f : expf(l - m) * rz;
      f = a.scale * (sum - s * A);
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

static SelArgs make_args(const mm_moe_select* s) {
  SelArgs a{};
  a.T = static_cast<int>(s->T);
  a.E = static_cast<int>(s->E);
  a.k = static_cast<int>(s->k);
  a.G = s->topk_groups < s->groups ? s->groups : 1;
  a.keep = s->topk_groups;
  a.gs = a.E / a.G;
  int p = 1;
  while (p < a.G) p *= 2;
  a.lpg = 32 / p;
  a.c = (a.gs + a.lpg - 1) / a.lpg;
  a.sigmoid = s->score == MM_MOE_SCORE_SIGMOID;
  a.top2 = s->group_score == MM_MOE_GROUP_TOP2;
  a.renorm = s->renormalise != 0;
  a.scale = s->scale;
  return a;
}

static unsigned blocks_of(int T) {
  return static_cast<unsigned>((static_cast<int64_t>(T) + SEL_THREADS / 32 - 1) /
                               (SEL_THREADS / 32));
}

template <typename T, int PL>
static cudaError_t launch_fwd(const Ctx& c, SelArgs a, const T* logits, const float* bias,
                              int32_t* idx, float* w) {
  constexpr int BYTES = PL * static_cast<int>(sizeof(T)), V = BYTES < 16 ? BYTES : 16;
  a.vec = a.c == PL && a.gs % PL == 0 && BYTES >= 4 && al(logits, V) &&
          a.E * sizeof(T) % V == 0;
  constexpr int D = PL < 9 ? PL : 9;  // (k up to 8)
  auto* kern = a.k < D || D == PL ? (bias != nullptr ? select_fwd_kernel<T, PL, D, true>
                                                     : select_fwd_kernel<T, PL, D, false>)
                                  : (bias != nullptr ? select_fwd_kernel<T, PL, PL, true>
                                                     : select_fwd_kernel<T, PL, PL, false>);
  return launch_k(c.stream, kern, dim3(blocks_of(a.T)), dim3(SEL_THREADS), 0, logits, bias, a, idx,
                  w);
}

cudaError_t launch_select_fwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const float* bias, int32_t* idx, float* w) {
  const SelArgs a = make_args(s);
  prof_begin(c, K_SELECT_FWD);
  const cudaError_t e = with_dtype(s->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const T* l = static_cast<const T*>(logits);
    if (a.c <= 1) return launch_fwd<T, 1>(c, a, l, bias, idx, w);
    if (a.c <= 2) return launch_fwd<T, 2>(c, a, l, bias, idx, w);
    if (a.c <= 4) return launch_fwd<T, 4>(c, a, l, bias, idx, w);
    if (a.c <= 8) return launch_fwd<T, 8>(c, a, l, bias, idx, w);
    if (a.c <= 16) return launch_fwd<T, 16>(c, a, l, bias, idx, w);
    if (a.c <= 32) return launch_fwd<T, 32>(c, a, l, bias, idx, w);
    return launch_fwd<T, 64>(c, a, l, bias, idx, w);
  });
  prof_end(c, K_SELECT_FWD);
  return e;
}

template <typename T, typename O>
static cudaError_t launch_bwd(const Ctx& c, const SelArgs& a, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out) {
  constexpr int U = VN<O>;
  const bool dense = !a.sigmoid && !a.renorm;
  const bool vec = a.E % U == 0 && a.E * sizeof(T) % 16 == 0 && al(logits, 16) && al(out, 16) &&
                   (aux == nullptr || al(aux, 16));
  auto* kern = vec ? (dense ? select_bwd_kernel<T, O, U, true> : select_bwd_kernel<T, O, U, false>)
                   : (dense ? select_bwd_kernel<T, O, 1, true> : select_bwd_kernel<T, O, 1, false>);
  return launch_k(c.stream, kern, dim3(blocks_of(a.T)), dim3(SEL_THREADS), 0,
                  static_cast<const T*>(logits), idx, dw, aux, a, static_cast<O*>(out));
}

cudaError_t launch_select_bwd(const Ctx& c, const mm_moe_select* s, const void* logits,
                              const int32_t* idx, const float* dw, const float* aux, void* out) {
  const SelArgs a = make_args(s);
  prof_begin(c, K_SELECT_BWD);
  const cudaError_t e = with_dtype(s->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    if (s->grad_dtype == s->dtype) return launch_bwd<T, T>(c, a, logits, idx, dw, aux, out);
    return launch_bwd<T, __nv_bfloat16>(c, a, logits, idx, dw, aux, out);
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

// whether [a, a + an) and [b, b + bn) share a byte
static bool meet(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_select_backward(
    const mm_moe_select* select, const void* logits, const int32_t* topk_idx,
    const float* dtopk_w, const float* dlogits_aux, void* dlogits, void* stream) {
  if (!select_ok(select) || !al(logits, dtype_bytes(select->dtype)) || !al(topk_idx, 4) ||
      !al(dtopk_w, 4) || (dlogits_aux != nullptr && !al(dlogits_aux, 4)) ||
      !al(dlogits, dtype_bytes(select->grad_dtype)))
    return MM_MOE_EINVAL;
  const size_t n = static_cast<size_t>(select->T * select->E);
  const size_t out = n * dtype_bytes(select->grad_dtype);
  if (meet(dlogits, out, logits, n * dtype_bytes(select->dtype)) ||
      (dlogits_aux != nullptr && meet(dlogits, out, dlogits_aux, n * 4)))
    return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  return op_status(
      launch_select_bwd(c, select, logits, topk_idx, dtopk_w, dlogits_aux, dlogits));
}
