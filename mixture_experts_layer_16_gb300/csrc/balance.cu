// balance.cu -- the router's auxiliary losses and per-expert counts, with the gradient
// of the logits.
//
// The tokens are split into G sequences (ragged, in order; by default one).  A token
// counts when its mask is set and its logits are not all -inf.  With p = softmax(logits),
// lse = log sum exp(logits), n_s the counting tokens of sequence s, S the sequences with
// n_s > 0 and N = sum n_s:
//   counts[s, e] = the (token, slot) pairs of s routed to e (an index outside [0, E) is
//                  dropped)
//   f[s, e] = E / (k n_s) counts[s, e],      P[s, e] = 1 / n_s sum_t p[t, e]
//   seq_loss[s] = sum_e f[s, e] P[s, e],     balance = 1 / S sum_s seq_loss[s]
//   z = 1 / N sum_t lse_t^2
// The counts are constants of the gradient:
//   dlogits[t, e] = p_e (c_e - sum_j p_j c_j) + dz 2 lse_t / N p_e,
//   c_e = dbalance E / (k n_s^2 S) counts[s, e]
//
// Both passes read the logits once: a token's row sits in the registers of 8 to 32 lanes
// (few lanes, several values each, so that a reduction over the experts takes few
// shuffles), and the sums over tokens stay in registers until a sequence or the CTA's
// range of tokens ends.  No floating-point atomics: every sum has a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dtype.cuh"
#include "internal.h"

namespace mmmoe {

constexpr int BAL_THREADS = 256;
constexpr int BAL_WARPS = BAL_THREADS / 32;

// Four consecutive logits; past E they read as -inf.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int e0, int E, bool vec, float (&v)[4]) {
  if (vec) {
    if (e0 < E) {
      if constexpr (sizeof(T) == 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(row + e0));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
      } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + e0));
        const T* h = reinterpret_cast<const T*>(&q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f32(h[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* row, int e0, int E, bool vec, const float (&v)[4]) {
  if (vec) {
    if (e0 >= E) return;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(row + e0) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 q;
      T* h = reinterpret_cast<T*>(&q);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint2*>(row + e0) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E) row[e0 + i] = from_f32<T>(v[i]);
  }
}

// The larger of two values; NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Walks a CTA's range [t0, t1) of tokens sequence by sequence.  Offsets may hold empty
// sequences and may leave tokens before the first or after the last one in none.
struct SeqWalk {
  const int32_t* off;  // [G + 1], or null: one sequence of all tokens
  int G;
  int s;               // sequence of the current piece, or -1: in none
  int64_t a, b;        // the current piece [a, b)
  int64_t t1;
  __device__ __forceinline__ int64_t at(int g) const { return __ldg(off + g); }
  __device__ __forceinline__ void start(const int32_t* off_, int G_, int64_t t0, int64_t t1_) {
    off = off_;
    G = G_;
    t1 = t1_;
    b = t0;
    s = 0;
    if (off == nullptr) return;
    int lo = 0, hi = G;  // the first sequence that ends past t0
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid + 1) > t0)
        hi = mid;
      else
        lo = mid + 1;
    }
    next_seq = lo;
  }
  int next_seq;
  // false when the range is done
  __device__ __forceinline__ bool next() {
    a = b;
    if (a >= t1) return false;
    if (off == nullptr) {
      b = t1;
      return true;
    }
    for (; next_seq < G; ++next_seq) {
      const int64_t lo = at(next_seq), hi = min(at(next_seq + 1), t1);
      if (hi <= a) continue;
      if (lo > a) {  // a gap in front of it
        b = min(lo, t1);
        s = -1;
        return true;
      }
      b = hi;
      s = next_seq;
      return true;
    }
    b = t1;
    s = -1;
    return true;
  }
};

// Partial results of one (CTA, sequence) piece, at row CTA + sequence of each array
// (unique: the next piece has a larger CTA or a larger sequence).
struct BalParts {
  float* stats;   // [2]: sequences with a counting token, counting tokens
  float* p;       // [pieces, E]
  int32_t* cnt;   // [pieces, E]
  int32_t* n;     // [pieces]
  float* z;       // [pieces]
  float* seq_z;   // [G]
};

template <typename T, int L, int NV>
__global__ void __launch_bounds__(BAL_THREADS) balance_fwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, int64_t T_, int E, int k,
    int G, int chunk, bool vec, float* __restrict__ lse_out, BalParts parts) {
  extern __shared__ char smem[];
  float* s_p = reinterpret_cast<float*>(smem);              // [BAL_WARPS][E]
  int* s_cnt = reinterpret_cast<int*>(s_p + BAL_WARPS * E);  // [E]
  __shared__ float s_z[BAL_WARPS];
  __shared__ int s_n[BAL_WARPS];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int l = lane % L;                    // lane within its token's group
  constexpr int GROUPS = BAL_THREADS / L;
  const int grp = tid / L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = min(T_, t0 + chunk);
  for (int e = tid; e < E; e += BAL_THREADS) s_cnt[e] = 0;
  __syncthreads();
  SeqWalk w;
  w.start(off, G, t0, t1);
  while (w.next()) {
    if (w.s < 0) {  // tokens in no sequence
      for (int64_t t = w.a + tid; t < w.b; t += BAL_THREADS) lse_out[t] = 0.f;
      continue;
    }
    float acc[NV * 4];
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) acc[i] = 0.f;
    float z = 0.f;
    int n = 0;
    for (int64_t base = w.a; base < w.b; base += GROUPS) {
      const int64_t t = base + grp;
      bool on = t < w.b;
      if (on && mask != nullptr) on = __ldg(mask + t) != 0;
      float v[NV][4];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (on) {
          load4(logits + t * E, 4 * (l + i * L), E, vec, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = -INFINITY;
        }
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max_nan(m, v[i][j]);
      m = lanes_max<L>(m);
      on = on && m != -INFINITY;  // (a NaN counts, and shows in the losses)
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] = on ? expf(v[i][j] - m) : 0.f;
          sum += v[i][j];
        }
      sum = lanes_sum<L>(sum);
      if (on) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[4 * i + j] = fmaf(v[i][j], inv, acc[4 * i + j]);
        for (int j = l; j < k; j += L) {
          const int e = __ldg(topk_idx + t * k + j);
          if (e >= 0 && e < E) atomicAdd(s_cnt + e, 1);
        }
      }
      if (l == 0 && t < w.b) {
        const float lse = on ? m + logf(sum) : 0.f;
        lse_out[t] = lse;
        z = fmaf(lse, lse, z);
        n += on ? 1 : 0;
      }
    }
    // join the groups of the warp, then the warps (in order)
#pragma unroll
    for (int i = 0; i < NV * 4; ++i)
#pragma unroll
      for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    z = warp_sum(z);
    n = warp_sum(n);
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * (l + i * L) + j;
          if (e < E) s_p[wid * E + e] = acc[4 * i + j];
        }
    }
    if (lane == 0) {
      s_z[wid] = z;
      s_n[wid] = n;
    }
    __syncthreads();
    const int64_t piece = static_cast<int64_t>(blockIdx.x) + w.s;
    for (int e = tid; e < E; e += BAL_THREADS) {
      float t = s_p[e];
#pragma unroll
      for (int i = 1; i < BAL_WARPS; ++i) t += s_p[i * E + e];
      parts.p[piece * E + e] = t;
      parts.cnt[piece * E + e] = s_cnt[e];
      s_cnt[e] = 0;
    }
    if (tid == 0) {
      float tz = 0.f;
      int tn = 0;
      for (int i = 0; i < BAL_WARPS; ++i) {
        tz += s_z[i];
        tn += s_n[i];
      }
      parts.z[piece] = tz;
      parts.n[piece] = tn;
    }
    __syncthreads();
  }
}

// One CTA per sequence: its pieces joined in order.
__global__ void __launch_bounds__(256) balance_seq_kernel(const int32_t* __restrict__ off,
                                                          int64_t T_, int E, int k, int chunk,
                                                          BalParts parts,
                                                          float* __restrict__ seq_loss,
                                                          int32_t* __restrict__ counts,
                                                          int32_t* __restrict__ tokens) {
  __shared__ float s[8];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x;
  const int64_t a = off != nullptr ? max(0, __ldg(off + g)) : 0;
  const int64_t b = off != nullptr ? min(T_, static_cast<int64_t>(__ldg(off + g + 1))) : T_;
  const int64_t c0 = a / chunk, c1 = b > a ? (b - 1) / chunk + 1 : c0;
  float dot = 0.f;
  for (int e = threadIdx.x; e < E; e += 256) {
    float p = 0.f;
    int cnt = 0;
    for (int64_t c = c0; c < c1; ++c) {
      p += parts.p[(c + g) * E + e];
      cnt += parts.cnt[(c + g) * E + e];
    }
    counts[static_cast<int64_t>(g) * E + e] = cnt;
    dot = fmaf(static_cast<float>(cnt), p, dot);
  }
  dot = block_sum(dot, s);
  float z = 0.f, n = 0.f;
  int ni = 0;
  for (int64_t c = c0 + threadIdx.x; c < c1; c += 256) {
    z += parts.z[c + g];
    ni += parts.n[c + g];
  }
  z = block_sum(z, s);
  ni = block_sum(ni, reinterpret_cast<int*>(s));
  n = static_cast<float>(ni);
  if (threadIdx.x == 0) {
    tokens[g] = ni;
    seq_loss[g] = ni > 0 ? dot * (static_cast<float>(E) / static_cast<float>(k)) / (n * n) : 0.f;
    parts.seq_z[g] = z;
  }
}

__global__ void __launch_bounds__(256) balance_total_kernel(int G, BalParts parts,
                                                            const float* __restrict__ seq_loss,
                                                            const int32_t* __restrict__ tokens,
                                                            float* __restrict__ losses) {
  __shared__ float s[8];
  pdl_wait();
  pdl_trigger();
  float a = 0.f, z = 0.f;
  int n = 0, live = 0;
  for (int g = threadIdx.x; g < G; g += 256) {
    a += seq_loss[g];
    z += parts.seq_z[g];
    n += tokens[g];
    live += tokens[g] > 0 ? 1 : 0;
  }
  a = block_sum(a, s);
  z = block_sum(z, s);
  n = block_sum(n, reinterpret_cast<int*>(s));
  live = block_sum(live, reinterpret_cast<int*>(s));
  if (threadIdx.x == 0) {
    losses[0] = live > 0 ? a / static_cast<float>(live) : 0.f;
    losses[1] = n > 0 ? z / static_cast<float>(n) : 0.f;
    parts.stats[0] = static_cast<float>(live);
    parts.stats[1] = static_cast<float>(n);
  }
}

template <typename T, int L, int NV>
__global__ void __launch_bounds__(BAL_THREADS) balance_bwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ off,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, const float* __restrict__ stats,
    const float* __restrict__ dlosses, int64_t T_, int E, int k, int G, int chunk, bool vec,
    T* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int l = lane % L;
  constexpr int GROUPS = BAL_THREADS / L;
  const int grp = tid / L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = min(T_, t0 + chunk);
  const float live = __ldg(stats), n_all = __ldg(stats + 1);
  const float db = __ldg(dlosses);
  const float dz = n_all > 0.f ? __ldg(dlosses + 1) * 2.f / n_all : 0.f;
  SeqWalk w;
  w.start(off, G, t0, t1);
  while (w.next()) {
    float c[NV][4];
    const float ns = w.s >= 0 ? static_cast<float>(__ldg(tokens + w.s)) : 0.f;
    const float scale =
        ns > 0.f ? db * (static_cast<float>(E) / static_cast<float>(k)) / (ns * ns * live) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * (l + i * L) + j;
        c[i][j] = ns > 0.f && e < E
                      ? scale * static_cast<float>(__ldg(counts + static_cast<int64_t>(w.s) * E + e))
                      : 0.f;
      }
    for (int64_t base = w.a; base < w.b; base += GROUPS) {
      const int64_t t = base + grp;
      bool on = t < w.b && ns > 0.f;
      if (on && mask != nullptr) on = __ldg(mask + t) != 0;
      float v[NV][4];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (on) {
          load4(logits + t * E, 4 * (l + i * L), E, vec, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = -INFINITY;
        }
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max_nan(m, v[i][j]);
      m = lanes_max<L>(m);
      on = on && m != -INFINITY;
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] = on ? expf(v[i][j] - m) : 0.f;
          sum += v[i][j];
          dot = fmaf(v[i][j], c[i][j], dot);
        }
      sum = lanes_sum<L>(sum);
      dot = lanes_sum<L>(dot);
      const float inv = on ? 1.f / sum : 0.f;
      const float shift = on ? dz * (m + logf(sum)) - dot * inv : 0.f;
      if (t < w.b) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = on ? v[i][j] * inv * (c[i][j] + shift) : 0.f;
          store4(dlogits + t * E, 4 * (l + i * L), E, vec, d);
        }
      }
    }
  }
}

// The split of T tokens over CTAs, and the workspace's arrays.
struct BalPlan {
  int chunk, nb;
  size_t stats, seq_z, n, z, cnt, p, bytes;
};

// Lanes per token (L) and 4-element vectors per lane (NV) by the number of experts.
static int bal_lanes(int E) { return E <= 128 ? 8 : E <= 256 ? 16 : 32; }

static BalPlan bal_plan(int64_t T, int E, int G) {
  BalPlan b{};
  const int groups = BAL_THREADS / bal_lanes(E);
  const int64_t per = (T + 607) / 608;  // about four CTAs on each of 152 SMs
  b.chunk = static_cast<int>((per + groups - 1) / groups * groups);
  b.nb = static_cast<int>((T + b.chunk - 1) / b.chunk);
  const size_t pieces = static_cast<size_t>(b.nb) + G;
  const auto take = [&](size_t bytes) {
    const size_t at = b.bytes;
    b.bytes += (bytes + 255) / 256 * 256;
    return at;
  };
  b.stats = take(8);
  b.seq_z = take(4 * static_cast<size_t>(G));
  b.n = take(4 * pieces);
  b.z = take(4 * pieces);
  b.cnt = take(4 * pieces * E);
  b.p = take(4 * pieces * E);
  return b;
}

static BalParts bal_parts(const BalPlan& b, void* ws) {
  char* p = static_cast<char*>(ws);
  return BalParts{reinterpret_cast<float*>(p + b.stats),   reinterpret_cast<float*>(p + b.p),
                  reinterpret_cast<int32_t*>(p + b.cnt),   reinterpret_cast<int32_t*>(p + b.n),
                  reinterpret_cast<float*>(p + b.z),       reinterpret_cast<float*>(p + b.seq_z)};
}

static bool bal_shape_ok(const mm_moe_balance_shape* s) {
  return s != nullptr && s->T >= 1 && s->T < (int64_t{1} << 31) - 65536 && s->E >= 1 &&
         s->E <= MAX_E && s->k >= 1 && s->k <= s->E && s->G >= 1 && s->G <= (1 << 24) &&
         dtype_ok(s->dtype);
}

static bool al(const void* p, uintptr_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

// f(lanes, vectors) as compile-time constants.
template <typename F>
static cudaError_t with_lanes(int E, F f) {
  using std::integral_constant;
  if (E <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (E <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  if (E <= 128) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  if (E <= 256) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
}

template <typename T>
static bool bal_vec(const void* p, int E) {
  return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_balance_workspace_size(
    const mm_moe_balance_shape* shape, size_t* bytes) {
  if (!bal_shape_ok(shape) || bytes == nullptr) return MM_MOE_EINVAL;
  *bytes = bal_plan(shape->T, static_cast<int>(shape->E), static_cast<int>(shape->G)).bytes;
  return MM_MOE_OK;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_balance_forward(
    const mm_moe_balance_shape* shape, const void* logits, const int32_t* topk_idx,
    const int32_t* seq_offsets, const uint8_t* mask, float* losses, float* seq_loss,
    int32_t* counts, int32_t* tokens, float* lse, void* workspace, void* stream) {
  if (!bal_shape_ok(shape)) return MM_MOE_EINVAL;
  if (!al(logits, dtype_bytes(shape->dtype)) || !al(topk_idx, 4) || !al(losses, 4) ||
      !al(seq_loss, 4) || !al(counts, 4) || !al(tokens, 4) || !al(lse, 4) || !al(workspace, 16) ||
      (seq_offsets == nullptr ? shape->G != 1 : !al(seq_offsets, 4)))
    return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int E = static_cast<int>(shape->E), k = static_cast<int>(shape->k),
            G = static_cast<int>(shape->G);
  const BalPlan b = bal_plan(shape->T, E, G);
  const BalParts parts = bal_parts(b, workspace);
  const size_t smem = static_cast<size_t>(BAL_WARPS + 1) * E * 4;
  prof_begin(c, K_BALANCE_FWD);
  cudaError_t e = with_dtype(shape->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const T* lg = static_cast<const T*>(logits);
    return with_lanes(E, [&](auto l, auto nv) {
      return launch_k(c.stream, balance_fwd_kernel<T, decltype(l)::value, decltype(nv)::value>,
                      dim3(b.nb), dim3(BAL_THREADS), smem, lg, topk_idx, seq_offsets, mask,
                      shape->T, E, k, G, b.chunk, bal_vec<T>(lg, E), lse, parts);
    });
  });
  prof_end(c, K_BALANCE_FWD);
  if (e != cudaSuccess) return MM_MOE_ECUDA;
  prof_begin(c, K_BALANCE_FINISH);
  e = launch_k(c.stream, balance_seq_kernel, dim3(G), dim3(256), 0, seq_offsets, shape->T, E, k,
               b.chunk, parts, seq_loss, counts, tokens);
  prof_end(c, K_BALANCE_FINISH);
  if (e != cudaSuccess) return MM_MOE_ECUDA;
  prof_begin(c, K_BALANCE_FINISH);
  e = launch_k(c.stream, balance_total_kernel, dim3(1), dim3(256), 0, G, parts,
               static_cast<const float*>(seq_loss), static_cast<const int32_t*>(tokens), losses);
  prof_end(c, K_BALANCE_FINISH);
  return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ECUDA;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_balance_backward(
    const mm_moe_balance_shape* shape, const void* logits, const int32_t* seq_offsets,
    const uint8_t* mask, const int32_t* counts, const int32_t* tokens, const float* dlosses,
    void* dlogits, const void* workspace, void* stream) {
  if (!bal_shape_ok(shape)) return MM_MOE_EINVAL;
  const size_t es = dtype_bytes(shape->dtype);
  if (!al(logits, es) || !al(dlogits, es) || !al(counts, 4) || !al(tokens, 4) ||
      !al(dlosses, 4) || !al(workspace, 16) ||
      (seq_offsets == nullptr ? shape->G != 1 : !al(seq_offsets, 4)))
    return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int E = static_cast<int>(shape->E), k = static_cast<int>(shape->k),
            G = static_cast<int>(shape->G);
  const BalPlan b = bal_plan(shape->T, E, G);
  const float* stats = bal_parts(b, const_cast<void*>(workspace)).stats;
  prof_begin(c, K_BALANCE_BWD);
  const cudaError_t e = with_dtype(shape->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const T* lg = static_cast<const T*>(logits);
    T* out = static_cast<T*>(dlogits);
    return with_lanes(E, [&](auto l, auto nv) {
      return launch_k(c.stream, balance_bwd_kernel<T, decltype(l)::value, decltype(nv)::value>,
                      dim3(b.nb), dim3(BAL_THREADS), 0, lg, seq_offsets, mask, counts, tokens,
                      stats, dlosses, shape->T, E, k, G, b.chunk,
                      bal_vec<T>(lg, E) && bal_vec<T>(out, E), out);
    });
  });
  prof_end(c, K_BALANCE_BWD);
  return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ECUDA;
}
