// select_fwd.cuh -- the choice of experts: the forward's kernel (formulas in select.cu), for the
// translation units of its logits' types.
//
// W = 8, 16 or 32 lanes take a token, as few as hold its row with 32 experts a lane (what a warp does
// once it does for all of its tokens; fewer tokens than fill the SMs: more lanes, up to 64 experts
// each).  A row comes to shared memory by cp.async in whole lines; a lane's experts belong to one
// group, whose lanes take its 16-byte pieces (or, unaligned, its experts) in turn.  A lower bound of
// the k-th largest key is the k-th largest of the lanes' two largest.  What lies above it, a dozen or
// two, goes to shared memory; each lane counts for its candidates how many keys are larger, which is
// their place.
//
// The order is that of the keys in 64 bits.  The fp32 keys decide where they lie further apart than
// their errors.  A closer pair is told apart by the difference of its keys, from the logits' own
// difference; groups in doubt, three keys together and pairs that are still too close are ranked by
// fp64 keys (131072 tokens x 256 experts of unit variance: some 80 pairs, a dozen groups).  So the indices
// do not depend on how a kernel rounds.  Without a bias the keys are the logits as they are.
//
// 131072 x 256 fp32: 72 us with a bias and four of eight groups, 59 without groups, 47 without a bias
// (the row's bytes take 20): 410 instructions a token, issued in 64% of the cycles, the ALU pipe
// (comparisons, selections) busy in 46%.  By rounds of a warp's largest head over sorted
// lanes, a warp a token, it took 139; with 16 lanes a token 98; with the next row on its way meanwhile 87
// (more shared memory, so less L1), in one CTA an SM less 73.  Up to 16 experts without groups have a kernel
// of their own below.
#pragma once
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

// Warps an SM below which a launch takes more lanes a token (us for 2048, 4096 and 8192 tokens of 256
// experts with bias and groups, at 2, 4, 8, 16 warps: 6.5, 7.5, 11.0; 7.4, 7.5, 11.1; 5.5, 12.3, 10.9;
// 5.5, 7.6, 18.9).
constexpr int SEL_FILL = 4;

__device__ __forceinline__ float low_nan(float f) { return fmaxf(f, -INFINITY); }
// For the choice and the sum under a softmax (whose terms' errors, weighted by the terms, stay within 2^-19
// of it), with the hardware's approximations (each within 2 ulp, the exponential's
// argument rounded): e^d within (|d| + 4) 2^-23 of itself, the sigmoid within 2^-21 of 1.
__device__ __forceinline__ float exp_key(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float sigmoid_key(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_key(-l)));
  return r;
}

// s(x) - s(y), exact to `tol` (some 2^-18 of itself, not of the scores), from the larger logit h and the
// smaller one l: s(h) (1 - s(l)) (1 - e^(l - h)) for the sigmoid, s(h) (1 - e^(l - h)) for the softmax.  (From
// s(l) and e^(h - l) a factor would be lost below fp32's range while the other leaves it above.)  What
// underflows here is below 2^-120.  score: s; terms: the errors of a softmax's sum, in 2^-24 of it.
template <typename F>
__device__ __forceinline__ float score_difference(float x, float y, bool sigmoid, float m, float terms,
                                                  F score, float& tol) {
  const float h = fmaxf(x, y), l = fminf(x, y), dl = x - y;
  float d = score(h) * -expm1f(-fabsf(dl));
  if (sigmoid) d *= sigmoid32(-l);
  tol = (sigmoid ? 64.f : terms + fabsf(h - m)) * 0x1p-24f * d + 0x1p-120f;
  return dl < 0.f ? -d : d;
}

// Reductions over aligned sets of n lanes.
template <typename F>
__device__ __forceinline__ float lanes(float v, int n, F f) {
  for (int o = 1; o < n; o <<= 1) v = f(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

__device__ __forceinline__ bool lanes_any(bool v, int n) {
  const uint32_t all = __ballot_sync(FULL, v);
  const int first = threadIdx.x & 31 & ~(n - 1);
  return (all >> first & (n == 32 ? FULL : (1u << n) - 1u)) != 0u;
}

// (key, e) to shared memory at `to`, which moves on, where the key comes up to `from`
__device__ __forceinline__ void put_from(uint32_t& to, float key, float from, int e) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t@p st.shared.v2.b32 [%0], {%3, %4};\n\t"
      "@p add.u32 %0, %0, 8;\n\t}"
      : "+r"(to)
      : "f"(key), "f"(from), "r"(__float_as_uint(key)), "r"(e)
      : "memory");
}

// The two larger of two pairs (descending).
__device__ __forceinline__ void merge2(float& a0, float& a1, float b0, float b1) {
  a1 = fmaxf(fminf(a0, b0), fmaxf(a1, b1));
  a0 = fmaxf(a0, b0);
}
template <int N>
__device__ __forceinline__ void top2_of(const float (&v)[N], float& t0, float& t1) {
  if constexpr (N == 1) {
    t0 = v[0], t1 = -INFINITY;
  } else {
    t0 = fmaxf(v[0], v[1]), t1 = fminf(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) merge2(t0, t1, fmaxf(v[i], v[i + 1]), fminf(v[i], v[i + 1]));
  }
}

// A lane's experts: the first, how many, and the others' places.  vec: 16-byte pieces of the row (NP a
// lane, taken from the group's number on, so that lanes of different groups read different banks).
template <typename T, int PL>
struct Mine {
  static constexpr int V = VN<T>, NP = PL / V > 0 ? PL / V : 1;
  int e0, cnt, lpg, turn;
  bool vec;
  __device__ __forceinline__ int piece(int p) const { return e0 + ((p + turn) & (NP - 1)) * V * lpg; }
  __device__ __forceinline__ int of(int i) const {
    return vec ? piece(i / V) + i % V : e0 + i * lpg;
  }
};

// An expert whose key comes up to the k-th.
struct __align__(8) Cand {
  float key;
  int e;
};

// A row's pieces to shared memory (each of the W lanes every W-th), or the lane's experts from there.
template <typename T, int W, int PL>
__device__ __forceinline__ void stage_row(const T* row, int pieces, uint32_t to) {
  const int lane = threadIdx.x & (W - 1);
#pragma unroll
  for (int i = 0; i < Mine<T, PL>::NP; ++i) {
    const int p = i * W + lane;
    if (p < pieces)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + p * 16),
                   "l"(row + p * VN<T>)
                   : "memory");
  }
}
template <typename T, int PL>
__device__ __forceinline__ void read_row(const unsigned char* from, const Mine<T, PL>& x,
                                         float (&l)[PL]) {
  constexpr int V = VN<T>;
  if constexpr (PL % V == 0) {
#pragma unroll
    for (int p = 0; p < PL / V; ++p) {
      float f[V];
      const uint4 q = x.cnt > 0 ? *reinterpret_cast<const uint4*>(from + x.piece(p) * sizeof(T))
                                : make_uint4(0, 0, 0, 0);
      unpack(q, f, static_cast<const T*>(nullptr));
#pragma unroll
      for (int j = 0; j < V; ++j) l[p * V + j] = f[j];
    }
  }
}

// ------------------------------------------------------------- the choice in 64 bits
// (b, i) in front of (a, j)
template <typename K>
__device__ __forceinline__ bool ahead(K a, int i, K b, int j) {
  return a > b || (a == b && i < j);
}

// The expert of place `lane` (of W), from keys in 64 bits or, without a bias, from the logits, for a
// token with more candidates than there is room for; kept: the lane's experts take part.
template <typename T, int W, int PL, bool BIAS>
__device__ __noinline__ int choose(const T* __restrict__ row, const float* __restrict__ bias,
                                   const SelArgs a, const Mine<T, PL> x, bool kept) {
  using K = std::conditional_t<BIAS, double, float>;
  const int lane = threadIdx.x & (W - 1), cnt = x.cnt;
  K key[PL];
  if constexpr (BIAS) {
    double m = -INFINITY, z = 0.0;
    if (!a.sigmoid) {
      for (int i = 0; i < cnt; ++i) m = fmax(m, static_cast<double>(to_f32(row[x.of(i)])));
      for (int o = W / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(FULL, m, o));
      m = finite_max(m);
      for (int i = 0; i < cnt; ++i) z += exp(static_cast<double>(to_f32(row[x.of(i)])) - m);
      z = sum_of<W>(z);
    }
    for (int i = 0; i < cnt; ++i) {
      const double l = to_f32(row[x.of(i)]);
      const double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : z == 0.0 ? 0.0 : exp(l - m) / z;
      key[i] = s + static_cast<double>(bias[x.of(i)]);
    }
  } else {
    for (int i = 0; i < cnt; ++i) key[i] = to_f32(row[x.of(i)]);
  }
  for (int i = 0; i < cnt; ++i)
    if (key[i] != key[i]) key[i] = -INFINITY;
  unsigned long long taken = 0;
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    K b = -INFINITY;
    int e = 0x7fffffff;
    if (kept)
      for (int i = 0; i < cnt; ++i) {
        const int o = x.of(i);
        if (!(taken >> i & 1u) && ahead(key[i], o, b, e)) b = key[i], e = o;
      }
    for (int o = W / 2; o > 0; o >>= 1) {
      const K ob = __shfl_xor_sync(FULL, b, o);
      const int oe = __shfl_xor_sync(FULL, e, o);
      if (ahead(ob, oe, b, e)) b = ob, e = oe;
    }
    for (int i = 0; i < cnt; ++i)
      if (x.of(i) == e) taken |= 1ull << i;
    if (lane == j) mine = e;
  }
  return mine;
}

// Places of the N candidates from keys in 64 bits; the first ones' experts into `at`.
template <typename T, int W>
__device__ __noinline__ void places64(const T* __restrict__ row, const float* __restrict__ bias,
                                      const SelArgs a, const Cand* cand, int N, double* keys,
                                      uint16_t* at) {
  const int lane = threadIdx.x & (W - 1);
  double m = -INFINITY, z = 1.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += W) m = fmax(m, static_cast<double>(to_f32(row[e])));
    for (int o = W / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(FULL, m, o));
    m = finite_max(m);
    z = 0.0;
    for (int e = lane; e < a.E; e += W) z += exp(static_cast<double>(to_f32(row[e])) - m);
    z = sum_of<W>(z);
  }
  for (int c = lane; c < N; c += W) {
    const double l = to_f32(row[cand[c].e]);
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : z == 0.0 ? 0.0 : exp(l - m) / z;
    const double key = s + static_cast<double>(bias[cand[c].e]);
    keys[c] = key != key ? -INFINITY : key;
  }
  __syncwarp();
  for (int c = lane; c < N; c += W) {
    int place = 0;
    for (int i = 0; i < N; ++i) place += ahead(keys[i], cand[i].e, keys[c], cand[c].e);
    if (place < a.k) at[place] = static_cast<uint16_t>(cand[c].e);
  }
  __syncwarp();
}

// Whether the lane's group is kept, from scores in 64 bits; `mask`: the lane's experts that can be
// among the two of its largest keys.
template <typename T, int W, int PL>
__device__ __noinline__ bool groups64(const T* __restrict__ row, const float* __restrict__ bias,
                                      const SelArgs a, const Mine<T, PL> x, unsigned long long mask) {
  const int lane = threadIdx.x & (W - 1), base = threadIdx.x & 31 & ~(W - 1);
  double m = -INFINITY, z = 1.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += W) m = fmax(m, static_cast<double>(to_f32(row[e])));
    for (int o = W / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(FULL, m, o));
    m = finite_max(m);
    if (bias != nullptr) {  // (without one, a common factor does not matter)
      z = 0.0;
      for (int e = lane; e < a.E; e += W) z += exp(static_cast<double>(to_f32(row[e])) - m);
      z = sum_of<W>(z);
    }
  }
  double t0 = -INFINITY, t1 = -INFINITY;
  while (mask != 0) {  // two at a time, for their chains of operations are long
    double s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = mask != 0 ? x.of(__ffsll(static_cast<long long>(mask)) - 1) : -1;
      mask &= mask - 1;  // (of none: none)
      double l = e >= 0 ? to_f32(row[e]) : 0.f;
      if (bias == nullptr && l != l) l = -INFINITY;  // (the logits rank)
      s[j] = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : z == 0.0 ? 0.0 : exp(l - m) / z;
      if (bias != nullptr && e >= 0) s[j] += static_cast<double>(bias[e]);
      if (e < 0 || s[j] != s[j]) s[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      t1 = fmax(t1, fmin(t0, s[j]));
      t0 = fmax(t0, s[j]);
    }
  }
  __syncwarp();
  for (int o = 1; o < a.lpg; o <<= 1) {
    const double o0 = __shfl_xor_sync(FULL, t0, o), o1 = __shfl_xor_sync(FULL, t1, o);
    t1 = fmax(fmin(t0, o0), fmax(t1, o1));
    t0 = fmax(t0, o0);
  }
  double g = a.top2 && a.gs > 1 ? t0 + t1 : t0;
  if (g != g) g = -INFINITY;  // (both infinities)
  const int mine = lane / a.lpg, within = lane % a.lpg;
  int rank = 0;
  for (int o = 0; o < a.G; o += a.lpg) {
    const int other = o + within;
    const double v = __shfl_sync(FULL, g, base + (other < a.G ? other : 0) * a.lpg);
    rank += other < a.G && ahead(v, other, g, mine);
  }
  for (int o = 1; o < a.lpg; o <<= 1) rank += __shfl_xor_sync(FULL, rank, o);
  return mine < a.G && rank < a.keep;
}

template <int PL>
constexpr int sel_warps = PL <= 8 ? 8 : 4;  // warps of a CTA
template <int PL>
constexpr int sel_ctas = PL <= 8 ? 4 : PL <= 16 ? 6 : PL <= 32 ? 5 : 3;  // CTAs an SM, all resident

// PL: experts a lane holds (at least c); W: lanes a token.
template <typename T, int W, int PL, bool BIAS>
__global__ void __launch_bounds__(32 * sel_warps<PL>, sel_ctas<PL>) select_fwd_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const SelArgs a,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr int WARPS = sel_warps<PL>, TOKENS = WARPS * 32 / W;
  constexpr int CAP = 8 * W;  // candidates at most
  constexpr int ROW = PL > 32 ? 512 : std::max(W * PL * static_cast<int>(sizeof(T)), PL > 8 ? 512 : 256);
  constexpr int STEP = 32 / W;  // tokens of a warp
  __shared__ __align__(16) unsigned char s_row[TOKENS][ROW];
  __shared__ __align__(16) Cand s_cand[TOKENS][CAP + 4];
  __shared__ float s_best[TOKENS][W + 2];  // by place, up to the (k + 2)th
  __shared__ uint16_t s_at[TOKENS][W + 2];
  __shared__ int s_turn;
  __shared__ __align__(16) float2 s_part[W == 8 ? TOKENS : 1][W];
  // the bias by lane, four of its experts at a time: [PL / 4][W][4]
  __shared__ __align__(16) float s_bias[BIAS ? W * PL : 4];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (W - 1), base = threadIdx.x & 31 & ~(W - 1);
  const int slot = threadIdx.x / W;
  const int group = lane / a.lpg, within = lane % a.lpg;
  Mine<T, PL> x;
  x.lpg = a.lpg;
  x.vec = a.vec;
  x.turn = group;
  x.e0 = group * a.gs + within * (a.vec ? VN<T> : 1);
  x.cnt = group >= a.G ? 0 : a.vec ? PL : max(0, (a.gs - within + a.lpg - 1) / a.lpg);
  const int cnt = x.cnt;
  const bool real = group < a.G;
  Cand* const cand = s_cand[slot];
  if constexpr (BIAS) {
    static_assert(PL % 4 == 0);
    for (int i = threadIdx.x / W; i < PL; i += TOKENS)
      s_bias[(i / 4 * W + lane) * 4 + i % 4] = i < cnt ? __ldg(bias + x.of(i)) : -INFINITY;
  }
  // The CTA's tokens come in steps of a warp's STEP, which its warps take as they get to them: a token
  // that needs 64 bits holds up its warp, not the CTA.  (A warp's tokens loop together.)
  const int steps = static_cast<int>((static_cast<int64_t>(a.T) + STEP - 1) / STEP);
  int turn = threadIdx.x >> 5;
  unsigned char* const here = s_row[slot];
  if (threadIdx.x == 0) s_turn = WARPS;
  __syncthreads();
  for (;;) {
    const int64_t step = static_cast<int64_t>(turn) * gridDim.x + blockIdx.x;
    if (step >= steps) break;
    const int64_t t = step * STEP + slot % STEP;
    const bool live = t < a.T;
    const T* const row = logits + (live ? t : 0) * a.E;
    if ((threadIdx.x & 31) == 0) turn = atomicAdd(&s_turn, 1);
    turn = __shfl_sync(FULL, turn, 0);  // the next one's
    float v[PL];
    if (a.vec) {
      stage_row<T, W, PL>(row, a.E / VN<T>,
                          static_cast<uint32_t>(__cvta_generic_to_shared(here)));
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      read_row<T, PL>(here, x, v);
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        v[i] = i < cnt ? to_f32(__ldg(row + x.e0 + i * x.lpg)) : -INFINITY;
    }
    float m = -INFINITY, rz = 0.f;  // the row's largest logit and 1 / sum exp(l - m)
    if (!a.sigmoid && (BIAS || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < PL; ++i) m = fmaxf(m, v[i]);
      m = finite_max(max_of<W>(cnt > 0 ? m : -INFINITY));
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) z += exp_key(v[i] - m);
      z = sum_of<W>(cnt > 0 ? z : 0.f);
      rz = z == 0.f ? 0.f : 1.f / z;
    }
    if constexpr (BIAS) {
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PL; ++i) v[i] = sigmoid_key(v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) v[i] = exp_key(v[i] - m) * rz;
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) v[i] += s_bias[(i / 4 * W + lane) * 4 + i % 4];
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = low_nan(v[i]);

    // the errors of two scores under the keys
    const float bound = BIAS ? (a.sigmoid ? 0x1p-19f : rz * ((2 * PL + 64) * 0x1p-24f)) : 0.f;
    bool kept = cnt > 0;
    float t0, t1 = -INFINITY;  // the lane's largest, and its second (or, of all, the other half's)
    if (a.G > 1) {
      top2_of(v, t0, t1);
    } else {
      t0 = v[0];
      if constexpr (PL > 1) {
        t1 = v[PL / 2];
#pragma unroll
        for (int i = 1; i < PL / 2; ++i) t0 = fmaxf(t0, v[i]), t1 = fmaxf(t1, v[i + PL / 2]);
      }
    }
    if (a.G > 1) {
      float g0 = real ? t0 : -INFINITY, g1 = real ? t1 : -INFINITY;
      for (int o = 1; o < a.lpg; o <<= 1)
        merge2(g0, g1, __shfl_xor_sync(FULL, g0, o), __shfl_xor_sync(FULL, g1, o));
      float lost = 1.f;  // by how much a score's relative error exceeds its key's
      if (!BIAS && a.top2) {  // scores of logits (the softmax's common factor does not matter)
        const float far = fmaxf(g0 == -INFINITY ? 0.f : fabsf(g0), g1 == -INFINITY ? 0.f : fabsf(g1));
        lost += max_of<W>(far);
        const float big = a.sigmoid ? 0.f : max_of<W>(g0);
        g0 = a.sigmoid ? sigmoid32(g0) : big == -INFINITY ? 0.f : expf(g0 - big);
        g1 = a.sigmoid ? sigmoid32(g1) : big == -INFINITY ? 0.f : expf(g1 - big);
      }
      const bool two = a.top2 && a.gs > 1;
      const float gs = low_nan(two ? g0 + g1 : g0);
      int rank = 0;  // a group's lanes share the comparisons
      for (int o = 0; o < a.G; o += a.lpg) {
        const int other = o + within;
        const float w = __shfl_sync(FULL, gs, base + (other < a.G ? other : 0) * a.lpg);
        rank += other < a.G && (w > gs || (w == gs && other < group));
      }
      for (int o = 1; o < a.lpg; o <<= 1) rank += __shfl_xor_sync(FULL, rank, o);
      kept = real && rank < a.keep;
      if (BIAS || a.top2) {  // (else the logits have told)
        const float least = min_of<W>(kept ? gs : INFINITY);
        const float best = max_of<W>(real && !kept ? gs : -INFINITY);
        // the errors of both sums: their scores' and the roundings, of the largest there is
        float size = (g0 == -INFINITY ? 0.f : fabsf(g0)) + (two && g1 != -INFINITY ? fabsf(g1) : 0.f);
        size = max_of<W>(real ? size : 0.f);
        const bool doubt =
            !(least - best > (BIAS ? 2.f * bound + size * 0x1p-22f : size * lost * 0x1p-20f));
        if (__any_sync(FULL, doubt)) {
          const float last = a.top2 ? t1 : t0;
          const float from = last - bound - fabsf(last) * 0x1p-21f;
          unsigned long long mask = 0;
#pragma unroll
          for (int i = 0; i < PL; ++i)
            if (i < cnt && !(v[i] < from)) mask |= 1ull << i;
          kept = groups64<T, W, PL>(row, BIAS ? bias : nullptr, a, x, mask);
        }
      }
      kept = kept && cnt > 0;
    }

    // The candidates: nothing else comes up to the k-th key, not by the keys' errors either.
    float least = -INFINITY;
    if (a.bounded) {
      if constexpr (W == 8) {  // the k-th of the lanes' two
        float2* const part = s_part[slot];
        part[lane] = kept ? make_float2(t0, t1) : make_float2(-INFINITY, -INFINITY);
        __syncwarp();
        float c0 = 0.f, c1 = 0.f;  // how many are larger
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          const float4 q = *reinterpret_cast<const float4*>(part + i);
          c0 += q.x > t0 ? 1.f : 0.f, c1 += q.x > t1 ? 1.f : 0.f;
          c0 += q.y > t0 ? 1.f : 0.f, c1 += q.y > t1 ? 1.f : 0.f;
          c0 += q.z > t0 ? 1.f : 0.f, c1 += q.z > t1 ? 1.f : 0.f;
          c0 += q.w > t0 ? 1.f : 0.f, c1 += q.w > t1 ? 1.f : 0.f;
        }
        const float k = static_cast<float>(a.k);
        least = fminf(c0 < k ? t0 : INFINITY, c1 < k ? t1 : INFINITY);
        least = min_of<W>(kept ? least : INFINITY);
      } else {  // the least of the sets' largest
        const bool any = lanes_any(kept, a.set);
        const float best =
            lanes(kept ? fmaxf(t0, t1) : -INFINITY, a.set, [](float p, float q) { return fmaxf(p, q); });
        least = min_of<W>(any ? best : INFINITY);
      }
      if constexpr (BIAS) {
        const float lower = least - (bound + fabsf(least) * 0x1p-21f);
        if (lower < least) least = lower;  // (not for what is not finite)
      }
    }
    const float none = __uint_as_float(0x7fffffffu);  // a NaN: no key comes up to it
    const float from = kept ? least : none;
    int n = 0;
    if (a.vec) {  // (a lane's places hold experts, or it is not kept)
#pragma unroll
      for (int i = 0; i < PL; ++i) n += v[i] >= from;
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) n += v[i] >= (i < cnt ? from : none);
    }
    int at = n;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      const int y = __shfl_up_sync(FULL, at, o, W);
      if (lane >= o) at += y;
    }
    const int all = __shfl_sync(FULL, at, base + W - 1);
    const bool over = all > CAP;  // (many equal keys)
    const int N = over ? 0 : all;
    {
      const float from_ = over ? none : from;
      uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(cand + at - n));
      if (a.vec) {
#pragma unroll
        for (int p = 0; p < PL / VN<T>; ++p) {
          const int e = x.piece(p);
#pragma unroll
          for (int j = 0; j < VN<T>; ++j) put_from(to, v[p * VN<T> + j], from_, e + j);
        }
      } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) put_from(to, v[i], i < cnt ? from_ : none, x.e0 + i * x.lpg);
      }
    }
    if (lane < 4) cand[N + lane].key = -INFINITY;
    for (int j = lane; j < a.k + 2; j += W) s_at[slot][j] = 0xffff;
    __syncwarp();
    // Each one's place: as many as are no smaller, without itself.  Equal ones come to the same
    // place and leave another empty.
    const auto settle = [&](int c, float key, float above) {
      // (the padding behind the last one is no smaller than -inf)
      const int place = static_cast<int>(above) - (key == -INFINITY ? -N & 3 : 0);
      if (c < N && place < a.k + 2) {
        s_best[slot][place] = key;
        s_at[slot][place] = static_cast<uint16_t>(cand[c].e);
      }
    };
    for (int c = lane; c < N; c += 3 * W) {  // three of the lane's at a time
      const float k0 = cand[c].key, k1 = c + W < N ? cand[c + W].key : INFINITY,
                  k2 = c + 2 * W < N ? cand[c + 2 * W].key : INFINITY;
      float p0 = -1.f, p1 = -1.f, p2 = -1.f;
      for (int i = 0; i < N; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(cand + i);
        const float4 r = *reinterpret_cast<const float4*>(cand + i + 2);
        p0 += q.x >= k0 ? 1.f : 0.f, p1 += q.x >= k1 ? 1.f : 0.f, p2 += q.x >= k2 ? 1.f : 0.f;
        p0 += q.z >= k0 ? 1.f : 0.f, p1 += q.z >= k1 ? 1.f : 0.f, p2 += q.z >= k2 ? 1.f : 0.f;
        p0 += r.x >= k0 ? 1.f : 0.f, p1 += r.x >= k1 ? 1.f : 0.f, p2 += r.x >= k2 ? 1.f : 0.f;
        p0 += r.z >= k0 ? 1.f : 0.f, p1 += r.z >= k1 ? 1.f : 0.f, p2 += r.z >= k2 ? 1.f : 0.f;
      }
      settle(c, k0, p0);
      settle(c + W, k1, p1);
      settle(c + 2 * W, k2, p2);
    }
    __syncwarp();
    bool hole = false;
    for (int j = lane; j < a.k + 2 && j < N; j += W) hole = hole || s_at[slot][j] == 0xffff;
    if (__any_sync(FULL, hole)) {  // equal keys: of them the first in front
      for (int c = lane; c < N; c += W) {
        const Cand mine = cand[c];
        int place = 0;
        for (int i = 0; i < N; ++i) {
          const Cand o = cand[i];
          place += o.key > mine.key || (o.key == mine.key && o.e < mine.e);
        }
        if (place < a.k + 2) {
          s_best[slot][place] = mine.key;
          s_at[slot][place] = static_cast<uint16_t>(mine.e);
        }
      }
      __syncwarp();
    }

    const bool mine = lane < a.k;
    int e = mine ? min(static_cast<int>(s_at[slot][lane]), a.E - 1) : 0;
    const auto logit = [&](int i) {
      return a.vec ? to_f32(reinterpret_cast<const T*>(here)[i]) : to_f32(__ldg(row + i));
    };
    float lj = logit(e);
    const auto score = [&](float x) { return a.sigmoid ? sigmoid32(x) : expf(x - m) * rz; };
    float sj = BIAS || a.sigmoid || !a.renorm ? score(lj) : 0.f;
    if constexpr (BIAS) {
      // Pairs in doubt, each lane's with the next place's, the last one's with the first left out
      // (the empty place behind the last candidate: nothing else comes up to it).
      const int after = mine ? s_at[slot][lane + 1] : 0xffff, behind = mine ? s_at[slot][lane + 2] : 0xffff;
      const float key = mine ? s_best[slot][lane] : 0.f;
      const auto close = [&](int at, int place) {
        const float k = at != 0xffff ? s_best[slot][place] : 0.f;
        return at != 0xffff && !(key - k > bound + 0x1p-22f * (fabsf(key) + fabsf(k)));
      };
      const bool near = close(after, lane + 1);
      if (__any_sync(FULL, near)) {
        bool swap = false, doubt = false;
        if (near) {
          const float ln = logit(after);
          const float db = __ldg(bias + e) - __ldg(bias + after);
          float tol;
          const float d = score_difference(lj, ln, a.sigmoid, m, 2 * PL + 64.f, score, tol);
          tol += 0x1p-23f * fabsf(db);
          const bool tie = lj == ln && db == 0.f;  // (in order then)
          swap = d + db < -tol;
          doubt = !(fabsf(d + db) > tol) && !tie;
          // three keys close together: only where they are the same
          if (close(behind, lane + 2)) {
            doubt = doubt || !(tie && logit(behind) == ln &&
                               __ldg(bias + behind) == __ldg(bias + after));
            // ... and behind the last place, where no lane looks further, only where all close ones are
            if (lane == a.k - 1 && !doubt) {
              const float b = __ldg(bias + e);
              for (int i = 0; i < N && !doubt; ++i) {
                const Cand o = cand[i];
                doubt = !(fabsf(key - o.key) > bound + 0x1p-22f * (fabsf(key) + fabsf(o.key))) &&
                        !(logit(o.e) == lj && __ldg(bias + o.e) == b);
              }
            }
          }
        }
        const int other = __shfl_up_sync(FULL, e, 1, W);
        const bool from_above = __shfl_up_sync(FULL, swap, 1, W) && lane > 0;
        doubt = (__ballot_sync(FULL, mine && doubt) >> base & (FULL >> (32 - W))) != 0;
        if (!doubt && mine && (swap || from_above)) {
          e = swap ? after : other;
          lj = logit(e);
          sj = score(lj);
        }
        // a few candidates are ranked anew, for many the whole row
        const bool many = doubt && N > ROW / 8, few = doubt && !many;
        if (__any_sync(FULL, few)) {
          places64<T, W>(row, bias, a, cand, few ? N : 0,
                         reinterpret_cast<double*>(here), s_at[slot]);
          if (few) e = mine ? min(static_cast<int>(s_at[slot][lane]), a.E - 1) : 0;
        }
        if (__any_sync(FULL, many)) {
          const int other = choose<T, W, PL, BIAS>(row, bias, a, x, kept);
          if (many) e = mine ? other : 0;
        }
        if (doubt) {
          lj = to_f32(__ldg(row + e));
          sj = score(lj);
        }
      }
    }
    if (__any_sync(FULL, over)) {
      const int other = choose<T, W, PL, BIAS>(row, bias, a, x, kept);
      if (over) {
        e = mine ? other : 0;
        lj = to_f32(__ldg(row + e));
        if (BIAS || a.sigmoid || !a.renorm) sj = score(lj);
      }
    }
    float w;
    if (!a.renorm) {
      w = sj * a.scale;
    } else if (a.sigmoid) {
      w = a.scale * (sj / (sum_of<W>(mine ? sj : 0.f) + SUM_EPS));
    } else {  // the softmax over the chosen
      const float big = max_of<W>(mine ? lj : -INFINITY);
      const float ex = mine && !(lj == -INFINITY) ? expf(lj - big) : 0.f;  // (of a NaN a NaN)
      const float sum = sum_of<W>(ex);
      w = sum == 0.f ? 0.f : a.scale * (ex / sum);
      if (BIAS && sj != sj) w = sj;  // (a row whose scores are NaN)
    }
    if (mine && live) {
      topk_idx[t * a.k + lane] = e;
      topk_w[t * a.k + lane] = w;
    }
    __syncwarp();  // (the next token's candidates go to the same place)
  }
}

// ------------------------------------------------------------------------ few experts
// The largest logit and the sum of e^(l - m) in 64 bits (of a softmax), and a key from them.
struct Row64 {
  double m, z;
};
template <typename T>
__device__ __forceinline__ Row64 row64(const T* __restrict__ row, const SelArgs& a) {
  Row64 r{-INFINITY, 0.0};
  if (a.sigmoid) return r;
  for (int e = 0; e < a.E; ++e) r.m = fmax(r.m, static_cast<double>(to_f32(row[e])));
  r.m = finite_max(r.m);
  for (int e = 0; e < a.E; ++e) r.z += exp(static_cast<double>(to_f32(row[e])) - r.m);
  return r;
}
template <typename T>
__device__ __forceinline__ double key64(const T* __restrict__ row, const float* __restrict__ bias,
                                        const SelArgs& a, const Row64& r, int e) {
  const double l = to_f32(row[e]);
  const double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : r.z == 0.0 ? 0.0 : exp(l - r.m) / r.z;
  const double key = s + static_cast<double>(bias[e]);
  return key != key ? -INFINITY : key;
}

// Whether expert j's key (bias and all) lies above expert i's, for keys that fp32 does not tell apart: by
// the difference of the logits (as in select_fwd_kernel), else in 64 bits.
template <typename T>
__device__ __noinline__ bool above(const T* __restrict__ row, const float* __restrict__ bias,
                                   const SelArgs a, float m, float rz, int i, int j) {
  const float li = to_f32(__ldg(row + i)), lj = to_f32(__ldg(row + j));
  const float db = __ldg(bias + j) - __ldg(bias + i);
  if (lj == li && db == 0.f) return false;
  float tol;
  const float d = score_difference(
      lj, li, a.sigmoid, m, 128.f,
      [&](float x) { return a.sigmoid ? sigmoid32(x) : expf(x - m) * rz; }, tol);
  tol += 0x1p-23f * fabsf(db);
  if (fabsf(d + db) > tol) return d + db > 0.f;
  const Row64 r = row64(row, a);
  return key64(row, bias, a, r, j) > key64(row, bias, a, r, i);
}

// The experts' places by keys in 64 bits, four bits each.
template <typename T>
__device__ __noinline__ unsigned long long small_places64(const T* __restrict__ row,
                                                          const float* __restrict__ bias,
                                                          const SelArgs a) {
  const Row64 r = row64(row, a);
  double key[16];
  for (int e = 0; e < a.E; ++e) key[e] = key64(row, bias, a, r, e);
  unsigned long long places = 0;
  for (int e = 0; e < a.E; ++e) {
    int place = 0;
    for (int o = 0; o < a.E; ++o) place += ahead(key[o], o, key[e], e);
    places |= static_cast<unsigned long long>(place) << 4 * e;
  }
  return places;
}

// Up to N experts, all groups taking part: a thread a token, its keys in registers, every expert's
// place the number of keys in front of its own; pairs within each other's errors are compared anew.
// 131072 x 8 fp32 4.0 us (27 in eight lanes a token), 131072 x 16 9.4; with a bias 7.0 and 24 (sigmoid),
// 8.2 and 35 (softmax).
template <typename T, int N, bool BIAS>
__global__ void __launch_bounds__(128) select_small_kernel(
    const T* __restrict__ logits, const float* __restrict__ bias, const SelArgs a,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  pdl_wait();
  pdl_trigger();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (t >= a.T) return;
  const T* const row = logits + t * a.E;
  float l[N];
  if (a.vec) {  // (N experts)
#pragma unroll
    for (int i = 0; i < N; i += VN<T>) {
      float f[VN<T>];
      unpack(__ldg(reinterpret_cast<const uint4*>(row + i)), f, row);
#pragma unroll
      for (int j = 0; j < VN<T>; ++j) l[i + j] = f[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = i < a.E ? to_f32(__ldg(row + i)) : -INFINITY;
  }
  float m = -INFINITY, rz = 0.f;
  if (!a.sigmoid && (BIAS || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
    m = finite_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) z += i < a.E ? expf(l[i] - m) : 0.f;
    rz = z == 0.f ? 0.f : 1.f / z;
  }
  const auto score = [&](float x) { return a.sigmoid ? sigmoid32(x) : expf(x - m) * rz; };
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = BIAS ? score(l[i]) + (i < a.E ? __ldg(bias + i) : 0.f) : l[i];
    v[i] = i < a.E ? low_nan(v[i]) : -INFINITY;
  }
  int place[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = i + 1; j < N; ++j) {
      const bool behind = v[j] > v[i];
      place[i] += behind;
      place[j] += !behind;
    }
  if constexpr (BIAS) {
    // the errors of two scores (16 2^-24 of each: a sum of N terms besides), and the sums' own
    const float bound = (2 * N + 64) * 0x1p-24f * (a.sigmoid ? 1.f : rz);
    // by expert, those of higher index that are in doubt (all of them, once one bears on the choice: the
    // places are right together or not at all)
    uint32_t near[N];
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      near[i] = 0;
#pragma unroll
      for (int j = i + 1; j < N; ++j) {
        const bool apart = fabsf(v[i] - v[j]) > bound + 0x1p-22f * (fabsf(v[i]) + fabsf(v[j]));
        if (j < a.E && !apart) {
          near[i] |= 1u << j;
          any = any || min(place[i], place[j]) < a.k;
        }
      }
    }
    if (any) {
      unsigned long long packed = 0;  // the places, four bits each
#pragma unroll
      for (int i = 0; i < N; ++i) packed |= static_cast<unsigned long long>(place[i]) << 4 * i;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        while (near[i] != 0) {
          const int j = __ffs(near[i]) - 1;
          near[i] &= near[i] - 1;
          float vj = -INFINITY;
#pragma unroll
          for (int h = i + 1; h < N; ++h) vj = h == j ? v[h] : vj;
          const bool was = vj > v[i], is = above(row, bias, a, m, rz, i, j);
          if (was != is) {
            packed += is ? 1ull << 4 * i : 1ull << 4 * j;
            packed -= is ? 1ull << 4 * j : 1ull << 4 * i;
          }
        }
      }
      // A pair told apart by its difference, which can be finer than 64 bits of a key, and pairs that tie there
      // can form a circle: then all are ranked in 64 bits.
      uint32_t there = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) there |= i < a.E ? 1u << (packed >> 4 * i & 15u) : 0u;
      if (there != (1u << a.E) - 1u) packed = small_places64(row, bias, a);
#pragma unroll
      for (int i = 0; i < N; ++i)
        place[i] = i < a.E ? static_cast<int>(packed >> 4 * i & 15u) : N;
    }
  }
  // (absent experts come behind all: -inf, and of higher index)
  float big = -INFINITY, sum = 0.f;
  float w[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (place[i] < a.k) big = fmaxf(big, l[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = place[i] < a.k;
    w[i] = !in ? 0.f
           : a.renorm && !a.sigmoid ? (l[i] == -INFINITY ? 0.f : expf(l[i] - big))
                                    : score(l[i]);
    sum += w[i];
  }
  float c = !a.renorm ? a.scale : a.sigmoid ? 1.f / (sum + SUM_EPS) : sum == 0.f ? 0.f : 1.f / sum;
  if (BIAS && rz != rz) c = rz;  // (a row whose scores are NaN)
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (place[i] < a.k) {
      topk_idx[t * a.k + place[i]] = i;
      topk_w[t * a.k + place[i]] = a.renorm ? a.scale * (w[i] * c) : w[i] * c;
    }
}

// --------------------------------------------------------------------------- host side
template <typename T, int N>
cudaError_t sel_launch_small(const Ctx& c, SelArgs a, const T* logits, const float* bias,
                             int32_t* idx, float* w) {
  a.vec = a.E == N && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  auto* kern = bias != nullptr ? select_small_kernel<T, N, true> : select_small_kernel<T, N, false>;
  const int ctas = static_cast<int>((static_cast<int64_t>(a.T) + 127) / 128);
  return launch_k(c.stream, kern, dim3(ctas), dim3(128), 0, logits, bias, a, idx, w);
}

// The row over W lanes; false where they do not hold it.
inline bool sel_split(SelArgs* a, int W) {
  const auto up = [](int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
  };
  if (up(a->G) > W || a->k > W) return false;
  a->lpg = W / up(a->G);
  a->c = (a->gs + a->lpg - 1) / a->lpg;
  const int used = std::min(a->gs, a->lpg);  // lanes of a group that have experts
  if (W == 8) {
    // (every lane has two: in both halves of its places where all groups are one)
    const int half = a->G > 1 ? 1 : (a->c <= 4 ? 4 : a->c <= 8 ? 8 : a->c <= 16 ? 16 : 32) / 2;
    a->bounded = a->keep * used * (a->gs / a->lpg > half ? 2 : 1) >= a->k;
  } else {
    a->set = a->lpg;
    while (a->set > 0 && a->keep * ((used + a->set - 1) / a->set) < a->k) a->set /= 2;
    a->bounded = a->set > 0;
  }
  // (without a bound every expert that takes part is a candidate, of 8 W at most)
  if (!a->bounded && W < 32 && a->keep * a->gs > 8 * W) return false;
  return true;
}

template <typename T, int W, int PL>
cudaError_t sel_launch(const Ctx& c, SelArgs a, const T* logits, const float* bias, int32_t* idx,
                       float* w) {
  constexpr int TOKENS = sel_warps<PL> * 32 / W;
  a.vec = PL % VN<T> == 0 && a.gs == PL * a.lpg && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
          a.E * sizeof(T) % 16 == 0;
  auto* kern = bias != nullptr ? select_fwd_kernel<T, W, PL, true> : select_fwd_kernel<T, W, PL, false>;
  const int ctas = static_cast<int>((static_cast<int64_t>(a.T) + TOKENS - 1) / TOKENS);
  return launch_k(c.stream, kern, dim3(std::min(ctas, c.num_sms * sel_ctas<PL>)),
                  dim3(32 * sel_warps<PL>), 0, logits, bias, a, idx, w);
}

// As few lanes a token as hold its row, for what a warp does once it does for all its tokens; more where
// that leaves the SMs less than SEL_FILL warps.
template <typename T>
cudaError_t launch_select_fwd_of(const Ctx& c, const SelArgs& args, const T* logits,
                                 const float* bias, int32_t* idx, float* w) {
  SelArgs a = args;
  const auto fills = [&](int W) {
    return static_cast<int64_t>(a.T) * W >= static_cast<int64_t>(c.num_sms) * 32 * SEL_FILL;
  };
  if (a.G == 1 && a.E <= 16)
    return a.E <= 8 ? sel_launch_small<T, 8>(c, a, logits, bias, idx, w)
                    : sel_launch_small<T, 16>(c, a, logits, bias, idx, w);
  if (fills(8) && sel_split(&a, 8) && a.c <= 32) {
    if (a.c <= 4) return sel_launch<T, 8, 4>(c, a, logits, bias, idx, w);
    if (a.c <= 8) return sel_launch<T, 8, 8>(c, a, logits, bias, idx, w);
    if (a.c <= 16) return sel_launch<T, 8, 16>(c, a, logits, bias, idx, w);
    return sel_launch<T, 8, 32>(c, a, logits, bias, idx, w);
  }
  if (fills(16) && sel_split(&a, 16) && a.c <= 32) {
    if (a.c <= 8) return sel_launch<T, 16, 8>(c, a, logits, bias, idx, w);
    return sel_launch<T, 16, 32>(c, a, logits, bias, idx, w);
  }
  sel_split(&a, 32);  // (k and the groups are 32 at most)
  if (a.c <= 8) return sel_launch<T, 32, 8>(c, a, logits, bias, idx, w);
  if (a.c <= 32) return sel_launch<T, 32, 32>(c, a, logits, bias, idx, w);
  return sel_launch<T, 32, 64>(c, a, logits, bias, idx, w);
}

}  // namespace mmmoe
