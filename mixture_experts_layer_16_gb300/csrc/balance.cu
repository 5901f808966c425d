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
#include <type_traits>

#include "internal.h"
#include "ops.cuh"

namespace mmmoe {

// Threads of a token kernel's CTA at most: few large CTAs leave few pieces to join; with
// many short sequences, each of which ends with a barrier, smaller CTAs run side by side.
constexpr int BAL_THREADS = 384;
constexpr int BAL_SMALL = 128;
constexpr int BAL_WARPS = BAL_THREADS / 32;  // at most

// A token's row reaches its lanes through a ring in shared memory, STAGES - 1 tokens ahead,
// by cp.async: a lane copies its own four-logit quads (and its share of topk_idx) and reads
// nothing but what it copied, so no barrier guards the ring.  A quad past the last expert
// holds -inf from the start.
constexpr int BAL_STAGES = 3;

template <typename T, int L, int NV, bool VEC>
struct Ring {
  static constexpr int QUAD = 4 * static_cast<int>(sizeof(T));
  static constexpr int KS = L >= 8 ? 1 : 8 / L;  // topk_idx entries per lane (k <= 8; else read directly)
  static constexpr int BYTES = BAL_STAGES * (NV * QUAD + KS * 4);  // per thread
  // This thread's; its next one lies a quad (an int) of every thread further on, as a warp's
  // quads come from memory.  (A thread's quads side by side, which takes fewer address
  // instructions, cost 30% more time: the copies then scatter each line they bring.)
  uint32_t quads, idx, unit, idx_unit;
  int l, E, k;
  __device__ __forceinline__ void init(unsigned char* smem, int l_, int E_, int k_) {
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    unit = blockDim.x * QUAD;
    idx_unit = blockDim.x * 4;
    quads = base + threadIdx.x * QUAD;
    idx = base + BAL_STAGES * NV * unit + threadIdx.x * 4;
    l = l_;
    E = E_;
    k = k_;
    // what lies past the last expert
    if (E == 4 * L * NV) return;
#pragma unroll 1
    for (int st = 0; st < BAL_STAGES; ++st)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (expert(i) + j >= E) put(st, i, j, from_f32<T>(-INFINITY));
  }
  __device__ __forceinline__ int expert(int i) const { return 4 * (l + i * L); }
  __device__ __forceinline__ uint32_t quad(int st, int i) const { return quads + (st * NV + i) * unit; }
  __device__ __forceinline__ void put(int st, int i, int j, T v) const {
    const uint32_t at = quad(st, i) + j * static_cast<int>(sizeof(T));
    if constexpr (sizeof(T) == 4)
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
    else
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const uint16_t*>(&v))
                   : "memory");
  }
  template <int B>
  __device__ __forceinline__ static void copy(uint32_t dst, const void* src) {
    if constexpr (B == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B)
                   : "memory");
  }
  // A token's quads; p is its row from this lane's first expert on.  VEC: rows are whole
  // quads on their boundaries; others come element by element, 16-bit ones by plain loads.
  __device__ __forceinline__ void load(int st, const T* p) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC) {
        if (expert(i) < E) copy<QUAD>(quad(st, i), p + 4 * i * L);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (expert(i) + j < E) {
            if constexpr (sizeof(T) == 4)
              copy<4>(quad(st, i) + 4 * j, p + 4 * i * L + j);
            else
              put(st, i, j, p[4 * i * L + j]);
          }
      }
    }
  }
  // and of topk_idx; p is the row from this lane's first slot on
  __device__ __forceinline__ void load_idx(int st, const int32_t* p) const {
#pragma unroll
    for (int j = 0; j < KS; ++j)
      if (l + j * L < k) copy<4>(idx + (st * KS + j) * idx_unit, p + j * L);
  }
  __device__ __forceinline__ int slot(int st, int j) const {
    int e;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(e) : "r"(idx + (st * KS + j) * idx_unit) : "memory");
    return e;
  }
  __device__ __forceinline__ static void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ static void wait() {  // the oldest of STAGES rows has landed
    asm volatile("cp.async.wait_group %0;" ::"n"(BAL_STAGES - 1) : "memory");
  }
  __device__ __forceinline__ static void drain() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ void get(int st, f2 (&v)[2 * NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (sizeof(T) == 4) {
        asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
                     : "=l"(v[2 * i]), "=l"(v[2 * i + 1])
                     : "r"(quad(st, i))
                     : "memory");
      } else {
        uint2 q;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                     : "=r"(q.x), "=r"(q.y)
                     : "r"(quad(st, i))
                     : "memory");
        const T* h = reinterpret_cast<const T*>(&q);
        v[2 * i] = f2_make(to_f32(h[0]), to_f32(h[1]));
        v[2 * i + 1] = f2_make(to_f32(h[2]), to_f32(h[3]));
      }
    }
  }
};

// Mask bytes of a group's next L tokens, one a lane, read once for all of them.  p is the
// group's token of round `it`, of which `left` rounds' tokens remain.
template <int L>
struct MaskAhead {
  uint32_t mine = 1;
  __device__ __forceinline__ bool get(const uint8_t* p, int stride, int l, int it, int left) {
    if (it % L == 0) mine = l < left ? __ldg(p + static_cast<int64_t>(l) * stride) : 0;
    return __shfl_sync(0xffffffffu, mine, it % L, L) != 0;
  }
};

// Four values to o, where j < n of them exist (VEC: all or none).
template <bool VEC, typename T>
__device__ __forceinline__ void store4(T* o, int n, const float (&v)[4]) {
  if constexpr (VEC) {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 q;
      T* h = reinterpret_cast<T*>(&q);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint2*>(o) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] = from_f32<T>(v[i]);
  }
}

// The larger of two values; NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest and sum of a lane's values, in two chains.
template <int N>
__device__ __forceinline__ float pairs_max(const f2 (&v)[N]) {
  float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a, b;
    f2_split(v[i], a, b);
    m[i & 1] = max_nan(m[i & 1], max_nan(a, b));
  }
  return max_nan(m[0], m[1]);
}
template <int N>
__device__ __forceinline__ float pairs_sum(const f2 (&v)[N]) {
  f2 a = v[0], b = v[1];
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    a = f2_add(a, v[i]);
    b = f2_add(b, v[i + 1]);
  }
  return f2_sum(f2_add(a, b));
}

// 2^x; below 2^-126 zero (FLUSH) or the subnormal
template <bool FLUSH>
__device__ __forceinline__ float pow2(float x) {
  float r;
  if constexpr (FLUSH)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// ln x for x >= 1 (a softmax's sum), to 2^-22
__device__ __forceinline__ float ln_sum(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r * 0.69314718055994530942f;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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
// sequences and may leave tokens before the first or after the last one in none.  The
// offsets around the range come into shared memory; every thread of the CTA walks along.
struct SeqWalk {
  static constexpr int WINDOW = BAL_SMALL;
  const int32_t* off;  // [G + 1], or null: one sequence of all tokens
  int* win;            // shared [WINDOW + 1]: offsets from off[base] on
  int G;
  int s;               // sequence of the current piece, or -1: in none
  int64_t a, b;        // the current piece [a, b)
  int64_t t1;
  int next_seq, base;

  __device__ __forceinline__ void fill() {
    __syncthreads();
    base = next_seq;
    for (int i = threadIdx.x; i <= WINDOW; i += blockDim.x)
      if (base + i <= G) win[i] = __ldg(off + base + i);
    __syncthreads();
  }
  __device__ __forceinline__ void start(const int32_t* off_, int* win_, int G_, int64_t t0,
                                        int64_t t1_) {
    off = off_;
    win = win_;
    G = G_;
    t1 = t1_;
    b = t0;
    s = 0;
    if (off == nullptr) return;
    next_seq = 0;
    if (G <= WINDOW) {  // all offsets fit: one trip to memory
      fill();
      const int i = threadIdx.x;
      next_seq = __syncthreads_count(i < G && win[i < G ? i + 1 : 0] <= t0);
      return;
    }
    // the first sequence that ends past t0: each round, the threads test as many
    // sequences at equal distances and leave one distance to search
    int lo = 0, n = G;  // it is in [lo, lo + n], lo + n = G: none
    while (n > 0) {
      const int threads = blockDim.x, d = (n + threads - 1) / threads;
      const int g = lo + static_cast<int>(threadIdx.x + 1) * d - 1;  // last of my distance
      const int before = __syncthreads_count(g < lo + n && __ldg(off + g + 1) <= t0);
      const int nlo = lo + before * d;
      n = d == 1 ? 0 : min(d - 1, lo + n - nlo);
      lo = nlo;
    }
    next_seq = min(lo, G);
    fill();
  }
  // false when the range is done
  __device__ __forceinline__ bool next() {
    a = b;
    if (a >= t1) return false;
    if (off == nullptr) {
      b = t1;
      return true;
    }
    for (; next_seq < G; ++next_seq) {
      if (next_seq - base >= WINDOW) fill();
      const int64_t lo = win[next_seq - base], 
                    hi = min(static_cast<int64_t>(win[next_seq - base + 1]), t1);
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

// e^(l - m) as 2^((l - m) log2(e)): the difference comes first, so that rows of the type's
// lowest value, whose product with log2(e) overflows, keep their (even) distribution.
constexpr float LOG2_E = 1.44269504088896340736f;
template <bool FLUSH, int N>
__device__ __forceinline__ void pairs_exp(f2 (&v)[N], float m) {
  const f2 nm = f2_make(-m, -m), s = f2_make(LOG2_E, LOG2_E);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a, b;
    f2_split(f2_mul(f2_add(v[i], nm), s), a, b);
    v[i] = f2_make(pow2<FLUSH>(a), pow2<FLUSH>(b));
  }
}

// Partial results of one (CTA, sequence) piece, at row CTA + sequence of each array
// (unique: the next piece has a larger CTA or a larger sequence).
struct BalParts {
  float* stats;   // [2]: sequences with a counting token, counting tokens
  float* p;       // [pieces, E]
  int32_t* cnt;   // [pieces, E]
  int32_t* n;     // [pieces]
  float* z;       // [pieces]
  float* seq_z;   // [G]
  float* dot;     // [G, expert blocks of the joining kernel]
  int* arrived;   // CTAs of the joining kernel that are done
  float* cta_f;   // [CTAs of balance_join_many_kernel, 2]: sums of sequence losses, of lse^2
  int* cta_n;     // [.., 2]: tokens, sequences with a token
};

// What the sequences of a thread, a CTA or the whole call add up to.
struct BalTotals {
  float sum, z;
  int n, live;
  __device__ __forceinline__ void add(float v, float zg, int ng) {
    sum += v;
    z += zg;
    n += ng;
    live += ng > 0 ? 1 : 0;
  }
  // the CTA's threads together (`one_warp`: the others have nothing), then the results
  __device__ __forceinline__ void finish(bool one_warp, const BalParts& parts, float* losses) {
    __shared__ float s_f[32][2];
    __shared__ int s_i[32][2];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    sum = warp_sum(sum);
    z = warp_sum(z);
    n = warp_sum(n);
    live = warp_sum(live);
    if (!one_warp) {
      if (lane == 0) {
        s_f[wid][0] = sum;
        s_f[wid][1] = z;
        s_i[wid][0] = n;
        s_i[wid][1] = live;
      }
      __syncthreads();
      const bool in = lane < static_cast<int>(blockDim.x) / 32;
      sum = warp_sum(in ? s_f[lane][0] : 0.f);
      z = warp_sum(in ? s_f[lane][1] : 0.f);
      n = warp_sum(in ? s_i[lane][0] : 0);
      live = warp_sum(in ? s_i[lane][1] : 0);
    }
    if (threadIdx.x == 0) {
      losses[0] = live > 0 ? sum / static_cast<float>(live) : 0.f;
      losses[1] = n > 0 ? z / static_cast<float>(n) : 0.f;
      parts.stats[0] = static_cast<float>(live);
      parts.stats[1] = static_cast<float>(n);
    }
  }
};
__device__ __forceinline__ float sequence_loss(float dot, int n, float per) {
  const float nf = static_cast<float>(n);
  return n > 0 ? dot * per / (nf * nf) : 0.f;
}

// Sequences up to which a single CTA gives the call's results by itself.  (One token makes one CTA
// at any G: with more sequences the joining launch writes their results.)
constexpr int BAL_ALONE_SEQS = 2;

// What the call returns.
struct BalOut {
  float* losses;     // [2]
  float* seq_loss;   // [G]
  int32_t* counts;   // [G, E]
  int32_t* tokens;   // [G]
};

// The tokens' pass: 131072 x 256 logits in 28 us of the call's 31, 0.73 of the copy rate; HBM and
// 59% of the issue slots.  In bf16, half the bytes, the call takes 26 us: bound by issue and by the
// chain of a token's reductions.
template <typename T, int L, int NV, bool VEC>
__global__ void __launch_bounds__(BAL_THREADS, NV >= 8 ? 1 : 2) balance_fwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, int64_t T_, int E, int k,
    int G, int chunk, float* __restrict__ lse_out, BalParts parts, BalOut out) {
  using R = Ring<T, L, NV, VEC>;
  const int nt = blockDim.x, warps = nt / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  float* s_p = reinterpret_cast<float*>(smem + R::BYTES * nt);  // [warps][E]
  int* s_cnt = reinterpret_cast<int*>(s_p + warps * E);  // [E]
  __shared__ float s_z[BAL_WARPS], s_dot[BAL_WARPS];
  __shared__ int s_n[BAL_WARPS];
  __shared__ int s_win[SeqWalk::WINDOW + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int l = lane % L;  // lane within its token's group
  const int GROUPS = nt / L;
  const int grp = tid / L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = min(T_, t0 + chunk);
  R ring;
  ring.init(smem, l, E, k);
  const bool alone = gridDim.x == 1 && G <= BAL_ALONE_SEQS;  // (then its results are the call's)
  const float per = static_cast<float>(E) / static_cast<float>(k);
  BalTotals all{};
  if (blockIdx.x == 0 && tid == 0) *parts.arrived = 0;
  for (int e = tid; e < E; e += nt) s_cnt[e] = 0;
  if (alone && off != nullptr)  // sequences without tokens
    for (int i = tid; i < G * (E + 1); i += nt) {
      if (i < G) {
        out.seq_loss[i] = 0.f;
        out.tokens[i] = 0;
      } else {
        out.counts[i - G] = 0;
      }
    }
  __syncthreads();
  SeqWalk w;
  w.start(off, s_win, G, t0, t1);
  while (w.next()) {
    if (w.s < 0) {  // tokens in no sequence
      for (int64_t t = w.a + tid; t < w.b; t += nt) lse_out[t] = 0.f;
      continue;
    }
    f2 acc[2 * NV] = {};
    float z = 0.f;
    int n = 0;
    MaskAhead<L> ahead;
    // rounds of the CTA, and those in which this group has a token
    const int len = static_cast<int>(w.b - w.a), rounds = (len + GROUPS - 1) / GROUPS;
    const int mine = grp < len ? (len - 1 - grp) / GROUPS + 1 : 0;
    const int64_t first = w.a + grp;
    const T* row = logits + first * E + 4 * l;   // of the token to copy next
    const int32_t* idx = topk_idx + first * k + l;
    const int64_t row_step = static_cast<int64_t>(GROUPS) * E, idx_step = static_cast<int64_t>(GROUPS) * k;
    int left = mine;
    const auto issue = [&](int st) {
      if (left > 0) {  // (a masked row is read like any other: no load waits for another)
        ring.load(st, row);
        ring.load_idx(st, idx);
      }
      R::commit();
      --left;
      row += row_step;
      idx += idx_step;
    };
#pragma unroll
    for (int i = 0; i < BAL_STAGES - 1; ++i) issue(i);
    float* lse_at = lse_out + first;
    const uint8_t* mask_at = mask != nullptr ? mask + first : nullptr;
    int st = 0;
    for (int it = 0; it < rounds; ++it) {
      issue(st == 0 ? BAL_STAGES - 1 : st - 1);
      bool on = it < mine;
      if (mask != nullptr) {
        on = ahead.get(mask_at, GROUPS, l, it, mine - it) && on;
        mask_at += GROUPS;
      }
      R::wait();
      f2 v[2 * NV];
      ring.get(st, v);
      const float m = lanes_max<L>(pairs_max(v));
      on = on && m != -INFINITY;  // (a NaN counts, and shows in the losses)
      pairs_exp<true>(v, m);
      const float sum = lanes_sum<L>(pairs_sum(v));
      if (on) {
        const float inv = reciprocal(sum);
        const f2 inv2 = f2_make(inv, inv);
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) acc[i] = f2_fma(v[i], inv2, acc[i]);
#pragma unroll
        for (int j = 0; j < R::KS; ++j) {
          const int e = l + j * L < k ? ring.slot(st, j) : -1;
          if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(s_cnt + e, 1);
        }
        if (k > R::KS * L) {
          const int32_t* rest = topk_idx + (first + static_cast<int64_t>(it) * GROUPS) * k;
          for (int j = l + R::KS * L; j < k; j += L) {
            const int e = __ldg(rest + j);
            if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(s_cnt + e, 1);
          }
        }
      }
      if (l == 0 && it < mine) {
        const float lse = on ? m + ln_sum(sum) : 0.f;
        *lse_at = lse;
        z = fmaf(lse, lse, z);
        n += on ? 1 : 0;
      }
      lse_at += GROUPS;
      st = st + 1 == BAL_STAGES ? 0 : st + 1;
    }
    R::drain();
    // join the groups of the warp, then the warps (in order)
    z = warp_sum(z);
    n = warp_sum(n);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float q[4];
      f2_split(acc[2 * i], q[0], q[1]);
      f2_split(acc[2 * i + 1], q[2], q[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 16; o >= L; o >>= 1) q[j] += __shfl_xor_sync(0xffffffffu, q[j], o);
        const int e = 4 * (l + i * L) + j;
        if (lane < L && e < E) s_p[wid * E + e] = q[j];
      }
    }
    if (lane == 0) {
      s_z[wid] = z;
      s_n[wid] = n;
    }
    __syncthreads();
    const int64_t piece = static_cast<int64_t>(blockIdx.x) + w.s;
    int32_t* cnt_at = alone ? out.counts + static_cast<int64_t>(w.s) * E : parts.cnt + piece * E;
    float dot = 0.f;
    for (int e = tid; e < E; e += nt) {
      float t = s_p[e];
#pragma unroll 4
      for (int i = 1; i < warps; ++i) t += s_p[i * E + e];
      if (!alone) parts.p[piece * E + e] = t;
      cnt_at[e] = s_cnt[e];
      dot = fmaf(static_cast<float>(s_cnt[e]), t, dot);
      s_cnt[e] = 0;
    }
    if (alone) {
      dot = warp_sum(dot);
      if (lane == 0) s_dot[wid] = dot;
      __syncthreads();
    }
    if (tid == 0) {
      float tz = 0.f;
      int tn = 0;
      for (int i = 0; i < warps; ++i) {
        tz += s_z[i];
        tn += s_n[i];
      }
      if (alone) {
        for (int i = 1; i < warps; ++i) dot += s_dot[i];
        const float v = sequence_loss(dot, tn, per);
        out.seq_loss[w.s] = v;
        out.tokens[w.s] = tn;
        all.add(v, tz, tn);
      } else {
        parts.z[piece] = tz;
        parts.n[piece] = tn;
      }
    }
    __syncthreads();
  }
  if (alone && wid == 0) all.finish(true, parts, out.losses);
}

// ---------------------------------------------------------------- joining the pieces
// The CTAs whose tokens sequence g reaches: [c0, c1).
struct PieceRange {
  uint32_t c0, c1;
  __device__ __forceinline__ PieceRange(const int32_t* off, int g, int64_t T_, int chunk) {
    const int n = static_cast<int>(T_), a = off != nullptr ? max(0, __ldg(off + g)) : 0;
    const int b = off != nullptr ? min(n, __ldg(off + g + 1)) : n;
    c0 = static_cast<uint32_t>(a) / static_cast<uint32_t>(chunk);
    c1 = b > a ? static_cast<uint32_t>(b - 1) / static_cast<uint32_t>(chunk) + 1 : c0;
  }
};

// Counts a CTA (whose results thread 0 wrote) in; true in all threads of the last one, with
// the others' results visible.  What is then added, and in which order, does not depend on
// which CTA that is.
__device__ __forceinline__ bool last_cta(int* arrived) {
  __shared__ int s_before;
  if (threadIdx.x == 0) {
    int before = 0;
    if (gridDim.x > 1)
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                   : "=r"(before)
                   : "l"(arrived)
                   : "memory");
    s_before = before;
  }
  __syncthreads();
  return s_before == static_cast<int>(gridDim.x) - 1;
}

// Few sequences: a CTA per sequence and 32 experts; its warps take every 32nd piece, ten
// loads of each kind in flight.
constexpr int JOIN_THREADS = 1024;
constexpr int JOIN_WARPS = JOIN_THREADS / 32;
__global__ void __launch_bounds__(JOIN_THREADS, 1) balance_join_few_kernel(
    const int32_t* __restrict__ off, int64_t T_, int E, int k, int G, int chunk, BalParts parts,
    BalOut out) {
  constexpr int BATCH = 10;
  __shared__ float s_p[JOIN_WARPS][33], s_z[JOIN_WARPS];
  __shared__ int s_c[JOIN_WARPS][33], s_n[JOIN_WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int blocks = (E + 31) / 32;
  const int g = blockIdx.x / blocks, eb = blockIdx.x - g * blocks;
  const int e = eb * 32 + lane;
  const PieceRange r(off, g, T_, chunk);
  float p = 0.f, z = 0.f;
  int cnt = 0, n = 0;
  // (the first of these loads are in flight beside the pieces' own)
  const uint32_t cz = r.c0 + threadIdx.x;
  const bool first = eb == 0 && cz < r.c1;
  const float z0 = first ? __ldcg(parts.z + cz + g) : 0.f;
  const int n0 = first ? __ldcg(parts.n + cz + g) : 0;
  if (e < E) {
    const int64_t at = static_cast<int64_t>(r.c0 + wid + g) * E + e;
    const float* pp = parts.p + at;
    const int32_t* pc = parts.cnt + at;
    const int step = JOIN_WARPS * E;
    for (uint32_t c = r.c0 + wid; c < r.c1; c += BATCH * JOIN_WARPS) {
      float fp[BATCH];
      int fc[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i, pp += step, pc += step) {
        const bool in = c + i * JOIN_WARPS < r.c1;
        fp[i] = in ? __ldcg(pp) : 0.f;
        fc[i] = in ? __ldcg(pc) : 0;
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        p += fp[i];
        cnt += fc[i];
      }
    }
  }
  s_p[wid][lane] = p;
  s_c[wid][lane] = cnt;
  if (eb == 0) {
    z = z0;
    n = n0;
#pragma unroll 1
    for (uint32_t c = cz + JOIN_THREADS; c < r.c1; c += JOIN_THREADS) {
      z += __ldcg(parts.z + c + g);
      n += __ldcg(parts.n + c + g);
    }
    z = warp_sum(z);
    n = warp_sum(n);
    if (lane == 0) {
      s_z[wid] = z;
      s_n[wid] = n;
    }
  }
  __syncthreads();
  // a warp per expert: lanes are the pieces' warps
  p = warp_sum(s_p[lane][wid]);
  cnt = warp_sum(s_c[lane][wid]);
  if (eb == 0 && wid == 0) {
    z = warp_sum(s_z[lane]);
    n = warp_sum(s_n[lane]);
  }
  __syncthreads();
  if (lane == 0) {
    s_p[0][wid] = static_cast<float>(cnt) * p;
    if (eb * 32 + wid < E) out.counts[static_cast<int64_t>(g) * E + eb * 32 + wid] = cnt;
  }
  __syncthreads();
  if (wid == 0) {
    const float dot = warp_sum(s_p[0][lane]);
    if (lane == 0) {
      parts.dot[blockIdx.x] = dot;
      if (eb == 0) {
        parts.seq_z[g] = z;
        out.tokens[g] = n;
      }
    }
  }
  if (!last_cta(parts.arrived)) return;
  const float per = static_cast<float>(E) / static_cast<float>(k);
  BalTotals all{};
  for (int i = threadIdx.x; i < G; i += JOIN_THREADS) {
    const int ni = __ldcg(out.tokens + i);
    const float zi = __ldcg(parts.seq_z + i);
    const float* dots = parts.dot + static_cast<int64_t>(i) * blocks;
    float q[4];  // (beside the loads above)
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = j < blocks ? __ldcg(dots + j) : 0.f;
    float d = (q[0] + q[1]) + (q[2] + q[3]);
    for (int j = 4; j < blocks; ++j) d += __ldcg(dots + j);
    const float v = sequence_loss(d, ni, per);
    out.seq_loss[i] = v;
    all.add(v, zi, ni);
  }
  all.finish(G <= 32, parts, out.losses);
}

// Many sequences, with few pieces each: a CTA of up to 8 warps takes a sequence at a time, an
// expert a thread, eight pieces at once.
constexpr int JOIN_MANY_THREADS = 256;
constexpr int JOIN_MANY_CTAS = 152 * 4;
__global__ void __launch_bounds__(JOIN_MANY_THREADS) balance_join_many_kernel(
    const int32_t* __restrict__ off, int64_t T_, int E, int k, int G, int chunk, BalParts parts,
    BalOut out) {
  constexpr int BATCH = 8;
  __shared__ float s_dot[JOIN_MANY_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nt = blockDim.x;
  const float per = static_cast<float>(E) / static_cast<float>(k);
  BalTotals mine{};
  for (int g = blockIdx.x; g < G; g += gridDim.x) {
    const PieceRange r(off, g, T_, chunk);
    float dot = 0.f, z = 0.f;
    int n = 0;
    if (wid == 0 && r.c0 + lane < r.c1) {
      z = __ldcg(parts.z + r.c0 + lane + g);
      n = __ldcg(parts.n + r.c0 + lane + g);
    }
    for (int e = threadIdx.x; e < E; e += nt) {
      float p = 0.f;
      int cnt = 0;
      const int64_t at = static_cast<int64_t>(r.c0 + g) * E + e;
      const float* pp = parts.p + at;
      const int32_t* pc = parts.cnt + at;
      for (uint32_t c = r.c0; c < r.c1; c += BATCH) {
        float fp[BATCH];
        int fc[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i, pp += E, pc += E) {
          const bool in = c + i < r.c1;
          fp[i] = in ? __ldcg(pp) : 0.f;
          fc[i] = in ? __ldcg(pc) : 0;
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          p += fp[i];
          cnt += fc[i];
        }
      }
      out.counts[static_cast<int64_t>(g) * E + e] = cnt;
      dot = fmaf(static_cast<float>(cnt), p, dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) s_dot[wid] = dot;
    if (wid == 0) {
#pragma unroll 1
      for (uint32_t c = r.c0 + 32 + lane; c < r.c1; c += 32) {
        z += __ldcg(parts.z + c + g);
        n += __ldcg(parts.n + c + g);
      }
      z = warp_sum(z);
      n = warp_sum(n);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < nt / 32; ++i) dot += s_dot[i];
      const float v = sequence_loss(dot, n, per);
      out.tokens[g] = n;
      out.seq_loss[g] = v;
      mine.add(v, z, n);
    }
    __syncthreads();  // (s_dot is read)
  }
  if (threadIdx.x == 0) {
    parts.cta_f[2 * blockIdx.x] = mine.sum;
    parts.cta_f[2 * blockIdx.x + 1] = mine.z;
    parts.cta_n[2 * blockIdx.x] = mine.n;
    parts.cta_n[2 * blockIdx.x + 1] = mine.live;
  }
  if (!last_cta(parts.arrived)) return;
  BalTotals all{};
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += nt) {
    all.sum += __ldcg(parts.cta_f + 2 * i);
    all.z += __ldcg(parts.cta_f + 2 * i + 1);
    all.n += __ldcg(parts.cta_n + 2 * i);
    all.live += __ldcg(parts.cta_n + 2 * i + 1);
  }
  all.finish(false, parts, out.losses);
}

// The gradient: the softmax again, one read and one write; 131072 x 256 in 45.3 us, 0.87 of the
// copy rate; in bf16 24.1 us, 0.82.  (Above 512 experts in fp32 one register is spilled.)
template <typename T, int L, int NV, bool VEC>
__global__ void __launch_bounds__(BAL_THREADS, NV >= 8 ? 1 : 2) balance_bwd_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ off,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, const float* __restrict__ stats,
    const float* __restrict__ dlosses, int64_t T_, int E, int k, int G, int chunk,
    T* __restrict__ dlogits) {
  using R = Ring<T, L, NV, VEC>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int s_win[SeqWalk::WINDOW + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int l = lane % L;
  const int GROUPS = blockDim.x / L;
  const int grp = tid / L;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = min(T_, t0 + chunk);
  R ring;
  ring.init(smem, l, E, 0);
  const float live = __ldg(stats), n_all = __ldg(stats + 1);
  const float db = __ldg(dlosses);
  const float dz = n_all > 0.f ? __ldg(dlosses + 1) * 2.f / n_all : 0.f;
  SeqWalk w;
  w.start(off, s_win, G, t0, t1);
  while (w.next()) {
    MaskAhead<L> ahead;
    const int len = static_cast<int>(w.b - w.a), rounds = (len + GROUPS - 1) / GROUPS;
    const int mine = grp < len ? (len - 1 - grp) / GROUPS + 1 : 0;
    const int64_t first = w.a + grp, row_step = static_cast<int64_t>(GROUPS) * E;
    const T* row = logits + first * E + 4 * l;
    int left = mine;
    const auto issue = [&](int st) {
      if (left > 0) ring.load(st, row);
      R::commit();
      --left;
      row += row_step;
    };
#pragma unroll
    for (int i = 0; i < BAL_STAGES - 1; ++i) issue(i);
    T* out = dlogits + first * E + 4 * l;
    const uint8_t* mask_at = mask != nullptr ? mask + first : nullptr;
    f2 c[2 * NV];
    const float ns = w.s >= 0 ? static_cast<float>(__ldg(tokens + w.s)) : 0.f;
    const float scale =
        ns > 0.f ? db * (static_cast<float>(E) / static_cast<float>(k)) / (ns * ns * live) : 0.f;
    const auto coef = [&](int e) {
      return w.s >= 0 && e < E
                 ? scale * static_cast<float>(__ldg(counts + static_cast<int64_t>(w.s) * E + e))
                 : 0.f;
    };
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) {
      const int e = 4 * (l + i / 2 * L) + i % 2 * 2;
      c[i] = f2_make(coef(e), coef(e + 1));
    }
    int st = 0;
    for (int it = 0; it < rounds; ++it, out += row_step) {
      issue(st == 0 ? BAL_STAGES - 1 : st - 1);
      bool on = it < mine && ns > 0.f;
      if (mask != nullptr) {
        on = ahead.get(mask_at, GROUPS, l, it, mine - it) && on;
        mask_at += GROUPS;
      }
      R::wait();
      f2 v[2 * NV];
      ring.get(st, v);
      const float m = lanes_max<L>(pairs_max(v));
      on = on && m != -INFINITY;
      pairs_exp<false>(v, m);
      const float sum = lanes_sum<L>(pairs_sum(v));
      f2 dot2 = 0;
#pragma unroll
      for (int i = 0; i < 2 * NV; ++i) dot2 = f2_fma(v[i], c[i], dot2);
      const float dot = lanes_sum<L>(f2_sum(dot2));
      const float inv = reciprocal(sum);
      const float shift = dz * (m + ln_sum(sum)) - dot * inv;
      const f2 inv2 = f2_make(inv, inv), shift2 = f2_make(shift, shift);
      if (it < mine) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float d[4] = {};
          if (on) {
            f2_split(f2_mul(f2_mul(v[2 * i], inv2), f2_add(c[2 * i], shift2)), d[0], d[1]);
            f2_split(f2_mul(f2_mul(v[2 * i + 1], inv2), f2_add(c[2 * i + 1], shift2)), d[2], d[3]);
          }
          store4<VEC>(out + 4 * i * L, E - 4 * (l + i * L), d);
        }
      }
      st = st + 1 == BAL_STAGES ? 0 : st + 1;
    }
    R::drain();
  }
}

// The split of T tokens over CTAs, and the workspace's arrays.
struct BalPlan {
  int threads, chunk, nb;
  size_t stats, arrived, seq_z, dot, cta_f, cta_n, n, z, cnt, p, bytes;
};

// Lanes per token (L) and 4-element vectors per lane (NV) by the number of experts.
static int bal_lanes(int E) {
  return E <= 8 ? 2 : E <= 16 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : 32;
}

static BalPlan bal_plan(int64_t T, int E, int G, bool forward) {
  BalPlan b{};
  // (131072 tokens, 128 experts: 4096 sequences 83.8 us forward in large CTAs, 52.4 in small
  // ones; one sequence 22.3 and 25.4)
  b.threads = T / G < 1024 && G > 152 ? BAL_SMALL : BAL_THREADS;
  // (above 512 experts the registers allow one large CTA on an SM)
  const int ctas = 152 * (E <= 512 ? 2 : 1) * (BAL_THREADS / b.threads);
  const int groups = b.threads / bal_lanes(E);
  const int64_t per = (T + ctas - 1) / ctas;
  b.chunk = static_cast<int>((per + groups - 1) / groups * groups);
  // a CTA takes its sequences one after the other: where whole rounds of it would hold
  // several, and there are CTAs to spare, about one each
  if (b.chunk > T / G) b.chunk = static_cast<int>(std::max(per, T / G));
  // few tokens: one CTA takes them all and no launch follows (us, two launches and one: 64 x 8
  // 5.1 and 3.0, 192 x 128 6.4 and 5.7, 288 x 128 6.3 and 6.9; two sequences in 64 x 128 9.1
  // and 7.2, three in 128 x 128 9.2 and 9.6).  Gradients have no second launch to save.
  if (forward && T <= static_cast<int64_t>(std::max(0, 6 - 2 * G)) * groups)
    b.chunk = static_cast<int>(T);
  b.nb = static_cast<int>((T + b.chunk - 1) / b.chunk);
  const size_t pieces = static_cast<size_t>(b.nb) + G;
  const auto take = [&](size_t bytes) {
    const size_t at = b.bytes;
    b.bytes += (bytes + 255) / 256 * 256;
    return at;
  };
  b.stats = take(8);
  b.arrived = take(4);
  b.cta_f = take(8 * JOIN_MANY_CTAS);
  b.cta_n = take(8 * JOIN_MANY_CTAS);
  b.dot = take(4 * static_cast<size_t>(G) * ((E + 31) / 32));
  b.seq_z = take(4 * static_cast<size_t>(G));
  b.n = take(4 * pieces);
  b.z = take(4 * pieces);
  b.cnt = take(4 * pieces * E);
  b.p = take(4 * pieces * E);
  return b;
}

static BalParts bal_parts(const BalPlan& b, void* ws) {
  char* p = static_cast<char*>(ws);
  return BalParts{reinterpret_cast<float*>(p + b.stats),  reinterpret_cast<float*>(p + b.p),
                  reinterpret_cast<int32_t*>(p + b.cnt),  reinterpret_cast<int32_t*>(p + b.n),
                  reinterpret_cast<float*>(p + b.z),      reinterpret_cast<float*>(p + b.seq_z),
                  reinterpret_cast<float*>(p + b.dot),    reinterpret_cast<int*>(p + b.arrived),
                  reinterpret_cast<float*>(p + b.cta_f),  reinterpret_cast<int*>(p + b.cta_n)};
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
  if (E <= 8) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (E <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
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
  *bytes = bal_plan(shape->T, static_cast<int>(shape->E), static_cast<int>(shape->G), false).bytes;
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
  const BalPlan b = bal_plan(shape->T, E, G, true);
  const BalParts parts = bal_parts(b, workspace);
  const BalOut out{losses, seq_loss, counts, tokens};
  prof_begin(c, K_BALANCE_FWD);
  cudaError_t e = with_dtype(shape->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const T* lg = static_cast<const T*>(logits);
    return with_lanes(E, [&](auto l, auto nv) {
      constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
      auto* kern = bal_vec<T>(lg, E) ? balance_fwd_kernel<T, L, NV, true>
                                     : balance_fwd_kernel<T, L, NV, false>;
      const size_t smem = static_cast<size_t>(Ring<T, L, NV, true>::BYTES) * b.threads +
                          static_cast<size_t>(b.threads / 32 + 1) * E * 4;
      const cudaError_t r = allow_smem(kern, smem);
      if (r != cudaSuccess) return r;
      return launch_k(c.stream, kern, dim3(b.nb), dim3(b.threads), smem, lg, topk_idx,
                      seq_offsets, mask, shape->T, E, k, G, b.chunk, lse, parts, out);
    });
  });
  prof_end(c, K_BALANCE_FWD);
  if (e != cudaSuccess) return op_status(e);
  if (b.nb == 1 && G <= BAL_ALONE_SEQS) return MM_MOE_OK;
  // The first kernel where a sequence has many pieces and all its CTAs run at once (us, first
  // and second: 131072 x 128 16 sequences, 19 pieces each, 21.3 and 23.7, 64 sequences, 5
  // pieces, 26.0 and 23.1; 32768 x 256 in 32, 256 CTAs, 19.8 and 17.6; one sequence, whose
  // second kernel is one CTA with no other to wait for, 21 pieces 7.0 and 6.4)
  const int64_t units = static_cast<int64_t>(G) * ((E + 31) / 32);
  const bool few = G == 1 ? b.nb > 24 : b.nb > 6 * static_cast<int64_t>(G) && units <= sms;
  prof_begin(c, K_BALANCE_FINISH);
  e = launch_k(c.stream, few ? balance_join_few_kernel : balance_join_many_kernel,
               dim3(static_cast<unsigned>(few ? units : std::min(G, JOIN_MANY_CTAS))),
               dim3(few ? JOIN_THREADS : std::min(JOIN_MANY_THREADS, (E + 31) / 32 * 32)), 0,
               seq_offsets, shape->T, E, k, G, b.chunk, parts, out);
  prof_end(c, K_BALANCE_FINISH);
  return op_status(e);
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
  const auto lg_at = reinterpret_cast<uintptr_t>(logits), d_at = reinterpret_cast<uintptr_t>(dlogits);
  const uintptr_t size = static_cast<uintptr_t>(shape->T) * shape->E * es;
  if (d_at < lg_at + size && lg_at < d_at + size) return MM_MOE_EINVAL;
  const int sms = sm_count_103();
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int E = static_cast<int>(shape->E), k = static_cast<int>(shape->k),
            G = static_cast<int>(shape->G);
  const BalPlan b = bal_plan(shape->T, E, G, false);
  const float* stats = bal_parts(b, const_cast<void*>(workspace)).stats;
  prof_begin(c, K_BALANCE_BWD);
  const cudaError_t e = with_dtype(shape->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const T* lg = static_cast<const T*>(logits);
    T* out = static_cast<T*>(dlogits);
    return with_lanes(E, [&](auto l, auto nv) {
      constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
      auto* kern = bal_vec<T>(lg, E) && bal_vec<T>(out, E) ? balance_bwd_kernel<T, L, NV, true>
                                                           : balance_bwd_kernel<T, L, NV, false>;
      const size_t smem = static_cast<size_t>(Ring<T, L, NV, true>::BYTES) * b.threads;
      const cudaError_t r = allow_smem(kern, smem);
      if (r != cudaSuccess) return r;
      return launch_k(c.stream, kern, dim3(b.nb), dim3(b.threads), smem, lg, seq_offsets, mask,
                      counts, tokens, stats, dlosses, shape->T, E, k, G, b.chunk, out);
    });
  });
  prof_end(c, K_BALANCE_BWD);
  return op_status(e);
}
