// norm.cuh -- layer normalisation: what its forward (norm.cu) and its backward (norm_bwd.cu)
// share, the rows' way through a CTA and the checks of the arguments.
//
//   mu = 1/H sum_i x_i,  var = 1/H sum_i (x_i - mu)^2,  r = (var + eps)^(-1/2)
//   xh = (x - mu) r,     y = w xh + b
//   g = w dy,            dx = r (g - mean(g) - xh mean(g xh)) [+ dx_add]
//   dw = sum_t dy xh,    db = sum_t dy
//
// x, y, dy, dx are bf16, fp16 or fp32; everything is computed in fp32 and rounded once
// where it is stored.  The variance is taken from the centred values (a second pass
// over the row), never as a difference of moments.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "internal.h"
#include "ops.cuh"

namespace mmmoe {

// One row operand: base pointer and elements from one row to the next.
template <typename T>
struct Rows {
  T* p;
  int64_t ld;
  __device__ __forceinline__ T* row(int64_t t) const { return p + t * ld; }
};

// The elements of 16 bytes as fp32 pairs, and back.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4& q, f2 (&v)[VN<T> / 2]) {
  float f[VN<T>];
  unpack(q, f, static_cast<const T*>(nullptr));
#pragma unroll
  for (int i = 0; i < VN<T> / 2; ++i) v[i] = f2_make(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const f2 (&v)[VN<T> / 2]) {
  float f[VN<T>];
#pragma unroll
  for (int i = 0; i < VN<T> / 2; ++i) f2_split(v[i], f[2 * i], f[2 * i + 1]);
  return pack(f, static_cast<const T*>(nullptr));
}

// ---------------------------------------------------------------- rows over a group
// Both passes split a CTA into groups of GT threads (a power of two up to 32, or whole
// warps); a group takes every gridDim * groups-th row.  A row is cut into units of 16
// bytes at the 16-byte boundaries of memory, so its first unit may begin up to 15 bytes in
// front of the row (of the row before it: read, and masked) and its last one may end past it
// (copied with a shorter source size).  The cut repeats every 8 rows at most, and a grid
// of more than one round has a multiple of 8 CTAs, so a group sees the same cut in all
// its rows and each of its threads the same columns: unit j + i GT, i < NU.
//
// Units come through a ring in shared memory, S - 1 rows ahead, by cp.async: a thread
// copies its own units and reads nothing but what it copied, so no barrier guards the ring.
constexpr int NORM_THREADS = 512;

// Steps of ROWS rows in the ring: 64 to 192 KB of it.
template <int NU, int ROWS>
constexpr int norm_fwd_steps = ROWS == 2 ? 3 : NU <= 4 ? 4 : NU <= 5 ? 3 : 2;
template <int NU, bool ADD, int ROWS>
constexpr int norm_bwd_steps = (NU <= 2 ? 4 : 2) / ROWS + (NU <= 2 && !ADD && ROWS == 2 ? 1 : 0);
// Parameters stay in registers up to 16 columns a thread, else in shared memory.
template <typename T, int NU>
constexpr bool norm_params_shared = NU * VN<T> > 16;

__device__ __forceinline__ void async_copy(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copy(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ ulonglong2 lds16_f2(uint32_t a) {
  ulonglong2 v;
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds8(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16_zero(uint32_t a) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
}
__device__ __forceinline__ void group_bar(int g, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(threads) : "memory");
}

// What a row is like: ANY; whole units (EVEN: it starts and ends on a 16-byte boundary, so
// nothing is masked or cut short); FULL: whole units, NU of them for every thread.
enum Cut { ANY, EVEN, FULL };

// A thread's place: its group and its columns.
template <typename T, int NU, Cut CUT>
struct Place {
  static constexpr int U = VN<T>;
  int GT, g, j, groups, H;
  int shift;  // elements the row's first unit begins in front of the row
  int units;
  __device__ __forceinline__ void init(int GT_, int H_) {
    GT = GT_;
    H = H_;
    g = threadIdx.x / GT;
    j = threadIdx.x - g * GT;
    groups = blockDim.x / GT;
  }
  // the first row of the warp's groups (they loop together)
  __device__ __forceinline__ uint32_t first_of_warp(uint32_t t) const {
    return GT < 32 ? t - (g & (32 / GT - 1)) : t;
  }
  template <typename V>
  __device__ __forceinline__ void cut(const Rows<V>& r, int64_t t) {
    shift = CUT != ANY ? 0
                       : static_cast<int>((reinterpret_cast<uintptr_t>(r.p + t * r.ld) & 15) / sizeof(T));
    units = CUT != ANY ? H / U : (H + shift + U - 1) / U;
  }
  // first column of unit i (may be negative, or past the row)
  __device__ __forceinline__ int col(int i) const { return (j + i * GT) * U - shift; }
  __device__ __forceinline__ bool has(int i) const { return CUT == FULL || j + i * GT < units; }
  // the whole unit lies in the row
  __device__ __forceinline__ bool whole(int i) const {
    return CUT != ANY ? has(i) : col(i) >= 0 && col(i) + U <= H;
  }
  __device__ __forceinline__ bool in(int c) const { return c >= 0 && c < H; }
  // The thread's first unit of a row (unit i lies i GT units further on).
  template <typename V>
  __device__ __forceinline__ V* at(const Rows<V>& r, int64_t t) const {
    return r.p + t * r.ld + col(0);
  }
  // unit i of the row whose first unit of this thread is at p; what lies past the row
  // arrives as zero
  __device__ __forceinline__ void copy(uint32_t slot, const T* p, int i) const {
    if constexpr (CUT != ANY)
      async_copy(slot, p + i * GT * U);
    else
      async_copy(slot, p + i * GT * U, min(U, H - col(i)) * static_cast<int>(sizeof(T)));
  }
  // zero in front of the row
  __device__ __forceinline__ void mask(uint4& q, int i) const {
    if (CUT != ANY || i != 0) return;
    if (j == 0 && shift != 0) {
      T* h = reinterpret_cast<T*>(&q);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k < shift) h[k] = from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void store(T* p, int i, const uint4& q) const {
    T* o = p + i * GT * U;
    if (whole(i)) {
      *reinterpret_cast<uint4*>(o) = q;
    } else if constexpr (CUT == ANY) {
      const T* h = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (in(col(i) + k)) o[k] = h[k];
    }
  }
  // parameters of the thread's columns as pairs, zero outside the row
  template <typename P>
  __device__ __forceinline__ void params(const P* p, f2 (&v)[NU * U / 2]) const {
    if constexpr (CUT != ANY) {
      if (p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {  // whole vectors
        constexpr int N = VN<P> < U ? VN<P> : U;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int k = 0; k < U; k += N) {
            f2 t[VN<P> / 2] = {};
            if (has(i)) unpack2<P>(__ldg(reinterpret_cast<const uint4*>(p + col(i) + k)), t);
#pragma unroll
            for (int q = 0; q < N / 2; ++q) v[(i * U + k) / 2 + q] = t[q];
          }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int k = 0; k < U; k += 2) {
        const int c = col(i) + k;
        const float a = p != nullptr && in(c) ? to_f32(p[c]) : 0.f;
        const float b = p != nullptr && in(c + 1) ? to_f32(p[c + 1]) : 0.f;
        v[(i * U + k) / 2] = f2_make(a, b);
      }
  }
  // f(column, value) for the thread's pairs of values, inside the row
  template <typename F>
  __device__ __forceinline__ void each(const f2 (&v)[NU * U / 2], F f) const {
#pragma unroll
    for (int k = 0; k < NU * U / 2; ++k) {
      const int c = col(2 * k / U) + 2 * k % U;
      float lo, hi;
      f2_split(v[k], lo, hi);
      if (in(c)) f(c, lo);
      if (in(c + 1)) f(c + 1, hi);
    }
  }
};

// Sums over a group, the same in each of its threads: within a warp by shuffles, across
// a group's warps through s (one entry per warp of the CTA, not in use from an earlier sum),
// added in order after one barrier.
__device__ __forceinline__ float lanes_sum(float v, int GT) {
  if (GT >= 32) return warp_sum(v);
  for (int o = GT >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int N>
struct alignas(4 * N) Sums {  // one shared-memory access
  float v[N];
};
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], Sums<N>* s, int g, int GT) {
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = lanes_sum(v[q], GT);
  if (GT <= 32) return;
  const int gw = GT >> 5;
  if ((threadIdx.x & 31) == 0) {
    Sums<N> mine;
#pragma unroll
    for (int q = 0; q < N; ++q) mine.v[q] = v[q];
    s[threadIdx.x >> 5] = mine;
  }
  group_bar(g, GT);
  s += g * gw;
  Sums<N> t = s[0];
  for (int i = 1; i < gw; ++i) {
    const Sums<N> o = s[i];
#pragma unroll
    for (int q = 0; q < N; ++q) t.v[q] += o.v[q];
  }
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = t.v[q];
}

// --------------------------------------------------------------- looped, any width
// For rows that no CTA holds in its ring, and operands whose rows are cut differently.  VEC:
// every row is whole 16-byte units and the parameters lie on 16-byte boundaries; else
// element by element.
constexpr int LOOP_THREADS = 512;
template <typename T, bool VEC>
constexpr int loop_unit = VEC ? VN<T> : 1;

template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* p, int u, float (&f)[loop_unit<T, VEC>]) {
  if constexpr (VEC)
    unpack(reinterpret_cast<const uint4*>(p)[u], f, p);
  else
    f[0] = to_f32(p[u]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* p, int u, const float (&f)[loop_unit<T, VEC>]) {
  if constexpr (VEC)
    reinterpret_cast<uint4*>(p)[u] = pack(f, p);
  else
    p[u] = from_f32<T>(f[0]);
}
// U parameters from column c on
template <typename P, int U>
__device__ __forceinline__ void load_params(const P* p, int c, float (&f)[U]) {
  if constexpr (U == 1) {
    f[0] = to_f32(p[c]);
  } else {
    constexpr int N = VN<P> < U ? VN<P> : U;  // (fp32 parameters of 16-bit rows: two loads)
#pragma unroll
    for (int i = 0; i < U; i += N) {
      float t[VN<P>];
      unpack(__ldg(reinterpret_cast<const uint4*>(p + c + i)), t, p);
#pragma unroll
      for (int j = 0; j < N; ++j) f[i + j] = t[j];
    }
  }
}

// ------------------------------------------------------------------------ host side
// Rows of partial column sums a backward of T rows writes at most (the workspace's size).
constexpr int NORM_MAX_PARTS = 152 * 2;
inline int norm_parts(int64_t T) { return static_cast<int>(std::min<int64_t>(T, NORM_MAX_PARTS)); }

inline bool norm_shape_ok(const mm_moe_norm_shape* s) {
  return s != nullptr && s->T >= 1 && s->T < (int64_t{1} << 31) && s->H >= 1 &&
         s->H <= (1 << 20) && dtype_ok(s->dtype) &&
         (s->param_dtype == s->dtype || s->param_dtype == MM_MOE_DT_F32) && s->eps >= 0.f;
}

// aligned to its element, and (rows) a stride of at least the row
inline bool rows_ok(const void* p, int64_t ld, const mm_moe_norm_shape* s) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % dtype_bytes(s->dtype) == 0 &&
         (ld >= s->H || s->T == 1) && ld < (int64_t{1} << 40);
}
// Whether operands a and b of T rows of H elements share memory: b's rows (a's, where they begin
// first) against the other's.  Exact for rows equally far apart and for dense ones; of others, the
// first row of the operand that begins later.
inline bool rows_overlap(const void* a, int64_t lda, const void* b, int64_t ldb,
                         const mm_moe_norm_shape* s) {
  if (s->T == 1) lda = ldb = s->H;
  if (reinterpret_cast<uintptr_t>(b) < reinterpret_cast<uintptr_t>(a)) {
    std::swap(a, b);
    std::swap(lda, ldb);
  }
  const int64_t d = static_cast<int64_t>(
      (reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / dtype_bytes(s->dtype));
  // (2^31 rows 2^40 elements apart leave 64 bits)
  if (d >= static_cast<__int128>(s->T - 1) * lda + s->H) return false;
  const int64_t row = d / lda;  // where b begins
  if (d - row * lda < s->H) return true;
  return row + 1 < s->T && (row + 1) * lda < d + (ldb == s->H ? s->T * s->H : s->H);
}
// the same rows: what is written over them element by element
inline bool same_rows(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t T) {
  return a == b && (T == 1 || lda == ldb);
}

inline bool vec_ok(const void* p, size_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

inline bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The cut of an operand's rows (see Place): the same for rows that start on a 16-byte
// boundary and lie equally far apart modulo 16 bytes.
template <typename A, typename B>
bool same_cut(const Rows<A>& a, const Rows<B>& b, int64_t rows) {
  if (a.p == nullptr) return true;
  return al16(a.p) && al16(b.p) &&
         (rows == 1 || (a.ld - b.ld) * sizeof(A) % 16 == 0);
}

// Threads of a group that holds a row of H elements of T in NU units a thread, whatever
// its cut (`even`: every row starts on a 16-byte boundary); 0 when no CTA does.
template <typename T, int NU>
int group_threads(int H, bool even) {
  const int units = (H + (even ? 1 : 2) * (VN<T> - 1)) / VN<T>;
  const int n = (units + NU - 1) / NU;
  if (n > NORM_THREADS) return 0;
  if (n > 32) return (n + 31) / 32 * 32;
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

// a / b rounded up (the rows go up to 2^31 - 1, so the sum does not fit 32 bits)
inline int div_up(int a, int b) {
  return static_cast<int>((static_cast<int64_t>(a) + b - 1) / b);
}

struct NormGrid {
  int GT, groups, ctas;
};

// Rows spread over every SM first, then over the groups of a CTA (all of a warp's groups).
// A grid of several rounds has a multiple of 8 CTAs (see Place).
inline NormGrid norm_grid(int GT, int T, int sms, int most_groups = NORM_THREADS) {
  sms = std::max(8, sms / 8 * 8);
  const int per_warp = GT < 32 ? 32 / GT : 1;
  const int most = std::min(most_groups, NORM_THREADS / GT);
  int groups = std::min(most, div_up(T, sms));
  groups = (groups + per_warp - 1) / per_warp * per_warp;
  return NormGrid{GT, groups, std::min(sms, div_up(T, groups))};
}

template <typename T>
bool even_rows(const Rows<T>& r, int64_t rows) {
  return rows == 1 || r.ld * sizeof(T) % 16 == 0;
}

}  // namespace mmmoe
