// norm.cu -- layer normalisation in front of the layer: forward, and the backward with
// the reduction of the parameters' gradients.
//
//   mu = 1/H sum_i x_i,  var = 1/H sum_i (x_i - mu)^2,  r = (var + eps)^(-1/2)
//   xh = (x - mu) r,     y = w xh + b
//   g = w dy,            dx = r (g - mean(g) - xh mean(g xh)) [+ dx_add]
//   dw = sum_t dy xh,    db = sum_t dy
//
// x, y, dy, dx are bf16, fp16 or fp32; everything is computed in fp32 and rounded once
// where it is stored.  The variance is taken from the centred values (a second pass
// over the row), never as a difference of moments.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

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

// ------------------------------------------------------------------------- forward
// A thread with up to 16 columns holds its parameters in registers; with more columns a
// row needs fewer threads, so fewer sums across warps (none up to 2048 columns of 16 bits:
// 16384 x 2048 bf16 takes 31.8 us with 128 threads a row, 16 columns each, 22.6 us with a
// warp a row), and the parameters come from shared memory.  Where several warps share a
// row and registers allow it, a group takes two rows at a time (ROWS), so that two share
// the two barriers.
template <typename T, typename P, int NU, Cut CUT, int ROWS>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_fwd_kernel(
    Rows<const T> x, Rows<T> y, int T_, int H, int GT, const P* __restrict__ w,
    const P* __restrict__ b, float eps, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int U = VN<T>, C2 = NU * U / 2, S = norm_fwd_steps<NU, ROWS>;
  constexpr bool PS = norm_params_shared<T, NU>;
  static_assert(CUT != ANY || !PS, "a shifted row's columns do not line up with the parameters");
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  __shared__ Sums<ROWS> s_sum[2][NORM_THREADS / 32];
  const int nt = blockDim.x;
  const uint32_t ring =
      static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)) + threadIdx.x * 16;
  const uint32_t unit_bytes = nt * 16, row_bytes = NU * unit_bytes, step_bytes = ROWS * row_bytes;
  pdl_wait();
  pdl_trigger();
  Place<T, NU, CUT> p;
  p.init(GT, H);
  const float inv = 1.f / static_cast<float>(H);
  const uint32_t n = T_, step = gridDim.x * p.groups;
  uint32_t t = blockIdx.x * p.groups + p.g;
  uint32_t tw = p.first_of_warp(t);
  p.cut(x, t);
  uint32_t ta = t;  // the row to copy next
  const auto issue = [&](uint32_t at) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r, ta += step) {
      if (ta >= n) continue;
      const T* px = p.at(x, ta);
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (p.has(i)) p.copy(at + r * row_bytes + i * unit_bytes, px, i);
    }
    async_commit();
  };
  for (int i = 0; i < S * ROWS * NU; ++i)
    if (!p.has(i % NU)) sts16_zero(ring + i * unit_bytes);
  issue(ring);
  f2 wv[PS ? 1 : C2], bv[PS ? 1 : C2];
  // shared: weight then bias in fp32, the two halves of the units apart (16-byte reads of
  // consecutive units then meet no bank twice)
  const uint32_t sw = ring - threadIdx.x * 16 + S * step_bytes;
  if constexpr (PS) {
    float* s = reinterpret_cast<float*>(ring_bytes + S * step_bytes);
    for (int c = threadIdx.x; c < H; c += nt) {
      const int at = ((c % U / 4) * p.units + c / U) * 4 + c % 4;
      s[at] = to_f32(w[c]);
      s[H + at] = b != nullptr ? to_f32(b[c]) : 0.f;
    }
    __syncthreads();
  } else {
    p.params(w, wv);
    p.params(b, bv);
  }
  // (behind the parameters, which the first row already needs)
#pragma unroll
  for (int i = 1; i < S - 1; ++i) issue(ring + i * step_bytes);
  bool full = true;
#pragma unroll
  for (int i = 0; i < NU; ++i) full = full && p.whole(i);
  uint32_t st = ring, st_in = ring + (S - 1) * step_bytes;
  const uint32_t ring_end = ring + S * step_bytes;
  for (; tw < n; t += ROWS * step, tw += ROWS * step) {
    issue(st_in);
    async_wait<S - 1>();
    f2 v[ROWS][C2];
    float mu[ROWS], q[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      f2 a2 = 0;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        uint4 raw = lds16(st + r * row_bytes + i * unit_bytes);
        p.mask(raw, i);
        f2 u[U / 2];
        unpack2<T>(raw, u);
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
          v[r][i * U / 2 + k] = u[k];
          a2 = f2_add(a2, u[k]);
        }
      }
      mu[r] = f2_sum(a2);
    }
    st_in = st;
    st += step_bytes;
    if (st == ring_end) st = ring;
    group_sum<ROWS>(mu, s_sum[0], p.g, GT);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      mu[r] *= inv;
      const f2 nmu = f2_make(-mu[r], -mu[r]);
#pragma unroll
      for (int k = 0; k < C2; ++k) v[r][k] = f2_add(v[r][k], nmu);
      if (!full) {  // what is not in the row has no deviation either
#pragma unroll
        for (int k = 0; k < C2; ++k) {
          const int c = p.col(2 * k / U) + 2 * k % U;
          float lo, hi;
          f2_split(v[r][k], lo, hi);
          v[r][k] = f2_make(p.in(c) ? lo : 0.f, p.in(c + 1) ? hi : 0.f);
        }
      }
      f2 a2 = 0;
#pragma unroll
      for (int k = 0; k < C2; ++k) a2 = f2_fma(v[r][k], v[r][k], a2);
      q[r] = f2_sum(a2);
    }
    group_sum<ROWS>(q, s_sum[1], p.g, GT);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint32_t tr = t + r * step;
      if (tr >= n) continue;
      T* const py = p.at(y, tr);
      const float rs = rsqrtf(q[r] * inv + eps);
      const f2 r2 = f2_make(rs, rs);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (!p.has(i)) break;
        f2 u[U / 2];
        if constexpr (PS) {
          const uint32_t at = sw + (p.j + i * GT) * 16;
#pragma unroll
          for (int h = 0; h < U / 4; ++h) {
            const ulonglong2 w4 = lds16_f2(at + h * p.units * 16),
                             b4 = lds16_f2(at + H * 4 + h * p.units * 16);
            const int e = i * U / 2 + 2 * h;
            u[2 * h] = f2_fma(f2_mul(v[r][e], r2), w4.x, b4.x);
            u[2 * h + 1] = f2_fma(f2_mul(v[r][e + 1], r2), w4.y, b4.y);
          }
        } else {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            const int e = i * U / 2 + k;
            u[k] = f2_fma(f2_mul(v[r][e], r2), wv[e], bv[e]);
          }
        }
        p.store(py, i, pack2<T>(u));
      }
      if (p.j == 0) {
        mean[tr] = mu[r];
        rstd[tr] = rs;
      }
    }
  }
  async_wait<0>();
}

// ------------------------------------------------------------------------ backward
// dx and the CTA's column sums in one read of x, dy (and dx_add): the column sums stay
// in the registers of the threads that own the columns.  A group takes ROWS rows at a time,
// whose sums meet at one barrier: two where shared memory holds two steps of them.  Their
// x and dy are then read from the ring and unpacked a second time, which costs fewer
// cycles than the barrier's wait with one row in flight.
template <typename T, int NU, Cut CUT, bool ADD, int ROWS>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_bwd_kernel(
    Rows<const T> dy, Rows<const T> x, Rows<const T> add, Rows<T> dx, const void* __restrict__ w,
    bool w32, const float* __restrict__ mean, const float* __restrict__ rstd, int T_, int H, int GT,
    float* __restrict__ part, void* __restrict__ dweight, void* __restrict__ dbias) {
  constexpr int U = VN<T>, C2 = NU * U / 2, S = norm_bwd_steps<NU, ADD, ROWS>;
  constexpr int ARRAYS = ADD ? 3 : 2;
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  __shared__ Sums<2 * ROWS> s_sum[2][NORM_THREADS / 32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)) + tid * 16;
  const uint32_t unit_bytes = nt * 16, array_bytes = NU * unit_bytes,
                 row_bytes = ARRAYS * array_bytes, step_bytes = ROWS * row_bytes;
  pdl_wait();
  pdl_trigger();
  Place<T, NU, CUT> p;
  p.init(GT, H);
  const float inv = 1.f / static_cast<float>(H);
  const uint32_t n = T_, step = gridDim.x * p.groups;
  uint32_t t = blockIdx.x * p.groups + p.g;
  uint32_t tw = p.first_of_warp(t);
  p.cut(x, t);
  uint32_t ta = t;  // the row to copy next
  const auto issue = [&](uint32_t at) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r, ta += step) {
      if (ta >= n) continue;
      const T *px = p.at(x, ta), *pg = p.at(dy, ta);
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (p.has(i)) {
          p.copy(at + r * row_bytes + i * unit_bytes, px, i);
          p.copy(at + r * row_bytes + array_bytes + i * unit_bytes, pg, i);
        }
      if constexpr (ADD) {
        const T* pa = p.at(add, ta);
#pragma unroll
        for (int i = 0; i < NU; ++i)
          if (p.has(i)) p.copy(at + r * row_bytes + 2 * array_bytes + i * unit_bytes, pa, i);
      }
    }
    async_commit();
  };
  for (int i = 0; i < S * ROWS * ARRAYS * NU; ++i)
    if (!p.has(i % NU)) sts16_zero(ring + i * unit_bytes);
  // the parameters' loads stand behind the first step's, not behind the whole ring's
  issue(ring);
  f2 wv[C2], dw[C2], db[C2];
  if (w32)
    p.params(static_cast<const float*>(w), wv);
  else
    p.params(static_cast<const T*>(w), wv);
#pragma unroll
  for (int i = 1; i < S - 1; ++i) issue(ring + i * step_bytes);
#pragma unroll
  for (int k = 0; k < C2; ++k) dw[k] = db[k] = 0;
  float mu_n[ROWS], r_n[ROWS];
  const auto stats = [&](uint32_t from) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint32_t q = from + r * step;
      mu_n[r] = q < n ? __ldg(mean + q) : 0.f;
      r_n[r] = q < n ? __ldg(rstd + q) : 0.f;
    }
  };
  stats(t);
  int buf = 0;  // (one barrier a step: two buffers keep the next sums off these)
  uint32_t st = ring, st_in = ring + (S - 1) * step_bytes;
  const uint32_t ring_end = ring + S * step_bytes;
  for (; tw < n; t += ROWS * step, tw += ROWS * step) {
    issue(st_in);
    f2 r2[ROWS], m2[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      r2[r] = f2_make(r_n[r], r_n[r]);
      m2[r] = f2_make(-mu_n[r], -mu_n[r]);
    }
    stats(t + ROWS * step);
    async_wait<S - 1>();
    // xh and g = w dy of unit i of row r
    const auto unit = [&](int r, int i, f2 (&xh)[U / 2], f2 (&g)[U / 2], bool sums) {
      uint4 qx = lds16(st + r * row_bytes + i * unit_bytes),
            qg = lds16(st + r * row_bytes + array_bytes + i * unit_bytes);
      p.mask(qx, i);
      p.mask(qg, i);  // (a zero dy takes the column out of every sum)
      f2 fx[U / 2], fg[U / 2];
      unpack2<T>(qx, fx);
      unpack2<T>(qg, fg);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) {
        const int e = i * U / 2 + k;
        xh[k] = f2_mul(f2_add(fx[k], m2[r]), r2[r]);
        g[k] = f2_mul(fg[k], wv[e]);
        if (sums) {
          dw[e] = f2_fma(fg[k], xh[k], dw[e]);
          db[e] = f2_add(db[e], fg[k]);
        }
      }
    };
    f2 xh1[ROWS == 1 ? NU : 1][U / 2], g1[ROWS == 1 ? NU : 1][U / 2];
    float ac[2 * ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      f2 a2 = 0, c2 = 0;
      if (t + r * step < n) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          f2 xh[U / 2], g[U / 2];
          unit(r, i, xh, g, true);
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            a2 = f2_add(a2, g[k]);
            c2 = f2_fma(g[k], xh[k], c2);
            if constexpr (ROWS == 1) {
              xh1[i][k] = xh[k];
              g1[i][k] = g[k];
            }
          }
        }
      }
      ac[2 * r] = f2_sum(a2);
      ac[2 * r + 1] = f2_sum(c2);
    }
    group_sum<2 * ROWS>(ac, s_sum[buf], p.g, GT);
    buf ^= 1;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (t + r * step >= n) continue;
      T* const pd = p.at(dx, t + r * step);
      const float a = -ac[2 * r] * inv, c = -ac[2 * r + 1] * inv;
      const f2 na = f2_make(a, a), nc = f2_make(c, c);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (!p.has(i)) break;
        f2 xh[U / 2], g[U / 2], u[U / 2];
        if constexpr (ROWS > 1) unit(r, i, xh, g, false);
        if constexpr (ADD) {
          unpack2<T>(lds16(st + r * row_bytes + 2 * array_bytes + i * unit_bytes), u);
        } else {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) u[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
          const f2 h = ROWS > 1 ? xh[k] : xh1[ROWS > 1 ? 0 : i][k];
          const f2 gg = ROWS > 1 ? g[k] : g1[ROWS > 1 ? 0 : i][k];
          u[k] = f2_fma(f2_fma(h, nc, f2_add(gg, na)), r2[r], u[k]);
        }
        p.store(pd, i, pack2<T>(u));
      }
    }
    st_in = st;
    st += step_bytes;
    if (st == ring_end) st = ring;
  }
  async_wait<0>();

  // the groups' column sums, added in order: the CTA's partial ones, or from the only CTA
  // the gradients themselves
  float* const p0 = part + static_cast<int64_t>(blockIdx.x) * 2 * H;
  const auto put = [&](int which, int c, float v) {
    if (gridDim.x > 1) {
      p0[which * H + c] = v;
    } else {
      void* const o = which == 0 ? dweight : dbias;
      if (o == nullptr) return;
      if (w32)
        static_cast<float*>(o)[c] = v;
      else
        static_cast<T*>(o)[c] = from_f32<T>(v);
    }
  };
  if (p.groups == 1) {
    p.each(dw, [&](int c, float v) { put(0, c, v); });
    p.each(db, [&](int c, float v) { put(1, c, v); });
    return;
  }
  // Groups may cut their rows differently, so the sums meet by column.
  float* const sj = reinterpret_cast<float*>(ring_bytes);  // [groups][2][H]
  __syncthreads();
  if constexpr (CUT != ANY) {
    float* const q = sj + 2 * p.g * H;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (!p.has(i)) break;
      ulonglong2* const o = reinterpret_cast<ulonglong2*>(q + p.col(i));
      ulonglong2* const ob = reinterpret_cast<ulonglong2*>(q + H + p.col(i));
#pragma unroll
      for (int k = 0; k < U / 4; ++k) {
        o[k] = make_ulonglong2(dw[i * U / 2 + 2 * k], dw[i * U / 2 + 2 * k + 1]);
        ob[k] = make_ulonglong2(db[i * U / 2 + 2 * k], db[i * U / 2 + 2 * k + 1]);
      }
    }
  } else {
    p.each(dw, [&](int c, float v) { sj[2 * p.g * H + c] = v; });
    p.each(db, [&](int c, float v) { sj[(2 * p.g + 1) * H + c] = v; });
  }
  __syncthreads();
  for (int i = tid; i < 2 * H; i += nt) {
    float v = sj[i];
#pragma unroll 4
    for (int k = 1; k < p.groups; ++k) v += sj[2 * k * H + i];
    put(i >= H, i < H ? i : i - H, v);
  }
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

// One CTA per row; the row is read three times (sum, centred squares, output), the
// second and third time from L1/L2.
template <typename T, typename P, bool VEC>
__global__ void __launch_bounds__(LOOP_THREADS) norm_fwd_loop_kernel(
    Rows<const T> x, Rows<T> y, int T_, int H, const P* __restrict__ w, const P* __restrict__ b,
    float eps, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int U = loop_unit<T, VEC>;
  __shared__ float s[LOOP_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(H);
  const int units = H / U;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
    const T* xr = x.row(t);
    float a = 0.f;
#pragma unroll 4
    for (int u = threadIdx.x; u < units; u += LOOP_THREADS) {
      float f[U];
      load_unit<T, VEC>(xr, u, f);
#pragma unroll
      for (int k = 0; k < U; ++k) a += f[k];
    }
    const float mu = block_sum(a, s) * inv;
    a = 0.f;
#pragma unroll 4
    for (int u = threadIdx.x; u < units; u += LOOP_THREADS) {
      float f[U];
      load_unit<T, VEC>(xr, u, f);
#pragma unroll
      for (int k = 0; k < U; ++k) a = fmaf(f[k] - mu, f[k] - mu, a);
    }
    const float r = rsqrtf(block_sum(a, s) * inv + eps);
    T* yr = y.row(t);
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += LOOP_THREADS) {
      float f[U], wf[U], bf[U] = {};
      load_unit<T, VEC>(xr, u, f);
      load_params(w, u * U, wf);
      if (b != nullptr) load_params(b, u * U, bf);
#pragma unroll
      for (int k = 0; k < U; ++k) f[k] = fmaf((f[k] - mu) * r, wf[k], bf[k]);
      store_unit<T, VEC>(yr, u, f);
    }
    if (threadIdx.x == 0) {
      mean[t] = mu;
      rstd[t] = r;
    }
  }
}

template <typename T, typename P, bool VEC>
__global__ void __launch_bounds__(LOOP_THREADS) norm_dx_loop_kernel(
    Rows<const T> dy, Rows<const T> x, const P* __restrict__ w, const float* __restrict__ mean,
    const float* __restrict__ rstd, Rows<const T> add, Rows<T> dx, int T_, int H) {
  constexpr int U = loop_unit<T, VEC>;
  __shared__ float s[LOOP_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(H);
  const int units = H / U;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
    const T* xr = x.row(t);
    const T* gr = dy.row(t);
    const float mu = mean[t], r = rstd[t];
    float a = 0.f, c = 0.f;
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += LOOP_THREADS) {
      float fx[U], fg[U], wf[U];
      load_unit<T, VEC>(xr, u, fx);
      load_unit<T, VEC>(gr, u, fg);
      load_params(w, u * U, wf);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        a = fmaf(fg[k], wf[k], a);
        c = fmaf(fg[k] * wf[k], (fx[k] - mu) * r, c);
      }
    }
    a = block_sum(a, s) * inv;
    c = block_sum(c, s) * inv;
    T* o = dx.row(t);
#pragma unroll 2
    for (int u = threadIdx.x; u < units; u += LOOP_THREADS) {
      float fx[U], fg[U], wf[U], d[U] = {};
      load_unit<T, VEC>(xr, u, fx);
      load_unit<T, VEC>(gr, u, fg);
      load_params(w, u * U, wf);
      if (add.p != nullptr) load_unit<T, VEC>(add.row(t), u, d);
#pragma unroll
      for (int k = 0; k < U; ++k)
        d[k] = fmaf(fg[k] * wf[k] - a - (fx[k] - mu) * r * c, r, d[k]);
      store_unit<T, VEC>(o, u, d);
    }
  }
}

// Column sums of one range of rows per blockIdx.y: a thread owns a unit's columns.
// part[(blockIdx.y * 2 + {0, 1}) * H + i] = {sum dy xh, sum dy} over the range.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) norm_cols_loop_kernel(Rows<const T> dy, Rows<const T> x,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             int T_, int H, int rows,
                                                             float* __restrict__ part) {
  constexpr int U = loop_unit<T, VEC>;
  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x * 256 + threadIdx.x;
  if (u >= H / U) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t t1 = min(static_cast<int64_t>(T_), t0 + rows);
  float a[U] = {}, c[U] = {};
#pragma unroll 4
  for (int64_t t = t0; t < t1; ++t) {
    float fx[U], fg[U];
    load_unit<T, VEC>(x.row(t), u, fx);
    load_unit<T, VEC>(dy.row(t), u, fg);
    const float mu = __ldg(mean + t), r = __ldg(rstd + t);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      a[k] = fmaf(fg[k], (fx[k] - mu) * r, a[k]);
      c[k] += fg[k];
    }
  }
  float* const p = part + static_cast<int64_t>(blockIdx.y) * 2 * H + u * U;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    p[k] = a[k];
    p[H + k] = c[k];
  }
}

// dweight (blockIdx.y 0) / dbias (1) from n partial rows: 16 warps take every 16th row of
// 32 columns, ten loads in flight each, and are added in order.
template <typename P>
__global__ void __launch_bounds__(512) norm_cols_finish_kernel(const float* __restrict__ part,
                                                               int n, int H, P* __restrict__ dw,
                                                               P* __restrict__ db) {
  constexpr int W = 16, B = 10;
  pdl_wait();
  pdl_trigger();
  __shared__ float s[W][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (i < H) {
    const float* p = part + static_cast<int64_t>(blockIdx.y) * H + i;
    for (int j = w; j < n; j += W * B) {
      float v[B];
#pragma unroll
      for (int b = 0; b < B; ++b)
        v[b] = j + b * W < n ? __ldcg(p + static_cast<int64_t>(j + b * W) * 2 * H) : 0.f;
#pragma unroll
      for (int b = 0; b < B; ++b) a += v[b];
    }
  }
  s[w][lane] = a;
  __syncthreads();
  if (w == 0 && i < H) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) t += s[j][lane];
    P* out = blockIdx.y == 0 ? dw : db;
    out[i] = from_f32<P>(t);
  }
}

// Rows of partial column sums a backward of T rows writes at most (the workspace's size).
constexpr int NORM_MAX_PARTS = 152 * 2;
static int norm_parts(int64_t T) { return static_cast<int>(std::min<int64_t>(T, NORM_MAX_PARTS)); }

static bool norm_shape_ok(const mm_moe_norm_shape* s) {
  return s != nullptr && s->T >= 1 && s->T < (int64_t{1} << 31) && s->H >= 1 &&
         s->H <= (1 << 20) && dtype_ok(s->dtype) &&
         (s->param_dtype == s->dtype || s->param_dtype == MM_MOE_DT_F32) && s->eps >= 0.f;
}

// aligned to its element, and (rows) a stride of at least the row
static bool rows_ok(const void* p, int64_t ld, const mm_moe_norm_shape* s) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % dtype_bytes(s->dtype) == 0 &&
         (ld >= s->H || s->T == 1) && ld < (int64_t{1} << 40);
}
static bool vec_ok(const void* p, size_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

static bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The cut of an operand's rows (see Place): the same for rows that start on a 16-byte
// boundary and lie equally far apart modulo 16 bytes.
template <typename A, typename B>
static bool same_cut(const Rows<A>& a, const Rows<B>& b, int64_t rows) {
  if (a.p == nullptr) return true;
  return al16(a.p) && al16(b.p) &&
         (rows == 1 || (a.ld - b.ld) * sizeof(A) % 16 == 0);
}

// Threads of a group that holds a row of H elements of T in NU units a thread, whatever
// its cut (`even`: every row starts on a 16-byte boundary); 0 when no CTA does.
template <typename T, int NU>
static int group_threads(int H, bool even) {
  const int units = (H + (even ? 1 : 2) * (VN<T> - 1)) / VN<T>;
  const int n = (units + NU - 1) / NU;
  if (n > NORM_THREADS) return 0;
  if (n > 32) return (n + 31) / 32 * 32;
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

struct NormGrid {
  int GT, groups, ctas;
};

// Rows spread over every SM first, then over the groups of a CTA (all of a warp's groups).
// A grid of several rounds has a multiple of 8 CTAs (see Place).
static NormGrid norm_grid(int GT, int T, int sms, int most_groups = NORM_THREADS) {
  sms = std::max(8, sms / 8 * 8);
  const int per_warp = GT < 32 ? 32 / GT : 1;
  const int most = std::min(most_groups, NORM_THREADS / GT);
  int groups = std::min(most, (T + sms - 1) / sms);
  groups = (groups + per_warp - 1) / per_warp * per_warp;
  return NormGrid{GT, groups, std::min(sms, (T + groups - 1) / groups)};
}

template <typename T>
static bool even_rows(const Rows<T>& r, int64_t rows) {
  return rows == 1 || r.ld * sizeof(T) % 16 == 0;
}

template <typename T, typename P, int NU, int ROWS>
static cudaError_t fwd_launch(const Ctx& c, Rows<const T> x, Rows<T> y, int T_, int H, const P* w,
                              const P* b, float eps, float* mean, float* rstd) {
  const int GT = group_threads<T, NU>(H, even_rows(x, T_));
  constexpr int RING = norm_fwd_steps<NU, ROWS> * ROWS * NU * 16;  // bytes per thread
  // the ring and shared parameters have to fit beside each other
  const int fit = norm_params_shared<T, NU> ? (224 * 1024 - 8 * H) / (RING * GT) : NORM_THREADS;
  const NormGrid n = norm_grid(GT, T_, c.num_sms, fit);
  const int nt = n.GT * n.groups;
  size_t smem = static_cast<size_t>(RING) * nt;
  const bool even = even_rows(x, T_) && H % VN<T> == 0;
  auto* kern = norm_fwd_kernel<T, P, NU, EVEN, ROWS>;
  if constexpr (norm_params_shared<T, NU>)
    smem += sizeof(float) * 2 * H;
  else if (!even)
    kern = norm_fwd_kernel<T, P, NU, ANY, ROWS>;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_k(c.stream, kern, dim3(n.ctas), dim3(nt), smem, x, y, T_, H, n.GT, w, b, eps, mean,
                  rstd);
}

template <typename T, typename P>
static mm_moe_status norm_forward(const Ctx& c, const mm_moe_norm_shape* s, const void* x_,
                                  int64_t ldx, const void* w_, const void* b_, void* y_,
                                  int64_t ldy, float* mean, float* rstd) {
  const int T_ = static_cast<int>(s->T), H = static_cast<int>(s->H);
  const Rows<const T> x{static_cast<const T*>(x_), ldx};
  const Rows<T> y{static_cast<T*>(y_), ldy};
  const P* w = static_cast<const P*>(w_);
  const P* b = static_cast<const P*>(b_);
  constexpr int MOST = 16 / VN<T>;  // units of 16 columns
  const bool even = even_rows(x, T_);
  const auto go = [&](auto nu, auto rows) {
    return fwd_launch<T, P, decltype(nu)::value, decltype(rows)::value>(c, x, y, T_, H, w, b,
                                                                        s->eps, mean, rstd);
  };
  const auto pick = [&]() -> cudaError_t {
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, MOST> most{};
    if (same_cut(x, y, T_)) {
      if (T_ <= c.num_sms && group_threads<T, 1>(H, even) != 0)
        return go(one, one);  // one row a CTA: spread it wide
      if constexpr (sizeof(T) == 2) {
        if (even && H % VN<T> == 0 && H > 512 && H <= 8192) {
          // as few warps as hold the row in 8 units a thread, and as few units as they need
          // (12000 x 2560 in five units 23.9 us, in eight 31.3; 8192 x 4096 in eight units
          // 25.2 us, in four, two rows a barrier, 26.8)
          const int units = H / VN<T>, lanes = (units + 255) / 256 * 32;
          switch ((units + lanes - 1) / lanes) {
            case 3: return go(std::integral_constant<int, 3>{}, one);
            case 4: return go(std::integral_constant<int, 4>{}, one);
            case 5: return go(std::integral_constant<int, 5>{}, one);
            case 6: return go(std::integral_constant<int, 6>{}, one);
            case 7: return go(std::integral_constant<int, 7>{}, one);
            default: return go(std::integral_constant<int, 8>{}, one);
          }
        }
      }
      const int GT = group_threads<T, MOST>(H, even);
      if (GT > 32) return go(most, two);
      if (GT != 0) return go(most, one);
    }
    const bool vec = even && even_rows(y, T_) && H % VN<T> == 0 && al16(x.p) && al16(y.p) &&
                     al16(w) && (b == nullptr || al16(b));
    return launch_k(c.stream,
                    vec ? norm_fwd_loop_kernel<T, P, true> : norm_fwd_loop_kernel<T, P, false>,
                    dim3(std::min(T_, c.num_sms * 4)), dim3(LOOP_THREADS), 0, x, y, T_, H, w, b,
                    s->eps, mean, rstd);
  };
  prof_begin(c, K_NORM_FWD);
  const cudaError_t e = pick();
  prof_end(c, K_NORM_FWD);
  return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ECUDA;
}

// One backward's operands.
template <typename T>
struct BwdArgs {
  Rows<const T> dy, x, add;
  Rows<T> dx;
  const void* w;
  bool w32;
  const float *mean, *rstd;
  int T_, H;
  float* part;
  void *dw, *db;
};

// So few rows that a single CTA's groups hold them in two rounds (rows of differing cuts: in
// one, see Place): nothing is left to join after it.
static bool one_cta(int GT, int T, bool even) {
  return T <= (even ? 2 : 1) * (NORM_THREADS / GT);
}

template <typename T, int NU, int ROWS>
static cudaError_t bwd_launch(const Ctx& c, const BwdArgs<T>& a, int* n_part) {
  const int GT = group_threads<T, NU>(a.H, even_rows(a.x, a.T_));
  NormGrid n = norm_grid(GT, a.T_, c.num_sms);
  if (one_cta(GT, a.T_, even_rows(a.x, a.T_))) n = NormGrid{GT, NORM_THREADS / GT, 1};
  const int nt = n.GT * n.groups;
  size_t smem = static_cast<size_t>(ROWS) * NU * 16 * nt *
                (a.add.p != nullptr ? 3 * norm_bwd_steps<NU, true, ROWS>
                                    : 2 * norm_bwd_steps<NU, false, ROWS>);
  if (n.groups > 1) smem = std::max(smem, sizeof(float) * 2 * n.groups * a.H);
  const bool even = even_rows(a.x, a.T_) && a.H % VN<T> == 0;
  const Cut cut = !even ? ANY : NU <= 2 && a.H == n.GT * NU * VN<T> ? FULL : EVEN;
  auto* kern = a.add.p != nullptr
                   ? (cut == ANY    ? norm_bwd_kernel<T, NU, ANY, true, ROWS>
                      : cut == EVEN ? norm_bwd_kernel<T, NU, EVEN, true, ROWS>
                                    : norm_bwd_kernel<T, NU, FULL, true, ROWS>)
                   : (cut == ANY    ? norm_bwd_kernel<T, NU, ANY, false, ROWS>
                      : cut == EVEN ? norm_bwd_kernel<T, NU, EVEN, false, ROWS>
                                    : norm_bwd_kernel<T, NU, FULL, false, ROWS>);
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  *n_part = n.ctas;
  return launch_k(c.stream, kern, dim3(n.ctas), dim3(nt), smem, a.dy, a.x, a.add,
                  a.dx, a.w, a.w32, a.mean, a.rstd, a.T_, a.H, n.GT, a.part, a.dw, a.db);
}

template <typename T, typename P>
static mm_moe_status norm_backward(const Ctx& c, const mm_moe_norm_shape* s, const void* dy,
                                   int64_t lddy, const void* x, int64_t ldx, const void* w,
                                   const float* mean, const float* rstd, const void* add,
                                   int64_t ldadd, void* dx, int64_t lddx, void* dw, void* db,
                                   float* part) {
  const int T_ = static_cast<int>(s->T), H = static_cast<int>(s->H);
  const BwdArgs<T> a{{static_cast<const T*>(dy), lddy},
                     {static_cast<const T*>(x), ldx},
                     {static_cast<const T*>(add), ldadd},
                     {static_cast<T*>(dx), lddx},
                     w,
                     sizeof(P) == 4,
                     mean,
                     rstd,
                     T_,
                     H,
                     part,
                     dw,
                     db};
  constexpr int MOST = 16 / VN<T>;
  const bool even = even_rows(a.x, T_);
  cudaError_t e;
  int n = 0;
  if (same_cut(a.dy, a.x, T_) && same_cut(a.add, a.x, T_) && same_cut(a.dx, a.x, T_) &&
      group_threads<T, MOST>(H, even) != 0) {
    prof_begin(c, K_NORM_BWD);
    const auto pick = [&]() -> cudaError_t {
      constexpr int WIDE = sizeof(T) == 2 ? 2 : 4;
      if (T_ <= c.num_sms && !one_cta(group_threads<T, WIDE>(H, even), T_, even) &&
          group_threads<T, 1>(H, even) != 0)
        return bwd_launch<T, 1, 1>(c, a, &n);
      if constexpr (sizeof(T) == 2) {
        // 16 bits: two rows a barrier where more than two warps share a row (8191 x 4096
        // 43.8 -> 40.2 us, 20011 x 1111 47.5 -> 41.0 us; 30000 x 1000, two warps a row, 44.5
        // -> 46.3 us)
        return group_threads<T, 2>(H, even) > 64 ? bwd_launch<T, 2, 2>(c, a, &n)
                                                 : bwd_launch<T, 2, 1>(c, a, &n);
      } else {
        return group_threads<T, 2>(H, even) != 0 ? bwd_launch<T, 2, 1>(c, a, &n)
                                                 : bwd_launch<T, 4, 1>(c, a, &n);
      }
    };
    e = pick();
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
    if (n == 1) return MM_MOE_OK;  // (the only CTA has written them)
  } else {
    const bool vec = even && even_rows(a.dy, T_) && even_rows(a.dx, T_) && H % VN<T> == 0 &&
                     al16(x) && al16(dy) && al16(dx) && al16(w) &&
                     (add == nullptr || (al16(add) && even_rows(a.add, T_)));
    prof_begin(c, K_NORM_BWD);
    e = launch_k(c.stream,
                 vec ? norm_dx_loop_kernel<T, P, true> : norm_dx_loop_kernel<T, P, false>,
                 dim3(std::min(T_, c.num_sms * 4)), dim3(LOOP_THREADS), 0, a.dy, a.x,
                 static_cast<const P*>(w), mean, rstd, a.add, a.dx, T_, H);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
    const int cols = (H / (vec ? VN<T> : 1) + 255) / 256;
    const int want = std::min(norm_parts(T_), std::max(1, c.num_sms * 8 / cols));
    const int rows = (T_ + want - 1) / want;
    n = (T_ + rows - 1) / rows;
    prof_begin(c, K_NORM_BWD);
    e = launch_k(c.stream, vec ? norm_cols_loop_kernel<T, true> : norm_cols_loop_kernel<T, false>,
                 dim3(cols, n), dim3(256), 0, a.dy, a.x, mean, rstd, T_, H, rows, part);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
  }
  prof_begin(c, K_NORM_BWD_FINISH);
  e = launch_k(c.stream, norm_cols_finish_kernel<P>, dim3((H + 31) / 32, db != nullptr ? 2 : 1),
               dim3(512), 0, static_cast<const float*>(part), n, H, static_cast<P*>(dw),
               static_cast<P*>(db));
  prof_end(c, K_NORM_BWD_FINISH);
  return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ECUDA;
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_norm_workspace_size(const mm_moe_norm_shape* shape,
                                                               size_t* bytes) {
  if (!norm_shape_ok(shape) || bytes == nullptr) return MM_MOE_EINVAL;
  *bytes = static_cast<size_t>(norm_parts(shape->T)) * 2 * shape->H * sizeof(float);
  return MM_MOE_OK;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_norm_forward(const mm_moe_norm_shape* shape,
                                                        const void* x, int64_t ldx,
                                                        const void* weight, const void* bias,
                                                        void* y, int64_t ldy, float* mean,
                                                        float* rstd, void* stream) {
  if (!norm_shape_ok(shape)) return MM_MOE_EINVAL;
  const size_t pb = dtype_bytes(shape->param_dtype);
  if (!rows_ok(x, ldx, shape) || !rows_ok(y, ldy, shape) || !vec_ok(weight, pb) ||
      (bias != nullptr && !vec_ok(bias, pb)) || !vec_ok(mean, 4) || !vec_ok(rstd, 4))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  return with_dtype(shape->dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (shape->param_dtype == shape->dtype)
      return norm_forward<T, T>(c, shape, x, ldx, weight, bias, y, ldy, mean, rstd);
    return norm_forward<T, float>(c, shape, x, ldx, weight, bias, y, ldy, mean, rstd);
  });
}

extern "C" MM_MOE_API mm_moe_status mm_moe_norm_backward(
    const mm_moe_norm_shape* shape, const void* dy, int64_t lddy, const void* x, int64_t ldx,
    const void* weight, const float* mean, const float* rstd, const void* dx_add, int64_t ldadd,
    void* dx, int64_t lddx, void* dweight, void* dbias, void* workspace, void* stream) {
  if (!norm_shape_ok(shape)) return MM_MOE_EINVAL;
  const size_t pb = dtype_bytes(shape->param_dtype);
  if (!rows_ok(dy, lddy, shape) || !rows_ok(x, ldx, shape) || !rows_ok(dx, lddx, shape) ||
      (dx_add != nullptr && !rows_ok(dx_add, ldadd, shape)) || !vec_ok(weight, pb) ||
      !vec_ok(mean, 4) || !vec_ok(rstd, 4) || !vec_ok(dweight, pb) ||
      (dbias != nullptr && !vec_ok(dbias, pb)) || !vec_ok(workspace, 16))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  float* part = static_cast<float*>(workspace);
  return with_dtype(shape->dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (shape->param_dtype == shape->dtype)
      return norm_backward<T, T>(c, shape, dy, lddy, x, ldx, weight, mean, rstd, dx_add, ldadd, dx,
                                 lddx, dweight, dbias, part);
    return norm_backward<T, float>(c, shape, dy, lddy, x, ldx, weight, mean, rstd, dx_add, ldadd,
                                   dx, lddx, dweight, dbias, part);
  });
}
