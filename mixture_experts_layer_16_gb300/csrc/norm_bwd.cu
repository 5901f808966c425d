// norm_bwd.cu -- layer normalisation: the backward, with the reduction of the parameters'
// gradients (formulas in norm.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "norm.cuh"
#include "ops.cuh"

namespace mmmoe {

// ------------------------------------------------------------------------ backward
// dx and the CTA's column sums in one read of x, dy (and dx_add): the column sums stay
// in the registers of the threads that own the columns.  A group takes ROWS rows at a time,
// whose sums meet at one barrier: two where shared memory holds two steps of them.  Their
// x and dy are then read from the ring and unpacked a second time, which costs fewer
// cycles than the barrier's wait with one row in flight.
// 16384 x 2048 bf16 with a residual gradient: 45.9 us together with the launch that ends it, 0.86
// of the copy rate (HBM, 6 us of ramps and that launch); 8191 x 4096 fp16 39.5 us, bound by the
// barrier of eight warps and by issue.
template <typename T, int NU, Cut CUT, bool ADD, int ROWS>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_bwd_kernel(
    Rows<const T> dy, Rows<const T> x, Rows<const T> add, Rows<T> dx, const void* __restrict__ w,
    bool w32, const float* __restrict__ mean, const float* __restrict__ rstd, int T_, int H, int GT,
    float* __restrict__ part, void* __restrict__ dweight, void* __restrict__ dbias) {
  constexpr int U = VN<T>, C2 = NU * U / 2, S = norm_bwd_steps<NU, ADD, ROWS>;
  constexpr int ARRAYS = ADD ? 3 : 2;
  constexpr bool KEEP = ROWS == 1 && NU * U <= 16;  // xh and g stay in registers
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
    f2 xh1[KEEP ? NU : 1][U / 2], g1[KEEP ? NU : 1][U / 2];
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
            if constexpr (KEEP) {
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
        if constexpr (!KEEP) unit(r, i, xh, g, false);
        if constexpr (ADD) {
          unpack2<T>(lds16(st + r * row_bytes + 2 * array_bytes + i * unit_bytes), u);
        } else {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) u[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < U / 2; ++k) {
          const f2 h = KEEP ? xh1[KEEP ? i : 0][k] : xh[k];
          const f2 gg = KEEP ? g1[KEEP ? i : 0][k] : g[k];
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
  // a thread's sums by whole units, dw's columns from q on and db's from q + H
  const auto put_units = [&](float* q) {
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
  };
  if (p.groups == 1) {
    if constexpr (CUT != ANY) {
      if (gridDim.x > 1) {
        put_units(p0);
        return;
      }
    }
    p.each(dw, [&](int c, float v) { put(0, c, v); });
    p.each(db, [&](int c, float v) { put(1, c, v); });
    return;
  }
  // Groups may cut their rows differently, so the sums meet by column.
  float* const sj = reinterpret_cast<float*>(ring_bytes);  // [groups][2][H]
  __syncthreads();
  if constexpr (CUT != ANY) {
    put_units(sj + 2 * p.g * H);
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

// dx, one CTA per row, x and dy read twice; with the column sums below, which read them a third
// time, 2048 x 16384 bf16 takes 106 us, 0.37 of the copy rate.
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
// 32 columns, ten loads in flight each, and are added in order.  About 3 us of latency for the
// 2.5 MB of 152 rows of 2048 columns.
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
    const float* p = part + static_cast<int64_t>(2 * w + blockIdx.y) * H + i;
    for (int j = w; j < n; j += W * B) {
      float v[B];
#pragma unroll
      for (int b = 0; b < B; ++b, p += 2 * W * H) v[b] = j + b * W < n ? __ldcg(p) : 0.f;
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
  constexpr Cut WHOLE = NU <= 2 ? FULL : EVEN;
  auto* kern = a.add.p != nullptr
                   ? (cut == ANY    ? norm_bwd_kernel<T, NU, ANY, true, ROWS>
                      : cut == EVEN ? norm_bwd_kernel<T, NU, EVEN, true, ROWS>
                                    : norm_bwd_kernel<T, NU, WHOLE, true, ROWS>)
                   : (cut == ANY    ? norm_bwd_kernel<T, NU, ANY, false, ROWS>
                      : cut == EVEN ? norm_bwd_kernel<T, NU, EVEN, false, ROWS>
                                    : norm_bwd_kernel<T, NU, WHOLE, false, ROWS>);
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
  constexpr int MOST = sizeof(T) == 2 ? 3 : 4;  // units a thread
  const bool even = even_rows(a.x, T_);
  cudaError_t e;
  int n = 0;
  if (same_cut(a.dy, a.x, T_) && same_cut(a.add, a.x, T_) && same_cut(a.dx, a.x, T_) &&
      group_threads<T, MOST>(H, even) != 0) {
    prof_begin(c, K_NORM_BWD);
    const auto pick = [&]() -> cudaError_t {
      // few rows: one unit a thread, in up to half of a CTA's groups (us, in two units and so:
      // 153 x 1024 bf16 5.1 and 4.3, 300 x 512 5.0 and 4.2; in all of them 300 x 2048 6.2 and
      // 6.6, 1200 x 512 5.1 and 6.2), unless a single CTA takes them in two units a thread.  (Not
      // in fp32's four, in which it would take twice as many rows: 16 x 1024 3.2 us in one unit,
      // 6.0 in one CTA; 9 x 1000 3.1 and 5.5; 5 x 2048 3.5 and 6.1.)
      const int g1 = group_threads<T, 1>(H, even), g2 = group_threads<T, 2>(H, even);
      if (g1 != 0 && T_ <= c.num_sms / 8 * 8 * std::max(1, NORM_THREADS / g1 / 2) &&
          !one_cta(g2, T_, even))
        return bwd_launch<T, 1, 1>(c, a, &n);
      if constexpr (sizeof(T) == 2) {
        // 16 bits: three units a thread where that doubles the CTA's groups, or no CTA holds the
        // row in two (us: 65536 x 511 101.8 and 65.2, 100000 x 333 81.5 and 58.5, 50000 x 600
        // 52.4 and 44.6; with 8 groups for 5, 5000 x 1111 18.4 and 21.5; narrow rows, 20000 x
        // 72 9.1 and 10.3; row by row and so 4096 x 8191 207.6 and 69.9, 2600 x 12288 106.2
        // and 48.5)
        const int g3 = group_threads<T, 3>(H, even);
        if (g2 == 0 || (H > 128 && NORM_THREADS / g3 >= 2 * (NORM_THREADS / g2)))
          return bwd_launch<T, 3, 1>(c, a, &n);
        // two rows a barrier where more than two warps share a row (8191 x 4096
        // 43.8 -> 40.2 us, 20011 x 1111 47.5 -> 41.0 us; 30000 x 1000, two warps a row, 44.5
        // -> 46.3 us)
        return g2 > 64 ? bwd_launch<T, 2, 2>(c, a, &n) : bwd_launch<T, 2, 1>(c, a, &n);
      } else {
        return g2 != 0 ? bwd_launch<T, 2, 1>(c, a, &n) : bwd_launch<T, 4, 1>(c, a, &n);
      }
    };
    e = pick();
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return op_status(e);
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
    if (e != cudaSuccess) return op_status(e);
    const int cols = (H / (vec ? VN<T> : 1) + 255) / 256;
    const int want = std::min(norm_parts(T_), std::max(1, c.num_sms * 8 / cols));
    const int rows = div_up(T_, want);
    n = div_up(T_, rows);
    prof_begin(c, K_NORM_BWD);
    e = launch_k(c.stream, vec ? norm_cols_loop_kernel<T, true> : norm_cols_loop_kernel<T, false>,
                 dim3(cols, n), dim3(256), 0, a.dy, a.x, mean, rstd, T_, H, rows, part);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return op_status(e);
  }
  prof_begin(c, K_NORM_BWD_FINISH);
  e = launch_k(c.stream, norm_cols_finish_kernel<P>, dim3((H + 31) / 32, db != nullptr ? 2 : 1),
               dim3(512), 0, static_cast<const float*>(part), n, H, static_cast<P*>(dw),
               static_cast<P*>(db));
  prof_end(c, K_NORM_BWD_FINISH);
  return op_status(e);
}

}  // namespace mmmoe

using namespace mmmoe;

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
  // (dx over dx_add is read and written element by element; x and dy are read again)
  if (rows_overlap(dx, lddx, x, ldx, shape) || rows_overlap(dx, lddx, dy, lddy, shape) ||
      (dx_add != nullptr && !same_rows(dx, lddx, dx_add, ldadd, shape->T) &&
       rows_overlap(dx, lddx, dx_add, ldadd, shape)))
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
