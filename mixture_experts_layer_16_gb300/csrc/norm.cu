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

#include "dtype.cuh"
#include "internal.h"

namespace mmmoe {

// One row operand: base pointer and elements from one row to the next.
template <typename T>
struct Rows {
  T* p;
  int64_t ld;
  __device__ __forceinline__ T* row(int64_t t) const { return p + t * ld; }
};

// A unit is V bytes of a row: 16 where the rows and the parameters allow it, else 4, else
// one 16-bit element.
template <int V>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int V>
__device__ __forceinline__ void unit_unpack(const typename Raw<V>::type& q,
                                            float (&f)[V / sizeof(T)]) {
  if constexpr (V == 16) {
    unpack(q, f, static_cast<const T*>(nullptr));
  } else {
    const T* h = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < V / static_cast<int>(sizeof(T)); ++i) f[i] = to_f32(h[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ typename Raw<V>::type unit_pack(const float (&f)[V / sizeof(T)]) {
  if constexpr (V == 16) {
    return pack(f, static_cast<const T*>(nullptr));
  } else {
    typename Raw<V>::type q;
    T* h = reinterpret_cast<T*>(&q);
#pragma unroll
    for (int i = 0; i < V / static_cast<int>(sizeof(T)); ++i) h[i] = from_f32<T>(f[i]);
    return q;
  }
}

// U consecutive parameters from column c on.
template <typename P, int U>
__device__ __forceinline__ void load_params(const P* __restrict__ p, int c, float (&f)[U]) {
  if constexpr (U * sizeof(P) >= 16) {
    constexpr int N = VN<P>;
#pragma unroll
    for (int i = 0; i < U / N; ++i) {
      float t[N];
      unpack(__ldg(reinterpret_cast<const uint4*>(p + c) + i), t, p);
#pragma unroll
      for (int j = 0; j < N; ++j) f[i * N + j] = t[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) f[i] = to_f32(p[c + i]);
  }
}

__device__ __forceinline__ void group_bar(int g, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(threads) : "memory");
}

// Sum over a group of GT threads (whole warps): the warps' sums meet in s[warps], each
// thread adds them in order.  One barrier; `s` must not be in use from the previous sum.
__device__ __forceinline__ float group_sum(float v, float* s, int g, int GT) {
  v = warp_sum(v);
  if (GT == 32) return v;
  const int w = (threadIdx.x >> 5) - g * (GT >> 5);
  if ((threadIdx.x & 31) == 0) s[w] = v;
  group_bar(g, GT);
  float t = s[0];
  for (int i = 1; i < (GT >> 5); ++i) t += s[i];
  return t;
}

// ------------------------------------------------------------------------- forward
// A row sits in the registers of GT threads (NU units each) from its one read to its
// output; the CTA holds blockDim / GT rows.
template <typename T, typename P, int V, int NU>
__global__ void __launch_bounds__(512) norm_fwd_kernel(Rows<const T> x, Rows<T> y, int T_, int H,
                                                       int GT, const P* __restrict__ w,
                                                       const P* __restrict__ b, float eps,
                                                       float* __restrict__ mean,
                                                       float* __restrict__ rstd) {
  constexpr int U = V / static_cast<int>(sizeof(T));
  using R = typename Raw<V>::type;
  __shared__ float s[2][16];
  pdl_wait();
  pdl_trigger();
  const int g = threadIdx.x / GT, j = threadIdx.x - g * GT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / GT) + g;
  if (t >= T_) return;  // a group leaves as a whole, and its barrier is its own
  const int units = H / U;
  const float inv = 1.f / static_cast<float>(H);
  float* const s0 = s[0] + g * (GT >> 5);
  float* const s1 = s[1] + g * (GT >> 5);
  const R* xr = reinterpret_cast<const R*>(x.row(t));
  R q[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = j + i * GT;
    if (u < units) q[i] = xr[u];
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (j + i * GT >= units) break;
    float f[U];
    unit_unpack<T, V>(q[i], f);
#pragma unroll
    for (int k = 0; k < U; ++k) a += f[k];
  }
  const float mu = group_sum(a, s0, g, GT) * inv;
  a = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (j + i * GT >= units) break;
    float f[U];
    unit_unpack<T, V>(q[i], f);
#pragma unroll
    for (int k = 0; k < U; ++k) a = fmaf(f[k] - mu, f[k] - mu, a);
  }
  const float r = rsqrtf(group_sum(a, s1, g, GT) * inv + eps);
  R* yr = reinterpret_cast<R*>(y.row(t));
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = j + i * GT;
    if (u >= units) break;
    float f[U], wf[U], bf[U] = {};
    unit_unpack<T, V>(q[i], f);
    load_params<P, U>(w, u * U, wf);
    if (b != nullptr) load_params<P, U>(b, u * U, bf);
#pragma unroll
    for (int k = 0; k < U; ++k) f[k] = fmaf((f[k] - mu) * r, wf[k], bf[k]);
    yr[u] = unit_pack<T, V>(f);
  }
  if (j == 0) {
    mean[t] = mu;
    rstd[t] = r;
  }
}

// ------------------------------------------------------------------------ backward
template <int V>
__device__ __forceinline__ void async_copy(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (V == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

constexpr int NORM_BWD_THREADS = 512;

// Rows in flight per group: three rows ahead for 32 bytes of a row per thread, one for 64
// (fp32, 16 columns a thread), so that the ring stays within 192 KB.
template <typename T, int V, int NU>
constexpr int norm_stages = V * NU <= 32 ? 4 : 2;

// dx and the CTA's column sums in one read of x, dy (and dx_add).  A group of GT threads
// takes a row at a time, its threads the same columns in every row, so the column sums
// stay in their registers.  A thread copies its own units of the next rows into shared
// memory with cp.async and reads nothing but what it copied itself: no barrier guards
// the ring, and the one barrier of a row is that of its two sums.
template <typename T, int V, int NU>
__global__ void __launch_bounds__(NORM_BWD_THREADS, 1) norm_bwd_kernel(
    Rows<const T> dy, Rows<const T> x, Rows<const T> add, Rows<T> dx, const void* __restrict__ w,
    bool w32, const float* __restrict__ mean, const float* __restrict__ rstd, int T_, int H, int GT,
    float* __restrict__ part) {
  constexpr int U = V / static_cast<int>(sizeof(T));
  constexpr int C = NU * U;  // columns per thread
  constexpr int S = norm_stages<T, V, NU>;
  using R = typename Raw<V>::type;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float2 s_sum[2][NORM_BWD_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, nt = blockDim.x;
  const int g = tid / GT, j = tid - g * GT, groups = nt / GT, gw = GT >> 5;
  const int units = H / U;
  const bool with_add = add.p != nullptr;
  const int arrays = with_add ? 3 : 2;
  const float inv = 1.f / static_cast<float>(H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + g;

  float wf[C], dw[C], db[C];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int c = (j + i * GT) * U + k;
      wf[i * U + k] = j + i * GT >= units ? 0.f
                      : w32               ? static_cast<const float*>(w)[c]
                                          : to_f32(static_cast<const T*>(w)[c]);
      dw[i * U + k] = db[i * U + k] = 0.f;
    }

  const auto slot = [&](int st, int arr, int i) {
    return reinterpret_cast<R*>(ring) + (static_cast<size_t>((st * arrays + arr) * NU + i) * nt + tid);
  };
  const auto issue = [&](int64_t row, int st) {
    if constexpr (V >= 4) {
      if (row < T_) {
        const R* xr = reinterpret_cast<const R*>(x.row(row));
        const R* gr = reinterpret_cast<const R*>(dy.row(row));
        const R* ar = with_add ? reinterpret_cast<const R*>(add.row(row)) : nullptr;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int u = j + i * GT;
          if (u < units) {
            async_copy<V>(slot(st, 0, i), xr + u);
            async_copy<V>(slot(st, 1, i), gr + u);
            if (with_add) async_copy<V>(slot(st, 2, i), ar + u);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  for (int p = 0; p < S - 1; ++p) issue(t + p * step, p);
  float mu_n = 0.f, r_n = 0.f;
  if (t < T_) {
    mu_n = __ldg(mean + t);
    r_n = __ldg(rstd + t);
  }
  int st = 0, buf = 0;
  for (; t < T_; t += step) {
    issue(t + (S - 1) * step, st == 0 ? S - 1 : st - 1);
    const float mu = mu_n, r = r_n;
    if (t + step < T_) {
      mu_n = __ldg(mean + t + step);
      r_n = __ldg(rstd + t + step);
    }
    if constexpr (V >= 4) asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    float xh[C], gv[C];
    float a = 0.f, c = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = j + i * GT;
      float fx[U] = {}, fg[U] = {};
      if (u < units) {
        if constexpr (V >= 4) {
          unit_unpack<T, V>(*slot(st, 0, i), fx);
          unit_unpack<T, V>(*slot(st, 1, i), fg);
        } else {
          unit_unpack<T, V>(reinterpret_cast<const R*>(x.row(t))[u], fx);
          unit_unpack<T, V>(reinterpret_cast<const R*>(dy.row(t))[u], fg);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int e = i * U + k;
          xh[e] = (fx[k] - mu) * r;
          dw[e] = fmaf(fg[k], xh[e], dw[e]);
          db[e] += fg[k];
          gv[e] = fg[k] * wf[e];
          a += gv[e];
          c = fmaf(gv[e], xh[e], c);
        }
      }
    }
    a = warp_sum(a);
    c = warp_sum(c);
    if (GT > 32) {
      float2* s = s_sum[buf] + g * gw;
      if ((tid & 31) == 0) s[(tid >> 5) - g * gw] = make_float2(a, c);
      group_bar(g, GT);
      a = c = 0.f;
      for (int i = 0; i < gw; ++i) {
        const float2 v = s[i];
        a += v.x;
        c += v.y;
      }
      buf ^= 1;
    }
    a *= inv;
    c *= inv;
    R* o = reinterpret_cast<R*>(dx.row(t));
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = j + i * GT;
      if (u >= units) break;
      float f[U] = {};
      if (with_add) {
        if constexpr (V >= 4)
          unit_unpack<T, V>(*slot(st, 2, i), f);
        else
          unit_unpack<T, V>(reinterpret_cast<const R*>(add.row(t))[u], f);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int e = i * U + k;
        f[k] = fmaf(gv[e] - a - xh[e] * c, r, f[k]);
      }
      o[u] = unit_pack<T, V>(f);
    }
    st = st + 1 == S ? 0 : st + 1;
  }
  if constexpr (V >= 4) asm volatile("cp.async.wait_group 0;" ::: "memory");

  // the groups' column sums, added in order
  float* const p0 = part + static_cast<int64_t>(blockIdx.x) * 2 * H;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = j + i * GT;
      if (u >= units) break;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        p0[u * U + k] = dw[i * U + k];
        p0[H + u * U + k] = db[i * U + k];
      }
    }
    return;
  }
  float* sj = reinterpret_cast<float*>(ring);
  __syncthreads();
#pragma unroll
  for (int e = 0; e < C; ++e) {
    sj[e * nt + tid] = dw[e];
    sj[(C + e) * nt + tid] = db[e];
  }
  __syncthreads();
  for (int e = g; e < C; e += groups) {
    const int u = j + e / U * GT;
    if (u >= units) break;
    float a = 0.f, c = 0.f;
    for (int q = 0; q < groups; ++q) {
      a += sj[e * nt + q * GT + j];
      c += sj[(C + e) * nt + q * GT + j];
    }
    p0[u * U + e % U] = a;
    p0[H + u * U + e % U] = c;
  }
}

// --------------------------------------------------------------- looped, any width
// One CTA per row; the row is read three times (sum, centred squares, output), the
// second and third time from L1/L2.
template <typename T, typename P>
__global__ void __launch_bounds__(256) norm_fwd_loop_kernel(Rows<const T> x, Rows<T> y, int T_,
                                                            int H, const P* __restrict__ w,
                                                            const P* __restrict__ b, float eps,
                                                            float* __restrict__ mean,
                                                            float* __restrict__ rstd) {
  __shared__ float s[8];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(H);
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
    const T* xr = x.row(t);
    float a = 0.f;
    for (int i = threadIdx.x; i < H; i += 256) a += to_f32(xr[i]);
    const float mu = block_sum(a, s) * inv;
    a = 0.f;
    for (int i = threadIdx.x; i < H; i += 256) {
      const float d = to_f32(xr[i]) - mu;
      a = fmaf(d, d, a);
    }
    const float r = rsqrtf(block_sum(a, s) * inv + eps);
    T* yr = y.row(t);
    for (int i = threadIdx.x; i < H; i += 256) {
      const float v = (to_f32(xr[i]) - mu) * r;
      yr[i] = from_f32<T>(fmaf(v, to_f32(w[i]), b != nullptr ? to_f32(b[i]) : 0.f));
    }
    if (threadIdx.x == 0) {
      mean[t] = mu;
      rstd[t] = r;
    }
  }
}

template <typename T, typename P>
__global__ void __launch_bounds__(256) norm_dx_loop_kernel(Rows<const T> dy, Rows<const T> x,
                                                           const P* __restrict__ w,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd,
                                                           Rows<const T> add, Rows<T> dx, int T_,
                                                           int H) {
  __shared__ float s[8];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(H);
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
    const T* xr = x.row(t);
    const T* gr = dy.row(t);
    const float mu = mean[t], r = rstd[t];
    float a = 0.f, c = 0.f;
    for (int i = threadIdx.x; i < H; i += 256) {
      const float g = to_f32(gr[i]) * to_f32(w[i]);
      a += g;
      c = fmaf(g, (to_f32(xr[i]) - mu) * r, c);
    }
    a = block_sum(a, s) * inv;
    c = block_sum(c, s) * inv;
    T* o = dx.row(t);
    for (int i = threadIdx.x; i < H; i += 256) {
      const float g = to_f32(gr[i]) * to_f32(w[i]);
      const float xh = (to_f32(xr[i]) - mu) * r;
      float d = (g - a - xh * c) * r;
      if (add.p != nullptr) d += to_f32(add.row(t)[i]);
      o[i] = from_f32<T>(d);
    }
  }
}

// Column sums of one range of rows per blockIdx.y: a thread owns a column.
// part[(blockIdx.y * 2 + {0, 1}) * H + i] = {sum dy xh, sum dy} over the range.
template <typename T>
__global__ void __launch_bounds__(256) norm_cols_loop_kernel(Rows<const T> dy, Rows<const T> x,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             int T_, int H, int rows,
                                                             float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= H) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t t1 = min(static_cast<int64_t>(T_), t0 + rows);
  float a = 0.f, c = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const float g = to_f32(dy.row(t)[i]);
    a = fmaf(g, (to_f32(x.row(t)[i]) - mean[t]) * rstd[t], a);
    c += g;
  }
  part[(static_cast<int64_t>(blockIdx.y) * 2) * H + i] = a;
  part[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * H + i] = c;
}

// dweight / dbias from n partial rows, added in order.
template <typename P>
__global__ void __launch_bounds__(256) norm_cols_finish_kernel(const float* __restrict__ part,
                                                               int n, int H, P* __restrict__ dw,
                                                               P* __restrict__ db) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[2][8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float a = 0.f, c = 0.f;
  if (i < H) {
    for (int j = w; j < n; j += 8) {
      a += part[(static_cast<int64_t>(j) * 2) * H + i];
      c += part[(static_cast<int64_t>(j) * 2 + 1) * H + i];
    }
  }
  s[0][w][lane] = a;
  s[1][w][lane] = c;
  __syncthreads();
  if (w < 2 && i < H) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += s[w][j][lane];
    if (w == 0)
      dw[i] = from_f32<P>(t);
    else if (db != nullptr)
      db[i] = from_f32<P>(t);
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

// Whether rows (null: absent) split into units of V bytes.
template <typename T>
static bool units_ok(const Rows<T>& r, int64_t rows, int H, size_t V) {
  return r.p == nullptr || (reinterpret_cast<uintptr_t>(r.p) % V == 0 && H * sizeof(T) % V == 0 &&
                            (rows == 1 || r.ld * sizeof(T) % V == 0));
}

static int round32(int n) { return (n + 31) / 32 * 32; }

template <typename T, typename P, int V, int NU>
static cudaError_t fwd_launch(const Ctx& c, int GT, Rows<const T> x, Rows<T> y, int T_, int H,
                              const P* w, const P* b, float eps, float* mean, float* rstd) {
  const int groups = GT >= 256 ? 1 : 256 / GT;
  return launch_k(c.stream, norm_fwd_kernel<T, P, V, NU>, dim3((T_ + groups - 1) / groups),
                  dim3(groups * GT), 0, x, y, T_, H, GT, w, b, eps, mean, rstd);
}

template <typename T, typename P, int V>
static cudaError_t fwd_units(const Ctx& c, Rows<const T> x, Rows<T> y, int T_, int H, const P* w,
                             const P* b, float eps, float* mean, float* rstd) {
  const int units = H / (V / static_cast<int>(sizeof(T)));
  constexpr int NMAX = V == 16 ? 8 : 16;
  // few rows: a row over more threads ends sooner; many: fewer threads sum it more cheaply
  const int want = T_ <= c.num_sms * 4 ? NMAX / 8 : NMAX;
  const int GT = std::min(512, round32((units + want - 1) / want));
  const int nu = (units + GT - 1) / GT;
#define MM_FWD(N) \
  if (nu <= N) return fwd_launch<T, P, V, N>(c, GT, x, y, T_, H, w, b, eps, mean, rstd)
  if constexpr (V == 16) {
    MM_FWD(1);
    MM_FWD(2);
    MM_FWD(4);
    MM_FWD(8);
  } else {
    MM_FWD(2);
    MM_FWD(16);
  }
#undef MM_FWD
  return launch_k(c.stream, norm_fwd_loop_kernel<T, P>, dim3(std::min(T_, c.num_sms * 8)),
                  dim3(256), 0, x, y, T_, H, w, b, eps, mean, rstd);
}

template <typename T, typename P>
static mm_moe_status norm_forward(const Ctx& c, const mm_moe_norm_shape* s, const void* x,
                                  int64_t ldx, const void* w_, const void* b_, void* y,
                                  int64_t ldy, float* mean, float* rstd) {
  const int T_ = static_cast<int>(s->T), H = static_cast<int>(s->H);
  const Rows<const T> xr{static_cast<const T*>(x), ldx};
  const Rows<T> yr{static_cast<T*>(y), ldy};
  const P* w = static_cast<const P*>(w_);
  const P* b = static_cast<const P*>(b_);
  const auto ok = [&](size_t V) { return units_ok(xr, T_, H, V) && units_ok(yr, T_, H, V); };
  prof_begin(c, K_NORM_FWD);
  cudaError_t e;
  if (ok(16) && vec_ok(w, 16) && (b == nullptr || vec_ok(b, 16)))
    e = fwd_units<T, P, 16>(c, xr, yr, T_, H, w, b, s->eps, mean, rstd);
  else if (sizeof(T) == 4 || ok(4))
    e = fwd_units<T, P, 4>(c, xr, yr, T_, H, w, b, s->eps, mean, rstd);
  else
    e = fwd_units<T, P, sizeof(T)>(c, xr, yr, T_, H, w, b, s->eps, mean, rstd);
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
};

template <typename T, int V, int NU>
static cudaError_t bwd_launch(const Ctx& c, const BwdArgs<T>& a, int units, int* n_part) {
  constexpr int C = NU * V / static_cast<int>(sizeof(T));
  const int GT = round32((units + NU - 1) / NU);
  const int groups =
      std::min(NORM_BWD_THREADS / GT, (a.T_ + c.num_sms - 1) / c.num_sms);
  const int nt = GT * groups;
  size_t smem = groups > 1 ? static_cast<size_t>(2) * C * nt * sizeof(float) : 0;
  if (V >= 4)
    smem = std::max(smem, static_cast<size_t>(norm_stages<T, V, NU>) *
                              (a.add.p != nullptr ? 3 : 2) * NU * V * nt);
  auto* kern = norm_bwd_kernel<T, V, NU>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  *n_part = std::min(c.num_sms, (a.T_ + groups - 1) / groups);
  return launch_k(c.stream, kern, dim3(*n_part), dim3(nt), smem, a.dy, a.x, a.add, a.dx, a.w,
                  a.w32, a.mean, a.rstd, a.T_, a.H, GT, a.part);
}

// 16 columns a thread where a warp would otherwise not hold the row, else as few as fill it
template <typename T, int V>
static cudaError_t bwd_units(const Ctx& c, const BwdArgs<T>& a, int* n_part) {
  constexpr int U = V / static_cast<int>(sizeof(T));
  const int units = a.H / U;
  if (units <= 32) return bwd_launch<T, V, 1>(c, a, units, n_part);
  if constexpr (V == 16 && sizeof(T) == 4) {
    if (a.H <= 4096) return bwd_launch<T, V, 2>(c, a, units, n_part);
  }
  return bwd_launch<T, V, 16 / U>(c, a, units, n_part);
}

constexpr int NORM_BWD_MAX_H = NORM_BWD_THREADS * 16;

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
                     part};
  const auto ok = [&](size_t V) {
    return units_ok(a.dy, T_, H, V) && units_ok(a.x, T_, H, V) && units_ok(a.add, T_, H, V) &&
           units_ok(a.dx, T_, H, V);
  };
  cudaError_t e;
  int n = 0;
  if (H <= NORM_BWD_MAX_H) {
    prof_begin(c, K_NORM_BWD);
    if (ok(16))
      e = bwd_units<T, 16>(c, a, &n);
    else if (sizeof(T) == 4 || ok(4))
      e = bwd_units<T, 4>(c, a, &n);
    else
      e = bwd_units<T, sizeof(T)>(c, a, &n);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
  } else {
    prof_begin(c, K_NORM_BWD);
    e = launch_k(c.stream, norm_dx_loop_kernel<T, P>, dim3(std::min(T_, c.num_sms * 8)), dim3(256),
                 0, a.dy, a.x, static_cast<const P*>(w), mean, rstd, a.add, a.dx, T_, H);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
    const int want = std::min(norm_parts(T_), std::max(1, c.num_sms * 8 / ((H + 255) / 256)));
    const int rows = (T_ + want - 1) / want;
    n = (T_ + rows - 1) / rows;
    prof_begin(c, K_NORM_BWD);
    e = launch_k(c.stream, norm_cols_loop_kernel<T>, dim3((H + 255) / 256, n), dim3(256), 0, a.dy,
                 a.x, mean, rstd, T_, H, rows, part);
    prof_end(c, K_NORM_BWD);
    if (e != cudaSuccess) return MM_MOE_ECUDA;
  }
  prof_begin(c, K_NORM_BWD_FINISH);
  e = launch_k(c.stream, norm_cols_finish_kernel<P>, dim3((H + 31) / 32), dim3(256), 0,
               static_cast<const float*>(part), n, H, static_cast<P*>(dw), static_cast<P*>(db));
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
