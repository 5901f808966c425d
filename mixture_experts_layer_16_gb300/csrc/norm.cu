// norm.cu -- layer normalisation in front of the layer: the forward (formulas in norm.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "norm.cuh"
#include "ops.cuh"

namespace mmmoe {

// ------------------------------------------------------------------------- forward
// A thread with up to 16 columns holds its parameters in registers; with more columns a
// row needs fewer threads, so fewer sums across warps (none up to 2048 columns of 16 bits:
// 16384 x 2048 bf16 takes 31.8 us with 128 threads a row, 16 columns each, 22.4 us with a
// warp a row, 0.88 of the copy rate), and the parameters come from shared memory.  Where several warps share a
// row and registers allow it, a group takes two rows at a time (ROWS), so that two share
// the two barriers.
template <typename T, typename P, int NU, Cut CUT, int ROWS>
__global__ void __launch_bounds__(NORM_THREADS, 1) norm_fwd_kernel(
    Rows<const T> x, Rows<T> y, int T_, int H, int GT, const P* __restrict__ w,
    const P* __restrict__ b, float eps, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int U = VN<T>, C2 = NU * U / 2, S = norm_fwd_steps<NU, ROWS>;
  constexpr bool PS = norm_params_shared<T, NU>;
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
  // shared, rows of whole units: weight then bias in fp32, the two halves of the units apart
  // (16-byte reads of consecutive units then meet no bank twice); others, whose units begin at
  // any column: (weight, bias) by column modulo U, so that the k-th columns of consecutive
  // units are neighbours whatever the shift, with zeros around the row
  const uint32_t sw = ring - threadIdx.x * 16 + S * step_bytes;
  const int pitch = H / U + 3;  // of a residue
  if constexpr (PS && CUT == ANY) {
    float2* s = reinterpret_cast<float2*>(ring_bytes + S * step_bytes);
    for (int c = static_cast<int>(threadIdx.x) - U; c < (pitch - 1) * U; c += nt) {
      const bool in = p.in(c);
      s[(c + U) % U * pitch + (c + U) / U] = make_float2(
          in ? to_f32(w[c]) : 0.f, in && b != nullptr ? to_f32(b[c]) : 0.f);
    }
    __syncthreads();
  } else if constexpr (PS) {
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
  uint32_t cut = 0;  // units that lie in the row in part, or not at all
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    full = full && p.whole(i);
    cut |= p.whole(i) ? 0u : 1u << i;
  }
  uint32_t sk[PS && CUT == ANY ? U : 1];  // the k-th column of this thread's unit 0
  if constexpr (PS && CUT == ANY)
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int c = k - p.shift + U;
      sk[k] = sw + (c % U * pitch + c / U + p.j) * 8;
    }
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
      // what is not in the row has no deviation either
      if constexpr (CUT == ANY) {
#pragma unroll
        for (int i = 0; i < NU; ++i)
          if (cut & 1u << i) {
#pragma unroll
            for (int k = i * U / 2; k < (i + 1) * U / 2; ++k) {
              const int c = p.col(i) + 2 * k % U;
              float lo, hi;
              f2_split(v[r][k], lo, hi);
              v[r][k] = f2_make(p.in(c) ? lo : 0.f, p.in(c + 1) ? hi : 0.f);
            }
          }
      } else if (!full) {
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
        if constexpr (PS && CUT == ANY) {
#pragma unroll
          for (int k = 0; k < U / 2; ++k) {
            float lo, hi;
            f2_split(f2_mul(v[r][i * U / 2 + k], r2), lo, hi);
            const float2 a = lds8(sk[2 * k] + i * GT * 8), c = lds8(sk[2 * k + 1] + i * GT * 8);
            u[k] = f2_make(fmaf(lo, a.x, a.y), fmaf(hi, c.x, c.y));
          }
        } else if constexpr (PS) {
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

// One CTA per row; the row is read three times (sum, centred squares, output), the
// second and third time from L1/L2.  2048 x 16384 bf16: 34.0 us, 0.58 of the copy rate.
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

template <typename T, typename P, int NU, int ROWS>
static cudaError_t fwd_launch(const Ctx& c, Rows<const T> x, Rows<T> y, int T_, int H, const P* w,
                              const P* b, float eps, float* mean, float* rstd) {
  const int GT = group_threads<T, NU>(H, even_rows(x, T_));
  constexpr int RING = norm_fwd_steps<NU, ROWS> * ROWS * NU * 16;  // bytes per thread
  // the ring and shared parameters have to fit beside each other
  constexpr int U = VN<T>;
  const int shared = norm_params_shared<T, NU> ? 8 * (H + 4 * U) : 0;
  const int fit = (224 * 1024 - shared) / (RING * GT);
  const NormGrid n = norm_grid(GT, T_, c.num_sms, fit);
  const int nt = n.GT * n.groups;
  const size_t smem = static_cast<size_t>(RING) * nt + shared;
  const bool even = even_rows(x, T_) && H % VN<T> == 0;
  // (fp32 rows on 16-byte boundaries have at most four units a thread)
  constexpr Cut WHOLE = sizeof(T) == 4 && NU > 4 ? ANY : EVEN;
  auto* kern =
      even ? norm_fwd_kernel<T, P, NU, WHOLE, ROWS> : norm_fwd_kernel<T, P, NU, ANY, ROWS>;
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
  constexpr int U = VN<T>, MOST = 16 / U;  // units of 16 columns
  const bool even = even_rows(x, T_), any = !even || H % U != 0;
  const auto go = [&](auto nu, auto rows) {
    return fwd_launch<T, P, decltype(nu)::value, decltype(rows)::value>(c, x, y, T_, H, w, b,
                                                                        s->eps, mean, rstd);
  };
  // every group has one row at most
  const auto one_round = [&](int GT) {
    return GT != 0 && T_ <= c.num_sms / 8 * 8 * (NORM_THREADS / GT);
  };
  const auto pick = [&]() -> cudaError_t {
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, MOST> most{};
    if (same_cut(x, y, T_)) {
      // few rows: as many threads for each as there are (300 x 2048 bf16 2.6 us, with a warp a
      // row 4.0; two units a thread where they spare a second warp: 300 x 512 bf16 2.0 and 2.1)
      const int g1 = group_threads<T, 1>(H, even);
      if (one_round(g1) && !(sizeof(T) == 2 && g1 == 64)) return go(one, one);
      if (T_ <= 4 * c.num_sms && one_round(group_threads<T, 2>(H, even))) return go(two, one);
      const int GT = group_threads<T, MOST>(H, even);
      // the units a row may have, whatever its cut
      const int units = any ? (H + 2 * (U - 1)) / U : H / U;
      if constexpr (sizeof(T) == 2) {
        // As few warps as hold the row in 8 units a thread, and as few units as they need
        // (12000 x 2560 in five units 23.9 us, in eight 31.3; 8192 x 4096 in eight units
        // 25.2 us, in four, two rows a barrier, 26.8).  Rows on no boundary: also parts of a
        // warp, for what their ends cost is paid once for all rows of a warp (65536 x 511 in
        // 16 lanes 34.3 us, in 64 60.6; 8192 x 4095 31.8 and 50.1), once there are rows
        // enough for the parameters' way into shared memory (1216 x 1001 4.6 and 4.6, 600 x
        // 1001 5.3 and 3.7).
        // The same for rows above 8192 columns, up to what fits beside the parameters and
        // pays (row by row and so: 2600 x 12288 39.4 and 31.0, 2100 x 16001 69.4 and 53.1;
        // but 2048 x 16384 34.0 and 39.4, 600 x 9000 10.2 and 14.4).
        const bool many = T_ > 8 * c.num_sms;
        if (any || H > 8192 ? many && H > 128 && H <= (any ? 16384 : 12288) : H > 512) {
          int lanes = (units + 255) / 256 * 32;
          while (any && lanes <= 32 && lanes > 8 && units <= 4 * lanes) lanes /= 2;
          switch ((units + lanes - 1) / lanes) {
            case 1:
            case 2: break;
            case 3: return go(std::integral_constant<int, 3>{}, one);
            case 4: return go(std::integral_constant<int, 4>{}, one);
            case 5: return go(std::integral_constant<int, 5>{}, one);
            case 6: return go(std::integral_constant<int, 6>{}, one);
            case 7: return go(std::integral_constant<int, 7>{}, one);
            default: return go(std::integral_constant<int, 8>{}, one);
          }
        }
      } else if (any && H > 64 && H <= 8192) {
        // Where groups of four units a thread would leave over 30% of a CTA's slots empty: up to
        // 12 units a thread, with many rows, or where that makes a warp of two or more (us, in
        // four units and so: 65536 x 511 57.6 and 45.2, 30202 x 1111 49.8 and 45.3, 8192 x 4095
        // 55.2 and 46.9, 2000 x 511 4.6 and 3.7; but 5000 x 333 5.7 and 6.9, 4000 x 1111 10.5
        // and 10.9, and without empty slots 43690 x 767 44.7 and 46.8).
        const int slots = NORM_THREADS * MOST, used = GT == 0 ? 0 : NORM_THREADS / GT * units;
        if (used * 10 < slots * 7 &&
            ((units > 128 && units <= 256) || GT == 0 || T_ > 48 * c.num_sms)) {
          int lanes = (units + 383) / 384 * 32;
          while (lanes <= 32 && lanes > 8 && units <= 4 * lanes) lanes /= 2;
          const int n = (units + lanes - 1) / lanes;
          if (n <= 6) return go(std::integral_constant<int, 6>{}, one);
          if (n <= 8) return go(std::integral_constant<int, 8>{}, one);
          if (n <= 10) return go(std::integral_constant<int, 10>{}, one);
          return go(std::integral_constant<int, 12>{}, one);
        }
      }
      if (GT > 32 && !one_round(GT)) return go(most, two);
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
  return op_status(e);
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
  if (!same_rows(x, ldx, y, ldy, shape->T) && rows_overlap(x, ldx, y, ldy, shape))
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
