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

// Rows of partial column sums a backward of T rows writes (both the launch and the
// workspace size go by it).
constexpr int NORM_MAX_PARTS = 152 * 4;
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

template <typename T, typename P>
static mm_moe_status norm_forward(const Ctx& c, const mm_moe_norm_shape* s, const void* x,
                                  int64_t ldx, const void* w, const void* b, void* y, int64_t ldy,
                                  float* mean, float* rstd) {
  const int T_ = static_cast<int>(s->T), H = static_cast<int>(s->H);
  prof_begin(c, K_NORM_FWD);
  const cudaError_t e = launch_k(
      c.stream, norm_fwd_loop_kernel<T, P>, dim3(std::min(T_, c.num_sms * 8)), dim3(256), 0,
      Rows<const T>{static_cast<const T*>(x), ldx}, Rows<T>{static_cast<T*>(y), ldy}, T_, H,
      static_cast<const P*>(w), static_cast<const P*>(b), s->eps, mean, rstd);
  prof_end(c, K_NORM_FWD);
  return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ECUDA;
}

template <typename T, typename P>
static mm_moe_status norm_backward(const Ctx& c, const mm_moe_norm_shape* s, const void* dy,
                                   int64_t lddy, const void* x, int64_t ldx, const void* w,
                                   const float* mean, const float* rstd, const void* add,
                                   int64_t ldadd, void* dx, int64_t lddx, void* dw, void* db,
                                   float* part) {
  const int T_ = static_cast<int>(s->T), H = static_cast<int>(s->H);
  const Rows<const T> gr{static_cast<const T*>(dy), lddy}, xr{static_cast<const T*>(x), ldx},
      ar{static_cast<const T*>(add), ldadd};
  const Rows<T> dr{static_cast<T*>(dx), lddx};
  prof_begin(c, K_NORM_BWD);
  cudaError_t e = launch_k(c.stream, norm_dx_loop_kernel<T, P>, dim3(std::min(T_, c.num_sms * 8)),
                           dim3(256), 0, gr, xr, static_cast<const P*>(w), mean, rstd, ar, dr, T_,
                           H);
  prof_end(c, K_NORM_BWD);
  if (e != cudaSuccess) return MM_MOE_ECUDA;
  const int want = std::min(norm_parts(T_), std::max(1, c.num_sms * 8 / ((H + 255) / 256)));
  const int rows = (T_ + want - 1) / want, n = (T_ + rows - 1) / rows;
  prof_begin(c, K_NORM_BWD);
  e = launch_k(c.stream, norm_cols_loop_kernel<T>, dim3((H + 255) / 256, n), dim3(256), 0, gr, xr,
               mean, rstd, T_, H, rows, part);
  prof_end(c, K_NORM_BWD);
  if (e != cudaSuccess) return MM_MOE_ECUDA;
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
  const int sms = sm_count_103();
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
  const int sms = sm_count_103();
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
