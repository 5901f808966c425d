// gradclip.cu -- the global L2 norm of many gradient tensors, and clipping by it.
//
//   norm = (sum over tensors and elements of g^2)^(1/2)
//   coef = min(1, max_norm / (norm + eps)),   out = coef g
//
// The tensors' addresses travel in the kernels' parameters, so a call needs no copy to
// the device and holds nothing from one call to the next.  The tensors are cut into
// chunks of CHUNK elements; the CTAs of a launch take every gridDim.x-th chunk.  Squares
// are summed in fp32 inside a thread's share of a chunk and in fp64 from there on; a
// share whose fp32 sum leaves [1e-30, 1e36] (squares that overflow or vanish although
// their values do not) is summed again in fp64.  Every sum has a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ops.cuh"

namespace mmmoe {

constexpr int GC_THREADS = 256;
constexpr int GC_CHUNK = 16384;  // elements: 8 16-byte vectors per thread in 16 bits, 16 in fp32
constexpr int GC_SHORT = 4096;   // of few and small tensors, up to one for every SM (250,000
                                 // elements 5.4 us in long ones, 4.6 in short ones; 1 M 5.7, 6.4)
constexpr int GC_MAX = 384;      // tensors per launch (11 KB of parameters) ...
constexpr int GC_FEW = 32;       // ... and of a launch with few (1 KB)
constexpr int GC_CTAS = 4;       // CTAs per SM, all resident
// The first pass reads all but its last GC_KEEP chunks (64 MB of 16-bit gradients) as
// streaming data, so that L2 holds those when the second pass begins with them.
constexpr int GC_KEEP = 2000;

// The tensors of one launch.  Elements [0, head) of a tensor precede its first 16-byte
// boundary; chunk c covers head + [c, c + 1) CHUNK, the first chunk the head too.
template <int N, int CHUNK_>
struct GradList {
  static constexpr int CHUNK = CHUNK_;
  const void* in[N];
  void* out[N];
  int64_t n[N];
  int first[N + 1];  // first chunk of each tensor in the launch's numbering
  uint8_t dt[N];     // in | out << 4
  int count;
};

template <typename L>
__device__ __forceinline__ int find_tensor(const L& g, int chunk) {
  int lo = 0, hi = g.count - 1;  // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
  const int64_t h = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(T);
  return h < n ? h : n;
}

template <int CHUNK, typename T>
__device__ __forceinline__ double sq_chunk(const T* p, int64_t n, int64_t chunk, bool keep) {
  constexpr int N = VN<T>;
  constexpr int PER = CHUNK / N / GC_THREADS;
  constexpr int BATCH = PER < 8 ? PER : 8;  // vectors in flight per thread
  const int64_t head = head_of(p, n);
  const int64_t a = head + chunk * CHUNK;
  const int64_t len = n > a ? (n - a < CHUNK ? n - a : CHUNK) : 0;
  const uint4* v = reinterpret_cast<const uint4*>(p + a);
  const int nv = static_cast<int>(len / N);
  double acc = 0.0;
  for (int j0 = threadIdx.x; j0 < nv; j0 += BATCH * GC_THREADS) {
    uint4 q[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      q[i] = j0 + i * GC_THREADS >= nv ? make_uint4(0, 0, 0, 0)
             : keep                    ? __ldg(v + j0 + i * GC_THREADS)
                                       : __ldcs(v + j0 + i * GC_THREADS);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      float f[N];
      unpack(q[i], f, p);
#pragma unroll
      for (int j = 0; j < N; ++j) s = fmaf(f[j], f[j], s);
    }
    constexpr uint32_t MAGNITUDE = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
    bool again = !(s <= 1e36f);
    if (s < 1e-30f) {
      uint32_t bits = 0;  // (all zero: an expert without tokens, nothing to add again)
#pragma unroll
      for (int i = 0; i < BATCH; ++i) bits |= (q[i].x | q[i].y | q[i].z | q[i].w) & MAGNITUDE;
      again = bits != 0;
    }
    if (again) {
#pragma unroll 1
      for (int j = j0; j < nv && j < j0 + BATCH * GC_THREADS; j += GC_THREADS) {
        float f[N];
        unpack(__ldg(v + j), f, p);
#pragma unroll
        for (int t = 0; t < N; ++t) acc += static_cast<double>(f[t]) * static_cast<double>(f[t]);
      }
    } else {
      acc += s;
    }
  }
  // the elements before the first and after the last whole vector
  const int tail = static_cast<int>(len - static_cast<int64_t>(nv) * N);
  if (static_cast<int>(threadIdx.x) < tail) {
    const double f = to_f32(p[a + static_cast<int64_t>(nv) * N + threadIdx.x]);
    acc += f * f;
  }
  if (chunk == 0 && static_cast<int>(threadIdx.x) < head) {
    const double f = to_f32(p[threadIdx.x]);
    acc += f * f;
  }
  return acc;
}

// Sums in fp64 go through one warp: the SM adds two doubles a cycle, so an addition by
// every thread of its CTAs takes half a microsecond (all warps joining the partial sums and
// taking the root cost the second pass 6 us: 5 M gradients 15.4 us, so 9.1).
__device__ __forceinline__ double tile_sum(const double* s, int n) {
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += 32) a += s[i];
  return a;
}

// part[blockIdx.x] = the CTA's share of the sum of squares.  1.2 GB in 167 us (reads alone, a
// little above the copy rate).
template <typename L>
__global__ void __launch_bounds__(GC_THREADS, GC_CTAS) grad_sq_kernel(
    const __grid_constant__ L g, double* __restrict__ part) {
  __shared__ double s[GC_THREADS];
  pdl_wait();
  pdl_trigger();
  const int total = g.first[g.count];
  double acc = 0.0;
  int t = blockIdx.x < total ? find_tensor(g, blockIdx.x) : 0;
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    while (t + 1 < g.count && g.first[t + 1] <= c) ++t;
    const int64_t k = c - g.first[t];
    const int d = g.dt[t] & 15;
    const bool keep = c >= total - GC_KEEP;
    if (d == MM_MOE_DT_BF16)
      acc += sq_chunk<L::CHUNK>(static_cast<const __nv_bfloat16*>(g.in[t]), g.n[t], k, keep);
    else if (d == MM_MOE_DT_F16)
      acc += sq_chunk<L::CHUNK>(static_cast<const __half*>(g.in[t]), g.n[t], k, keep);
    else
      acc += sq_chunk<L::CHUNK>(static_cast<const float*>(g.in[t]), g.n[t], k, keep);
  }
  s[threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  acc = warp_sum(tile_sum(s, GC_THREADS));
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm from n partial sums, the same in every CTA (and in every thread of it).
__device__ __forceinline__ float norm_of(const double* part, int n) {
  // (a tile that held all of a launch's sums, 4 KB more a CTA, would leave less of L1 to the
  // scaling: 604 M gradients 544 us with this one, 624 with that)
  constexpr int TILE = GC_THREADS;
  __shared__ double s[TILE];
  __shared__ float s_norm;
  double a = 0.0;
  for (int i0 = 0; i0 < n; i0 += TILE) {
    if (i0 > 0) __syncthreads();
    if (i0 + static_cast<int>(threadIdx.x) < n) s[threadIdx.x] = __ldcg(part + i0 + threadIdx.x);
    __syncthreads();
    if (threadIdx.x < 32) a += tile_sum(s, min(TILE, n - i0));
  }
  if (threadIdx.x < 32) {
    a = warp_sum(a);
    if (threadIdx.x == 0) s_norm = static_cast<float>(sqrt(a));
  }
  __syncthreads();
  return s_norm;
}

__global__ void __launch_bounds__(GC_THREADS) grad_norm_kernel(const double* __restrict__ part,
                                                               int n, float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  const float v = norm_of(part, n);
  if (threadIdx.x == 0) *norm = v;
}

// One vector of TI (16 bytes, or 8 where 16 bits widen to fp32, so that a store is 16).
template <typename TI, typename TO>
__device__ __forceinline__ uint4 scale_vec(const std::conditional_t<sizeof(TI) == sizeof(TO), uint4, uint2>& q,
                                           float coef) {
  if constexpr (sizeof(TI) == sizeof(TO)) {
    float f[VN<TI>];
    unpack(q, f, static_cast<const TI*>(nullptr));
#pragma unroll
    for (int t = 0; t < VN<TI>; ++t) f[t] *= coef;
    return pack(f, static_cast<const TO*>(nullptr));
  } else {
    float f[8];
    unpack(make_uint4(q.x, q.y, 0, 0), f, static_cast<const TI*>(nullptr));
    return make_uint4(__float_as_uint(f[0] * coef), __float_as_uint(f[1] * coef),
                      __float_as_uint(f[2] * coef), __float_as_uint(f[3] * coef));
  }
}

template <int CHUNK, typename TI, typename TO>
__device__ __forceinline__ void scale_chunk(const TI* p, TO* o, int64_t n, int64_t chunk,
                                            float coef) {
  using V = std::conditional_t<sizeof(TI) == sizeof(TO), uint4, uint2>;
  constexpr int N = 16 / static_cast<int>(sizeof(TO));  // elements of a vector
  constexpr int PER = CHUNK / N / GC_THREADS;
  constexpr int BATCH = PER < 4 ? PER : 4;  // vectors in flight per thread (8 measured 1 to 6% slower)
  const int64_t head = head_of(p, n);
  const int64_t a = head + chunk * CHUNK;
  const int len = static_cast<int>(n > a ? (n - a < CHUNK ? n - a : CHUNK) : 0);
  const int tid = threadIdx.x;
  int done = 0;
  if (reinterpret_cast<uintptr_t>(o + a) % 16 == 0) {
    const V* v = reinterpret_cast<const V*>(p + a) + tid;
    uint4* w = reinterpret_cast<uint4*>(o + a) + tid;
    const int nv = len / N;
    done = nv * N;
    if (len == CHUNK) {
#pragma unroll 1
      for (int i0 = 0; i0 < PER; i0 += BATCH, v += BATCH * GC_THREADS, w += BATCH * GC_THREADS) {
        V q[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) q[i] = v[i * GC_THREADS];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) w[i * GC_THREADS] = scale_vec<TI, TO>(q[i], coef);
      }
    } else {
#pragma unroll 1
      for (int j0 = tid; j0 < nv; j0 += 4 * GC_THREADS, v += 4 * GC_THREADS, w += 4 * GC_THREADS) {
        V q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i * GC_THREADS < nv) q[i] = v[i * GC_THREADS];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i * GC_THREADS < nv) w[i * GC_THREADS] = scale_vec<TI, TO>(q[i], coef);
      }
    }
  }
  for (int j = done + tid; j < len; j += GC_THREADS)
    o[a + j] = from_f32<TO>(to_f32(p[a + j]) * coef);
  if (chunk == 0 && tid < head) o[tid] = from_f32<TO>(to_f32(p[tid]) * coef);
}

// Every CTA joins the partial sums by itself (a few KB from L2), so no launch and no
// counter stands between the two passes; the first one also stores the norm.  The chunks
// go backwards, from what the first pass left in L2.  The benchmark layer's gradients (604 M
// bf16, into bf16) took 561 us forwards, 555 backwards, 544 with the first pass's streaming
// loads: 3.6 GB moved at 6.65 TB/s.  Four CTAs an SM leave 64 registers a thread, of
// which the five type pairs spill 112 to 144 bytes; the pass runs at the copy rate all the same.
template <typename L>
__global__ void __launch_bounds__(GC_THREADS, GC_CTAS) grad_scale_kernel(
    const __grid_constant__ L g, const double* __restrict__ part, int n_part,
    float max_norm, float eps, bool all_in_place, float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  const float nrm = norm_of(part, n_part);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  const float ratio = max_norm / (nrm + eps);
  const float coef = ratio > 1.f ? 1.f : ratio;  // a NaN stays one
  if (all_in_place && coef == 1.f) return;  // nothing changes
  const int total = g.first[g.count];
  const int last = total - 1 - static_cast<int>(blockIdx.x);
  int t = last >= 0 ? find_tensor(g, last) : 0;
  for (int c = last; c >= 0; c -= gridDim.x) {
    while (g.first[t] > c) --t;
    const void* in = g.in[t];
    void* out = g.out[t];
    if (in == out && coef == 1.f) continue;
    const int64_t k = c - g.first[t], n = g.n[t];
    switch (g.dt[t]) {
      case MM_MOE_DT_BF16 | MM_MOE_DT_BF16 << 4:
        scale_chunk<L::CHUNK>(static_cast<const __nv_bfloat16*>(in), static_cast<__nv_bfloat16*>(out), n, k,
                    coef);
        break;
      case MM_MOE_DT_F16 | MM_MOE_DT_F16 << 4:
        scale_chunk<L::CHUNK>(static_cast<const __half*>(in), static_cast<__half*>(out), n, k, coef);
        break;
      case MM_MOE_DT_BF16 | MM_MOE_DT_F32 << 4:
        scale_chunk<L::CHUNK>(static_cast<const __nv_bfloat16*>(in), static_cast<float*>(out), n, k, coef);
        break;
      case MM_MOE_DT_F16 | MM_MOE_DT_F32 << 4:
        scale_chunk<L::CHUNK>(static_cast<const __half*>(in), static_cast<float*>(out), n, k, coef);
        break;
      default:
        scale_chunk<L::CHUNK>(static_cast<const float*>(in), static_cast<float*>(out), n, k, coef);
    }
  }
}

static bool al(const void* p, uintptr_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

// Elements of all tensors together: their chunks count in 32 bits.
constexpr int64_t MAX_TOTAL = int64_t{1} << 43;

static bool grads_ok(const mm_moe_grad* g, int64_t n, bool clip) {
  if (n < 0 || n > MM_MOE_MAX_GRADS || (n > 0 && g == nullptr)) return false;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (!dtype_ok(g[i].dtype) || g[i].numel < 0 || g[i].numel > MAX_TOTAL) return false;
    if ((total += g[i].numel) > MAX_TOTAL) return false;
    if (g[i].numel > 0 && !al(g[i].grad, dtype_bytes(g[i].dtype))) return false;
    if (!clip) continue;
    if (g[i].out_dtype != g[i].dtype && g[i].out_dtype != MM_MOE_DT_F32) return false;
    if (g[i].numel > 0 && !al(g[i].out, dtype_bytes(g[i].out_dtype))) return false;
    if (g[i].numel > 0 && g[i].out == g[i].grad && g[i].out_dtype != g[i].dtype) return false;
  }
  return true;
}

// Up to N tensors from i on into a list; returns the first one left out.
template <int N, int CHUNK>
static int64_t fill_list(GradList<N, CHUNK>* l, const mm_moe_grad* g, int64_t i, int64_t n) {
  l->count = 0;
  int chunks = 0;
  for (; i < n && l->count < N; ++i) {
    if (g[i].numel == 0) continue;
    l->in[l->count] = g[i].grad;
    l->out[l->count] = g[i].out;
    l->n[l->count] = g[i].numel;
    l->dt[l->count] = static_cast<uint8_t>(g[i].dtype | g[i].out_dtype << 4);
    l->first[l->count++] = chunks;
    chunks += static_cast<int>((g[i].numel + CHUNK - 1) / CHUNK);
  }
  l->first[l->count] = chunks;
  return i;
}

static int64_t max_lists(int64_t n) { return n / GC_MAX + 1; }

// f(list) over lists of all tensors; at least one call when `always`.
template <typename F>
static cudaError_t each_list(const mm_moe_grad* g, int64_t n, bool always, F f) {
  const auto once = [&](auto l) {
    fill_list(&l, g, 0, n);
    return l.count > 0 || always ? f(l) : cudaSuccess;
  };
  if (n <= GC_FEW) {
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) total += g[i].numel;
    // (up to a short chunk for every SM)
    if (total <= GC_SHORT * 152) return once(GradList<GC_FEW, GC_SHORT>{});
    return once(GradList<GC_FEW, GC_CHUNK>{});
  }
  GradList<GC_MAX, GC_CHUNK> l;
  cudaError_t e = cudaSuccess;
  for (int64_t i = 0; i < n && e == cudaSuccess; always = false) {
    i = fill_list(&l, g, i, n);
    if (l.count > 0 || always) e = f(l);
  }
  return e;
}

// Sum-of-squares launches over all tensors; *n_part partials are written.
static cudaError_t launch_sq(const Ctx& c, const mm_moe_grad* g, int64_t n, double* part,
                             int* n_part) {
  *n_part = 0;
  return each_list(g, n, false, [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    const int grid = std::min(c.num_sms * GC_CTAS, l.first[l.count]);
    prof_begin(c, K_GRAD_SQ);
    const cudaError_t e = launch_k(c.stream, grad_sq_kernel<L>, dim3(grid), dim3(GC_THREADS), 0, l,
                                   part + *n_part);
    prof_end(c, K_GRAD_SQ);
    *n_part += grid;
    return e;
  });
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_grad_workspace_size(int64_t n_tensors, size_t* bytes) {
  if (n_tensors < 0 || n_tensors > MM_MOE_MAX_GRADS || bytes == nullptr) return MM_MOE_EINVAL;
  *bytes = static_cast<size_t>(max_lists(n_tensors)) * 152 * GC_CTAS * sizeof(double);
  return MM_MOE_OK;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_grad_norm(const mm_moe_grad* grads, int64_t n_tensors,
                                                     float* norm, void* workspace, void* stream) {
  if (!grads_ok(grads, n_tensors, false) || !al(norm, 4) || !al(workspace, 16))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  double* part = static_cast<double*>(workspace);
  int n_part = 0;
  cudaError_t e = launch_sq(c, grads, n_tensors, part, &n_part);
  if (e != cudaSuccess) return op_status(e);
  prof_begin(c, K_GRAD_NORM);
  e = launch_k(c.stream, grad_norm_kernel, dim3(1), dim3(GC_THREADS), 0,
               static_cast<const double*>(part), n_part, norm);
  prof_end(c, K_GRAD_NORM);
  return op_status(e);
}

extern "C" MM_MOE_API mm_moe_status mm_moe_grad_clip(const mm_moe_grad* grads, int64_t n_tensors,
                                                     float max_norm, float eps, float* norm,
                                                     void* workspace, void* stream) {
  if (!grads_ok(grads, n_tensors, true) || !(max_norm >= 0.f) || !(eps >= 0.f) || !al(norm, 4) ||
      !al(workspace, 16))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  double* part = static_cast<double*>(workspace);
  int n_part = 0;
  cudaError_t e = launch_sq(c, grads, n_tensors, part, &n_part);
  if (e != cudaSuccess) return op_status(e);
  bool in_place = true;
  for (int64_t i = 0; i < n_tensors; ++i)
    in_place = in_place && (grads[i].numel == 0 || grads[i].out == grads[i].grad);
  e = each_list(grads, n_tensors, true, [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    const int grid = std::max(1, std::min(c.num_sms * GC_CTAS, l.first[l.count]));
    prof_begin(c, K_GRAD_SCALE);
    const cudaError_t r =
        launch_k(c.stream, grad_scale_kernel<L>, dim3(grid), dim3(GC_THREADS), 0, l,
                 static_cast<const double*>(part), n_part, max_norm, eps, in_place, norm);
    prof_end(c, K_GRAD_SCALE);
    return r;
  });
  return op_status(e);
}
