// resnorm_bwd.cu -- the norms before and after a block with its gate and residual scale: the
// backward, with the reduction of the parameters' gradients (formulas in resnorm.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "ops.cuh"
#include "resnorm.cuh"

namespace mmmoe {

template <typename T, typename R>
struct BwdOps {
  Rows<const R> dout;  // null: zero
  Rows<const T> dn;    // null: no norm in front of the next block
  Rows<const R> out;
  Rows<const T> f;  // null: neither f nor its gradient
  Rows<R> dx;
  Rows<T> df;
  const void *w_post, *gate_c, *gate_t, *w_pre;
  bool p32, sums_f;  // sums_f: K is wanted (a norm behind the block, or a gate of its channels)
  float scale;
  const float *rstd_f, *rstd_out;
  void* dgate_t;
  float* part;  // [CTA][2][H]: K, dw_pre
  float* mean_ov;  // [T] <oh v> (the looped kernels')
  int T_, H, GT;
  int steps, step_bytes;  // of the ring of single columns
};

// Bytes of a thread's share of a row in the ring.
template <typename T, typename R, int NU, int U>
constexpr int rn_bwd_bytes = 2 * (Operand<T, NU, U>::BYTES + Operand<R, NU, U>::BYTES);
// Steps of the ring: as many as fit beside so many bytes of parameters.
template <typename T, typename R, int NU>
constexpr int rn_bwd_steps(int params) {
  return std::max(1, std::min(4, (RN_SMEM - params) / (RN_THREADS * rn_bwd_bytes<T, R, NU, 8>)));
}

// What a launch has: any of the operands; dout, dn and f; these and the norm behind the block (asked for
// at run time that norm's term of df costs 3% of 16384 x 2048 bf16).
enum Have { SOME, ALL, ALL_POST };

// S: steps of the ring (units of 8).  dx, df and the CTA's column sums in one read; the column sums stay
// in the registers of the threads that own the columns, which leaves none for c and w: they are read from
// shared memory (in registers, with 72 bytes of spills: 16384 x 2048 bf16 92 us).
// 16384 x 2048 with the launch that ends it: 68.0 us in bf16 (0.87 of the copy rate), 99.3 with an fp32
// residual stream (0.89; its rows in halves of sectors 135, not on their way to L2 a row ahead 120); one
// unit a thread, eight warps a row: 93 and 130.
template <typename T, typename R, int NU, int U, int S, Have HAVE>
__global__ void __launch_bounds__(RN_THREADS, rn_ctas<NU, U>) resnorm_bwd_kernel(const BwdOps<T, R> a) {
  constexpr bool SHARED = U == 8, WHOLE = HAVE != SOME;
  using OT = Operand<T, NU, U>;
  using OR = Operand<R, NU, U>;
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  __shared__ float4 s_sum[2][RN_THREADS / 32];
  const uint32_t nt = blockDim.x, piece = nt * 16;
  const uint32_t step_bytes = U == 8 ? rn_bwd_bytes<T, R, NU, U> * nt : a.step_bytes;
  const int steps = U == 8 ? S : a.steps;
  pdl_wait();
  pdl_trigger();
  Cols<NU, U> c;
  c.init(a.GT, a.H);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)) +
                        (U == 8 ? threadIdx.x * 16 : c.g * (step_bytes / c.groups));
  const uint32_t out_at = U == 8 ? OR::BYTES * nt : single_bytes(a.H, sizeof(R)), dn_at = 2 * out_at,
                 f_at = dn_at + (U == 8 ? OT::BYTES * nt : single_bytes(a.H, sizeof(T)));
  const uint32_t n = a.T_, step = gridDim.x * c.groups;
  uint32_t t = blockIdx.x * c.groups + c.g, tw = c.first_of_warp(t), ta = t;
  const float inv = 1.f / static_cast<float>(a.H);
  const bool pre = WHOLE || a.dn.p != nullptr, has_f = WHOLE || a.f.p != nullptr,
             has_d = WHOLE || a.dout.p != nullptr;
  const bool post = HAVE == ALL_POST || a.w_post != nullptr;
  const auto issue = [&](uint32_t at) {
    if (ta < n) {
      if (has_d) OR::issue(c, a.dout.row(ta), at, piece);
      if (pre) {
        OR::issue(c, a.out.row(ta), at + out_at, piece);
        OT::issue(c, a.dn.row(ta), at + dn_at, piece);
      }
      if (has_f) OT::issue(c, a.f.row(ta), at + f_at, piece);
    }
    if constexpr (U == 8) {
      if (rn_prefetch<R> && c.j == 0) {
        const int64_t tp = static_cast<int64_t>(ta) + step;
        if (tp < n) {
          if (has_d) prefetch_row(a.dout.row(tp), a.H);
          if (pre) prefetch_row(a.out.row(tp), a.H), prefetch_row(a.dn.row(tp), a.H);
          if (has_f) prefetch_row(a.f.row(tp), a.H);
        }
      }
    }
    ta += step;
    async_commit();
  };
  for (int i = 0; i < steps - 1; ++i) issue(ring + i * step_bytes);
  constexpr int P = Cols<NU, U>::P, PIECES = Cols<NU, U>::PIECES;
  constexpr bool KEEP = U == 8 && NU == 1;  // x, out and f stay in registers between the two passes
  f2 K[NU * U / 2], dw[NU * U / 2];
  f2 cf1[SHARED ? 1 : NU * U / 2], w1[SHARED ? 1 : NU * U / 2];
  const uint32_t planes = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)) + steps * step_bytes,
                 plane = a.H / 8 * 16;
  {
    f2 cf[NU * U / 2], w[NU * U / 2];
    load_coef<T, NU, U>(c, a.w_post, a.gate_c, a.p32, a.scale, cf);
#pragma unroll
    for (int k = 0; k < NU * U / 2; ++k) w[k] = K[k] = dw[k] = 0;
    if (pre) load_params<T, NU, U>(c, a.w_pre, a.p32, w);
    if constexpr (SHARED) {
      if (c.g == 0) put_planes(c, planes, plane, cf, w);
      __syncthreads();
    } else {
#pragma unroll
      for (int k = 0; k < NU * U / 2; ++k) cf1[k] = cf[k], w1[k] = w[k];
    }
  }
  const auto params = [&](int i, f2 (&cf)[P], f2 (&w)[P]) {
    if constexpr (SHARED) {
      get_plane(c, planes, plane, i, cf);
      get_plane(c, planes + 2 * plane, plane, i, w);
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k) cf[k] = cf1[i * P + k], w[k] = w1[i * P + k];
    }
  };
  // the next row's gate and reciprocal norms, a row ahead
  float gt_n = 1.f, rf_n = 1.f, ro_n = 0.f;
  const auto stats = [&](uint32_t q) {
    if (q >= n) return;
    if (a.gate_t != nullptr) gt_n = param<T>(a.gate_t, a.p32, q);
    if (post) rf_n = __ldg(a.rstd_f + q);
    if (pre) ro_n = __ldg(a.rstd_out + q);
  };
  stats(t);
  int buf = 0;
  uint32_t st = ring, st_in = ring + (steps - 1) * step_bytes;
  const uint32_t ring_end = ring + steps * step_bytes;
  for (; tw < n; t += step, tw += step) {
    if constexpr (U == 8)
      issue(st_in);
    else
      single_turn(c.g, a.GT, steps, [&] { issue(st_in); });
    const bool live = t < n;
    const float gt = gt_n, rf = rf_n, ro = ro_n;
    stats(t + step);
    const f2 ro2 = f2_of(ro);
    if constexpr (U == 8) async_wait<S - 1>();
    const uint32_t at_d = OR::found(st, a.dout.row(t)), at_o = OR::found(st + out_at, a.out.row(t)),
                   at_n = OT::found(st + dn_at, a.dn.row(t)), at_f = OT::found(st + f_at, a.f.row(t));
    // piece i: x = dout + ro w dn, out, f, dn
    const auto get = [&](int i, f2 (&x)[P], f2 (&o)[P], f2 (&f)[P], f2 (&dn)[P]) {
#pragma unroll
      for (int k = 0; k < P; ++k) x[k] = o[k] = f[k] = dn[k] = 0;
      if (has_d) OR::get(c, at_d, piece, i, x);
      if (pre) {
        OR::get(c, at_o, piece, i, o);
        OT::get(c, at_n, piece, i, dn);
      }
      if (has_f) OT::get(c, at_f, piece, i, f);
    };
    f2 x1[KEEP ? P : 1], o1[KEEP ? P : 1], f1[KEEP ? P : 1];
    f2 a0 = 0, a1 = 0, a2 = 0;
    if (live)
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (c.has_piece(i)) {
          f2 x[P], o[P], f[P], dn[P], cf[P], w[P];
          get(i, x, o, f, dn);
          params(i, cf, w);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const int e = i * P + k;
            const f2 v = f2_mul(w[k], dn[k]), cfk = f2_mul(cf[k], f[k]);
            x[k] = f2_fma(ro2, v, x[k]);
            a0 = f2_fma(o[k], v, a0);
            a1 = f2_fma(cfk, x[k], a1);
            a2 = f2_fma(cfk, o[k], a2);
            dw[e] = f2_fma(f2_mul(dn[k], ro2), o[k], dw[e]);
            if constexpr (KEEP) x1[k] = x[k], o1[k] = o[k], f1[k] = f[k];
          }
        }
    float s[3] = {f2_sum(a0), f2_sum(a1), f2_sum(a2)};
    group_sum3(s, s_sum[buf], c.g, a.GT);
    buf ^= 1;
    const float k1 = ro * ro * (ro * s[0] * inv);
    const float cfd = rf * (pre ? s[1] - k1 * s[2] : s[1]);  // sum c fh D (f may be infinite)
    if (live) {
      if (c.j == 0 && a.dgate_t != nullptr) {
        if (a.p32)
          static_cast<float*>(a.dgate_t)[t] = cfd;
        else
          static_cast<T*>(a.dgate_t)[t] = from_f32<T>(cfd);
      }
      const f2 nk1 = f2_of(-k1), grf = f2_of(gt * rf);
      const f2 nm2 = f2_of(-(rf * rf) * (gt * cfd * inv));
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (c.has_piece(i)) {
          f2 x[P], o[P], f[P], dn[P], cf[P], w[P], q[P];
          params(i, cf, w);
          if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < P; ++k) x[k] = x1[k], o[k] = o1[k], f[k] = f1[k];
          } else {
            get(i, x, o, f, dn);
#pragma unroll
            for (int k = 0; k < P; ++k) x[k] = f2_fma(ro2, f2_mul(w[k], dn[k]), x[k]);
          }
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const int e = i * P + k;
            x[k] = f2_fma(nk1, o[k], x[k]);
            q[k] = f2_mul(grf, x[k]);
            K[e] = f2_fma(f[k], q[k], K[e]);
          }
          if (post) {
#pragma unroll
            for (int k = 0; k < P; ++k) f[k] = f2_fma(cf[k], q[k], f2_mul(nm2, f[k]));
          } else {  // (df holds no f, which may be infinite)
#pragma unroll
            for (int k = 0; k < P; ++k) f[k] = f2_mul(cf[k], q[k]);
          }
          put_piece<R>(c, a.dx.row(t), i, x);
          if (has_f) put_piece<T>(c, a.df.row(t), i, f);
        }
    }
    st_in = st;
    st += step_bytes;
    if (st == ring_end) st = ring;
  }
  async_wait<0>();
  if (!a.sums_f && !pre) return;
  // the CTA's groups' column sums, added in order
  float* const p0 = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  float* const sj = reinterpret_cast<float*>(ring_bytes);  // [groups][2][H]
  float* const q = c.groups == 1 ? p0 : sj + 2 * c.g * a.H;
  if (c.groups > 1) __syncthreads();  // (the ring is read no more)
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    if (c.has_piece(i)) {
      f2 k[P], d[P];
#pragma unroll
      for (int j = 0; j < P; ++j) k[j] = K[i * P + j], d[j] = dw[i * P + j];
      put_sums(c, q, i, k);
      put_sums(c, q + a.H, i, d);
    }
  if (c.groups == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.H; i += nt) {
    float v = sj[i];
    for (int k = 1; k < c.groups; ++k) v += sj[2 * k * a.H + i];
    p0[i] = v;
  }
}

// Any width: dx and df, a CTA a row, read twice; <oh v> is left for the column sums.
template <typename T, typename R, int U>
__global__ void __launch_bounds__(LOOP_THREADS) resnorm_dx_loop_kernel(const BwdOps<T, R> a) {
  __shared__ float s[LOOP_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(a.H);
  const bool pre = a.dn.p != nullptr, has_f = a.f.p != nullptr, post = a.w_post != nullptr;
  const bool whole = loop_whole(a.w_post, a.gate_c, a.w_pre);
  for (int64_t t = blockIdx.x; t < a.T_; t += gridDim.x) {
    const float gt = a.gate_t != nullptr ? param<T>(a.gate_t, a.p32, t) : 1.f;
    const float rf = post ? __ldg(a.rstd_f + t) : 1.f;
    const float ro = pre ? __ldg(a.rstd_out + t) : 0.f;
    const auto unit = [&](int i, float (&d)[U], float (&oh)[U], float (&v)[U], float (&fh)[U],
                          float (&cf)[U]) {
#pragma unroll
      for (int j = 0; j < U; ++j) d[j] = oh[j] = v[j] = fh[j] = cf[j] = 0.f;
      if (a.dout.p != nullptr) loop_get<R, U>(a.dout.row(t) + i, d);
      if (pre) {
        loop_get<R, U>(a.out.row(t) + i, oh);
        loop_get<T, U>(a.dn.row(t) + i, v);
        float w[U];
        loop_params<T, U>(a.w_pre, a.p32, whole, i, w);
#pragma unroll
        for (int j = 0; j < U; ++j) oh[j] *= ro, v[j] *= w[j];
      }
      if (has_f) {
        loop_get<T, U>(a.f.row(t) + i, fh);
        loop_coef<T, U>(a.w_post, a.gate_c, a.p32, whole, a.scale, i, cf);
#pragma unroll
        for (int j = 0; j < U; ++j) fh[j] *= rf;
      }
    };
    float s1 = 0.f, s2 = 0.f, s3 = 0.f;
    for (int i = threadIdx.x * U; i < a.H; i += LOOP_THREADS * U) {
      float d[U], oh[U], v[U], fh[U], cf[U];
      unit(i, d, oh, v, fh, cf);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float cfh = cf[j] * fh[j];
        s1 = fmaf(oh[j], v[j], s1);
        s2 = fmaf(cfh, fmaf(ro, v[j], d[j]), s2);
        s3 = fmaf(cfh, oh[j], s3);
      }
    }
    const float m1 = block_sum(s1, s) * inv;
    s2 = block_sum(s2, s);
    s3 = block_sum(s3, s);
    const float cfd = pre ? s2 - ro * m1 * s3 : s2;  // (f may be infinite)
    if (threadIdx.x == 0) {
      if (a.mean_ov != nullptr) a.mean_ov[t] = m1;
      if (a.dgate_t != nullptr) {
        if (a.p32)
          static_cast<float*>(a.dgate_t)[t] = cfd;
        else
          static_cast<T*>(a.dgate_t)[t] = from_f32<T>(cfd);
      }
    }
    const float m2 = gt * cfd * inv;
    for (int i = threadIdx.x * U; i < a.H; i += LOOP_THREADS * U) {
      float d[U], oh[U], v[U], fh[U], cf[U];
      unit(i, d, oh, v, fh, cf);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        d[j] = fmaf(ro, fmaf(-m1, oh[j], v[j]), d[j]);
        cf[j] *= gt * d[j];
      }
      if (post) {  // (without the norm df holds no f, which may be infinite)
#pragma unroll
        for (int j = 0; j < U; ++j) cf[j] = rf * fmaf(-m2, fh[j], cf[j]);
      }
      put_unit<R, U>(a.dx.row(t) + i, d);
      if (has_f) put_unit<T, U>(a.df.row(t) + i, cf);
    }
  }
}

// Column sums of one range of rows per blockIdx.y: a thread owns U columns.
template <typename T, typename R, int U>
__global__ void __launch_bounds__(256) resnorm_cols_loop_kernel(const BwdOps<T, R> a, int rows) {
  pdl_wait();
  pdl_trigger();
  const int i = (blockIdx.x * 256 + threadIdx.x) * U;
  if (i >= a.H) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t t1 = min(static_cast<int64_t>(a.T_), t0 + rows);
  const bool pre = a.dn.p != nullptr, post = a.w_post != nullptr;
  float w[U] = {}, K[U] = {}, dw[U] = {};
  if (pre) loop_params<T, U>(a.w_pre, a.p32, loop_whole(a.w_pre, nullptr, nullptr), i, w);
#pragma unroll 2
  for (int64_t t = t0; t < t1; ++t) {
    float d[U] = {};
    if (a.dout.p != nullptr) loop_get<R, U>(a.dout.row(t) + i, d);
    if (pre) {
      const float ro = __ldg(a.rstd_out + t), m1 = __ldcg(a.mean_ov + t);
      float oh[U], dn[U];
      loop_get<R, U>(a.out.row(t) + i, oh);
      loop_get<T, U>(a.dn.row(t) + i, dn);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        oh[j] *= ro;
        dw[j] = fmaf(dn[j], oh[j], dw[j]);
        d[j] = fmaf(ro, fmaf(-m1, oh[j], w[j] * dn[j]), d[j]);
      }
    }
    if (a.sums_f) {
      const float gt = a.gate_t != nullptr ? param<T>(a.gate_t, a.p32, t) : 1.f;
      const float rf = post ? __ldg(a.rstd_f + t) : 1.f;
      float f[U];
      loop_get<T, U>(a.f.row(t) + i, f);
#pragma unroll
      for (int j = 0; j < U; ++j) K[j] = fmaf(f[j] * rf, gt * d[j], K[j]);
    }
  }
  float* const p = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.H + i;
  put_unit<float, U>(p, K);
  put_unit<float, U>(p + a.H, dw);
}

// The parameters' gradients from n partial rows: 16 warps take every 16th row of 32 columns
// and are added in order; blockIdx.y 0: K's (dw_post, dgate_c), 1: dw_pre.
template <typename P>
__global__ void __launch_bounds__(512) resnorm_finish_kernel(
    const float* __restrict__ part, int n, int H, const P* __restrict__ w_post,
    const P* __restrict__ gate_c, float scale, P* __restrict__ dw_post, P* __restrict__ dgate_c,
    P* __restrict__ dw_pre) {
  constexpr int W = 16, B = 10;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.y == 0 ? dw_post == nullptr && dgate_c == nullptr : dw_pre == nullptr) return;
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
  if (w != 0 || i >= H) return;
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) t += s[j][lane];
  if (blockIdx.y == 1) {
    dw_pre[i] = from_f32<P>(t);
    return;
  }
  t *= scale;
  if (dw_post != nullptr) dw_post[i] = from_f32<P>(gate_c != nullptr ? t * to_f32(gate_c[i]) : t);
  if (dgate_c != nullptr) dgate_c[i] = from_f32<P>(w_post != nullptr ? t * to_f32(w_post[i]) : t);
}

template <typename T, typename R, int NU, int U, int S>
static cudaError_t bwd_launch_steps(const Ctx& c, const BwdOps<T, R>& a, const NormGrid& g,
                                    int params) {
  const int nt = g.GT * g.groups;
  size_t smem = U == 8 ? static_cast<size_t>(S) * nt * rn_bwd_bytes<T, R, NU, U> + params
                       : static_cast<size_t>(a.steps) * a.step_bytes;
  if (g.groups > 1) smem = std::max(smem, sizeof(float) * 2 * g.groups * a.H);
  const bool all = a.dout.p != nullptr && a.dn.p != nullptr && a.f.p != nullptr;
  auto* kern = all ? resnorm_bwd_kernel<T, R, NU, U, S, ALL> : resnorm_bwd_kernel<T, R, NU, U, S, SOME>;
  if constexpr (U == 8) {
    if (all && a.w_post != nullptr) kern = resnorm_bwd_kernel<T, R, NU, U, S, ALL_POST>;
  }
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_k(c.stream, kern, dim3(g.ctas), dim3(nt), smem, a);
}

template <typename T, typename R, int NU, int U>
static cudaError_t bwd_launch(const Ctx& c, BwdOps<T, R> a, int* n_part) {
  a.GT = rn_group_threads<NU, U>(a.H);
  const NormGrid g = rn_grid(a.GT, a.T_, c.num_sms * rn_ctas<NU, U>);
  *n_part = g.ctas;
  if constexpr (U == 1) {
    a.step_bytes = g.groups * 2 * (single_bytes(a.H, sizeof(T)) + single_bytes(a.H, sizeof(R)));
    a.steps = single_steps<NU>(a.step_bytes);
    return bwd_launch_steps<T, R, NU, U, 0>(c, a, g, 0);
  } else {
    const int params = 4 * (a.H / 8 * 16);
    constexpr int MOST = rn_bwd_steps<T, R, NU>(8 * 1024),
                  LEAST = rn_bwd_steps<T, R, NU>(NU * 32 * 1024);
    const int fit = rn_bwd_steps<T, R, NU>(params);
    if (fit >= MOST) return bwd_launch_steps<T, R, NU, U, MOST>(c, a, g, params);
    return bwd_launch_steps<T, R, NU, U, LEAST>(c, a, g, params);
  }
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_resnorm_backward(
    const mm_moe_resnorm* shape, const void* dout, int64_t lddout, const void* dn, int64_t lddn,
    const void* out, int64_t ldout, const void* f, int64_t ldf, const void* post_weight,
    const void* gate, const void* pre_weight, const float* rstd_f, const float* rstd_out, void* dx,
    int64_t lddx, void* df, int64_t lddf, void* dpost_weight, void* dgate, void* dpre_weight,
    void* workspace, void* stream) {
  if (!resnorm_shape_ok(shape)) return MM_MOE_EINVAL;
  const size_t b = dtype_bytes(shape->dtype), rb = dtype_bytes(shape->res_dtype),
               pb = dtype_bytes(shape->param_dtype);
  const bool pre = shape->pre != 0, has_f = f != nullptr, post = shape->post != 0 && has_f;
  const int gk = has_f ? shape->gate : MM_MOE_GATE_NONE;
  const RowSpan in[4] = {{dout, lddout, rb}, {pre ? dn : nullptr, lddn, b},
                         {pre ? out : nullptr, ldout, rb}, {f, ldf, b}};
  const RowSpan res[2] = {{dx, lddx, rb}, {has_f ? df : nullptr, lddf, b}};
  if ((dout == nullptr && !pre) || (!has_f && !pre) || (dout != nullptr && !span_ok(in[0], shape)) ||
      (pre && (!span_ok(in[1], shape) || !span_ok(in[2], shape) || !vec_ok(pre_weight, pb) ||
               !vec_ok(rstd_out, 4) || !vec_ok(dpre_weight, pb))) ||
      (has_f && (!span_ok(in[3], shape) || !span_ok(res[1], shape))) ||
      (post && (!vec_ok(post_weight, pb) || !vec_ok(rstd_f, 4) || !vec_ok(dpost_weight, pb))) ||
      (gk != MM_MOE_GATE_NONE && (!vec_ok(gate, pb) || !vec_ok(dgate, pb))) ||
      !span_ok(res[0], shape) || !vec_ok(workspace, 16))
    return MM_MOE_EINVAL;
  for (const RowSpan& r : res)
    for (const RowSpan& i : in)
      if (spans_meet(r, i, shape)) return MM_MOE_EINVAL;
  if (spans_meet(res[0], res[1], shape)) return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int T_ = static_cast<int>(shape->T), H = static_cast<int>(shape->H);
  bool even = H % 8 == 0;
  for (const RowSpan& r : {in[0], in[1], in[2], in[3], res[0], res[1]})
    even = even && span_even(r, shape);
  float* const part = static_cast<float*>(workspace);
  float* const mean_ov = part + static_cast<int64_t>(norm_parts(shape->T)) * 2 * H;
  const bool sums_f = post || gk == MM_MOE_GATE_CHANNEL;
  int parts = 0;
  cudaError_t e = with_types(shape, [&](auto* t, auto* r) -> cudaError_t {
    using T = std::remove_pointer_t<decltype(t)>;
    using R = std::remove_pointer_t<decltype(r)>;
    const BwdOps<T, R> a{{static_cast<const R*>(dout), lddout},
                         {static_cast<const T*>(pre ? dn : nullptr), lddn},
                         {static_cast<const R*>(out), ldout},
                         {static_cast<const T*>(f), ldf},
                         {static_cast<R*>(dx), lddx},
                         {static_cast<T*>(df), lddf},
                         post ? post_weight : nullptr,
                         gk == MM_MOE_GATE_CHANNEL ? gate : nullptr,
                         gk == MM_MOE_GATE_TOKEN ? gate : nullptr,
                         pre_weight,
                         shape->param_dtype == MM_MOE_DT_F32,
                         sums_f,
                         shape->scale,
                         rstd_f,
                         rstd_out,
                         gk == MM_MOE_GATE_TOKEN ? dgate : nullptr,
                         part,
                         mean_ov,
                         T_,
                         H,
                         0};
    cudaError_t err;
    prof_begin(c, K_RESNORM_BWD);
    if (even && H <= 16 * RN_THREADS) {
      const int g1 = rn_group_threads<1, 8>(H);
      if (g1 != 0 && T_ <= c.num_sms * std::max(1, RN_THREADS / g1))
        err = bwd_launch<T, R, 1, 8>(c, a, &parts);
      else
        err = bwd_launch<T, R, 2, 8>(c, a, &parts);
      prof_end(c, K_RESNORM_BWD);
      return err;
    }
    if (!even && H <= 16 * RN_THREADS) {
      err = H <= 4 * RN_THREADS   ? bwd_launch<T, R, 4, 1>(c, a, &parts)
            : H <= 8 * RN_THREADS ? bwd_launch<T, R, 8, 1>(c, a, &parts)
                                  : bwd_launch<T, R, 16, 1>(c, a, &parts);
      prof_end(c, K_RESNORM_BWD);
      return err;
    }
    err = launch_k(c.stream,
                   even ? resnorm_dx_loop_kernel<T, R, 8> : resnorm_dx_loop_kernel<T, R, 1>,
                   dim3(std::min(T_, c.num_sms * 4)), dim3(LOOP_THREADS), 0, a);
    prof_end(c, K_RESNORM_BWD);
    if (err != cudaSuccess || (!sums_f && !pre)) return err;
    const int cols = ((even ? H / 8 : H) + 255) / 256;
    const int want = std::min(norm_parts(T_), std::max(1, c.num_sms * 8 / cols));
    const int rows = div_up(T_, want);
    parts = div_up(T_, rows);
    prof_begin(c, K_RESNORM_BWD);
    err = launch_k(c.stream,
                   even ? resnorm_cols_loop_kernel<T, R, 8> : resnorm_cols_loop_kernel<T, R, 1>,
                   dim3(cols, parts), dim3(256), 0, a, rows);
    prof_end(c, K_RESNORM_BWD);
    return err;
  });
  if (e != cudaSuccess || (!sums_f && !pre)) return op_status(e);
  prof_begin(c, K_RESNORM_FINISH);
  e = with_dtype(shape->param_dtype, [&](auto* p) {
    using P = std::remove_pointer_t<decltype(p)>;
    return launch_k(c.stream, resnorm_finish_kernel<P>, dim3((H + 31) / 32, pre ? 2 : 1), dim3(512),
                    0, static_cast<const float*>(part), parts, H,
                    static_cast<const P*>(post ? post_weight : nullptr),
                    static_cast<const P*>(gk == MM_MOE_GATE_CHANNEL ? gate : nullptr), shape->scale,
                    static_cast<P*>(post ? dpost_weight : nullptr),
                    static_cast<P*>(gk == MM_MOE_GATE_CHANNEL ? dgate : nullptr),
                    static_cast<P*>(pre ? dpre_weight : nullptr));
  });
  prof_end(c, K_RESNORM_FINISH);
  return op_status(e);
}
