// resnorm.cu -- the norms before and after a block with its gate and residual scale: the
// forward (formulas in resnorm.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "ops.cuh"
#include "resnorm.cuh"

namespace mmmoe {

template <typename T, typename R>
struct FwdOps {
  Rows<const R> x;
  Rows<const T> f;  // null: out is x and not stored
  Rows<R> out;
  Rows<T> n;  // null: no norm in front of the next block
  const void *w_post, *gate_c, *gate_t, *w_pre;
  bool p32;
  float scale, eps;
  float *rstd_f, *rstd_out;
  int T_, H, GT;
  int steps, step_bytes;  // of the ring of single columns
};

// Bytes of a thread's share of a row in the ring.
template <typename T, typename R, int NU, int U>
constexpr int rn_fwd_bytes = Operand<T, NU, U>::BYTES + Operand<R, NU, U>::BYTES;
template <typename T, typename R, int NU, int THREADS>
constexpr int rn_fwd_steps =
    std::max(1, std::min(4, RN_SMEM / (THREADS * rn_fwd_bytes<T, R, NU, 8>)));

// JOINT (units of 8): the sum over the next row's f joins this row's over out, one barrier a row for two.
// That takes a step of the ring's lead, and pays where rows span warps and the lead is long or the warps
// are many (us at 16384 x 2048, without and with: bf16 47.8, 45.9; with an fp32 residual stream 67.2,
// 72.4; 32768 x 512, a warp a row, 24.3, 25.0; 6000 x 4608 with an fp32 stream 67.8, 57.3; 4096 x 8192
// bf16 53.8, 45.4).
// 16384 x 2048 in bf16 is at 0.86 of the copy rate, with an fp32 residual stream at 0.89 (62.0 to 67.2 us;
// its rows in 16-byte halves of sectors, and not on their way to L2 a row ahead: 80).  Two CTAs an SM with
// half of the ring and the parameters in shared memory: 49.9 and 71.6.
template <typename T, typename R, int NU, int U, bool JOINT, int THREADS = RN_THREADS>
__global__ void __launch_bounds__(THREADS, rn_ctas<NU, U>) resnorm_fwd_kernel(const FwdOps<T, R> a) {
  constexpr int S = U == 8 ? rn_fwd_steps<T, R, NU, THREADS> : 0;
  const int steps = U == 8 ? S : a.steps;
  using OF = Operand<T, NU, U>;
  using OX = Operand<R, NU, U>;
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  static_assert(!JOINT || S >= 2);
  constexpr int NSUM = JOINT ? 2 : 1;
  __shared__ Sums<NSUM> s_sum[2][THREADS / 32];
  const uint32_t piece = blockDim.x * 16;
  const uint32_t step_bytes = U == 8 ? rn_fwd_bytes<T, R, NU, U> * blockDim.x : a.step_bytes;
  pdl_wait();
  pdl_trigger();
  Cols<NU, U> c;
  c.init(a.GT, a.H);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_bytes)) +
                        (U == 8 ? threadIdx.x * 16 : c.g * (step_bytes / c.groups));
  const uint32_t x_at = U == 8 ? OF::BYTES * blockDim.x : single_bytes(a.H, sizeof(T));
  const uint32_t n = a.T_, step = gridDim.x * c.groups;
  uint32_t t = blockIdx.x * c.groups + c.g, tw = c.first_of_warp(t), ta = t;
  const float inv = 1.f / static_cast<float>(a.H);
  const auto issue = [&](uint32_t at) {
    if (ta < n) {
      if (a.f.p != nullptr) OF::issue(c, a.f.row(ta), at, piece);
      OX::issue(c, a.x.row(ta), at + x_at, piece);
    }
    if constexpr (U == 8) {
      if (rn_prefetch<R> && c.j == 0) {
        const int64_t tp = static_cast<int64_t>(ta) + step;
        if (tp < n) {
          if (a.f.p != nullptr) prefetch_row(a.f.row(tp), a.H);
          prefetch_row(a.x.row(tp), a.H);
        }
      }
    }
    ta += step;
    async_commit();
  };
  for (int i = 0; i < steps - 1; ++i) issue(ring + i * step_bytes);
  constexpr int P = Cols<NU, U>::P, PIECES = Cols<NU, U>::PIECES;
  f2 cf[NU * U / 2], w[NU * U / 2];
  if (a.f.p != nullptr) load_coef<T, NU, U>(c, a.w_post, a.gate_c, a.p32, a.scale, cf);
  if (a.n.p != nullptr) load_params<T, NU, U>(c, a.w_pre, a.p32, w);
  float gt_n = 1.f;  // the next row's gate, a row ahead
  const auto gate = [&](uint32_t q) {
    if (q < n && a.gate_t != nullptr) gt_n = param<T>(a.gate_t, a.p32, q);
  };
  gate(t);
  // Every sum takes the buffer that the one in front of it did not: with one barrier to a sum, a warp that
  // has its totals writes its part of the next sum while others still read the last one's.
  int buf = 0;
  const auto add_up = [&](float (&v)[NSUM]) {
    group_sum<NSUM>(v, s_sum[buf], c.g, a.GT);
    buf ^= 1;
  };
  uint32_t st = ring, st_in = ring + (steps - 1) * step_bytes;
  const uint32_t ring_end = ring + steps * step_bytes;
  const bool post = a.f.p != nullptr && a.w_post != nullptr;
  const auto sum_f = [&](uint32_t at, uint32_t q) {  // the thread's part of row q's sum over f
    at = OF::found(at, a.f.row(q));
    f2 s2 = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if (c.has_piece(i)) {
        f2 f[P];
        OF::get(c, at, piece, i, f);
#pragma unroll
        for (int k = 0; k < P; ++k) s2 = f2_fma(f[k], f[k], s2);
      }
    return f2_sum(s2);
  };
  float rf_n = 1.f;  // the next row's
  if constexpr (JOINT) {
    async_wait<S - 2>();
    if (post) {
      float ss[2] = {0.f, t < n ? sum_f(st, t) : 0.f};
      add_up(ss);
      rf_n = rsqrtf(fmaf(ss[1], inv, a.eps));
    }
  }
  for (; tw < n; t += step, tw += step) {
    if constexpr (U == 8)
      issue(st_in);
    else
      single_turn(c.g, a.GT, steps, [&] { issue(st_in); });
    const bool live = t < n;
    float gt = gt_n;
    gate(t + step);
    if constexpr (U == 8 && !JOINT) async_wait<S - 1>();
    f2 o[NU * U / 2];
    if (post) {
      float rf = rf_n;
      if constexpr (!JOINT) {
        float ss[1] = {live ? sum_f(st, t) : 0.f};
        add_up(ss);
        rf = rsqrtf(fmaf(ss[0], inv, a.eps));
      }
      if (live && c.j == 0) a.rstd_f[t] = rf;
      gt *= rf;
    }
    f2 s2 = 0;
    const f2 gt2 = f2_of(gt);
    const uint32_t at_x = OX::found(st + x_at, a.x.row(t)), at_f = OF::found(st, a.f.row(t));
    if (live)
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (c.has_piece(i)) {
          f2 x[P];
          OX::get(c, at_x, piece, i, x);
          if (a.f.p != nullptr) {
            f2 f[P];
            OF::get(c, at_f, piece, i, f);
#pragma unroll
            for (int k = 0; k < P; ++k) x[k] = f2_fma(f2_mul(cf[i * P + k], gt2), f[k], x[k]);
            put_piece<R>(c, a.out.row(t), i, x);
          }
#pragma unroll
          for (int k = 0; k < P; ++k) {
            o[i * P + k] = x[k];
            s2 = f2_fma(x[k], x[k], s2);
          }
        }
    const uint32_t st_next = st + step_bytes == ring_end ? ring : st + step_bytes;
    float so = f2_sum(s2);
    if constexpr (JOINT) {
      async_wait<S - 2>();
      float ss[2] = {so, post && t + step < n ? sum_f(st_next, t + step) : 0.f};
      if (post || a.n.p != nullptr) add_up(ss);
      so = ss[0];
      rf_n = rsqrtf(fmaf(ss[1], inv, a.eps));
    } else if (a.n.p != nullptr) {
      float ss[1] = {so};
      add_up(ss);
      so = ss[0];
    }
    if (a.n.p != nullptr) {
      const float ro = rsqrtf(fmaf(so, inv, a.eps));
      if (live) {
        if (c.j == 0) a.rstd_out[t] = ro;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if (c.has_piece(i)) {
            f2 y[P];
#pragma unroll
            for (int k = 0; k < P; ++k) y[k] = f2_mul(f2_mul(o[i * P + k], f2_of(ro)), w[i * P + k]);
            put_piece<T>(c, a.n.row(t), i, y);
          }
      }
    }
    st_in = st;
    st = st_next;
  }
  async_wait<0>();
}

// Any width: a CTA a row, read up to three times (from L1 and L2).
template <typename T, typename R, int U>
__global__ void __launch_bounds__(LOOP_THREADS) resnorm_fwd_loop_kernel(const FwdOps<T, R> a) {
  __shared__ float s[LOOP_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const float inv = 1.f / static_cast<float>(a.H);
  const bool has_f = a.f.p != nullptr, whole = loop_whole(a.w_post, a.gate_c, a.w_pre);
  for (int64_t t = blockIdx.x; t < a.T_; t += gridDim.x) {
    float k = a.gate_t != nullptr ? param<T>(a.gate_t, a.p32, t) : 1.f;
    if (has_f && a.w_post != nullptr) {
      float ss = 0.f;
      for (int i = threadIdx.x * U; i < a.H; i += LOOP_THREADS * U) {
        float f[U];
        loop_get<T, U>(a.f.row(t) + i, f);
#pragma unroll
        for (int j = 0; j < U; ++j) ss = fmaf(f[j], f[j], ss);
      }
      const float rf = rsqrtf(fmaf(block_sum(ss, s), inv, a.eps));
      if (threadIdx.x == 0) a.rstd_f[t] = rf;
      k *= rf;
    }
    const auto values = [&](int i, float (&x)[U]) {
      loop_get<R, U>(a.x.row(t) + i, x);
      if (!has_f) return;
      float f[U], cf[U];
      loop_get<T, U>(a.f.row(t) + i, f);
      loop_coef<T, U>(a.w_post, a.gate_c, a.p32, whole, a.scale, i, cf);
#pragma unroll
      for (int j = 0; j < U; ++j) x[j] = fmaf(cf[j] * k, f[j], x[j]);
    };
    float ro = 0.f;
    if (a.n.p != nullptr) {
      float ss = 0.f;
      for (int i = threadIdx.x * U; i < a.H; i += LOOP_THREADS * U) {
        float x[U];
        values(i, x);
#pragma unroll
        for (int j = 0; j < U; ++j) ss = fmaf(x[j], x[j], ss);
      }
      ro = rsqrtf(fmaf(block_sum(ss, s), inv, a.eps));
      if (threadIdx.x == 0) a.rstd_out[t] = ro;
    }
    // (out may lie over x: every element is written by the thread that read it last)
    for (int i = threadIdx.x * U; i < a.H; i += LOOP_THREADS * U) {
      float x[U];
      values(i, x);
      if (has_f) put_unit<R, U>(a.out.row(t) + i, x);
      if (a.n.p != nullptr) {
        float w[U];
        loop_params<T, U>(a.w_pre, a.p32, whole, i, w);
#pragma unroll
        for (int j = 0; j < U; ++j) x[j] *= ro * w[j];
        put_unit<T, U>(a.n.row(t) + i, x);
      }
    }
  }
}

template <typename T, typename R, int NU, int U>
static cudaError_t fwd_launch(const Ctx& c, FwdOps<T, R> a) {
  a.GT = rn_group_threads<NU, U>(a.H);
  constexpr bool MAY = U == 8 && NU > 1;  // (NU = 1: a row or two a group)
  const bool joint = MAY && a.GT > (sizeof(R) == 2 ? 32 : 128);
  // two groups of up to 384 threads (in 80 registers) where 512 threads would be one, which waits at its
  // barrier: 6000 x 5120 bf16 52.5 -> 41.5 us, x 6144 88.7 -> 60.8 (elsewhere 51.8); where more groups fit
  // anyway 512 threads are as fast (x 3584) or faster (16384 x 2048 45.9, 47.6 with six groups for four)
  constexpr int MORE = MAY && sizeof(R) == 2 ? 768 : RN_THREADS;
  const bool more = a.GT > RN_THREADS / 2 && 2 * a.GT <= MORE;
  const NormGrid g = rn_grid(a.GT, a.T_, c.num_sms * rn_ctas<NU, U>, more ? MORE : RN_THREADS);
  const int nt = g.GT * g.groups;
  size_t smem;
  if (U == 8) {
    smem = static_cast<size_t>(more ? rn_fwd_steps<T, R, NU, MORE> : rn_fwd_steps<T, R, NU, RN_THREADS>) *
           nt * rn_fwd_bytes<T, R, NU, U>;
  } else {
    a.step_bytes = g.groups * (single_bytes(a.H, sizeof(T)) + single_bytes(a.H, sizeof(R)));
    a.steps = single_steps<NU>(a.step_bytes);
    smem = static_cast<size_t>(a.steps) * a.step_bytes;
  }
  auto* kern = more    ? resnorm_fwd_kernel<T, R, NU, U, MAY, MORE>
               : joint ? resnorm_fwd_kernel<T, R, NU, U, MAY>
                       : resnorm_fwd_kernel<T, R, NU, U, false>;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_k(c.stream, kern, dim3(g.ctas), dim3(nt), smem, a);
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_resnorm_workspace_size(const mm_moe_resnorm* shape,
                                                                  size_t* bytes) {
  if (!resnorm_shape_ok(shape) || bytes == nullptr) return MM_MOE_EINVAL;
  *bytes = (static_cast<size_t>(norm_parts(shape->T)) * 2 * shape->H + shape->T) * sizeof(float);
  return MM_MOE_OK;
}

extern "C" MM_MOE_API mm_moe_status mm_moe_resnorm_forward(
    const mm_moe_resnorm* shape, const void* x, int64_t ldx, const void* f, int64_t ldf,
    const void* post_weight, const void* gate, const void* pre_weight, void* out, int64_t ldout,
    void* n, int64_t ldn, float* rstd_f, float* rstd_out, void* stream) {
  if (!resnorm_shape_ok(shape)) return MM_MOE_EINVAL;
  const size_t b = dtype_bytes(shape->dtype), rb = dtype_bytes(shape->res_dtype),
               pb = dtype_bytes(shape->param_dtype);
  const RowSpan sx{x, ldx, rb}, sf{f, ldf, b}, so{f != nullptr ? out : nullptr, ldout, rb},
      sn{shape->pre ? n : nullptr, ldn, b};
  if (!span_ok(sx, shape) || (f == nullptr && !shape->pre)) return MM_MOE_EINVAL;
  if (f != nullptr &&
      (!span_ok(sf, shape) || !span_ok(so, shape) ||
       (shape->post && (!vec_ok(post_weight, pb) || !vec_ok(rstd_f, 4))) ||
       (shape->gate != MM_MOE_GATE_NONE && !vec_ok(gate, pb))))
    return MM_MOE_EINVAL;
  if (shape->pre && (!span_ok(sn, shape) || !vec_ok(pre_weight, pb) || !vec_ok(rstd_out, 4)))
    return MM_MOE_EINVAL;
  const bool in_place = so.p == x && (shape->T == 1 || ldout == ldx);
  if ((!in_place && spans_meet(so, sx, shape)) || spans_meet(so, sf, shape) ||
      spans_meet(sn, sx, shape) || spans_meet(sn, sf, shape) || spans_meet(sn, so, shape))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int T_ = static_cast<int>(shape->T), H = static_cast<int>(shape->H);
  const bool even = H % 8 == 0 && span_even(sx, shape) && span_even(sf, shape) &&
                    span_even(so, shape) && span_even(sn, shape);
  prof_begin(c, K_RESNORM_FWD);
  const cudaError_t e = with_types(shape, [&](auto* t, auto* r) -> cudaError_t {
    using T = std::remove_pointer_t<decltype(t)>;
    using R = std::remove_pointer_t<decltype(r)>;
    const FwdOps<T, R> a{{static_cast<const R*>(x), ldx},
                         {static_cast<const T*>(f), ldf},
                         {static_cast<R*>(out), ldout},
                         {static_cast<T*>(shape->pre ? n : nullptr), ldn},
                         shape->post && f != nullptr ? post_weight : nullptr,
                         shape->gate == MM_MOE_GATE_CHANNEL && f != nullptr ? gate : nullptr,
                         shape->gate == MM_MOE_GATE_TOKEN && f != nullptr ? gate : nullptr,
                         pre_weight,
                         shape->param_dtype == MM_MOE_DT_F32,
                         shape->scale,
                         shape->eps,
                         rstd_f,
                         rstd_out,
                         T_,
                         H,
                         0};
    if (even && H <= 16 * RN_THREADS) {
      const int g1 = rn_group_threads<1, 8>(H);
      if (g1 != 0 && T_ <= c.num_sms * std::max(1, RN_THREADS / g1))
        return fwd_launch<T, R, 1, 8>(c, a);
      return fwd_launch<T, R, 2, 8>(c, a);
    }
    if (!even && H <= 4 * RN_THREADS) return fwd_launch<T, R, 4, 1>(c, a);
    if (!even && H <= 8 * RN_THREADS) return fwd_launch<T, R, 8, 1>(c, a);
    if (!even && H <= 16 * RN_THREADS) return fwd_launch<T, R, 16, 1>(c, a);
    return launch_k(c.stream,
                    even ? resnorm_fwd_loop_kernel<T, R, 8> : resnorm_fwd_loop_kernel<T, R, 1>,
                    dim3(std::min(T_, c.num_sms * 4)), dim3(LOOP_THREADS), 0, a);
  });
  prof_end(c, K_RESNORM_FWD);
  return op_status(e);
}
