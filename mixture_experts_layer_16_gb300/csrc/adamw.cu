// adamw.cu -- one AdamW step over many tensors, with moments in fp32 or in 8 bits.
//
//   g = coef grad,  coef = min(1, max_norm / (norm + clip_eps))   (1 without a norm)
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p - lr (m c1 / (sqrt(v) c2 + eps) + decay p),   c1 = 1 / (1 - b1^t), c2 = (1 - b2^t)^(-1/2)
//
// p is the fp32 master where there is one (the 16-bit parameter is then written as its
// rounding), else the parameter.  Everything is computed in fp32; the powers of the betas are kept
// in fp64 in a counter on the device, which the step's last launch advances, so that a captured
// step counts on at every replay and a skipped one (a norm that is not finite) does not count.
//
// Moments in 8 bits.  Blocks of 32 elements share a power of two 2^(c - 127), the smallest
// under which the block's largest value fits: m as e4m3 (sign, 4 exponent bits of bias 7, 3 fraction
// bits, up to 448), v, which has no sign, with 5 exponent bits of bias 15 and 3 fraction bits (up to
// 1.875 * 2^16).  An average that moves by 1 - b2 of itself a step would never leave a code under
// rounding to nearest (half a step is 3 to 6%), so both are rounded at random, up with the
// probability of the fraction: the averages keep their expectation.  The random bits are a hash of
// the step, the tensor's place in the call, the element and the seed: the same call gives the same
// bits, however it is launched.  A v above zero never rounds to zero (an m left beside it would
// be divided by eps).  A block with a value that is not finite has the scale's NaN.
//
// Bytes bound the step: a bf16 parameter with a master and a bf16 gradient moves 28 bytes with fp32
// moments, 16 with 8-bit ones.  The benchmark layer's 604 M parameters take 2.65 ms (0.94 of the copy
// rate), 200 M in 48 tensors with 8-bit moments 0.57 (0.84: 75 instructions an element, two thirds of
// the issue slots).  A tensor with an operand on no vector boundary goes element by element: these 200 M 0.81,
// 1.12 for 0.88 with fp32 moments.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>

#include "internal.h"
#include "ops.cuh"

namespace mmmoe {

constexpr int AW_THREADS = 256;
constexpr int AW_UNIT = 8;  // elements of a thread: 16 bytes of 16-bit types, 32 of fp32
constexpr int AW_CHUNK = AW_THREADS * AW_UNIT;
constexpr int AW_CTAS = 4;   // CTAs per SM
constexpr int AW_MAX = 256;  // tensors per launch (13 KB of parameters) ...
constexpr int AW_FEW = 32;   // ... and of a launch with few (1.6 KB)

// The device counter (mm_moe_adamw_step's `counter`): the steps behind, and b1, b2 to their power.
struct Counter {
  int64_t step;
  double pow1, pow2;
  unsigned int ticket;  // CTAs of the running launch that have read it
  unsigned int pad;
};

enum { AW_VEC = 64, AW_HAS_MASTER = 128 };  // flags beside the types: param | grad << 2

template <int N>
struct AdamList {
  void* param[N];
  float* master[N];
  const void* grad[N];
  int64_t n[N], at[N];  // elements; first one's place in the moments
  float decay[N];
  int first[N + 1];  // first chunk of each tensor in the launch's numbering
  uint16_t index[N];  // place in the call
  uint8_t flags[N];
  int count;
};

struct AdamArgs {
  float b1, a1, b2, a2, eps, lr;  // a = 1 - b
  double b1d, b2d;
  const float* lr_dev;
  const float* norm;
  float max_norm, clip_eps;
  uint32_t seed;
  bool last;  // the call's last launch
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  Counter* counter;
};

// A 32-bit hash: odd multipliers (from the golden ratio and from the root of two) between shifts.
__device__ __forceinline__ uint32_t mix32_open(uint32_t x) {  // all but the last shift
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  return x * 0x6A09E667u;
}
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = mix32_open(x);
  return x ^ (x >> 16);
}

__device__ __forceinline__ float sqrt_approx(float v) {  // within 2^-22 of itself
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float rcp_approx(float v) {  // within 2^-22 of itself (v is a normal number)
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// ------------------------------------------------------------------- eight elements
struct Raw8 {
  uint32_t w[8];
};
__device__ __forceinline__ void ld32(const void* p, Raw8& r) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                 "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const float (&f)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "r"(__float_as_uint(f[0])), "r"(__float_as_uint(f[1])), "r"(__float_as_uint(f[2])),
               "r"(__float_as_uint(f[3])), "r"(__float_as_uint(f[4])), "r"(__float_as_uint(f[5])),
               "r"(__float_as_uint(f[6])), "r"(__float_as_uint(f[7]))
               : "memory");
}
// Elements [i, i + n) of an array of type dt as they lie in memory (the others are zero).
__device__ __forceinline__ void load_raw(const void* p, int dt, int64_t i, int n, bool vec,
                                         Raw8& r) {
  if (vec && n == AW_UNIT) {
    if (dt == MM_MOE_DT_F32) {
      ld32(static_cast<const float*>(p) + i, r);
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
      r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < AW_UNIT; ++k) r.w[k] = 0;
  if (dt == MM_MOE_DT_F32) {
#pragma unroll
    for (int k = 0; k < AW_UNIT; ++k)
      if (k < n) r.w[k] = static_cast<const uint32_t*>(p)[i + k];
  } else {
#pragma unroll
    for (int k = 0; k < AW_UNIT; ++k)
      if (k < n)
        r.w[k / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + k]) << 16 * (k & 1);
  }
}
__device__ __forceinline__ void widen(const Raw8& r, int dt, float (&f)[8]) {
  if (dt == MM_MOE_DT_F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r.w[k]);
  } else {
    const uint4 q = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    if (dt == MM_MOE_DT_BF16)
      unpack(q, f, static_cast<const __nv_bfloat16*>(nullptr));
    else
      unpack(q, f, static_cast<const __half*>(nullptr));
  }
}
__device__ __forceinline__ void store8(void* p, int dt, int64_t i, int n, bool vec,
                                       const float (&f)[8]) {
  if (dt == MM_MOE_DT_F32) {
    float* o = static_cast<float*>(p) + i;
    if (vec && n == AW_UNIT) {
      st32(o, f);
      return;
    }
#pragma unroll
    for (int k = 0; k < AW_UNIT; ++k)
      if (k < n) o[k] = f[k];
    return;
  }
  const uint4 q = dt == MM_MOE_DT_BF16 ? pack(f, static_cast<const __nv_bfloat16*>(nullptr))
                                       : pack(f, static_cast<const __half*>(nullptr));
  uint16_t* o = static_cast<uint16_t*>(p) + i;
  if (vec && n == AW_UNIT) {
    *reinterpret_cast<uint4*>(o) = q;
    return;
  }
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < AW_UNIT; ++k)
    if (k < n) o[k] = static_cast<uint16_t>(w[k / 2] >> 16 * (k & 1));
}

// ------------------------------------------------------------------ moments in 8 bits
// The formats: exponent bias, fraction bits of the largest code (in fp32's place) and by how much
// a block's scale code lies below its largest value's exponent.
struct M8 {
  static constexpr int BIAS = 7, TOP = 0x600000, SHIFT = 8;
  static constexpr bool SIGNED = true;
};
struct V8 {
  static constexpr int BIAS = 15, TOP = 0x700000, SHIFT = 16;
  static constexpr bool SIGNED = false;
};
__device__ __forceinline__ float scale_of(uint32_t c) {  // 2^(c - 127), 255 is a NaN
  return __uint_as_float(c == 0 ? 0x00400000u : c == 255 ? 0x7fffffffu : c << 23);
}
// e4m3 is a conversion of the hardware's, exact in f16.  The other format's bits are those of an fp32
// number whose exponent runs from 0 (subnormals among them): one exact product moves it to the
// format's own bias, another applies the block's scale.
__device__ __forceinline__ void decode8(uint2 q, float scale, float (&f)[8], M8) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
        : "=r"(h)
        : "h"(static_cast<uint16_t>(w[k / 2] >> 16 * (k & 1))));
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f2_split(f2_mul(f2_make(t.x, t.y), f2_make(scale, scale)), f[2 * k], f[2 * k + 1]);
  }
}
__device__ __forceinline__ void decode8(uint2 q, float scale, float (&f)[8], V8) {
  const uint32_t w[2] = {q.x, q.y};
  // (a code's byte alone, at the top)
  const auto bits = [&](int k) {
    return __uint_as_float(__byte_perm(w[k / 4], 0, (k & 3) << 12 | 0x444) >> 4);
  };
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const f2 t = f2_mul(f2_make(bits(k), bits(k + 1)), f2_make(0x1p112f, 0x1p112f));
    f2_split(f2_mul(t, f2_make(scale, scale)), f[k], f[k + 1]);
  }
}
// Codes of a thread's eight values (four neighbouring lanes hold a block), rounded up where the
// bits that a code drops and 16 random ones carry.  `c`: the block's scale code.
template <typename F>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], const uint32_t (&rnd)[8], uint32_t& c) {
  constexpr float MOVE = F::BIAS == 7 ? 0x1p-120f : 0x1p-112f;
  // as integers: a NaN's bits lie above infinity's
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint32_t x = __float_as_uint(f[k]), y = __float_as_uint(f[k + 1]);
    top = F::SIGNED ? max(top, max(x & 0x7fffffffu, y & 0x7fffffffu)) : max(top, max(x, y));
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2)) & 0x7fffffffu;
  const int e = max(static_cast<int>((top + (0x7fffff - F::TOP)) >> 23) - F::SHIFT, 0);
  c = top >= 0x7f800000u ? 255u : static_cast<uint32_t>(e);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  float z[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2)  // (the code's bits are bits 20 to 27)
    f2_split(f2_mul(f2_mul(f2_make(f[k], f[k + 1]), f2_make(inv, inv)), f2_make(MOVE, MOVE)), z[k],
             z[k + 1]);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 7; k >= 0; --k) {
    const uint32_t up = (__float_as_uint(z[k]) + rnd[k] * 16) * 16;  // (now the top byte; the sign is gone)
    w[k / 4] = __funnelshift_l(up, w[k / 4], 8);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (F::SIGNED) {
      const uint32_t* b = reinterpret_cast<const uint32_t*>(f + 4 * h);  // the signs' bytes
      const uint32_t lo = __byte_perm(b[0], b[1], 0x0073), hi = __byte_perm(b[2], b[3], 0x0073);
      w[h] |= __byte_perm(lo, hi, 0x5410) & 0x80808080u;
    } else if (((w[h] - 0x01010101u) & ~w[h] & 0x80808080u) != 0) {  // a zero: only of a zero
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((w[h] >> 8 * k & 0xffu) == 0 && f[4 * h + k] > 0.f) w[h] |= 1u << 8 * k;
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename L>
__device__ __forceinline__ int tensor_of(const L& g, int chunk) {
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

template <typename L, bool BITS8>
__global__ void __launch_bounds__(AW_THREADS, AW_CTAS) adamw_kernel(const __grid_constant__ L g,
                                                                    const AdamArgs a) {
  __shared__ float s_c1, s_c2;
  __shared__ uint32_t s_key;
  pdl_wait();
  pdl_trigger();
  float coef = 1.f;
  if (a.norm != nullptr) {
    const float nrm = __ldcg(a.norm);
    if (!(fabsf(nrm) <= 3.4028235e38f)) return;  // nothing moves, and the step does not count
    coef = fminf(__frcp_rn(nrm + a.clip_eps) * a.max_norm, 1.f);  // (0 inf is a NaN: coef 1)
  }
  const float lr = a.lr_dev != nullptr ? __ldcg(a.lr_dev) : a.lr;
  if (threadIdx.x == 0) {
    Counter* const k = a.counter;
    const long long t = __ldcg(reinterpret_cast<const long long*>(&k->step)) + 1;
    const double p1 = __ldcg(&k->pow1) * a.b1d, p2 = __ldcg(&k->pow2) * a.b2d;
    s_c1 = static_cast<float>(1.0 / (1.0 - p1));
    s_c2 = static_cast<float>(1.0 / sqrt(1.0 - p2));
    s_key = mix32(a.seed + 0x9E3779B1u * static_cast<uint32_t>(t));
    if (a.last) {
      __threadfence();
      if (atomicAdd(&k->ticket, 1u) == gridDim.x - 1) {  // every CTA has read it
        k->step = t;
        k->pow1 = p1;
        k->pow2 = p2;
        k->ticket = 0;
      }
    }
  }
  const int total = g.first[g.count];
  int t = static_cast<int>(blockIdx.x) < total ? tensor_of(g, blockIdx.x) : 0;
  bool ready = false;
  for (int ch = blockIdx.x; ch < total; ch += gridDim.x) {
    while (t + 1 < g.count && g.first[t + 1] <= ch) ++t;
    const int flags = g.flags[t], dt = flags & 3, gdt = flags >> 2 & 3;
    const bool vec = flags & AW_VEC, has_master = flags & AW_HAS_MASTER;
    const int64_t n = g.n[t];
    const int64_t i = static_cast<int64_t>(ch - g.first[t]) * AW_CHUNK + threadIdx.x * AW_UNIT;
    const int mine = static_cast<int>(min(static_cast<int64_t>(AW_UNIT), max(n - i, int64_t{0})));
    const bool held = i < ((n + 31) & ~int64_t{31});  // the moments' blocks are whole
    const int64_t at = g.at[t] + i;
    void* const wide = has_master ? static_cast<void*>(g.master[t]) : g.param[t];
    const int wdt = has_master ? MM_MOE_DT_F32 : dt;
    Raw8 rg, rp, rm, rv;
    uint2 qm, qv;
    uint32_t cm = 0, cv = 0;
    load_raw(g.grad[t], gdt, i, mine, vec, rg);
    load_raw(wide, wdt, i, mine, vec, rp);
    if constexpr (BITS8) {
      qm = qv = make_uint2(0, 0);
      if (held) {
        qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + at);
        qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + at);
        cm = a.m_scale[at >> 5];
        cv = a.v_scale[at >> 5];
      }
    } else {
      if (held) {
        ld32(static_cast<const float*>(a.m) + at, rm);
        ld32(static_cast<const float*>(a.v) + at, rv);
      }
    }
    if (!ready) {  // (behind the first loads)
      __syncthreads();
      ready = true;
    }
    float fg[8], fp[8], m[8], v[8];
    widen(rg, gdt, fg);
    widen(rp, wdt, fp);
    if constexpr (BITS8) {
      decode8(qm, scale_of(cm), m, M8{});
      decode8(qv, scale_of(cv), v, V8{});
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = __uint_as_float(rm.w[k]);
        v[k] = __uint_as_float(rv.w[k]);
      }
    }
    const float c1 = s_c1, c2 = s_c2, decay = g.decay[t];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // Under 8 bits each product is rounded by itself, as elementwise fp32 arithmetic does: a value
      // beside the border between two codes falls to the same side wherever the step is computed.
      const float x = fg[k] * coef;
      m[k] = BITS8 ? __fadd_rn(__fmul_rn(m[k], a.b1), __fmul_rn(x, a.a1)) : fmaf(m[k], a.b1, x * a.a1);
      v[k] = BITS8 ? __fadd_rn(__fmul_rn(v[k], a.b2), __fmul_rn(__fmul_rn(x, x), a.a2))
                   : fmaf(v[k], a.b2, x * x * a.a2);
      const float u = m[k] * c1 * rcp_approx(fmaf(sqrt_approx(v[k]), c2, a.eps));
      fp[k] = fmaf(-lr, fmaf(decay, fp[k], u), fp[k]);
    }
    store8(wide, wdt, i, mine, vec, fp);
    if (has_master) store8(g.param[t], dt, i, mine, vec, fp);
    if (mine < AW_UNIT) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= mine) m[k] = v[k] = 0.f;
    }
    if constexpr (BITS8) {
      // 16 bits of each element's hash for either moment (i is a multiple of 8)
      uint32_t rm16[8], rv16[8];
      const uint32_t key = mix32(s_key ^ g.index[t]) ^ static_cast<uint32_t>(i >> 32) * 0x9E3779B1u ^
                           static_cast<uint32_t>(i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t x = mix32_open(key ^ k);
        rv16[k] = x >> 16;
        rm16[k] = (x ^ rv16[k]) & 0xffffu;
      }
      qm = encode8<M8>(m, rm16, cm);
      qv = encode8<V8>(v, rv16, cv);
      if (held) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at) = qm;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at) = qv;
        if ((threadIdx.x & 3) == 0) {
          a.m_scale[at >> 5] = static_cast<uint8_t>(cm);
          a.v_scale[at >> 5] = static_cast<uint8_t>(cv);
        }
      }
    } else if (held) {
      st32(static_cast<float*>(a.m) + at, m);
      st32(static_cast<float*>(a.v) + at, v);
    }
  }
}

// The values of 8-bit moments in bf16 (exact where a value is one of bf16's).
__global__ void __launch_bounds__(256) adamw_moments_kernel(
    const uint8_t* __restrict__ m, const uint8_t* __restrict__ m_scale,
    const uint8_t* __restrict__ v, const uint8_t* __restrict__ v_scale, int64_t n,
    __nv_bfloat16* __restrict__ om, __nv_bfloat16* __restrict__ ov) {
  pdl_wait();
  pdl_trigger();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256 * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8; i < n; i += stride) {
    const uint2 qm = __ldg(reinterpret_cast<const uint2*>(m + i));
    const uint2 qv = __ldg(reinterpret_cast<const uint2*>(v + i));
    const float sm = scale_of(__ldg(m_scale + (i >> 5))), sv = scale_of(__ldg(v_scale + (i >> 5)));
    float f[8];
    decode8(qm, sm, f, M8{});
    *reinterpret_cast<uint4*>(om + i) = pack(f, om);
    decode8(qv, sv, f, V8{});
    *reinterpret_cast<uint4*>(ov + i) = pack(f, ov);
  }
}

static bool al(const void* p, uintptr_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

constexpr int64_t AW_MAX_TOTAL = int64_t{1} << 41;  // elements: a launch's chunks count in 32 bits

static bool tensors_ok(const mm_moe_adamw_tensor* p, int64_t n, int64_t* elements) {
  if (n < 0 || n > MM_MOE_MAX_GRADS || (n > 0 && p == nullptr)) return false;
  int64_t& total = *elements = 0;
  for (int64_t i = 0; i < n; ++i) {
    const mm_moe_adamw_tensor& t = p[i];
    if (!dtype_ok(t.dtype) || (t.grad_dtype != t.dtype && t.grad_dtype != MM_MOE_DT_F32) ||
        t.numel < 0 || t.numel > AW_MAX_TOTAL || !(std::fabs(t.weight_decay) <= FLT_MAX) ||
        (total += t.numel) > AW_MAX_TOTAL)
      return false;
    if (t.numel == 0) continue;
    if (!al(t.param, dtype_bytes(t.dtype)) || !al(t.grad, dtype_bytes(t.grad_dtype))) return false;
    if (t.master != nullptr && (t.dtype == MM_MOE_DT_F32 || !al(t.master, 4))) return false;
  }
  return true;
}

// A range of memory that the step reads, or also writes.
struct Span {
  uintptr_t begin, end;
  bool written;
};
// Whether what is written lies apart from all the rest (two gradients may be the same).
static bool apart(Span* s, int64_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;  // where those in front end
  for (int64_t i = 0; i < n; ++i) {
    if (s[i].begin < (s[i].written ? any : written)) return false;
    any = std::max(any, s[i].end);
    if (s[i].written) written = std::max(written, s[i].end);
  }
  return true;
}
static mm_moe_status check_apart(const mm_moe_adamw_tensor* p, int64_t n) {
  Span few[3 * AW_FEW];
  Span* const s = n <= AW_FEW ? few : new (std::nothrow) Span[3 * n];
  if (s == nullptr) return MM_MOE_ECUDA;
  int64_t k = 0;
  const auto add = [&](const void* at, size_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    if (bytes != 0 && at != nullptr) s[k++] = Span{a, a + bytes, written};
  };
  for (int64_t i = 0; i < n; ++i) {
    const mm_moe_adamw_tensor& t = p[i];
    add(t.param, t.numel * dtype_bytes(t.dtype), true);
    add(t.master, t.numel * 4, true);
    add(t.grad, t.numel * dtype_bytes(t.grad_dtype), false);
  }
  const bool ok = apart(s, k);
  if (s != few) delete[] s;
  return ok ? MM_MOE_OK : MM_MOE_EINVAL;
}

template <int N>
static int64_t fill(AdamList<N>* l, const mm_moe_adamw_tensor* p, int64_t i, int64_t n,
                    int64_t* at) {
  l->count = 0;
  int chunks = 0;
  for (; i < n && l->count < N; ++i) {
    const mm_moe_adamw_tensor& t = p[i];
    if (t.numel == 0) continue;
    const int c = l->count++;
    const bool vec = al(t.param, t.dtype == MM_MOE_DT_F32 ? 32 : 16) &&
                     al(t.grad, t.grad_dtype == MM_MOE_DT_F32 ? 32 : 16) &&
                     (t.master == nullptr || al(t.master, 32));
    l->param[c] = t.param;
    l->master[c] = t.master;
    l->grad[c] = t.grad;
    l->n[c] = t.numel;
    l->at[c] = *at;
    l->decay[c] = t.weight_decay;
    l->index[c] = static_cast<uint16_t>(i);
    l->flags[c] = static_cast<uint8_t>(t.dtype | t.grad_dtype << 2 | (vec ? AW_VEC : 0) |
                                       (t.master != nullptr ? AW_HAS_MASTER : 0));
    l->first[c] = chunks;
    chunks += static_cast<int>((t.numel + AW_CHUNK - 1) / AW_CHUNK);
    *at += (t.numel + 31) / 32 * 32;
  }
  l->first[l->count] = chunks;
  return i;
}

template <typename L>
static cudaError_t launch_adamw(const Ctx& c, const L& l, const AdamArgs& a, bool bits8) {
  const int grid = std::max(1, std::min(c.num_sms * AW_CTAS, l.first[l.count]));
  prof_begin(c, K_ADAMW);
  const cudaError_t e =
      launch_k(c.stream, bits8 ? adamw_kernel<L, true> : adamw_kernel<L, false>, dim3(grid),
               dim3(AW_THREADS), 0, l, a);
  prof_end(c, K_ADAMW);
  return e;
}

}  // namespace mmmoe

using namespace mmmoe;

extern "C" MM_MOE_API mm_moe_status mm_moe_adamw_step(
    const mm_moe_adamw* opt, const mm_moe_adamw_tensor* tensors, int64_t n_tensors, void* m,
    uint8_t* m_scale, void* v, uint8_t* v_scale, void* counter, double lr, const float* lr_dev,
    const float* norm, void* stream) {
  if (opt == nullptr || !(opt->beta1 >= 0.0 && opt->beta1 < 1.0) ||
      !(opt->beta2 >= 0.0 && opt->beta2 < 1.0) || !(opt->eps >= FLT_MIN && opt->eps <= FLT_MAX) ||
      !(opt->max_norm >= 0.f) || !(opt->clip_eps >= 0.f) || opt->states < 0 || opt->states > 1 ||
      !(std::fabs(lr) <= FLT_MAX))
    return MM_MOE_EINVAL;
  int64_t elements;
  if (!tensors_ok(tensors, n_tensors, &elements)) return MM_MOE_EINVAL;
  const bool bits8 = opt->states == MM_MOE_STATES_8BIT;
  if ((elements > 0 && (!al(m, 32) || !al(v, 32) || (bits8 && (!m_scale || !v_scale)))) ||
      !al(counter, 16) || (norm != nullptr && !al(norm, 4)) ||
      (lr_dev != nullptr && !al(lr_dev, 4)))
    return MM_MOE_EINVAL;
  const mm_moe_status meet = check_apart(tensors, n_tensors);
  if (meet != MM_MOE_OK) return meet;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  AdamArgs a{};
  a.b1 = static_cast<float>(opt->beta1);
  a.a1 = static_cast<float>(1.0 - opt->beta1);
  a.b2 = static_cast<float>(opt->beta2);
  a.a2 = static_cast<float>(1.0 - opt->beta2);
  a.b1d = opt->beta1;
  a.b2d = opt->beta2;
  a.eps = static_cast<float>(opt->eps);
  a.lr = static_cast<float>(lr);
  a.lr_dev = lr_dev;
  a.norm = norm;
  a.max_norm = opt->max_norm;
  a.clip_eps = opt->clip_eps;
  a.seed = opt->seed;
  a.m = m;
  a.v = v;
  a.m_scale = m_scale;
  a.v_scale = v_scale;
  a.counter = static_cast<Counter*>(counter);
  int64_t at = 0;
  if (n_tensors <= AW_FEW) {
    AdamList<AW_FEW> l;
    fill(&l, tensors, 0, n_tensors, &at);
    a.last = true;
    return op_status(launch_adamw(c, l, a, bits8));
  }
  AdamList<AW_MAX> l;
  cudaError_t e = cudaSuccess;
  for (int64_t i = 0; i < n_tensors && e == cudaSuccess;) {
    i = fill(&l, tensors, i, n_tensors, &at);
    a.last = i == n_tensors;
    e = launch_adamw(c, l, a, bits8);
  }
  return op_status(e);
}

extern "C" MM_MOE_API mm_moe_status mm_moe_adamw_moments(const uint8_t* m, const uint8_t* m_scale,
                                                         const uint8_t* v, const uint8_t* v_scale,
                                                         int64_t n, uint16_t* m_out,
                                                         uint16_t* v_out, void* stream) {
  if (n < 0 || n % 32 != 0 || n > 2 * AW_MAX_TOTAL) return MM_MOE_EINVAL;
  if (n == 0) return MM_MOE_OK;
  if (!al(m, 16) || !al(v, 16) || !m_scale || !v_scale || !al(m_out, 16) || !al(v_out, 16))
    return MM_MOE_EINVAL;
  const int sms = std::min(152, sm_count_103());
  if (sms == 0) return MM_MOE_ENOTSUP;
  int launches = 0;
  const Ctx c{static_cast<cudaStream_t>(stream), sms, &launches};
  const int64_t ctas = (n / 8 + 255) / 256;
  prof_begin(c, K_ADAMW_MOMENTS);
  const cudaError_t e =
      launch_k(c.stream, adamw_moments_kernel,
               dim3(static_cast<unsigned>(std::min<int64_t>(ctas, sms * 8))), dim3(256), 0, m,
               m_scale, v, v_scale, n, reinterpret_cast<__nv_bfloat16*>(m_out),
               reinterpret_cast<__nv_bfloat16*>(v_out));
  prof_end(c, K_ADAMW_MOMENTS);
  return op_status(e);
}
