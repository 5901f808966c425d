// resnorm.cuh -- the norms before and after a block fused with its gate and residual scale: what
// the forward (resnorm.cu) and the backward (resnorm_bwd.cu) share.
//
//   u = w_post f rf,  rf = (1/H sum f^2 + eps)^(-1/2)          (u = f without a norm behind the block)
//   out = x + scale gate u                                     gate: per channel, per token or none
//   n = w_pre out ro,  ro = (1/H sum out^2 + eps)^(-1/2)       (the next block's norm)
// Backward, with oh = out ro, fh = f rf, c = scale gate w_post and v = w_pre dn:
//   D = dout + ro (v - oh <oh v>),   dx = D,                   <>: mean over the row
//   q = c D,  df = rf (q - fh <fh q>)                          (df = q without the norm)
//   dw_pre = sum_t dn oh;  K = sum_t [gate_t] fh D gives dw_post = scale gate_c K and
//   dgate_c = scale w_post K;  dgate_t = scale sum_h w_post fh D
// <fh q> needs D, which needs <oh v>; so that a row's sums meet at one barrier, the backward sums
//   s1 = sum out v,  s2 = sum c f x,  s3 = sum c f out   with x = dout + ro v, and has
//   k = ro^3 s1 / H,  D = x - k out,  sum c fh D = rf (s2 - k s3).
//
// f, n and their gradients are of one type, x and out (the residual stream) of it or fp32,
// the parameters and the gate of it or fp32.  Everything is computed in fp32 and rounded once where it
// is stored; n comes from out before its rounding.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "norm.cuh"
#include "ops.cuh"

namespace mmmoe {

constexpr int RN_THREADS = 512;
constexpr int RN_SMEM = 230400;  // bytes of the ring and the parameters at most (227 KB, less what is static)

// A row is cut into units of U = 8 columns (16 bytes of 16-bit types, 32 of fp32), dealt out to
// the threads of a group in turn, NU to each; rows on no 16-byte boundary, or of a width that is no
// multiple of 8, into single columns (U = 1).  Rows come through a ring in shared memory by
// cp.async, S - 1 rows ahead.  Of units of 8 a thread reads only what it copied itself; of single columns a
// group copies its row in the 16-byte pieces of memory that it touches, and meets at a barrier before
// it reads it (9000 x 3001 bf16 forward 113 us, backward 129; loaded into registers a row ahead, 2 bytes at
// a time, 146 and 226).  A thread's values are pairs for the packed fp32 arithmetic, in PIECES (its units,
// or four single columns, so that few registers hold the operands) of P pairs.
template <int NU, int U>
struct Cols {
  static constexpr int N = NU * U, PIECES = U == 8 ? NU : NU / 4, P = N / PIECES / 2;
  int GT, g, j, groups, H;
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
  __device__ __forceinline__ int col(int i) const { return (j + i * GT) * U; }
  __device__ __forceinline__ bool has(int i) const { return col(i) < H; }
  __device__ __forceinline__ bool has_piece(int i) const { return has(U == 8 ? i : i * 4); }
};

// Whether rows are sent for into L2 a row ahead of the ring: with an fp32 residual stream, whose ring is
// short (backward of 16384 x 2048 119.7 -> 100.5 us; all in bf16 68.4 -> 72.6).
template <typename R>
constexpr bool rn_prefetch = sizeof(R) == 4;

// A whole row on its way to L2 (16-byte aligned, a multiple of 16 bytes), by one thread.
template <typename V>
__device__ __forceinline__ void prefetch_row(const V* row, int H) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row),
               "r"(H * static_cast<int>(sizeof(V)))
               : "memory");
}

__device__ __forceinline__ void async_copy_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 32 bytes in one store: whole sectors
__device__ __forceinline__ void store32(float* p, const f2 (&f)[4]) {
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(f[0]), "l"(f[1]), "l"(f[2]),
               "l"(f[3])
               : "memory");
}
__device__ __forceinline__ void sts16_f2(uint32_t a, f2 x, f2 y) {
  asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(a), "l"(x), "l"(y) : "memory");
}
__device__ __forceinline__ f2 f2_of(float v) { return f2_make(v, v); }

template <typename V>
__device__ __forceinline__ float lds_one(uint32_t a) {
  if constexpr (sizeof(V) == 4) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
    return f;
  } else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    V v;
    memcpy(&v, &h, 2);
    return to_f32(v);
  }
}
// Bytes of the ring for one row in single columns: all the 16-byte pieces that it can touch.
__host__ __device__ inline int single_bytes(int H, int size) { return (H * size + 30) / 16 * 16; }

// One row operand of type V on its way to the thread's registers.
template <typename V, int NU, int U>
struct Operand {
  using C = Cols<NU, U>;
  static constexpr int PARTS = U == 8 ? 8 / VN<V> : 0;  // 16-byte pieces of a unit
  static constexpr int BYTES = PARTS * 16 * NU;         // of a thread's share of a row in the ring
  static __device__ __forceinline__ void issue(const C& c, const V* row, uint32_t at, uint32_t piece) {
    if constexpr (U == 8) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (c.has(i)) {
#pragma unroll
          for (int h = 0; h < PARTS; ++h) {
            // (the halves of 32 bytes meet in L1: past it each would fetch the whole sector)
            if constexpr (PARTS == 2)
              async_copy_l1(at + (i * PARTS + h) * piece, row + c.col(i) + h * VN<V>);
            else
              async_copy(at + (i * PARTS + h) * piece, row + c.col(i) + h * VN<V>);
          }
        }
    } else {
      const int head = reinterpret_cast<uintptr_t>(row) & 15;
      const char* const from = reinterpret_cast<const char*>(row) - head;
      const int bytes = head + c.H * static_cast<int>(sizeof(V));
      for (int k = c.j * 16; k < bytes; k += c.GT * 16)
        async_copy(at + k, from + k, min(16, bytes - k));  // (nothing behind the row's end)
    }
  }
  // where a row at p is found that was sent for to `at`
  static __device__ __forceinline__ uint32_t found(uint32_t at, const V* p) {
    return U == 8 ? at : at + (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15);
  }
  // piece i's values (single columns: zero where there is none)
  static __device__ __forceinline__ void get(const C& c, uint32_t at, uint32_t piece, int i,
                                             f2 (&f)[C::P]) {
    if constexpr (U == 8) {
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        f2 t[VN<V> / 2];
        unpack2<V>(lds16(at + (i * PARTS + h) * piece), t);
#pragma unroll
        for (int k = 0; k < VN<V> / 2; ++k) f[h * (VN<V> / 2) + k] = t[k];
      }
    } else {
      const auto one = [&](int k) {
        return c.has(k) ? lds_one<V>(at + c.col(k) * static_cast<uint32_t>(sizeof(V))) : 0.f;
      };
#pragma unroll
      for (int k = 0; k < C::P; ++k) f[k] = f2_make(one(i * 4 + 2 * k), one(i * 4 + 2 * k + 1));
    }
  }
};

__device__ __forceinline__ void group_meet(int g, int GT) {
  if (GT > 32)
    group_bar(g, GT);
  else
    __syncwarp();
}
// Single columns: when it returns the next row of the ring is there for the whole group.  issue() sends for a
// row in place of the one in front, which all of the group are done with (of a ring of one step: for the
// row itself).
template <typename F>
__device__ __forceinline__ void single_turn(int g, int GT, int steps, F issue) {
  if (steps == 1) {
    group_meet(g, GT);
    issue();
    async_wait<0>();
    group_meet(g, GT);
    return;
  }
  if (steps == 4)
    async_wait<2>();
  else if (steps == 3)
    async_wait<1>();
  else
    async_wait<0>();
  group_meet(g, GT);
  issue();
}

// U elements of a row from memory
template <typename V, int U>
__device__ __forceinline__ void loop_get(const V* p, float (&f)[U]) {
  if constexpr (U == 8) {
#pragma unroll
    for (int h = 0; h < 8 / VN<V>; ++h) {
      float t[VN<V>];
      unpack(reinterpret_cast<const uint4*>(p)[h], t, p);
#pragma unroll
      for (int k = 0; k < VN<V>; ++k) f[h * VN<V> + k] = t[k];
    }
  } else {
    f[0] = to_f32(*p);
  }
}

template <typename V, int U>
__device__ __forceinline__ void put_unit(V* p, const float (&f)[U]) {
  if constexpr (U == 8) {
#pragma unroll
    for (int h = 0; h < 8 / VN<V>; ++h) {
      float t[VN<V>];
#pragma unroll
      for (int k = 0; k < VN<V>; ++k) t[k] = f[h * VN<V> + k];
      reinterpret_cast<uint4*>(p)[h] = pack(t, p);
    }
  } else {
    *p = from_f32<V>(f[0]);
  }
}
// A piece's values to their columns of a row.
template <typename V, int NU, int U>
__device__ __forceinline__ void put_piece(const Cols<NU, U>& c, V* row, int i,
                                          const f2 (&f)[Cols<NU, U>::P]) {
  if constexpr (U == 8 && std::is_same_v<V, float>) {
    store32(row + c.col(i), f);
  } else if constexpr (U == 8) {
    uint4* const o = reinterpret_cast<uint4*>(row + c.col(i));
#pragma unroll
    for (int h = 0; h < 8 / VN<V>; ++h) {
      f2 t[VN<V> / 2];
#pragma unroll
      for (int k = 0; k < VN<V> / 2; ++k) t[k] = f[h * (VN<V> / 2) + k];
      o[h] = pack2<V>(t);
    }
  } else {
#pragma unroll
    for (int k = 0; k < Cols<NU, U>::P; ++k) {
      const int j = i * 4 + 2 * k;
      float lo, hi;
      f2_split(f[k], lo, hi);
      if (c.has(j)) row[c.col(j)] = from_f32<V>(lo);
      if (c.has(j + 1)) row[c.col(j + 1)] = from_f32<V>(hi);
    }
  }
}

// The same for fp32 sums, in shared or global memory, on 16-byte boundaries.
template <int NU, int U>
__device__ __forceinline__ void put_sums(const Cols<NU, U>& c, float* p, int i,
                                         const f2 (&f)[Cols<NU, U>::P]) {
  if constexpr (U == 8) {
    ulonglong2* const o = reinterpret_cast<ulonglong2*>(p + c.col(i));
    o[0] = make_ulonglong2(f[0], f[1]);
    o[1] = make_ulonglong2(f[2], f[3]);
  } else {
    put_piece<float>(c, p, i, f);
  }
}

// Parameters (of type T, or fp32) of the thread's columns; zero where it has none.
template <typename T, int NU, int U>
__device__ __forceinline__ void load_params(const Cols<NU, U>& c, const void* p, bool p32,
                                            f2 (&out)[NU * U / 2]) {
  float v[NU * U];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    float f[U] = {};
    if (c.has(i)) {
      const bool whole = U == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
      if (p32) {
        const float* q = static_cast<const float*>(p) + c.col(i);
        if constexpr (U == 8) {
          if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 t = __ldg(reinterpret_cast<const float4*>(q) + h);
              f[4 * h] = t.x, f[4 * h + 1] = t.y, f[4 * h + 2] = t.z, f[4 * h + 3] = t.w;
            }
          }
        }
        if (!whole)
#pragma unroll
          for (int k = 0; k < U; ++k) f[k] = __ldg(q + k);
      } else {
        const T* q = static_cast<const T*>(p) + c.col(i);
        if constexpr (U == 8) {
          if (whole) {
#pragma unroll
            for (int h = 0; h < 8 / VN<T>; ++h) {
              float t[VN<T>];
              unpack(__ldg(reinterpret_cast<const uint4*>(q) + h), t, q);
#pragma unroll
              for (int k = 0; k < VN<T>; ++k) f[h * VN<T> + k] = t[k];
            }
          }
        }
        if (!whole)
#pragma unroll
          for (int k = 0; k < U; ++k) f[k] = to_f32(q[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) v[i * U + k] = f[k];
  }
#pragma unroll
  for (int k = 0; k < NU * U / 2; ++k) out[k] = f2_make(v[2 * k], v[2 * k + 1]);
}

template <typename T>
__device__ __forceinline__ float param(const void* p, bool p32, int64_t i) {
  return p32 ? __ldg(static_cast<const float*>(p) + i) : to_f32(static_cast<const T*>(p)[i]);
}

// Parameters of columns [i, i + U) (`whole`: in 16-byte accesses).
template <typename T, int U>
__device__ __forceinline__ void loop_params(const void* p, bool p32, bool whole, int i, float (&f)[U]) {
  if (U == 8 && whole) {
    if (p32)
      loop_get<float, U>(static_cast<const float*>(p) + i, f);
    else
      loop_get<T, U>(static_cast<const T*>(p) + i, f);
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) f[j] = param<T>(p, p32, i + j);
  }
}
__device__ __forceinline__ bool loop_whole(const void* a, const void* b, const void* c) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
           reinterpret_cast<uintptr_t>(c)) & 15) == 0;
}
// c = scale [gate_c] [w_post] there
template <typename T, int U>
__device__ __forceinline__ void loop_coef(const void* w_post, const void* gate_c, bool p32, bool whole,
                                          float scale, int i, float (&c)[U]) {
  float p[U];
#pragma unroll
  for (int j = 0; j < U; ++j) c[j] = scale;
  if (w_post != nullptr) {
    loop_params<T, U>(w_post, p32, whole, i, p);
#pragma unroll
    for (int j = 0; j < U; ++j) c[j] *= p[j];
  }
  if (gate_c != nullptr) {
    loop_params<T, U>(gate_c, p32, whole, i, p);
#pragma unroll
    for (int j = 0; j < U; ++j) c[j] *= p[j];
  }
}

// c = scale [gate_c] [w_post] of the thread's columns
template <typename T, int NU, int U>
__device__ __forceinline__ void load_coef(const Cols<NU, U>& c, const void* w_post,
                                          const void* gate_c, bool p32, float scale,
                                          f2 (&v)[NU * U / 2]) {
  if (w_post != nullptr) {
    load_params<T, NU, U>(c, w_post, p32, v);
  } else {
#pragma unroll
    for (int k = 0; k < NU * U / 2; ++k) v[k] = f2_of(1.f);
  }
#pragma unroll
  for (int k = 0; k < NU * U / 2; ++k) v[k] = f2_mul(v[k], f2_of(scale));
  if (gate_c != nullptr) {
    f2 t[NU * U / 2];
    load_params<T, NU, U>(c, gate_c, p32, t);
#pragma unroll
    for (int k = 0; k < NU * U / 2; ++k) v[k] = f2_mul(v[k], t[k]);
  }
}

// The thread's c and w in shared memory: four planes of H / 8 entries, two pairs of a unit in each, so
// that a warp's lanes read 512 bytes in a row.
template <int NU>
__device__ __forceinline__ void put_planes(const Cols<NU, 8>& c, uint32_t planes, uint32_t plane,
                                           const f2 (&cf)[NU * 4], const f2 (&w)[NU * 4]) {
#pragma unroll
  for (int i = 0; i < NU; ++i)
    if (c.has(i)) {
      const uint32_t at = planes + (c.j + i * c.GT) * 16;
      sts16_f2(at, cf[4 * i], cf[4 * i + 1]);
      sts16_f2(at + plane, cf[4 * i + 2], cf[4 * i + 3]);
      sts16_f2(at + 2 * plane, w[4 * i], w[4 * i + 1]);
      sts16_f2(at + 3 * plane, w[4 * i + 2], w[4 * i + 3]);
    }
}
// Piece i's values of the two planes from `planes` on.
template <int NU>
__device__ __forceinline__ void get_plane(const Cols<NU, 8>& c, uint32_t planes, uint32_t plane, int i,
                                          f2 (&v)[4]) {
  const uint32_t at = planes + (c.j + i * c.GT) * 16;
  const ulonglong2 q = lds16_f2(at), r = lds16_f2(at + plane);
  v[0] = q.x, v[1] = q.y, v[2] = r.x, v[3] = r.y;
}
// Three sums over a group, as group_sum (a warp's in 16 bytes).
__device__ __forceinline__ void group_sum3(float (&v)[3], float4* s, int g, int GT) {
#pragma unroll
  for (int q = 0; q < 3; ++q) v[q] = lanes_sum(v[q], GT);
  if (GT <= 32) return;
  const int gw = GT >> 5;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float4(v[0], v[1], v[2], 0.f);
  group_bar(g, GT);
  s += g * gw;
  float4 t = s[0];
  for (int i = 1; i < gw; ++i) {
    const float4 o = s[i];
    t.x += o.x, t.y += o.y, t.z += o.z;
  }
  v[0] = t.x, v[1] = t.y, v[2] = t.z;
}

// ------------------------------------------------------------------------ host side
constexpr int RN_MAX_H = 1 << 20;

inline bool resnorm_shape_ok(const mm_moe_resnorm* s) {
  return s != nullptr && s->T >= 1 && s->T < (int64_t{1} << 31) && s->H >= 1 && s->H <= RN_MAX_H &&
         dtype_ok(s->dtype) && (s->res_dtype == s->dtype || s->res_dtype == MM_MOE_DT_F32) &&
         (s->param_dtype == s->dtype || s->param_dtype == MM_MOE_DT_F32) && s->post >= 0 &&
         s->post <= 1 && s->pre >= 0 && s->pre <= 1 && s->gate >= MM_MOE_GATE_NONE &&
         s->gate <= MM_MOE_GATE_TOKEN && s->eps >= 0.f && s->eps <= 3.4028235e38f &&
         s->scale >= -3.4028235e38f && s->scale <= 3.4028235e38f;
}

// An operand of T rows, `bytes` an element.
struct RowSpan {
  const void* p;
  int64_t ld;
  size_t bytes;
};
inline bool span_ok(const RowSpan& r, const mm_moe_resnorm* s) {
  return r.p != nullptr && reinterpret_cast<uintptr_t>(r.p) % r.bytes == 0 &&
         (r.ld >= s->H || s->T == 1) && r.ld < (int64_t{1} << 40);
}
// Whether two operands may share memory: exact for rows equally far apart, else by their extents.
inline bool spans_meet(const RowSpan& a, const RowSpan& b, const mm_moe_resnorm* s) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const auto end = [&](const RowSpan& r) {
    return reinterpret_cast<uintptr_t>(r.p) +
           static_cast<unsigned __int128>((s->T - 1) * static_cast<__int128>(s->T == 1 ? 0 : r.ld) + s->H) *
               r.bytes;
  };
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa >= end(b) || pb >= end(a)) return false;
  const uintptr_t la = static_cast<uintptr_t>(a.ld) * a.bytes, lb = static_cast<uintptr_t>(b.ld) * b.bytes;
  if (s->T == 1 || la != lb) return true;
  const uintptr_t ra = s->H * a.bytes, rb = s->H * b.bytes;
  const uintptr_t d = pb >= pa ? (pb - pa) % la : (la - (pa - pb) % la) % la;  // b's row within a's
  return d < ra || la - d < rb;
}
inline bool span_even(const RowSpan& r, const mm_moe_resnorm* s) {
  const size_t unit = 8 * r.bytes;  // (fp32 is stored 32 bytes at a time)
  return r.p == nullptr ||
         (reinterpret_cast<uintptr_t>(r.p) % unit == 0 && (s->T == 1 || r.ld * r.bytes % unit == 0));
}

// CTAs an SM: two where single columns leave the registers for it (four a thread; 5003 x 1111 bf16
// forward 33 us, backward 43; one CTA, when columns came through registers, 61 for 41 and 64 for 56).
template <int NU, int U>
constexpr int rn_ctas = U == 1 && NU <= 4 ? 2 : 1;

// Steps of the ring of single columns, `step` bytes each.
template <int NU>
int single_steps(size_t step) {
  return static_cast<int>(std::min<size_t>(4, RN_SMEM / rn_ctas<NU, 1> / step));
}

// How the rows are spread: GT threads a row, groups of them in a CTA.
template <int NU, int U>
int rn_group_threads(int H) {
  const int units = (H + U - 1) / U;
  const int n = (units + NU - 1) / NU;
  if (n > RN_THREADS) return 0;
  if (n > 32) return (n + 31) / 32 * 32;
  int g = 1;
  while (g < n) g *= 2;
  return g;
}
inline NormGrid rn_grid(int GT, int T, int sms, int threads = RN_THREADS) {
  const int per_warp = GT < 32 ? 32 / GT : 1;
  int groups = std::min(threads / GT, div_up(T, sms));
  groups = (groups + per_warp - 1) / per_warp * per_warp;
  return NormGrid{GT, groups, std::min(sms, div_up(T, groups))};
}

// f(tag of T, tag of R): the types of the block and of the residual stream
template <typename F>
auto with_types(const mm_moe_resnorm* s, F f) {
  return with_dtype(s->dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (s->res_dtype == s->dtype) return f(t, static_cast<T*>(nullptr));
    return f(t, static_cast<float*>(nullptr));
  });
}

}  // namespace mmmoe
