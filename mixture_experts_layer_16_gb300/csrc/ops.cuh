// ops.cuh -- what the operators around the layer (norm.cuh, balance.cu, gradclip.cu, adamw.cu,
// select.cu, resnorm.cuh) share:
// their kernel ids and typed element access, bf16, fp16 and fp32 in memory, fp32 in
// registers.  A value is rounded (to nearest even) only where it is stored.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "internal.h"

namespace mmmoe {

// Kernel ids of these operators, after the layer's (per-kernel timing).
enum OpKernelId {
  K_NORM_FWD = K_COUNT,
  K_NORM_BWD,
  K_NORM_BWD_FINISH,
  K_BALANCE_FWD,
  K_BALANCE_FINISH,
  K_BALANCE_BWD,
  K_GRAD_SQ,
  K_GRAD_NORM,
  K_GRAD_SCALE,
  K_ADAMW,
  K_ADAMW_MOMENTS,
  K_SELECT_FWD,
  K_SELECT_BWD,
  K_RESNORM_FWD,
  K_RESNORM_BWD,
  K_RESNORM_FINISH,
  K_ALL_COUNT
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Elements of T in 16 bytes.
template <typename T>
constexpr int VN = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4], const float*) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8], const __nv_bfloat16*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8], const __half*) {
  const __half2* p = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(p[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[4], const float*) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], const __nv_bfloat16*) {
  uint4 v;
  __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], const __half*) {
  uint4 v;
  __half2* p = reinterpret_cast<__half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  return v;
}

// ------------------------------------------------------------------ two fp32 in a pair
// Packed fp32 arithmetic: one instruction for two values (add, mul, fma .f32x2); 1 to 5% of the
// time of the kernels here against one value an instruction.
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_split(v, a, b);
  return a + b;
}

inline bool dtype_ok(int32_t d) { return d >= MM_MOE_DT_BF16 && d <= MM_MOE_DT_F32; }
inline size_t dtype_bytes(int32_t d) { return d == MM_MOE_DT_F32 ? 4 : 2; }

// f(tag) with a null pointer of the element type as the tag.
template <typename F>
auto with_dtype(int32_t d, F f) {
  if (d == MM_MOE_DT_F32) return f(static_cast<float*>(nullptr));
  if (d == MM_MOE_DT_F16) return f(static_cast<__half*>(nullptr));
  return f(static_cast<__nv_bfloat16*>(nullptr));
}

// The current device's SM count, or 0 off sm_103 (asked once per device).
inline int sm_count_103() {
  static std::atomic<int> known[64];  // count + 1; 0: not asked yet
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed) != 0)
    return known[dev].load(std::memory_order_relaxed) - 1;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  const int n = major == 10 && minor == 3 ? sms : 0;
  if (dev < 64) known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

// A call's status.  The error of a failed one is taken off the host thread, whose next CUDA call
// would report it as its own.
inline mm_moe_status op_status(cudaError_t e) {
  if (e == cudaSuccess) return MM_MOE_OK;
  cudaGetLastError();
  return MM_MOE_ECUDA;
}

// Lets `kern` be launched with so much dynamic shared memory.
template <typename K>
inline cudaError_t allow_smem(K* kern, size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;  // within the default 48 KB, static part included
  return raise_smem_limit(reinterpret_cast<const void*>(kern), bytes);
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Sum over the CTA's warps, the same value in every thread (warps added in order);
// `s` holds one V per warp.  The leading barrier frees `s` from an earlier use.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* s) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = s[0];
  const int n = blockDim.x >> 5;
  for (int i = 1; i < n; ++i) t += s[i];
  return t;
}

}  // namespace mmmoe
