// Shared pieces of the frame-encoder operators (fm_ops.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fm_ops.h"

struct fm_buckets {
  int device;
  int num_buckets, max_distance, bidirectional;
  int32_t* host;  // map [2 * max_distance + 1], then {first, last} offset of each bucket
  int32_t* map;   // the same on the device
  int32_t* ranges;  // its second part; a bucket that no offset has is {1, 0}
};

namespace fm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// VEC adjacent elements, moved as one access
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

inline int64_t item_size(int64_t dtype) { return dtype == FM_F32 ? 4 : 2; }
inline bool is_float_type(int64_t d) { return d == FM_F32 || d == FM_F16 || d == FM_BF16; }

// SMs of the current device, asked for once per device
int num_sms();
// FM_OK, or FM_ERR_CUDA if the last launch was refused
inline fm_status launch_status() { return cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA; }
// Lets `kernel` use `bytes` of dynamic shared memory (a plain attribute call,
// repeated on every launch: it costs well under a microsecond)
template <typename K>
inline bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 40 * 1024 ||  // static arrays count against the 48 KB that need no asking
         cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
             cudaSuccess;
}

// dtable[c][h] = sum over r < rows and the offsets o of bucket c of
// part[r * row_stride + h * head_stride + o - first], where the array holds
// the offsets first .. first + count - 1 and buckets that reach an end of the
// map reach on to the ends of the array. One block per bucket and head.
fm_status bucket_sums_launch(const fm_buckets* buckets, const float* part, long long rows, long long row_stride,
                             long long head_stride, int first, int count, int heads, void* dtable, int64_t dtype,
                             cudaStream_t stream);

}  // namespace fm
