// Row elements in fp32, bf16 or fp16 and vectors of them, computed on in fp32.
#pragma once

#include "nerf_internal.cuh"

namespace nerfb {

template <typename T> __device__ __forceinline__ float elem_to_f(T v);
template <> __device__ __forceinline__ float elem_to_f(float v) { return v; }
template <> __device__ __forceinline__ float elem_to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float elem_to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T elem_from_f(float v);
template <> __device__ __forceinline__ float elem_from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 elem_from_f(float v) { return __float2bfloat16(v); }
template <> __device__ __forceinline__ __half elem_from_f(float v) { return __float2half(v); }

template <int BYTES> struct VecRaw;
template <> struct VecRaw<16> { using type = uint4; };
template <> struct VecRaw<4> { using type = uint32_t; };
template <> struct VecRaw<2> { using type = uint16_t; };

// N elements of T in one load or store of `BYTES` bytes.
template <typename T, int BYTES>
struct Vec {
  static constexpr int N = BYTES / (int)sizeof(T);
  using Raw = typename VecRaw<BYTES>::type;
  union { Raw raw; T e[N]; };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const Raw* p) { raw = __ldg(p); }
  __device__ __forceinline__ float get(int i) const { return elem_to_f<T>(e[i]); }
  __device__ __forceinline__ void set(int i, float v) { e[i] = elem_from_f<T>(v); }
};

}  // namespace nerfb
