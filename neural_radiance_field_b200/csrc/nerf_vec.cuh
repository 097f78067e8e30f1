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

// two 16-bit elements as one word
template <typename T> __device__ __forceinline__ uint32_t pair_from_f(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pair_from_f<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <> __device__ __forceinline__ uint32_t pair_from_f<__half>(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int BYTES> struct VecRaw;
template <> struct VecRaw<16> { using type = uint4; };
template <> struct VecRaw<4> { using type = uint32_t; };
template <> struct VecRaw<2> { using type = uint16_t; };

// N elements of T in one load or store of `BYTES` bytes.
template <typename T, int BYTES>
struct Vec {
  static constexpr int N = BYTES / (int)sizeof(T);
  using Raw = typename VecRaw<BYTES>::type;
  union { Raw raw; T e[N]; uint32_t words[BYTES >= 4 ? BYTES / 4 : 1]; };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const Raw* p) { raw = __ldg(p); }
  __device__ __forceinline__ float get(int i) const { return elem_to_f<T>(e[i]); }
  __device__ __forceinline__ void pack(const float* v) {
    if constexpr (sizeof(T) == 2 && BYTES >= 4) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) words[i] = pair_from_f<T>(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = elem_from_f<T>(v[i]);
    }
  }
};

}  // namespace nerfb
