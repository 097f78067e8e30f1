// Row elements in fp32, bf16 or fp16 and vectors of them, computed on in fp32.
#pragma once

#include <string.h>

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

// element i of a word of one fp32 or two 16-bit elements
template <typename T> __device__ __forceinline__ float word_elem(uint32_t w, int i);
template <> __device__ __forceinline__ float word_elem<float>(uint32_t w, int) { return __uint_as_float(w); }
template <> __device__ __forceinline__ float word_elem<__nv_bfloat16>(uint32_t w, int i) {
  return __uint_as_float(i ? w & 0xffff0000u : w << 16);
}
template <> __device__ __forceinline__ float word_elem<__half>(uint32_t w, int i) {
  return __half2float(__ushort_as_half((unsigned short)(i ? w >> 16 : w & 0xffffu)));
}
// the word of one fp32 element (lo) or of two 16-bit ones
template <typename T> __device__ __forceinline__ uint32_t word_from_f(float lo, float hi);
template <> __device__ __forceinline__ uint32_t word_from_f<float>(float lo, float) { return __float_as_uint(lo); }
template <> __device__ __forceinline__ uint32_t word_from_f<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &p, 4);
  return w;
}
template <> __device__ __forceinline__ uint32_t word_from_f<__half>(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &p, 4);
  return w;
}

// the larger of each element of two words; a NaN stays
template <typename T> __device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t word_max<float>(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <> __device__ __forceinline__ uint32_t word_max<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <> __device__ __forceinline__ uint32_t word_max<__half>(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// -inf in every element of a word
template <typename T> constexpr uint32_t kNegInf = 0xff800000u;
template <> constexpr uint32_t kNegInf<__nv_bfloat16> = 0xff80ff80u;
template <> constexpr uint32_t kNegInf<__half> = 0xfc00fc00u;

// Two fp32 values in one register pair: one instruction for both.
struct F2 {
  uint64_t v;
  static __device__ __forceinline__ F2 of(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ void split(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// N elements of T in one load or store of 16, 8, 4 or 2 bytes, held as 32-bit words
// (kept as single 16-bit elements they would take a register each).
template <typename T, int BYTES>
struct Vec {
  static constexpr int N = BYTES / (int)sizeof(T), W = BYTES >= 4 ? BYTES / 4 : 1, PER = 4 / (int)sizeof(T);
  uint32_t words[W];
  // vector v of the row or rows that start at p
  __device__ __forceinline__ void load(const void* p, int64_t v) {
    if constexpr (BYTES == 16) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(p) + v);
      words[0] = r.x, words[1 % W] = r.y, words[2 % W] = r.z, words[3 % W] = r.w;
    } else if constexpr (BYTES == 8) {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(p) + v);
      words[0] = r.x, words[1 % W] = r.y;
    } else if constexpr (BYTES == 4) {
      words[0] = __ldg(reinterpret_cast<const uint32_t*>(p) + v);
    } else {
      words[0] = __ldg(reinterpret_cast<const uint16_t*>(p) + v);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t v) const {
    if constexpr (BYTES == 16)
      reinterpret_cast<uint4*>(p)[v] = make_uint4(words[0], words[1 % W], words[2 % W], words[3 % W]);
    else if constexpr (BYTES == 8)
      reinterpret_cast<uint2*>(p)[v] = make_uint2(words[0], words[1 % W]);
    else if constexpr (BYTES == 4)
      reinterpret_cast<uint32_t*>(p)[v] = words[0];
    else
      reinterpret_cast<uint16_t*>(p)[v] = (uint16_t)words[0];
  }
  static __device__ __forceinline__ Vec of(const uint4& r) {
    static_assert(BYTES == 16, "a whole vector");
    Vec v;
    v.words[0] = r.x, v.words[1 % W] = r.y, v.words[2 % W] = r.z, v.words[3 % W] = r.w;
    return v;
  }
  __device__ __forceinline__ void fill(uint32_t w) {
#pragma unroll
    for (int i = 0; i < W; ++i) words[i] = w;
  }
  __device__ __forceinline__ float get(int i) const { return word_elem<T>(words[i / PER], i % PER); }
  // elements 2i and 2i + 1
  __device__ __forceinline__ F2 pair(int i) const { return F2::of(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ void pack(const float* v) {
#pragma unroll
    for (int i = 0; i < W; ++i) words[i] = word_from_f<T>(v[PER * i], N > 1 ? v[(PER * i + 1) % N] : 0.0f);
  }
};

}  // namespace nerfb
