// Rows taken to the experts' order and back, with weights, and the weights'
// gradients. One thread per (point, column); the dot products of a weight
// gradient one warp per pair.
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half(v); }

template <typename T>
__global__ void scatter_kernel(const T* __restrict__ x, int64_t n, int width,
                               const int32_t* __restrict__ pos, int k, const float* __restrict__ w,
                               T* __restrict__ rows) {
  const int64_t m = n * k;
  for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < n * width;
       q += (int64_t)gridDim.x * blockDim.x) {
    const int64_t i = q / width, c = q - i * width;
    const float v = to_f(x[q]);
    for (int j = 0; j < k; ++j) {
      const int32_t p = pos[i * k + j];
      if (p >= 0 && p < m) rows[p * (int64_t)width + c] = from_f<T>(w ? w[i * k + j] * v : v);
    }
  }
}

template <typename T>
__global__ void gather_kernel(const T* __restrict__ rows, int64_t n, int width,
                              const int32_t* __restrict__ pos, int k, const float* __restrict__ w,
                              T* __restrict__ out) {
  const int64_t m = n * k;
  for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < n * width;
       q += (int64_t)gridDim.x * blockDim.x) {
    const int64_t i = q / width, c = q - i * width;
    float s = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int32_t p = pos[i * k + j];
      if (p >= 0 && p < m) s = fmaf(w ? w[i * k + j] : 1.0f, to_f(rows[p * (int64_t)width + c]), s);
    }
    out[q] = from_f<T>(s);
  }
}

template <typename T>
__global__ void dots_kernel(const T* __restrict__ rows, const T* __restrict__ x, int64_t n, int width,
                            const int32_t* __restrict__ pos, int k, float* __restrict__ dw) {
  const int64_t m = n * k;
  const int lane = threadIdx.x & 31;
  for (int64_t q = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32; q < m;
       q += (int64_t)gridDim.x * blockDim.x / 32) {
    const int32_t p = pos[q];
    float s = 0.0f;
    if (p >= 0 && p < m)
      for (int c = lane; c < width; c += 32)
        s = fmaf(to_f(x[q / k * width + c]), to_f(rows[p * (int64_t)width + c]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dw[q] = s;
  }
}

unsigned blocks_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 148 * 32 ? b : 148 * 32);
}

template <typename T>
void scatter_t(const void* x, const void* other, int64_t n, int width, const int32_t* pos, int k,
               const float* w, void* rows, float* dw, cudaStream_t st) {
  if (rows) scatter_kernel<T><<<blocks_for(n * width), 256, 0, st>>>((const T*)x, n, width, pos, k, w, (T*)rows);
  if (dw) dots_kernel<T><<<blocks_for(n * k * 32), 256, 0, st>>>((const T*)other, (const T*)x, n, width, pos, k, dw);
}
template <typename T>
void gather_t(const void* rows, const void* x, int64_t n, int width, const int32_t* pos, int k,
              const float* w, void* out, float* dw, cudaStream_t st) {
  if (out) gather_kernel<T><<<blocks_for(n * width), 256, 0, st>>>((const T*)rows, n, width, pos, k, w, (T*)out);
  if (dw) dots_kernel<T><<<blocks_for(n * k * 32), 256, 0, st>>>((const T*)rows, (const T*)x, n, width, pos, k, dw);
}

}  // namespace

cudaError_t launch_rows_scatter(const void* x, const void* other, int dtype, int64_t n, int width,
                                const int32_t* pos, int k, const float* w, void* rows, float* dw,
                                cudaStream_t st) {
  if (dtype == NERF_DTYPE_FP32) scatter_t<float>(x, other, n, width, pos, k, w, rows, dw, st);
  else if (dtype == NERF_DTYPE_BF16) scatter_t<__nv_bfloat16>(x, other, n, width, pos, k, w, rows, dw, st);
  else scatter_t<__half>(x, other, n, width, pos, k, w, rows, dw, st);
  return cudaGetLastError();
}

cudaError_t launch_rows_gather(const void* rows, const void* x, int dtype, int64_t n, int width,
                               const int32_t* pos, int k, const float* w, void* out, float* dw,
                               cudaStream_t st) {
  if (dtype == NERF_DTYPE_FP32) gather_t<float>(rows, x, n, width, pos, k, w, out, dw, st);
  else if (dtype == NERF_DTYPE_BF16) gather_t<__nv_bfloat16>(rows, x, n, width, pos, k, w, out, dw, st);
  else gather_t<__half>(rows, x, n, width, pos, k, w, out, dw, st);
  return cudaGetLastError();
}

}  // namespace nerfb
