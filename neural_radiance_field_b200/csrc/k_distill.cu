// Distillation of student logits against a teacher's kept top logits, loss and
// gradient. One CTA per row: a pass with the running maximum and sum of the
// softmax over the row, the teacher's k entries in shared memory, and a second
// pass over the row (from L2) that writes the gradient.
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

constexpr int DT = 256;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half(v); }

template <typename F>
__device__ __forceinline__ float block_fold(float v, float* sm, F f) {
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x / 32] = v;
  __syncthreads();
  v = sm[0];
  for (int i = 1; i < DT / 32; ++i) v = f(v, sm[i]);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(DT)
distill_kernel(const T* __restrict__ student, int64_t n, int classes, const float* __restrict__ tl,
               const int32_t* __restrict__ ti, int k, float temperature,
               const float* __restrict__ scale, float* __restrict__ loss, T* __restrict__ grad) {
  __shared__ float red[DT / 32], p_s[DISTILL_MAX_K];
  __shared__ int32_t id_s[DISTILL_MAX_K];
  const int t = threadIdx.x;
  const float inv_t = 1.0f / temperature;
  auto fmx = [](float a, float b) { return (a != a || b != b) ? a + b : fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T* s = student + i * classes;
    float m = -INFINITY;
    for (int c = t; c < classes; c += DT) m = fmx(m, to_f(s[c]) * inv_t);
    m = block_fold(m, red, fmx);
    float z = 0.0f;
    for (int c = t; c < classes; c += DT) z += expf(to_f(s[c]) * inv_t - m);
    z = block_fold(z, red, add);
    int32_t id = -1;
    float y = -INFINITY;
    if (t < k) {
      id = ti[i * k + t];
      y = tl[i * k + t];
      if (id < 0 || id >= classes || y == -INFINITY) id = -1;
      y = id < 0 ? -INFINITY : y * inv_t;
    }
    const float top = block_fold(y, red, fmx);
    const float e = id < 0 ? 0.0f : expf(y - top);
    const float norm = block_fold(e, red, add);
    float l = 0.0f, p = 0.0f;
    if (id >= 0) {
      p = e / norm;
      if (p != 0.0f) l = p * ((y - top - logf(norm)) - (to_f(s[id]) * inv_t - m - logf(z)));
    }
    if (t < k) { id_s[t] = id; p_s[t] = p; }
    l = block_fold(l, red, add);
    const int some = __syncthreads_or(id >= 0);
    if (t == 0) loss[i] = some ? temperature * temperature * l : 0.0f;
    if (grad) {
      T* g = grad + i * classes;
      const float a = temperature * (scale ? scale[i] : 1.0f), iz = 1.0f / z;
      for (int c = t; c < classes; c += DT)
        g[c] = from_f<T>(some ? a * (expf(to_f(s[c]) * inv_t - m) * iz) : 0.0f);
      __syncthreads();
      // the kept classes again, less the teacher's probability (summed where an
      // id comes twice; its first entry writes)
      if (id >= 0) {
        float sum = 0.0f;
        bool first = true;
        for (int j = 0; j < k; ++j)
          if (id_s[j] == id) {
            first = first && j >= t;
            sum += p_s[j];
          }
        if (first) g[id] = from_f<T>(a * (expf(to_f(s[id]) * inv_t - m) * iz - sum));
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_distill(const void* student, int dtype, int64_t n, int classes,
                           const float* tl, const int32_t* ti, int k, float temperature,
                           const float* scale, float* loss, void* grad, cudaStream_t st) {
  const unsigned grid = (unsigned)(n < 148 * 8 ? n : 148 * 8);
  if (dtype == NERF_DTYPE_FP32)
    distill_kernel<float><<<grid, DT, 0, st>>>((const float*)student, n, classes, tl, ti, k, temperature, scale, loss, (float*)grad);
  else if (dtype == NERF_DTYPE_BF16)
    distill_kernel<__nv_bfloat16><<<grid, DT, 0, st>>>((const __nv_bfloat16*)student, n, classes, tl, ti, k, temperature, scale, loss, (__nv_bfloat16*)grad);
  else
    distill_kernel<__half><<<grid, DT, 0, st>>>((const __half*)student, n, classes, tl, ti, k, temperature, scale, loss, (__half*)grad);
  return cudaGetLastError();
}

}  // namespace nerfb
