// Distillation of student logits against a teacher's kept top logits, loss and
// gradient in one launch. With c = log2(e) / T, m the row's largest logit and
// Z = sum_i 2^(c (s_i - m)):  q_i = 2^(c (s_i - m)) / Z  and
// log q_i = (s_i - m) / T - log Z. (The difference is taken first: a row of
// masks of the type's lowest value must not overflow.)
//
// Bound by memory: the logits are read once and the gradient is written once.
// A row that fits the registers of a warp (rows up to 4 KB) or of a CTA of 256
// threads (up to 32 KB) stays there between the statistics and the gradient. A
// longer row is streamed twice, the second time from L2, by a cluster of CTAs
// that share the row's statistics through distributed shared memory: with few
// rows the cluster is what fills the GPU, with many it keeps the rows in flight
// (clusters x row bytes) inside L2. A row's 16-byte vectors start wherever its
// address allows; up to 14 elements before and after them go one by one.
#include <cooperative_groups.h>

#include "nerf_experts.cuh"
#include "nerf_vec.cuh"

namespace nerfb {
namespace {

namespace cg = cooperative_groups;

struct DistillArgs {
  const void* student;
  int64_t n;
  int classes;
  const float* tl;
  const int32_t* ti;
  int k;
  float temperature;
  const float* scale;
  float* loss;
  void* grad;
};

// 2^x within 2^-22 of its value; 0 below the normal range
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
template <typename F>
__device__ __forceinline__ float warp_fold(float v, F f) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The threads that share a row: a warp, or a CTA of NT threads.
template <int NT>
struct Team {
  float* red;                                // [NT / 32] for a CTA
  __device__ __forceinline__ int rank() const { return NT == 32 ? threadIdx.x & 31 : threadIdx.x; }
  __device__ __forceinline__ void sync() const { if (NT == 32) __syncwarp(); else __syncthreads(); }
  template <typename F>
  __device__ __forceinline__ float fold(float v, F f) const {
    v = warp_fold(v, f);
    if (NT == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < NT / 32; ++i) v = f(v, red[i]);
    return v;
  }
  __device__ __forceinline__ float max(float v) const { return fold(v, [](float a, float b) { return max_nan(a, b); }); }
  __device__ __forceinline__ float sum(float v) const { return fold(v, [](float a, float b) { return a + b; }); }
};

// The teacher's side of a row, from its statistics: every thread gets whether an
// entry is kept; `probs` ([k] of this team) the entries' probabilities.
template <typename T, int NT>
__device__ __forceinline__ bool teacher_row(const DistillArgs& A, const Team<NT>& team, int64_t i, const T* s,
                                            float m, float z, float* probs, bool write_loss) {
  const float inv_t = 1.0f / A.temperature;
  const float* tl = A.tl + i * A.k;
  const int32_t* ti = A.ti + i * A.k;
  const int r = team.rank();
  auto kept = [&](int j) { return (unsigned)__ldg(ti + j) < (unsigned)A.classes && __ldg(tl + j) != -INFINITY; };
  float top = -INFINITY;
  for (int j = r; j < A.k; j += NT)
    if (kept(j)) top = max_nan(top, __ldg(tl + j));
  top = team.max(top);
  const bool some = top != -INFINITY;
  float norm = 0.0f;
  for (int j = r; j < A.k; j += NT) {
    const float e = kept(j) ? expf((__ldg(tl + j) - top) * inv_t) : 0.0f;
    probs[j] = e;
    norm += e;
  }
  norm = team.sum(norm);
  const float log_norm = logf(norm), log_z = logf(z);
  float l = 0.0f;
  for (int j = r; j < A.k; j += NT) {
    const float p = kept(j) ? probs[j] / norm : 0.0f;
    probs[j] = p;
    if (p != 0.0f)
      l += p * (((__ldg(tl + j) - top) * inv_t - log_norm) - ((elem_to_f<T>(s[__ldg(ti + j)]) - m) * inv_t - log_z));
  }
  l = team.sum(l);
  if (write_loss && r == 0) A.loss[i] = some ? A.temperature * A.temperature * l : 0.0f;
  return some;
}

// The gradient of the kept classes in [lo, hi), which the row's pass wrote as q
// alone: less the teacher's probability, summed where an id comes twice (its
// first entry writes).
template <typename T, int NT>
__device__ __forceinline__ void kept_gradients(const DistillArgs& A, const Team<NT>& team, int64_t i, const T* s,
                                               T* g, float m, float c, float a, float iz, const float* probs,
                                               int lo, int hi) {
  const int32_t* ti = A.ti + i * A.k;
  for (int j = team.rank(); j < A.k; j += NT) {
    const int32_t id = __ldg(ti + j);
    if (id < lo || id >= hi) continue;
    float p = 0.0f;
    bool first = true;
    for (int q = 0; q < A.k; ++q)
      if (__ldg(ti + q) == id) {
        first = first && q >= j;
        p += probs[q];
      }
    if (first) g[id] = elem_from_f<T>(a * (exp2_fast((elem_to_f<T>(s[id]) - m) * c) * iz - p));
  }
}

constexpr float kLog2e = 1.44269504f;

// Rows in registers: NV vectors a thread (and one single element).
template <typename T, int NT, int NV>
__global__ void __launch_bounds__(256)
distill_rows_kernel(DistillArgs A) {
  using V = Vec<T, 16>;
  constexpr int TEAMS = 256 / NT;
  __shared__ float red[8], probs_s[TEAMS * DISTILL_MAX_K];
  const Team<NT> team{red};
  const int r = team.rank();
  float* probs = probs_s + (NT == 32 ? threadIdx.x / 32 : 0) * DISTILL_MAX_K;
  const float c = kLog2e / A.temperature;
  for (int64_t i = (int64_t)blockIdx.x * TEAMS + (NT == 32 ? threadIdx.x / 32 : 0); i < A.n;
       i += (int64_t)gridDim.x * TEAMS) {
    const T* s = (const T*)A.student + i * A.classes;
    T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
    const int head = min((int)((0 - (uintptr_t)s) % 16 / sizeof(T)), A.classes);
    const int nv = (A.classes - head) / V::N, single = r < head ? r : nv * V::N + r;
    const bool has = single < A.classes && (r < head || single >= head + nv * V::N);
    const uint4* sv = reinterpret_cast<const uint4*>(s + head);
    V v[NV];
    float one = -INFINITY, m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if (r + q * NT < nv) v[q].load(sv + r + q * NT);
    if (has) one = elem_to_f<T>(s[single]);
    m = one;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if (r + q * NT < nv)
#pragma unroll
        for (int e = 0; e < V::N; ++e) m = max_nan(m, v[q].get(e));
    m = team.max(m);
    float z = has ? exp2_fast((one - m) * c) : 0.0f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if (r + q * NT < nv)
#pragma unroll
        for (int e = 0; e < V::N; ++e) z += exp2_fast((v[q].get(e) - m) * c);
    z = team.sum(z);
    const bool some = teacher_row<T, NT>(A, team, i, s, m, z, probs, true);
    if (g) {
      const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f), iz = 1.0f / z;
      uint4* gv = reinterpret_cast<uint4*>(g + head);
#pragma unroll
      for (int q = 0; q < NV; ++q)
        if (r + q * NT < nv) {
          V o;
#pragma unroll
          for (int e = 0; e < V::N; ++e)
            o.set(e, some ? a * (exp2_fast((v[q].get(e) - m) * c) * iz) : 0.0f);
          gv[r + q * NT] = o.raw;
        }
      if (has) g[single] = elem_from_f<T>(some ? a * (exp2_fast((one - m) * c) * iz) : 0.0f);
      team.sync();
      if (some) kept_gradients<T, NT>(A, team, i, s, g, m, c, a, iz, probs, 0, A.classes);
    }
    team.sync();
  }
}

// Long rows, streamed by clusters: CTA `rank` of a cluster takes the rank-th
// part of the row's vectors (the last one also the single elements after them,
// the first one those before).
constexpr int DW_T = 512;
template <typename T, int BYTES>
__global__ void __launch_bounds__(DW_T, 2)
distill_wide_kernel(DistillArgs A) {
  using V = Vec<T, BYTES>;
  using Raw = typename V::Raw;
  __shared__ float red[DW_T / 32], probs[DISTILL_MAX_K];
  __shared__ float2 stat;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), t = threadIdx.x;
  const Team<DW_T> team{red};
  const float c = kLog2e / A.temperature;
  for (int64_t i = blockIdx.x / C; i < A.n; i += gridDim.x / C) {
    const T* s = (const T*)A.student + i * A.classes;
    T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
    const int head = BYTES == 16 ? min((int)((0 - (uintptr_t)s) % 16 / sizeof(T)), A.classes) : 0;
    const int nv = (A.classes - head) / V::N;
    const int v0 = (int)((int64_t)nv * rank / C), v1 = (int)((int64_t)nv * (rank + 1) / C);
    const int lo = rank == 0 ? 0 : head + v0 * V::N, hi = rank == C - 1 ? A.classes : head + v1 * V::N;
    const int before = rank == 0 ? head : 0, after = rank == C - 1 ? A.classes - head - nv * V::N : 0;
    const int single = t < before ? t : head + nv * V::N + t - before;
    const bool has = t < before + after;
    const Raw* sv = reinterpret_cast<const Raw*>(s + head);
    // running maximum and sum: the sum is rescaled once per four vectors
    float m = has ? elem_to_f<T>(s[single]) : -INFINITY, z = has ? 1.0f : 0.0f;
    for (int q0 = v0 + t; q0 < v1; q0 += 4 * DW_T) {
      V v[4];
      float top = m;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < v1) v[u].load(sv + q0 + u * DW_T);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < v1)
#pragma unroll
          for (int e = 0; e < V::N; ++e) top = max_nan(top, v[u].get(e));
      // nothing above -inf yet: any shift does, and -inf - (-inf) must not arise
      const float shift = top == -INFINITY ? 0.0f : top;
      z *= m == -INFINITY ? 0.0f : exp2_fast((m - shift) * c);
      m = top;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < v1)
#pragma unroll
          for (int e = 0; e < V::N; ++e) z += exp2_fast((v[u].get(e) - shift) * c);
    }
    const float mine = m;
    m = team.max(m);
    z = team.sum(mine == -INFINITY ? 0.0f : z * exp2_fast((mine - m) * c));
    if (C > 1) {
      if (t == 0) stat = make_float2(m, z);
      cluster.sync();
      float mm = -INFINITY;
      for (int q = 0; q < C; ++q) mm = max_nan(mm, cluster.map_shared_rank(&stat, q)->x);
      float zz = 0.0f;
      for (int q = 0; q < C; ++q) {
        const float2 o = *cluster.map_shared_rank(&stat, q);
        zz += o.x == -INFINITY ? 0.0f : o.y * exp2_fast((o.x - mm) * c);
      }
      m = mm;
      z = zz;
      cluster.sync();                        // every CTA has read the others' before one writes again or ends
    }
    const bool some = teacher_row<T, DW_T>(A, team, i, s, m, z, probs, rank == 0);
    if (g) {
      const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f), iz = 1.0f / z;
      Raw* gv = reinterpret_cast<Raw*>(g + head);
      for (int q0 = v0 + t; q0 < v1; q0 += 4 * DW_T) {
        V v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q0 + u * DW_T < v1) v[u].load(sv + q0 + u * DW_T);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q0 + u * DW_T < v1) {
            V o;
#pragma unroll
            for (int e = 0; e < V::N; ++e)
              o.set(e, some ? a * (exp2_fast((v[u].get(e) - m) * c) * iz) : 0.0f);
            gv[q0 + u * DW_T] = o.raw;
          }
      }
      if (has) g[single] = elem_from_f<T>(some ? a * (exp2_fast((elem_to_f<T>(s[single]) - m) * c) * iz) : 0.0f);
      __syncthreads();
      if (some) kept_gradients<T, DW_T>(A, team, i, s, g, m, c, a, iz, probs, lo, hi);
    }
    __syncthreads();
  }
}

template <typename T, int NT, int NV>
cudaError_t run_rows(const DistillArgs& A, cudaStream_t st) {
  const int64_t want = (A.n + 256 / NT - 1) / (256 / NT), most = 148 * 32;
  distill_rows_kernel<T, NT, NV><<<(unsigned)(want < most ? want : most), 256, 0, st>>>(A);
  return cudaGetLastError();
}

template <typename T, int BYTES>
cudaError_t run_wide(const DistillArgs& A, cudaStream_t st) {
  // CTAs of a row: as many as fill 148 SMs twice (few rows), and with many rows
  // enough to keep 296 CTAs' rows within about 32 MB of L2
  int C = 1;
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  while (C < 8 && bytes / C > 32768 && (A.n * C < 296 || 296 / C * bytes > (32 << 20))) C *= 2;
  int64_t rows = 296 / C;
  if (rows > A.n) rows = A.n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(DW_T);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_wide_kernel<T, BYTES>, A);
}

template <typename T>
cudaError_t run_t(const DistillArgs& A, cudaStream_t st) {
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  // the vectors of student and gradient rows coincide when both start alike
  if (A.grad && ((uintptr_t)A.grad - (uintptr_t)A.student) % 16) return run_wide<T, (int)sizeof(T)>(A, st);
  if (bytes <= 512) return run_rows<T, 32, 1>(A, st);
  if (bytes <= 1024) return run_rows<T, 32, 2>(A, st);
  if (bytes <= 4096) return run_rows<T, 32, 8>(A, st);
  if (bytes <= 8192) return run_rows<T, 256, 2>(A, st);
  if (bytes <= 16384) return run_rows<T, 256, 4>(A, st);
  if (bytes <= 32768) return run_rows<T, 256, 8>(A, st);
  return run_wide<T, 16>(A, st);
}

}  // namespace

cudaError_t launch_distill(const void* student, int dtype, int64_t n, int classes,
                           const float* tl, const int32_t* ti, int k, float temperature,
                           const float* scale, float* loss, void* grad, cudaStream_t st) {
  const DistillArgs A{student, n, classes, tl, ti, k, temperature, scale, loss, grad};
  if (dtype == NERF_DTYPE_FP32) return run_t<float>(A, st);
  if (dtype == NERF_DTYPE_BF16) return run_t<__nv_bfloat16>(A, st);
  return run_t<__half>(A, st);
}

}  // namespace nerfb
