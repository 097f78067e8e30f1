// Launchers of the expert operators (sort, rows there and back, distillation,
// per-cell networks). Each returns the launch status.
#pragma once

#include "nerf_internal.cuh"

namespace nerfb {

constexpr int EXPERT_MAX = 4096;            // experts of one sort (the 16^3 cells)
constexpr int EXPERT_MAX_K = 64;            // experts of one point
constexpr int DISTILL_MAX_K = 256;          // kept teacher logits of one row
constexpr int64_t EXPERT_MAX_PAIRS = int64_t(1) << 30;
constexpr int CELL_NP = 3317;               // parameters of one cell's network

int64_t expert_sort_workspace(int64_t pairs, int n_experts);
cudaError_t launch_expert_sort(const int32_t* ids, int64_t pairs, int n_experts, int32_t* offset,
                               int32_t* order, int32_t* pos, void* work, cudaStream_t st);

// rows[pos] = w x (rows NULL: not written); dw = <x, other[pos]> (dw NULL: not computed)
cudaError_t launch_rows_scatter(const void* x, const void* other, int dtype, int64_t n, int width,
                                const int32_t* pos, int k, const float* w, void* rows, float* dw,
                                cudaStream_t st);
// out = sum_j w rows[pos] (out NULL: not written); dw = <x, rows[pos]> (dw NULL: not computed)
cudaError_t launch_rows_gather(const void* rows, const void* x, int dtype, int64_t n, int width,
                               const int32_t* pos, int k, const float* w, void* out, float* dw,
                               cudaStream_t st);

cudaError_t launch_distill(const void* student, int dtype, int64_t n, int classes,
                           const float* t_logits, const int32_t* t_ids, int k, float temperature,
                           const float* scale, float* loss, void* grad, cudaStream_t st);

cudaError_t launch_cells_forward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                 int n_cells, const float* cell_w, float* raw, float* hidden,
                                 cudaStream_t st);
int64_t cells_backward_workspace(int64_t n, int n_cells);
cudaError_t launch_cells_backward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                  int n_cells, const float* cell_w, const float* hidden,
                                  const float* d_raw, float* grad, void* work, cudaStream_t st);

// A launch that may start while the launch before it in the stream still runs. Its
// kernel waits for that one's end (cudaGridDependencySynchronize) in every block
// before it reads a result of it, writes what it reads, or ends; and it takes those
// results without const __restrict__, whose loads assume data that no one writes.
template <typename K, typename... Args>
cudaError_t launch_early(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nerfb
