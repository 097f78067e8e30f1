// The C ABI of the expert operators: argument validation, then one launcher each.
#include <cstdio>

#include "nerf_experts.cuh"

namespace nerfb {
void set_global_error(const char* msg);
}

using namespace nerfb;

namespace {

nerf_status refuse(const char* fn, const char* why) {
  char buf[160];
  snprintf(buf, sizeof buf, "%s: %s", fn, why);
  set_global_error(buf);
  return NERF_ERR_INVALID_ARG;
}

nerf_status launched(const char* fn, cudaError_t e) {
  if (e == cudaSuccess) return NERF_OK;
  char buf[160];
  snprintf(buf, sizeof buf, "%s: %s", fn, cudaGetErrorString(e));
  set_global_error(buf);
  return NERF_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t dtype_size(int dtype) { return dtype == NERF_DTYPE_FP32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype >= NERF_DTYPE_FP32 && dtype <= NERF_DTYPE_FP16; }

// n points of k pairs each; nullptr when the sizes are in range.
const char* bad_pairs(int64_t n, int k) {
  if (n < 1 || k < 1) return "n and k must be at least 1";
  if (k > EXPERT_MAX_K) return "k above 64";
  if (n > EXPERT_MAX_PAIRS / k) return "more than 2^30 pairs";
  return nullptr;
}
const char* bad_experts(int n_experts) {
  return n_experts < 1 || n_experts > EXPERT_MAX ? "n_experts must be in 1..4096" : nullptr;
}
const char* bad_rows(int dtype, int64_t n, int width, const void* pos, int k, const void* weights,
                     const void* dw) {
  if (const char* why = bad_pairs(n, k)) return why;
  if (!dtype_ok(dtype)) return "unknown dtype";
  if (width < 1 || width > (1 << 20)) return "width must be in 1..2^20";
  if (!pos) return "pos is NULL";
  if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(dw, 4)) return "misaligned pointer";
  return nullptr;
}
const char* bad_cells(const void* x, const void* d, int64_t n, const void* offset, int n_cells,
                      const void* cell_w) {
  if (!x || !d || !offset || !cell_w) return "NULL pointer";
  if (n < 1 || n > EXPERT_MAX_PAIRS) return "n_rows must be in 1..2^30";
  if (n_cells < 1 || n_cells > EXPERT_MAX) return "n_cells must be in 1..4096";
  if (!aligned(x, 4) || !aligned(d, 4) || !aligned(offset, 4) || !aligned(cell_w, 4))
    return "misaligned pointer";
  return nullptr;
}

}  // namespace

extern "C" {

nerf_status nerf_expert_sort_workspace(int64_t n, int k, int n_experts, int64_t* out_bytes) {
  static const char fn[] = "nerf_expert_sort_workspace";
  if (!out_bytes) return refuse(fn, "out_bytes is NULL");
  if (const char* why = bad_pairs(n, k)) return refuse(fn, why);
  if (const char* why = bad_experts(n_experts)) return refuse(fn, why);
  *out_bytes = expert_sort_workspace(n * k, n_experts);
  return NERF_OK;
}

nerf_status nerf_expert_sort(const int32_t* ids, int64_t n, int k, int n_experts,
                             int32_t* out_offset, int32_t* out_order, int32_t* out_pos,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  static const char fn[] = "nerf_expert_sort";
  if (!ids || !out_offset || !out_pos || !workspace) return refuse(fn, "NULL pointer");
  if (const char* why = bad_pairs(n, k)) return refuse(fn, why);
  if (const char* why = bad_experts(n_experts)) return refuse(fn, why);
  if (!aligned(ids, 4) || !aligned(out_offset, 4) || !aligned(out_order, 4) ||
      !aligned(out_pos, 4) || !aligned(workspace, 16))
    return refuse(fn, "misaligned pointer");
  if (workspace_bytes < expert_sort_workspace(n * k, n_experts))
    return refuse(fn, "workspace too small");
  return launched(fn, launch_expert_sort(ids, n * k, n_experts, out_offset, out_order, out_pos,
                                         workspace, (cudaStream_t)stream));
}

nerf_status nerf_expert_dispatch(const void* x, int dtype, int64_t n, int width,
                                 const int32_t* pos, int k, const float* weights, void* rows,
                                 void* stream) {
  static const char fn[] = "nerf_expert_dispatch";
  if (const char* why = bad_rows(dtype, n, width, pos, k, weights, nullptr)) return refuse(fn, why);
  if (!x || !rows) return refuse(fn, "NULL pointer");
  if (!aligned(x, dtype_size(dtype)) || !aligned(rows, dtype_size(dtype)))
    return refuse(fn, "misaligned pointer");
  return launched(fn, launch_rows_scatter(x, nullptr, dtype, n, width, pos, k, weights, rows,
                                          nullptr, (cudaStream_t)stream));
}

nerf_status nerf_expert_dispatch_backward(const void* d_rows, const void* x, int dtype, int64_t n,
                                          int width, const int32_t* pos, int k,
                                          const float* weights, void* d_x, float* d_weights,
                                          void* stream) {
  static const char fn[] = "nerf_expert_dispatch_backward";
  if (const char* why = bad_rows(dtype, n, width, pos, k, weights, d_weights)) return refuse(fn, why);
  if (!d_rows) return refuse(fn, "d_rows is NULL");
  if (!d_x && !d_weights) return refuse(fn, "nothing to compute: d_x and d_weights are NULL");
  if (d_weights && !x) return refuse(fn, "d_weights needs x");
  const size_t a = dtype_size(dtype);
  if (!aligned(d_rows, a) || !aligned(x, a) || !aligned(d_x, a)) return refuse(fn, "misaligned pointer");
  return launched(fn, launch_rows_gather(d_rows, x, dtype, n, width, pos, k, weights, d_x, d_weights,
                                         (cudaStream_t)stream));
}

nerf_status nerf_expert_combine(const void* rows, int dtype, int64_t n, int width,
                                const int32_t* pos, int k, const float* weights, void* out,
                                void* stream) {
  static const char fn[] = "nerf_expert_combine";
  if (const char* why = bad_rows(dtype, n, width, pos, k, weights, nullptr)) return refuse(fn, why);
  if (!rows || !out) return refuse(fn, "NULL pointer");
  if (!aligned(rows, dtype_size(dtype)) || !aligned(out, dtype_size(dtype)))
    return refuse(fn, "misaligned pointer");
  return launched(fn, launch_rows_gather(rows, nullptr, dtype, n, width, pos, k, weights, out,
                                         nullptr, (cudaStream_t)stream));
}

nerf_status nerf_expert_combine_backward(const void* d_out, const void* rows, int dtype, int64_t n,
                                         int width, const int32_t* pos, int k,
                                         const float* weights, void* d_rows, float* d_weights,
                                         void* stream) {
  static const char fn[] = "nerf_expert_combine_backward";
  if (const char* why = bad_rows(dtype, n, width, pos, k, weights, d_weights)) return refuse(fn, why);
  if (!d_out) return refuse(fn, "d_out is NULL");
  if (!d_rows && !d_weights) return refuse(fn, "nothing to compute: d_rows and d_weights are NULL");
  if (d_weights && !rows) return refuse(fn, "d_weights needs rows");
  const size_t a = dtype_size(dtype);
  if (!aligned(d_out, a) || !aligned(rows, a) || !aligned(d_rows, a))
    return refuse(fn, "misaligned pointer");
  return launched(fn, launch_rows_scatter(d_out, rows, dtype, n, width, pos, k, weights, d_rows,
                                          d_weights, (cudaStream_t)stream));
}

nerf_status nerf_distill_topk(const void* student, int dtype, int64_t n, int n_classes,
                              const float* teacher_logits, const int32_t* teacher_ids, int k,
                              float temperature, const float* row_scale, float* out_loss,
                              void* out_grad, void* stream) {
  static const char fn[] = "nerf_distill_topk";
  if (!student || !teacher_logits || !teacher_ids || !out_loss) return refuse(fn, "NULL pointer");
  if (!dtype_ok(dtype)) return refuse(fn, "unknown dtype");
  if (n < 1 || n > (int64_t(1) << 40)) return refuse(fn, "n must be in 1..2^40");
  if (n_classes < 1 || n_classes > (1 << 30)) return refuse(fn, "n_classes must be in 1..2^30");
  if (k < 1 || k > DISTILL_MAX_K) return refuse(fn, "k must be in 1..256");
  // T, log2(e) / T and T^2 stay normal numbers
  if (!(temperature >= 0x1p-60f && temperature <= 0x1p60f))
    return refuse(fn, "temperature must be in 2^-60..2^60");
  const size_t a = dtype_size(dtype);
  if (!aligned(student, a) || !aligned(out_grad, a) || !aligned(teacher_logits, 4) ||
      !aligned(teacher_ids, 4) || !aligned(row_scale, 4) || !aligned(out_loss, 4))
    return refuse(fn, "misaligned pointer");
  return launched(fn, launch_distill(student, dtype, n, n_classes, teacher_logits, teacher_ids, k,
                                     temperature, row_scale, out_loss, out_grad,
                                     (cudaStream_t)stream));
}

nerf_status nerf_cells_forward(const float* x, const float* d, int64_t n_rows,
                               const int32_t* offset, int n_cells, const float* cell_w,
                               float* out_raw, float* out_hidden, void* stream) {
  static const char fn[] = "nerf_cells_forward";
  if (const char* why = bad_cells(x, d, n_rows, offset, n_cells, cell_w)) return refuse(fn, why);
  if (!out_raw) return refuse(fn, "NULL pointer");
  if (!aligned(out_raw, 16) || !aligned(out_hidden, 16))
    return refuse(fn, "out_raw and out_hidden must be 16-byte aligned");
  return launched(fn, launch_cells_forward(x, d, n_rows, offset, n_cells, cell_w, out_raw,
                                           out_hidden, (cudaStream_t)stream));
}

nerf_status nerf_cells_backward_workspace(int64_t n_rows, int n_cells, int64_t* out_bytes) {
  static const char fn[] = "nerf_cells_backward_workspace";
  if (!out_bytes) return refuse(fn, "out_bytes is NULL");
  if (n_rows < 1 || n_rows > EXPERT_MAX_PAIRS) return refuse(fn, "n_rows must be in 1..2^30");
  if (const char* why = bad_experts(n_cells)) return refuse(fn, why);
  *out_bytes = cells_backward_workspace(n_rows, n_cells);
  return NERF_OK;
}

nerf_status nerf_cells_backward(const float* x, const float* d, int64_t n_rows,
                                const int32_t* offset, int n_cells, const float* cell_w,
                                const float* hidden, const float* d_raw, float* grad_cell_w,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  static const char fn[] = "nerf_cells_backward";
  if (const char* why = bad_cells(x, d, n_rows, offset, n_cells, cell_w)) return refuse(fn, why);
  if (!hidden || !d_raw || !grad_cell_w || !workspace) return refuse(fn, "NULL pointer");
  if (!aligned(hidden, 16) || !aligned(d_raw, 16) || !aligned(grad_cell_w, 4) || !aligned(workspace, 16))
    return refuse(fn, "hidden, d_raw and workspace must be 16-byte aligned");
  if (workspace_bytes < cells_backward_workspace(n_rows, n_cells))
    return refuse(fn, "workspace too small");
  return launched(fn, launch_cells_backward(x, d, n_rows, offset, n_cells, cell_w, hidden, d_raw,
                                            grad_cell_w, workspace, (cudaStream_t)stream));
}

}  // extern "C"
