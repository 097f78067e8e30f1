// The KiloNeRF cell networks on rows sorted by cell, forward and weight gradient:
//   z1 = W1 gamma(x) + b1, h1 = relu(z1); z2 = W2 h1 + b2, h2 = relu(z2);
//   (r, g, b) = Wc [h2; gamma(d/|d|)] + bc, sigma = ws . h2 + bs.
// Backward, with g = d raw: g2 = (Wc_h^T g_rgb + ws g_sigma) (h2 > 0),
// g1 = (W2^T g2) (h1 > 0), and each weight's gradient the sum over the cell's
// rows of (its output's gradient) x (its input).
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

constexpr int CT = 256;
// parameter offsets inside a cell's blob
constexpr int O_W1 = 0, O_B1 = 2016, O_W2 = 2048, O_B2 = 3072, O_WS = 3104, O_BS = 3136, O_WC = 3137,
              O_BC = 3314;
constexpr int CF_ROWS = 8;      // rows of one CTA at a time

// unit direction: one rounded division per coordinate by the rounded norm
__device__ __forceinline__ void unit3(const float* d, float* u) {
  const float len = sqrtf(fmaf(d[0], d[0], fmaf(d[1], d[1], d[2] * d[2])));
  u[0] = d[0] / len;
  u[1] = d[1] / len;
  u[2] = d[2] / len;
}
__device__ __forceinline__ float pe_value(const float* v, int octaves, int j) {
  if (j < 3) return v[j];
  const int q = (j - 3) % (3 * octaves);
  float s, c;
  pe_sincos(v[q / octaves], q % octaves, &s, &c);
  return j - 3 < 3 * octaves ? s : c;
}

// One CTA per cell, CF_ROWS rows at a time, thread = (row, output).
__global__ void __launch_bounds__(CT)
cells_forward_kernel(const float* __restrict__ x, const float* __restrict__ d, int64_t n,
                     const int32_t* __restrict__ offset, const float* __restrict__ cell_w,
                     float* __restrict__ raw, float* __restrict__ hidden) {
  __shared__ float w[CELL_NP], px[CF_ROWS][63], pd[CF_ROWS][27], h1[CF_ROWS][32], h2[CF_ROWS][32];
  const int cell = blockIdx.x, t = threadIdx.x;
  const int64_t a = max(offset[cell], 0), b = min((int64_t)offset[cell + 1], n);
  if (a >= b) return;
  for (int q = t; q < CELL_NP; q += CT) w[q] = cell_w[(int64_t)cell * CELL_NP + q];
  const int r = t / 32, o = t & 31;
  for (int64_t i0 = a; i0 < b; i0 += CF_ROWS) {
    __syncthreads();
    const bool on = i0 + r < b;
    if (on) {
      const float* v = x + (i0 + r) * 3;
      float u[3];
      unit3(d + (i0 + r) * 3, u);
      for (int j = o; j < 63; j += 32) px[r][j] = pe_value(v, 10, j);
      if (o < 27) pd[r][o] = pe_value(u, 4, o);
    }
    __syncthreads();
    if (on) {
      float s = w[O_B1 + o];
      for (int k = 0; k < 63; ++k) s = fmaf(w[O_W1 + o * 63 + k], px[r][k], s);
      h1[r][o] = fmaxf(s, 0.0f);
    }
    __syncthreads();
    if (on) {
      float s = w[O_B2 + o];
      for (int k = 0; k < 32; ++k) s = fmaf(w[O_W2 + o * 32 + k], h1[r][k], s);
      h2[r][o] = fmaxf(s, 0.0f);
      if (hidden) {
        hidden[(i0 + r) * 64 + o] = h1[r][o];
        hidden[(i0 + r) * 64 + 32 + o] = h2[r][o];
      }
    }
    __syncthreads();
    if (on && o < 4) {
      float s = o < 3 ? w[O_BC + o] : w[O_BS];
      const float* wr = o < 3 ? w + O_WC + o * 59 : w + O_WS;
      for (int k = 0; k < 32; ++k) s = fmaf(wr[k], h2[r][k], s);
      if (o < 3)
        for (int k = 0; k < 27; ++k) s = fmaf(wr[32 + k], pd[r][k], s);
      raw[(i0 + r) * 4 + o] = s;
    }
  }
}

// One CTA per cell; the row's vectors in shared memory, every thread the
// running sums of its parameters.
__global__ void __launch_bounds__(CT)
cells_backward_kernel(const float* __restrict__ x, const float* __restrict__ d, int64_t n,
                      const int32_t* __restrict__ offset, const float* __restrict__ cell_w,
                      const float* __restrict__ hidden, const float* __restrict__ d_raw,
                      float* __restrict__ grad) {
  // one row: [gamma(x) 63 | 1 | h1 32 | h2 32 | gamma(d) 27] and [g1 32 | g2 32 | g 4]
  __shared__ float w2[1024], wh[4][32], in[155], out[68];
  const int cell = blockIdx.x, t = threadIdx.x;
  const int64_t a = max(offset[cell], 0), b = min((int64_t)offset[cell + 1], n);
  constexpr int PER = (CELL_NP + CT - 1) / CT;
  float acc[PER];
  int ia[PER], ib[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int q = t + j * CT;
    acc[j] = 0.0f;
    ia[j] = ib[j] = 0;
    if (q < O_B1) { ia[j] = q % 63; ib[j] = q / 63; }
    else if (q < O_W2) { ia[j] = 63; ib[j] = q - O_B1; }
    else if (q < O_B2) { ia[j] = 64 + (q - O_W2) % 32; ib[j] = 32 + (q - O_W2) / 32; }
    else if (q < O_WS) { ia[j] = 63; ib[j] = 32 + q - O_B2; }
    else if (q < O_BS) { ia[j] = 96 + q - O_WS; ib[j] = 67; }
    else if (q < O_WC) { ia[j] = 63; ib[j] = 67; }
    else if (q < O_BC) { ia[j] = 96 + (q - O_WC) % 59; ib[j] = 64 + (q - O_WC) / 59; }
    else if (q < CELL_NP) { ia[j] = 63; ib[j] = 64 + q - O_BC; }
  }
  if (a < b) {
    const float* W = cell_w + (int64_t)cell * CELL_NP;
    for (int q = t; q < 1024; q += CT) w2[q] = W[O_W2 + q];
    if (t < 128) wh[t / 32][t & 31] = t < 96 ? W[O_WC + t / 32 * 59 + (t & 31)] : W[O_WS + t - 96];
  }
  for (int64_t i = a; i < b; ++i) {
    __syncthreads();
    if (t < 63) in[t] = pe_value(x + i * 3, 10, t);
    else if (t == 63) in[t] = 1.0f;
    else if (t < 128) in[t] = hidden[i * 64 + t - 64];
    else if (t < 155) {
      float u[3];
      unit3(d + i * 3, u);
      in[t] = pe_value(u, 4, t - 128);
    } else if (t >= 160 && t < 164) out[64 + t - 160] = d_raw[i * 4 + t - 160];
    __syncthreads();
    if (t < 32) {
      float s = 0.0f;
      for (int c = 0; c < 4; ++c) s = fmaf(wh[c][t], out[64 + c], s);
      out[32 + t] = in[96 + t] > 0.0f ? s : 0.0f;
      __syncwarp();
      s = 0.0f;
      for (int k = 0; k < 32; ++k) s = fmaf(w2[k * 32 + t], out[32 + k], s);
      out[t] = in[64 + t] > 0.0f ? s : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = fmaf(in[ia[j]], out[ib[j]], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (t + j * CT < CELL_NP) grad[(int64_t)cell * CELL_NP + t + j * CT] = acc[j];
}

}  // namespace

cudaError_t launch_cells_forward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                 int n_cells, const float* cell_w, float* raw, float* hidden,
                                 cudaStream_t st) {
  cells_forward_kernel<<<n_cells, CT, 0, st>>>(x, d, n, offset, cell_w, raw, hidden);
  return cudaGetLastError();
}

int64_t cells_backward_workspace(int64_t, int) { return 16; }

cudaError_t launch_cells_backward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                  int n_cells, const float* cell_w, const float* hidden,
                                  const float* d_raw, float* grad, void*, cudaStream_t st) {
  cells_backward_kernel<<<n_cells, CT, 0, st>>>(x, d, n, offset, cell_w, hidden, d_raw, grad);
  return cudaGetLastError();
}

}  // namespace nerfb
