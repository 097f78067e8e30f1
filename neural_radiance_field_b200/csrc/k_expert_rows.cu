// Rows taken to the experts' order and back, with weights, and the weights'
// gradients:
//   scatter: rows[pos] = w x, with <x, other[pos]>   (dispatch, combine's backward)
//   gather:  out = sum_j w rows[pos], with <x, rows[pos]>   (combine, dispatch's backward)
//
// Bound by memory: every row is read or written once. A group of lanes takes one
// point and holds the point's own row in registers while its k sorted rows pass,
// so the point's row moves once whatever k is, and the weight gradient comes from
// the vectors that the row's own pass has in registers. A group has at most eight
// lanes, which take several vectors of a wide row at once: that keeps more loads
// in flight and spreads the pairs' index work over them. Rows move in vectors of
// 16, 8 or 4 bytes, the widest that their size and the buffers allow, else by
// element. On the device, 262,144 points of 256 bf16 with two pairs each: dispatch
// 62 us (6.2 TB/s, 0.96 of the measured copy rate), combine's backward with its weight
// gradient 100 us (0.99); 786,432 points of 4 fp32 with eight pairs: combine 30 us
// (0.79; its pairs' positions and weights are a third of the bytes). The grid covers
// points: few points with wide rows leave most of the GPU idle (300 points of 131,072
// fp32 with three pairs: 2.0 ms of 0.12).
#include "nerf_experts.cuh"
#include "nerf_vec.cuh"

namespace nerfb {
namespace {

constexpr int RT = 256;

// A lane's dot products are summed in runs of RUN terms and the runs' sums in order: a
// chain of 2^17 roundings, a lane's share of the widest row, was off by 7e-4 where
// equal terms round one way. The sums of the runs wait in shared memory.
constexpr int RUN = 512;
template <int KC>
struct Runs {
  float sum[KC][RT];
  // `done` vectors of the row lie behind the lanes, `run` make a run
  __device__ __forceinline__ void next(float* dot, int done, int run) {
    if (done == 0 || (done & (run - 1)) != 0) return;
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      sum[j][threadIdx.x] = done == run ? dot[j] : sum[j][threadIdx.x] + dot[j];
      dot[j] = 0.0f;
    }
  }
  // behind the last of the row's `nv` vectors
  __device__ __forceinline__ void end(float* dot, int lane, int nv, int run) {
    if (lane + run < nv)
#pragma unroll
      for (int j = 0; j < KC; ++j) dot[j] += sum[j][threadIdx.x];
  }
};
template <>
struct Runs<0> {                             // one run
  __device__ __forceinline__ void next(float*, int, int) {}
  __device__ __forceinline__ void end(float*, int, int, int) {}
};
// What a kernel does about the weights' gradients. Rows of one run (up to 4,096
// elements on eight lanes) have a form of their own: with the runs' code the other
// takes up to 127 registers for 80.
enum Dots { NO_DOTS, ONE_RUN, MANY_RUNS };

// a chunk of at most KC of a point's pairs: sorted rows (-1: none) and weights
template <int KC>
struct Pairs {
  int32_t p[KC];
  float w[KC];
  __device__ __forceinline__ void load(const int32_t* __restrict__ pos, const float* __restrict__ weights,
                                       int64_t i, int k, int j0, int64_t m, bool on) {
    const int64_t at = i * k + j0;
    if (KC == 8 && k == 8) {               // 16-byte loads where the caller's buffers have them aligned
      if ((((uintptr_t)pos | (uintptr_t)weights) & 15) == 0) {
        const int4 a = on ? __ldg(reinterpret_cast<const int4*>(pos + at)) : make_int4(-1, -1, -1, -1);
        const int4 b = on ? __ldg(reinterpret_cast<const int4*>(pos + at) + 1) : make_int4(-1, -1, -1, -1);
        p[0] = a.x, p[1 % KC] = a.y, p[2 % KC] = a.z, p[3 % KC] = a.w;
        p[4 % KC] = b.x, p[5 % KC] = b.y, p[6 % KC] = b.z, p[7 % KC] = b.w;
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), e = c;
        if (weights && on) {
          c = __ldg(reinterpret_cast<const float4*>(weights + at));
          e = __ldg(reinterpret_cast<const float4*>(weights + at) + 1);
        }
        w[0] = c.x, w[1 % KC] = c.y, w[2 % KC] = c.z, w[3 % KC] = c.w;
        w[4 % KC] = e.x, w[5 % KC] = e.y, w[6 % KC] = e.z, w[7 % KC] = e.w;
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if ((uint64_t)(int64_t)p[j] >= (uint64_t)m) p[j] = -1;
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const bool in = on && j0 + j < k;
      p[j] = in ? __ldg(pos + at + j) : -1;
      w[j] = in && weights ? __ldg(weights + at + j) : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < KC; ++j)
      if ((uint64_t)(int64_t)p[j] >= (uint64_t)m) p[j] = -1;
  }
};

// dw of a chunk from each lane's partial dot products
template <int KC>
__device__ __forceinline__ void store_dots(float* dot, int G, int lane, bool on, int64_t i, int k, int j0,
                                           float* __restrict__ dw) {
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    if (j0 + j >= k) break;                // uniform over the grid
    float s = dot[j];
    for (int o = G >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (on && lane == 0) dw[i * k + j0 + j] = s;
  }
}

template <typename T, int BYTES, int KC, Dots DOTS>
__global__ void __launch_bounds__(RT)
rows_scatter_kernel(const T* __restrict__ x, const T* __restrict__ other, int64_t n, int nv, int G,
                    const int32_t* __restrict__ pos, int k, const float* __restrict__ weights,
                    T* __restrict__ rows, float* __restrict__ dw) {
  using V = Vec<T, BYTES>;
  constexpr bool DW = DOTS != NO_DOTS;
  __shared__ Runs<DOTS == MANY_RUNS ? KC : 0> runs;
  constexpr int U = 4;                  // vectors of a row that a lane has in flight
  const int lane = threadIdx.x & (G - 1);
  const int64_t i = (int64_t)blockIdx.x * (RT / G) + threadIdx.x / G, m = n * k;
  const bool on = i < n;
  for (int j0 = 0; j0 < k; j0 += KC) {
    Pairs<KC> q;
    q.load(pos, weights, i, k, j0, m, on);
    float dot[KC] = {};
    if (on)
      for (int v0 = lane; v0 < nv; v0 += U * G) {
        runs.next(dot, v0 - lane, RUN / V::N * G);
        V a[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * G < nv) a[u].load(x, i * nv + v0 + u * G);
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          if (q.p[j] < 0) continue;
          const int64_t row = (int64_t)q.p[j] * nv + v0;
          V b[U];
          if (DW) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (v0 + u * G < nv) b[u].load(other, row + u * G);
          }
          if (rows) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (v0 + u * G < nv) {
                V o = a[u];
                if (weights) {
                  float f[V::N];
#pragma unroll
                  for (int c = 0; c < V::N; ++c) f[c] = q.w[j] * a[u].get(c);
                  o.pack(f);
                }
                o.store(rows, row + u * G);
              }
          }
          if (DW) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (v0 + u * G < nv)
#pragma unroll
                for (int c = 0; c < V::N; ++c) dot[j] = fmaf(a[u].get(c), b[u].get(c), dot[j]);
          }
        }
      }
    if (on) runs.end(dot, lane, nv, RUN / V::N * G);
    if (DW) store_dots<KC>(dot, G, lane, on, i, k, j0, dw);
  }
}

template <typename T, int BYTES, int KC, Dots DOTS>
__global__ void __launch_bounds__(RT)
rows_gather_kernel(const T* __restrict__ rows, const T* __restrict__ x, int64_t n, int nv, int G,
                   const int32_t* __restrict__ pos, int k, const float* __restrict__ weights,
                   T* __restrict__ out, float* __restrict__ dw) {
  using V = Vec<T, BYTES>;
  constexpr bool DW = DOTS != NO_DOTS;
  __shared__ Runs<DOTS == MANY_RUNS ? KC : 0> runs;
  constexpr int U = KC == 2 || BYTES <= 4 ? 4 : KC == 4 ? 2 : 1;                  // vectors of a row that a lane has in flight
  const int lane = threadIdx.x & (G - 1);
  const int64_t i = (int64_t)blockIdx.x * (RT / G) + threadIdx.x / G, m = n * k;
  const bool on = i < n;
  Pairs<KC> q;
  if (k <= KC) {                             // one pass for the sum and the dot products
    q.load(pos, weights, i, k, 0, m, on);
    float dot[KC] = {};
    if (on)
      for (int v0 = lane; v0 < nv; v0 += U * G) {
        runs.next(dot, v0 - lane, RUN / V::N * G);
        V a[U], b[U][KC];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * G < nv) {
#pragma unroll
            for (int j = 0; j < KC; ++j)
              if (q.p[j] >= 0) b[u][j].load(rows, (int64_t)q.p[j] * nv + v0 + u * G);
            if (DW) a[u].load(x, i * nv + v0 + u * G);
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * G < nv) {
            float s[V::N] = {};
#pragma unroll
            for (int j = 0; j < KC; ++j) {
              if (q.p[j] < 0) continue;
#pragma unroll
              for (int c = 0; c < V::N; ++c) {
                const float f = b[u][j].get(c);
                s[c] = fmaf(q.w[j], f, s[c]);
                if (DW) dot[j] = fmaf(a[u].get(c), f, dot[j]);
              }
            }
            if (out) {
              V o;
              o.pack(s);
              o.store(out, i * nv + v0 + u * G);
            }
          }
      }
    if (on) runs.end(dot, lane, nv, RUN / V::N * G);
    if (DW) store_dots<KC>(dot, G, lane, on, i, k, 0, dw);
    return;
  }
  if (out && on)                             // more pairs than a chunk: the sum over all of them first
    for (int v = lane; v < nv; v += G) {
      float s[V::N] = {};
      for (int j0 = 0; j0 < k; j0 += KC) {
        q.load(pos, weights, i, k, j0, m, true);
        V b[KC];
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (q.p[j] >= 0) b[j].load(rows, (int64_t)q.p[j] * nv + v);
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (q.p[j] >= 0) {
#pragma unroll
            for (int c = 0; c < V::N; ++c) s[c] = fmaf(q.w[j], b[j].get(c), s[c]);
          }
      }
      V o;
      o.pack(s);
      o.store(out, i * nv + v);
    }
  if (DW)
    for (int j0 = 0; j0 < k; j0 += KC) {
      q.load(pos, nullptr, i, k, j0, m, on);
      float dot[KC] = {};
      if (on)
        for (int v = lane; v < nv; v += G) {
          runs.next(dot, v - lane, RUN / V::N * G);
          V a;
          a.load(x, i * nv + v);
#pragma unroll
          for (int j = 0; j < KC; ++j) {
            if (q.p[j] < 0) continue;
            V b;
            b.load(rows, (int64_t)q.p[j] * nv + v);
#pragma unroll
            for (int c = 0; c < V::N; ++c) dot[j] = fmaf(a.get(c), b.get(c), dot[j]);
          }
        }
      if (on) runs.end(dot, lane, nv, RUN / V::N * G);
      store_dots<KC>(dot, G, lane, on, i, k, j0, dw);
    }
}

struct RowArgs {
  const void *a, *b;           // scatter: x, other; gather: rows, x
  int64_t n;
  int nv, G;
  const int32_t* pos;
  int k;
  const float* w;
  void* out;                   // scatter: rows; gather: out
  float* dw;
  cudaStream_t st;
};

template <bool SCATTER, typename T, int BYTES, int KC, Dots DOTS>
void run(const RowArgs& A) {
  const unsigned grid = (unsigned)((A.n + RT / A.G - 1) / (RT / A.G));
  if (SCATTER)
    rows_scatter_kernel<T, BYTES, KC, DOTS><<<grid, RT, 0, A.st>>>((const T*)A.a, (const T*)A.b, A.n, A.nv, A.G, A.pos,
                                                                 A.k, A.w, (T*)A.out, A.dw);
  else
    rows_gather_kernel<T, BYTES, KC, DOTS><<<grid, RT, 0, A.st>>>((const T*)A.a, (const T*)A.b, A.n, A.nv, A.G, A.pos,
                                                                A.k, A.w, (T*)A.out, A.dw);
}
// Pairs in chunks of two for k <= 2, of four for k <= 4, else of eight: an unused
// place of a chunk costs its predicates and registers. 200,000 points of 256 bf16,
// dispatch / combine / combine's backward: k 2 in chunks of two 49 / 46 / 78 us, of
// four 49 / 54 / 84, of eight 51 / 120 / 86; k 4 of four 83 / 75 / 146, of eight
// 83 / 131 / 148.
template <bool SCATTER, typename T, int BYTES, Dots DOTS>
void run_k(const RowArgs& A) {
  if (A.k <= 2) run<SCATTER, T, BYTES, 2, DOTS>(A);
  else if (A.k <= 4) run<SCATTER, T, BYTES, 4, DOTS>(A);
  else run<SCATTER, T, BYTES, 8, DOTS>(A);
}
template <bool SCATTER, typename T, int BYTES>
void run_dots(const RowArgs& A) {
  if (!A.dw) run_k<SCATTER, T, BYTES, NO_DOTS>(A);
  else if (A.nv <= RUN / Vec<T, BYTES>::N * A.G) run_k<SCATTER, T, BYTES, ONE_RUN>(A);
  else run_k<SCATTER, T, BYTES, MANY_RUNS>(A);
}
template <bool SCATTER, typename T>
cudaError_t run_t(RowArgs A, int width) {
  const uintptr_t all = (uintptr_t)A.a | (uintptr_t)A.b | (uintptr_t)A.out | (uintptr_t)(width * sizeof(T));
  const int bytes = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : (int)sizeof(T);
  A.nv = (int)(width * sizeof(T)) / bytes;
  // Lanes of a point. Of wide vectors up to sixteen go to four lanes, more to eight
  // (64 fp16 x 4 pairs of 429,740 points: four lanes 47 us, eight 62, two 55;
  // 1000 fp32 x 4 of 30,000: four 142, eight 99). Of small words a lane takes four,
  // so that a row of up to four is one lane's (90 bf16: eight lanes 61 us, sixteen 77).
  const int widest = bytes >= 8 && A.nv <= 16 ? 4 : 8, lanes = bytes >= 8 ? A.nv : (A.nv + 3) / 4;
  A.G = 1;
  while (A.G < lanes && A.G < widest) A.G *= 2;
  if (bytes == 16) run_dots<SCATTER, T, 16>(A);
  else if (bytes == 8) run_dots<SCATTER, T, 8>(A);
  else if (bytes == 4) run_dots<SCATTER, T, 4>(A);
  else run_dots<SCATTER, T, (int)sizeof(T)>(A);
  return cudaGetLastError();
}
template <bool SCATTER>
cudaError_t run_dtype(const RowArgs& A, int dtype, int width) {
  if (dtype == NERF_DTYPE_FP32) return run_t<SCATTER, float>(A, width);
  if (dtype == NERF_DTYPE_BF16) return run_t<SCATTER, __nv_bfloat16>(A, width);
  return run_t<SCATTER, __half>(A, width);
}

}  // namespace

cudaError_t launch_rows_scatter(const void* x, const void* other, int dtype, int64_t n, int width,
                                const int32_t* pos, int k, const float* w, void* rows, float* dw,
                                cudaStream_t st) {
  return run_dtype<true>(RowArgs{x, dw ? other : nullptr, n, 0, 0, pos, k, w, rows, dw, st}, dtype, width);
}

cudaError_t launch_rows_gather(const void* rows, const void* x, int dtype, int64_t n, int width,
                               const int32_t* pos, int k, const float* w, void* out, float* dw,
                               cudaStream_t st) {
  return run_dtype<false>(RowArgs{rows, dw ? x : nullptr, n, 0, 0, pos, k, w, out, dw, st}, dtype, width);
}

}  // namespace nerfb
