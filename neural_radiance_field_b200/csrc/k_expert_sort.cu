// Stable counting sort of (point, expert) pairs by expert.
//
// The pairs are cut into one contiguous chunk per warp. A counting pass fills
// count[chunk][expert]; a column scan turns it into every chunk's first row inside
// each expert, an expert scan into the experts' offsets; then every warp walks its
// chunk again in order, 32 pairs at a time. Equal ids among the 32 find each
// other with a match, a pair's rank among them is the number of lower lanes,
// and the chunk's running row of the expert advances by their number, so the
// rows of an expert come in pair order whatever the timing.
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

constexpr int ES_WARPS = 8;

int64_t sort_chunks(int64_t pairs) {
  const int64_t most = 148 * ES_WARPS, want = (pairs + 255) / 256;
  return want < most ? want : most;
}

__global__ void __launch_bounds__(ES_WARPS * 32)
es_count_kernel(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk, int64_t chunks, int n_experts,
                int32_t* __restrict__ count) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * ES_WARPS + threadIdx.x / 32;
  if (w >= chunks) return;
  int32_t* row = count + w * n_experts;
  for (int e = lane; e < n_experts; e += 32) row[e] = 0;
  __syncwarp();
  const int64_t end = min(pairs, (w + 1) * chunk);
  for (int64_t i0 = w * chunk; i0 < end; i0 += 32) {
    int id = i0 + lane < end ? ids[i0 + lane] : -1;
    if ((unsigned)id >= (unsigned)n_experts) id = -1;
    const unsigned peers = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && lane == __ffs(peers) - 1) row[id] += __popc(peers);
    __syncwarp();
  }
}

__global__ void es_columns_kernel(int32_t* __restrict__ count, int64_t chunks, int n_experts,
                                  int32_t* __restrict__ offset) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= n_experts) return;
  int32_t run = 0;
  for (int64_t w = 0; w < chunks; ++w) {
    const int32_t c = count[w * n_experts + e];
    count[w * n_experts + e] = run;
    run += c;
  }
  offset[e] = run;
}

__global__ void __launch_bounds__(1024) es_offsets_kernel(int32_t* __restrict__ offset, int n_experts) {
  __shared__ int32_t sums[1024];
  const int t = threadIdx.x;
  int32_t v[4], tot = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = 4 * t + j < n_experts ? offset[4 * t + j] : 0;
    tot += v[j];
  }
  sums[t] = tot;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int32_t u = t >= o ? sums[t - o] : 0;
    __syncthreads();
    sums[t] += u;
    __syncthreads();
  }
  int32_t run = sums[t] - tot;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (4 * t + j < n_experts) offset[4 * t + j] = run;
    run += v[j];
  }
  if (t == 1023) offset[n_experts] = sums[1023];
}

__global__ void __launch_bounds__(ES_WARPS * 32)
es_place_kernel(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk, int64_t chunks, int n_experts,
                const int32_t* __restrict__ offset, int32_t* __restrict__ count,
                int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * ES_WARPS + threadIdx.x / 32;
  if (w >= chunks) return;
  int32_t* row = count + w * n_experts;
  const int64_t end = min(pairs, (w + 1) * chunk);
  for (int64_t i0 = w * chunk; i0 < end; i0 += 32) {
    const int64_t i = i0 + lane;
    int id = i < end ? ids[i] : -1;
    if ((unsigned)id >= (unsigned)n_experts) id = -1;
    const unsigned peers = __match_any_sync(0xffffffffu, id);
    const int leader = __ffs(peers) - 1;
    int base = 0;
    if (id >= 0 && lane == leader) {
      base = row[id];
      row[id] = base + __popc(peers);
    }
    base = __shfl_sync(0xffffffffu, base, leader);
    __syncwarp();
    if (i < end) {
      int32_t p = -1;
      if (id >= 0) {
        p = offset[id] + base + __popc(peers & ((1u << lane) - 1u));
        if (order) order[p] = (int32_t)i;
      }
      pos[i] = p;
    }
  }
}

}  // namespace

int64_t expert_sort_workspace(int64_t pairs, int n_experts) {
  return (sort_chunks(pairs) * n_experts * 4 + 15) / 16 * 16;
}

cudaError_t launch_expert_sort(const int32_t* ids, int64_t pairs, int n_experts, int32_t* offset,
                               int32_t* order, int32_t* pos, void* work, cudaStream_t st) {
  const int64_t chunks = sort_chunks(pairs), chunk = (pairs + chunks - 1) / chunks;
  int32_t* count = (int32_t*)work;
  const unsigned grid = (unsigned)((chunks + ES_WARPS - 1) / ES_WARPS);
  es_count_kernel<<<grid, ES_WARPS * 32, 0, st>>>(ids, pairs, chunk, chunks, n_experts, count);
  es_columns_kernel<<<(n_experts + 63) / 64, 64, 0, st>>>(count, chunks, n_experts, offset);
  es_offsets_kernel<<<1, 1024, 0, st>>>(offset, n_experts);
  es_place_kernel<<<grid, ES_WARPS * 32, 0, st>>>(ids, pairs, chunk, chunks, n_experts, offset, count, order, pos);
  return cudaGetLastError();
}

}  // namespace nerfb
