// Stable counting sort of (point, expert) pairs by expert.
//
// Few pairs (ES_SMALL): one CTA; a pair's sorted row is the number of kept pairs
// before it in (expert, pair) order, counted directly (the ids sit in shared
// memory), and the offsets come from a binary search. One launch.
//
// Up to ES_ALONE: the place kernel below alone, in one CTA whose counts are the
// totals too. One launch.
//
// More: three launches over one contiguous chunk of pairs per CTA.
//   count:   the chunk's pairs of every expert (shared-memory atomics) -> table
//   columns: for every expert the prefix over the chunks, and its total
//   place:   a tile of the chunk at a time, every warp counts its own run of the
//            tile (16-bit counters, two experts a word), the counts are scanned
//            over the warps (and, before the first tile's, the totals over the
//            experts), and every warp walks its run in order, 32 pairs at a time.
//            Where experts are spread, every lane adds one to its expert's
//            counter and reads it again: it met no one if it finds its own sum,
//            and lanes that met are put in lane order. Where many meet, a match
//            instruction finds who shares an expert (a ballot per bit of the id
//            took longer) and one lane adds for all. Rows come out in pair order
//            whatever the timing.
// The launches overlap: place counts its first tile while columns still runs.
//
// 6.3 M pairs over 4,096 experts, eight neighbouring cells a point: 52 us on the device
// (55 call by call), 1.4 TB/s of the 75 MB that the sort has to read and write (0.22 of
// the copy rate); uniform ids: 37 us. Count takes 10 us, columns 5; place is bound by
// its chains through shared memory (counter, add, counter) at 16 warps an SM. The
// counters of 24 would fit (213 KB at 4,096 experts); that has not been tried.
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

// its work grows with the square of the pairs: 128 pairs of 64 experts take 2.6 us
// against 3.6 in the place kernel, 256 pairs 4.2 against 3.7
constexpr int ES_SMALL = 128, ES_SMALL_T = 1024;
constexpr int ES_WARPS = 16, ES_T = ES_WARPS * 32;
constexpr int ES_RUN = 4064;                 // pairs of a warp's run in one tile
constexpr int ES_TILE = ES_WARPS * ES_RUN;
static_assert(ES_TILE < 65536 && ES_RUN % 32 == 0, "a tile's counts are 16-bit");
// Pairs that one CTA sorts alone: 4,096 take 9.0 us against the three launches' 10.9
// with 4,096 experts and 8.5 against 7.7 with 64, where two launches less weigh more
// for the caller; 8,192 pairs of 64 experts 13.4 against 7.8.
constexpr int ES_ALONE = 4096;
static_assert(ES_ALONE <= ES_TILE, "in one tile");
// Pairs of a CTA at least, one per thread: 16,384 pairs of 64 experts take 7.0 us,
// with 1,024 to a CTA 7.9 and with 2,048 9.2.
constexpr int ES_CHUNK = ES_T;
constexpr int ES_MOST_CTAS = 148 * 2, ES_PER = (ES_MOST_CTAS + 15) / 16;
constexpr int ES_WORDS = (EXPERT_MAX / 2 + ES_T - 1) / ES_T;   // counter words of a thread in the scan

// Lanes that meet in a counter are put in order by a ballot per expert up to ES_FEW
// of them, by a match above (6.3 M uniform pairs of 256 experts: 38 us, 56 by the
// match alone); a warp goes over to matches where more than ES_MEET of its last 128
// pairs met (one expert for all: 51 us, 61 to 66 by adds; uniform over 4,096: 38 us
// by adds, 69 by matches; eight neighbouring cells a point: 52 either way). Both give
// the same ranks.
constexpr int ES_FEW = 4, ES_MEET = 16;
struct SortPlan {
  int ctas;
  int64_t chunk;                             // pairs of a CTA, a multiple of ES_T
};
// Small tables leave room for two CTAs to an SM. 6.3 M pairs of a gate, two and one: 64
// experts 65 and 65 us (uniform ids 51 and 53), 256: 63 and 83, 1,000: 66 and 84, 1,024:
// 66 and 84; only 100,000 points with two of 64 experts are quicker with one, 11.0 and
// 9.4. (The tables of up to 3,100 experts would fit twice as well: 2,048 experts take
// 88 us here, 68 with two.)
SortPlan sort_plan(int64_t pairs, int n_experts) {
  const int64_t most = n_experts <= 1024 ? ES_MOST_CTAS : 148, want = (pairs + ES_CHUNK - 1) / ES_CHUNK;
  const int64_t ctas = want < most ? want : most;
  const int64_t chunk = ((pairs + ctas - 1) / ctas + ES_T - 1) / ES_T * ES_T;
  return {(int)((pairs + chunk - 1) / chunk), chunk};
}

__global__ void __launch_bounds__(ES_SMALL_T)
sort_small_kernel(const int32_t* __restrict__ ids, int pairs, int n_experts, int32_t* __restrict__ offset,
                  int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  __shared__ __align__(16) int32_t id_s[ES_SMALL];
  __shared__ int32_t sorted[ES_SMALL];
  const int t = threadIdx.x, padded = (pairs + 3) & ~3;
  int id = INT32_MAX;                        // dropped pairs sort behind the kept ones
  if (t < pairs) {
    const int v = ids[t];
    if ((unsigned)v < (unsigned)n_experts) id = v;
  }
  if (t < padded) id_s[t] = id;
  const int kept = __syncthreads_count(id != INT32_MAX);
  if (t < pairs) {
    int row = 0;
    for (int q = 0; q < padded; q += 4) {
      const int4 v = *reinterpret_cast<const int4*>(id_s + q);
      row += (v.x < id || (v.x == id && q < t)) + (v.y < id || (v.y == id && q + 1 < t)) +
             (v.z < id || (v.z == id && q + 2 < t)) + (v.w < id || (v.w == id && q + 3 < t));
    }
    if (id != INT32_MAX) {
      sorted[row] = id;
      if (order) order[row] = t;
    }
    pos[t] = id != INT32_MAX ? row : -1;
  }
  __syncthreads();
  for (int e = t; e <= n_experts; e += ES_SMALL_T) {
    int lo = 0, hi = kept;                   // the first sorted pair of an expert >= e
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < e) lo = mid + 1; else hi = mid;
    }
    offset[e] = lo;
  }
}

// Calls f(id) for the ids [begin, end) by `n` threads, 16 loads in flight a
// thread. Neighbouring lanes take neighbouring pairs: pairs further apart are
// more often of one expert, whose counts a warp's atomics would add one by one.
template <typename F>
__device__ __forceinline__ void for_ids(const int32_t* __restrict__ ids, int64_t begin, int64_t end, int t, int n, F f) {
  for (int64_t i = begin + t; i < end; i += 16 * n) {
    int id[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) id[u] = i + u * n < end ? __ldg(ids + i + u * n) : -1;
#pragma unroll
    for (int u = 0; u < 16; ++u) f(id[u]);
  }
}

constexpr int ES_CT = 1024;
__global__ void __launch_bounds__(ES_CT)
sort_count_kernel(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk, int n_experts,
                  int32_t* __restrict__ table) {
  extern __shared__ int32_t hist[];
  cudaTriggerProgrammaticLaunchCompletion();
  for (int e = threadIdx.x; e < n_experts; e += ES_CT) hist[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk, end = min(pairs, begin + chunk);
  for_ids(ids, begin, end, threadIdx.x, ES_CT, [&](int id) {
    if ((unsigned)id < (unsigned)n_experts) atomicAdd(&hist[id], 1);
  });
  __syncthreads();
  for (int e = threadIdx.x; e < n_experts; e += ES_CT) table[(int64_t)blockIdx.x * n_experts + e] = hist[e];
}

// lane = expert, warp = a run of chunks: table becomes the exclusive prefix over
// the chunks, totals the experts' sums
constexpr int ES_COL_WARPS = 16;
__global__ void __launch_bounds__(ES_COL_WARPS * 32, 2)
sort_columns_kernel(int32_t* table, int chunks, int n_experts, int32_t* totals) {
  __shared__ int32_t part[ES_COL_WARPS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int per = (chunks + ES_COL_WARPS - 1) / ES_COL_WARPS, c0 = min(chunks, warp * per), n = min(chunks, c0 + per) - c0;
  int32_t* col = table + (int64_t)c0 * n_experts + e;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();           // the counts
  int32_t v[ES_PER], sum = 0;
#pragma unroll
  for (int c = 0; c < ES_PER; ++c) {
    v[c] = c < n && e < n_experts ? __ldcg(col + (int64_t)c * n_experts) : 0;
    sum += v[c];
  }
  part[warp][lane] = sum;
  __syncthreads();
  int32_t run = 0;
#pragma unroll
  for (int w = 0; w < ES_COL_WARPS - 1; ++w) run += w < warp ? part[w][lane] : 0;
  if (e < n_experts) {
    if (warp == ES_COL_WARPS - 1) totals[e] = run + sum;
#pragma unroll
    for (int c = 0; c < ES_PER; ++c) {
      if (c < n) col[(int64_t)c * n_experts] = run;
      run += v[c];
    }
  }
}

// 64 registers, so that its CTAs fit beside those of the launches before it.
// ALONE: one CTA has all pairs in one tile, and its own counts are the totals.
template <bool ALONE>
__global__ void __launch_bounds__(ES_T, 2)
sort_place_kernel(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk, int n_experts,
                  const int32_t* table, const int32_t* totals,
                  int32_t* __restrict__ offset, int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  // base[e]: the next sorted row of expert e for this CTA; words of two 16-bit
  // counters, [warp][words]: word w counts experts w (low half) and words + w (two
  // neighbours in a word would meet in it: a point's experts are often neighbours)
  extern __shared__ int32_t sm[];
  __shared__ int32_t sums[ES_WARPS];
  int32_t* base = sm;
  const int words = (n_experts + 1) / 2;
  uint32_t* counts = reinterpret_cast<uint32_t*>(sm + n_experts);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint32_t* mine = counts + warp * words;
  bool adds = true;
  const int64_t begin = blockIdx.x * chunk, end = min(pairs, begin + chunk);
  for (int64_t tile = begin; tile < end; tile += ES_TILE) {
    const int64_t left = min((int64_t)ES_TILE, end - tile);
    const int run = (int)((left + ES_WARPS * 32 - 1) / (ES_WARPS * 32)) * 32;   // pairs of a warp
    const int64_t r0 = tile + (int64_t)warp * run, r1 = min(tile + left, r0 + run);
    for (int q = lane; q < words; q += 32) mine[q] = 0;
    __syncwarp();
    for_ids(ids, r0, max(r0, r1), lane, 32, [&](int id) {
      if ((unsigned)id < (unsigned)n_experts)
        atomicAdd(&mine[id < words ? id : id - words], id < words ? 1u : 1u << 16);
    });
    // base and offset from the totals v of the thread's eight experts, 8 t .. 8 t + 7, and
    // before: their pairs in the chunks before this one
    const auto scan = [&](const int32_t* v, const int32_t* before) {
      int32_t tot = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) tot += v[j];
      int32_t first = tot;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, first, o);
        if (lane >= o) first += u;
      }
      if (lane == 31) sums[warp] = first;
      __syncthreads();
      first -= tot;
      for (int w = 0; w < warp; ++w) first += sums[w];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (8 * t + j < n_experts) {
          base[8 * t + j] = first + before[j];
          if (blockIdx.x == 0) offset[8 * t + j] = first;
        }
        first += v[j];
      }
      if (blockIdx.x == 0 && t == ES_T - 1) offset[n_experts] = first;
    };
    if (!ALONE && tile == begin) {
      cudaGridDependencySynchronize();       // the table and totals; the first tile's counts needed neither
      // both are written while this kernel may already run: loads from L2, never the non-coherent ones
      int32_t v[8], before[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = 8 * t + j < n_experts;
        v[j] = in ? __ldcg(totals + 8 * t + j) : 0;
        before[j] = in ? __ldcg(table + (int64_t)blockIdx.x * n_experts + 8 * t + j) : 0;
      }
      scan(v, before);
    }
    __syncthreads();
    // counts -> exclusive prefix over the warps, two experts a word
    uint32_t all[ES_WORDS];
#pragma unroll
    for (int u = 0; u < ES_WORDS; ++u) {
      const int q = t + u * ES_T;
      all[u] = 0;
      if (q < words)
#pragma unroll
        for (int w = 0; w < ES_WARPS; ++w) {
          const uint32_t v = counts[w * words + q];
          counts[w * words + q] = all[u];
          all[u] += v;
        }
      if (ALONE && q < words) {              // the totals, on their way to the threads that scan them
        base[q] = all[u] & 0xffffu;
        if (words + q < n_experts) base[words + q] = all[u] >> 16;
      }
    }
    __syncthreads();
    if (ALONE) {
      int32_t v[8];
      const int32_t before[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 8 * t + j < n_experts ? base[8 * t + j] : 0;
      scan(v, before);                       // a thread overwrites the entries that it read
      __syncthreads();
    }
    const uint32_t lower = (1u << lane) - 1u;
    int ahead[2][4];                         // the ids of the next 256 pairs, on their way
#pragma unroll
    for (int q = 0; q < 8; ++q)
      ahead[q >> 2][q & 3] = r0 + 32 * q + lane < r1 ? __ldg(ids + r0 + 32 * q + lane) : -1;
    for (int64_t i0 = r0; i0 < r1; i0 += 128) {
      const int left = (int)min((int64_t)128, r1 - i0) - lane;   // this lane's pairs: 32 q < left
      int id[4], p[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        id[q] = (unsigned)ahead[0][q] < (unsigned)n_experts ? ahead[0][q] : -1;
        ahead[0][q] = ahead[1][q];
        ahead[1][q] = i0 + 256 + 32 * q + lane < r1 ? __ldg(ids + i0 + 256 + 32 * q + lane) : -1;
      }
      int met = 0;                           // of the 128 pairs those with a later one of their expert in their 32
      if (adds) {
        int now[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {        // p: the counter before this lane's add; now: after all lanes'
          const int at = id[q] < words ? id[q] : id[q] - words, shift = id[q] < words ? 0 : 16;
          p[q] = 0, now[q] = 1;
          if (id[q] >= 0) p[q] = (int)((atomicAdd(&mine[at], 1u << shift) >> shift) & 0xffffu);
          __syncwarp();
          if (id[q] >= 0) now[q] = (int)((reinterpret_cast<volatile uint32_t*>(mine)[at] >> shift) & 0xffffu);
          __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {        // lanes that met in a counter: in lane order, not in that of their adds
          uint32_t meet = __ballot_sync(0xffffffffu, now[q] != p[q] + 1);
          met += __popc(meet);
          if (__popc(meet) > ES_FEW) {
            const uint32_t peers = __match_any_sync(0xffffffffu, id[q]);
            if (id[q] >= 0) p[q] = now[q] - __popc(peers) + __popc(peers & lower);
          } else {
            while (meet) {
              const int one = __shfl_sync(0xffffffffu, id[q], __ffs(meet) - 1);
              const uint32_t peers = __ballot_sync(0xffffffffu, id[q] == one);
              if (id[q] == one) p[q] = now[q] - __popc(peers) + __popc(peers & lower);
              meet &= ~peers;
            }
          }
        }
      } else {
        uint32_t peers[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) peers[q] = __match_any_sync(0xffffffffu, id[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = id[q] < words ? id[q] : id[q] - words, shift = id[q] < words ? 0 : 16;
          p[q] = 0;
          if (id[q] >= 0) p[q] = (int)((mine[at] >> shift) & 0xffffu) + __popc(peers[q] & lower);
          met += __popc(__ballot_sync(0xffffffffu, id[q] >= 0 && (peers[q] & lower) != 0));
          __syncwarp();                      // every lane has read its counter before one lane adds to it
          // one lane a peer group; the word's other expert may have one too, so the add is atomic
          if (id[q] >= 0 && (peers[q] & lower) == 0) atomicAdd(&mine[at], (uint32_t)__popc(peers[q]) << shift);
          __syncwarp();
        }
      }
      adds = met <= ES_MEET;
      int32_t* dst = pos + i0 + lane;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int32_t row = id[q] >= 0 ? base[id[q]] + p[q] : -1;
        if (id[q] >= 0 && order) order[row] = (int32_t)i0 + lane + 32 * q;
        if (32 * q < left) dst[32 * q] = row;
      }
    }
    if (ALONE) return;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < ES_WORDS; ++u) {
      const int q = t + u * ES_T;
      if (q < words) {
        base[q] += all[u] & 0xffffu;
        if (words + q < n_experts) base[words + q] += all[u] >> 16;
      }
    }
    __syncthreads();
  }
}

int64_t table_ints(const SortPlan& p, int n_experts) { return (int64_t)p.ctas * n_experts + n_experts; }

}  // namespace

int64_t expert_sort_workspace(int64_t pairs, int n_experts) {
  if (pairs <= ES_ALONE) return 16;
  return (table_ints(sort_plan(pairs, n_experts), n_experts) * 4 + 15) / 16 * 16;
}

cudaError_t launch_expert_sort(const int32_t* ids, int64_t pairs, int n_experts, int32_t* offset,
                               int32_t* order, int32_t* pos, void* work, cudaStream_t st) {
  if (pairs <= ES_SMALL) {
    sort_small_kernel<<<1, ES_SMALL_T, 0, st>>>(ids, (int)pairs, n_experts, offset, order, pos);
    return cudaGetLastError();
  }
  constexpr int most_sm = EXPERT_MAX * 4 + ES_WARPS * EXPERT_MAX * 2;
  const size_t place_sm = (size_t)n_experts * 4 + (size_t)ES_WARPS * ((n_experts + 1) / 2) * 4;
  cudaError_t e;
  if (pairs <= ES_ALONE) {
    e = cudaFuncSetAttribute(sort_place_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_sm);
    if (e != cudaSuccess) return e;
    sort_place_kernel<true><<<1, ES_T, place_sm, st>>>(ids, pairs, pairs, n_experts, nullptr, nullptr, offset, order, pos);
    return cudaGetLastError();
  }
  e = cudaFuncSetAttribute(sort_place_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most_sm);
  if (e != cudaSuccess) return e;
  const SortPlan plan = sort_plan(pairs, n_experts);
  int32_t* table = (int32_t*)work;
  int32_t* totals = table + (int64_t)plan.ctas * n_experts;
  sort_count_kernel<<<plan.ctas, ES_CT, n_experts * 4, st>>>(ids, pairs, plan.chunk, n_experts, table);
  // each of the other two may start while the one before it runs, and waits for
  // its results itself
  e = launch_early(sort_columns_kernel, (n_experts + 31) / 32, ES_COL_WARPS * 32, 0, st, table, plan.ctas, n_experts,
                   totals);
  if (e != cudaSuccess) return e;
  e = launch_early(sort_place_kernel<false>, plan.ctas, ES_T, place_sm, st, ids, pairs, plan.chunk, n_experts,
                   (const int32_t*)table, (const int32_t*)totals, offset, order, pos);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace nerfb
