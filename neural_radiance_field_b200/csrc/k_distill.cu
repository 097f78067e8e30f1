// Distillation of student logits against a teacher's kept top logits, loss and
// gradient in one launch. With c = log2(e) / T, m the row's largest logit and
// Z = sum_i 2^(c (s_i - m)):  q_i = 2^(c (s_i - m)) / Z  and
// log q_i = (s_i - m) / T - log Z. (The difference is taken first: a row of
// masks of the type's lowest value must not overflow.)
//
// Bound by memory: the logits are read once and the gradient is written once.
// The row stays in registers between its statistics and its gradient, held by a
// team: a warp (rows up to 16 KB, where there are rows enough to fill the GPU:
// no barrier anywhere), a CTA of 256 threads (up to 64 KB), or a cluster of two
// to eight such CTAs (up to 512 KB), which join their statistics through
// distributed shared memory. A CTA goes from row to row, and as soon as a vector
// of the gradient is written its register takes the next row's vector, so that
// row's loads run under this row's stores and barriers. Longer rows are streamed twice, the second time
// from L2, by clusters of eight. Warp 0 of a CTA works out the teacher's
// probabilities while the row's loads are in flight. A row's 16-byte vectors
// start wherever its address allows; up to 14 elements before and after them go
// one by one.
#include <cooperative_groups.h>

#include <atomic>

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

// (maximum, sum of 2^(c (v - maximum))) of the lanes' sets of logits together; the
// sum of an empty set or of -inf alone is 0, and no -inf is taken from -inf
__device__ __forceinline__ float2 warp_join(float2 v, float c) {
  const float m = warp_fold(v.x, [](float a, float b) { return max_nan(a, b); });
  const float z = m == -INFINITY ? 0.0f : v.y * exp2_fast((v.x - m) * c);
  return make_float2(m, warp_fold(z, [](float a, float b) { return a + b; }));
}
// The whole CTA's (maximum, sum); `red` holds two sets used in turn, so that one
// barrier a call is enough.
template <int NT>
__device__ __forceinline__ float2 cta_join(float2 v, float c, float2* red) {
  v = warp_join(v, c);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  constexpr int W = NT / 32;
  return warp_join((threadIdx.x & 31) < W ? red[threadIdx.x & 31] : make_float2(-INFINITY, 0.0f), c);
}

__device__ __forceinline__ float warp_sum(float v) { return warp_fold(v, [](float a, float b) { return a + b; }); }
__device__ __forceinline__ float warp_max(float v) { return warp_fold(v, [](float a, float b) { return max_nan(a, b); }); }

// What one warp knows of a row's teacher: of lane l, entry l's id (-1: not
// kept), logit, student logit and, once solved, probability; sum_j p_j log p_j,
// the same in every lane; whether an entry is kept. Entries past 32 are read
// from the arrays again where they are needed.
struct Teacher {
  int32_t id = -1;
  float y = -INFINITY, s = 0.0f, p = 0.0f, plogp = 0.0f;
  bool some = false;
};
// The loads alone, to be issued well before the rest.
template <typename T>
__device__ __forceinline__ Teacher teacher_load(const DistillArgs& A, int64_t i) {
  const int lane = threadIdx.x & 31;
  Teacher R;
  if (i < A.n && lane < A.k) {
    const int32_t id = __ldg(A.ti + i * A.k + lane);
    const float y = __ldg(A.tl + i * A.k + lane);
    if ((unsigned)id < (unsigned)A.classes && y != -INFINITY) {
      R.id = id;
      R.y = y;
      R.s = elem_to_f<T>(((const T*)A.student)[i * A.classes + id]);
    }
  }
  return R;
}
// The probabilities, also to probs[k], and the ids to ids[k] (-1: not kept).
__device__ __forceinline__ void teacher_solve(const DistillArgs& A, int64_t i, Teacher& R, float* probs, int32_t* ids) {
  const int lane = threadIdx.x & 31;
  const float inv_t = 1.0f / A.temperature;
  const float* tl = A.tl + i * A.k;
  const int32_t* ti = A.ti + i * A.k;
  auto kept = [&](int j) { return (unsigned)__ldg(ti + j) < (unsigned)A.classes && __ldg(tl + j) != -INFINITY; };
  float top = R.y;
  for (int j = lane + 32; j < A.k; j += 32)
    if (kept(j)) top = max_nan(top, __ldg(tl + j));
  top = warp_max(top);
  R.some = top != -INFINITY;
  const float z = (R.y - top) * inv_t;
  float norm = R.id >= 0 ? expf(z) : 0.0f;
  R.p = norm;
  for (int j = lane + 32; j < A.k; j += 32)
    if (kept(j)) norm += expf((__ldg(tl + j) - top) * inv_t);
  norm = warp_sum(norm);
  const float log_norm = logf(norm);
  R.p = R.id >= 0 ? R.p / norm : 0.0f;
  float l = R.p != 0.0f ? R.p * (z - log_norm) : 0.0f;
  if (lane < A.k) {
    probs[lane] = R.p;
    ids[lane] = R.id;
  }
  for (int j = lane + 32; j < A.k; j += 32) {
    const bool in = kept(j);
    const float w = (__ldg(tl + j) - top) * inv_t, p = in ? expf(w) / norm : 0.0f;
    probs[j] = p;
    ids[j] = in ? __ldg(ti + j) : -1;
    if (p != 0.0f) l += p * (w - log_norm);
  }
  R.plogp = warp_sum(l);
}

// The row's loss, by the warp that has its teacher.
template <typename T>
__device__ __forceinline__ void write_loss(const DistillArgs& A, int64_t i, const T* s, float m, float z,
                                           const float* probs, const int32_t* ids, const Teacher& R) {
  const int lane = threadIdx.x & 31;
  const float inv_t = 1.0f / A.temperature, log_z = logf(z);
  float l = R.p != 0.0f ? R.p * ((R.s - m) * inv_t - log_z) : 0.0f;
  for (int j = lane + 32; j < A.k; j += 32)
    if (probs[j] != 0.0f) l += probs[j] * ((elem_to_f<T>(s[ids[j]]) - m) * inv_t - log_z);
  l = warp_sum(l);
  if (lane == 0) A.loss[i] = R.some ? A.temperature * A.temperature * (R.plogp - l) : 0.0f;
}

// The gradient of the kept classes in [lo, hi), which the row's pass wrote as q
// alone: less the teacher's probability, summed where an id comes twice (its
// first entry writes). Thread `r` of `team`. aiz: row scale * T / Z.
template <typename T>
__device__ __forceinline__ void kept_gradients(int k, int r, int team, const T* s, T* g, float m, float c, float a,
                                               float aiz, const float* probs, const int32_t* ids, int lo, int hi) {
  for (int j = r; j < k; j += team) {
    const int32_t id = ids[j];
    if (id < lo || id >= hi) continue;
    const float v = elem_to_f<T>(s[id]);
    float p = 0.0f;
    bool first = true;
    for (int q = 0; q < k; ++q)
      if (ids[q] == id) {
        first = first && q >= j;
        p += probs[q];
      }
    if (first) g[id] = elem_from_f<T>(fmaf(exp2_fast((v - m) * c), aiz, -a * p));
  }
}
// The same by one warp that has the teacher's entries in registers (k <= 32):
// equal ids find each other by a match.
template <typename T>
__device__ __forceinline__ void kept_gradients_warp(const Teacher& R, T* g, float m, float c, float a, float aiz,
                                                    const float* probs) {
  const int lane = threadIdx.x & 31;
  const unsigned peers = __match_any_sync(0xffffffffu, R.id);
  if (R.id < 0 || lane != __ffs(peers) - 1) return;
  float p = 0.0f;
  for (unsigned left = peers; left; left &= left - 1) p += probs[__ffs(left) - 1];
  g[R.id] = elem_from_f<T>(fmaf(exp2_fast((R.s - m) * c), aiz, -a * p));
}

// A CTA's (maximum, sum) joined over its cluster: every CTA writes its own to all,
// and one cluster barrier later each has them all at hand. `stat` is one of two
// sets used in turn: a set is written again only after the next row's barrier,
// which no CTA passes before all have read it.
__device__ __forceinline__ float2 cluster_join(float2 v, float c, float2* stat, int rank, int C) {
  cg::cluster_group cluster = cg::this_cluster();
  if ((int)threadIdx.x < C) cluster.map_shared_rank(stat, threadIdx.x)[rank] = v;
  cluster.sync();
  const int lane = threadIdx.x & 31;
  return warp_join(lane < C ? stat[lane] : make_float2(-INFINITY, 0.0f), c);
}

constexpr float kLog2e = 1.44269504f;
// -inf, once or twice in a word
template <typename T> constexpr uint32_t kNegInf = 0xff800000u;
template <> constexpr uint32_t kNegInf<__nv_bfloat16> = 0xff80ff80u;
template <> constexpr uint32_t kNegInf<__half> = 0xfc00fc00u;

// The part of a row that CTA `rank` of `C` holds: vectors [v0, v1) of the row,
// and single elements (the first CTA those before the vectors, the last those after).
struct RowPart {
  int head, v0, v1, lo, hi, single;
  bool has;
  template <typename T, int N>
  static __device__ __forceinline__ RowPart of(const T* s, int classes, int rank, int C, int r) {
    RowPart p;
    p.head = N > 1 ? min((int)((0 - (uintptr_t)s) % 16 / sizeof(T)), classes) : 0;
    const int nv = (classes - p.head) / N;
    p.v0 = C == 1 ? 0 : (int)((int64_t)nv * rank / C);
    p.v1 = C == 1 ? nv : (int)((int64_t)nv * (rank + 1) / C);
    p.lo = rank == 0 ? 0 : p.head + p.v0 * N;
    p.hi = rank == C - 1 ? classes : p.head + p.v1 * N;
    const int before = rank == 0 ? p.head : 0, after = rank == C - 1 ? classes - p.head - nv * N : 0;
    p.single = r < before ? r : p.head + nv * N + r - before;
    p.has = r < before + after;
    return p;
  }
};

// Rows in registers: NV vectors a thread and one single element. TEAM 32: a warp
// a row, eight rows to a CTA; TEAM 256: a CTA, or a cluster of them, a row.
constexpr int rows_per_sm(int team, int nv) {
  return nv <= 2 ? 4 : nv <= 8 ? 3 : team == 32 && nv == 32 ? 1 : 2;
}
template <typename T, int TEAM, int NV>
__global__ void __launch_bounds__(256, rows_per_sm(TEAM, NV))
distill_rows_kernel(DistillArgs A, int C) {
  using V = Vec<T, 16>;
  constexpr int TEAMS = 256 / TEAM;
  constexpr bool AHEAD = TEAM != 32;         // load the next row early; other warps hide a warp's loads
  __shared__ float2 red[2][8], stat[2][8];
  // a team's probabilities and ids; a CTA's two sets are used in turn
  constexpr int SETS = TEAM == 32 ? TEAMS : 2;
  __shared__ float probs_s[SETS * DISTILL_MAX_K];
  __shared__ int32_t ids_s[SETS * DISTILL_MAX_K];
  __shared__ int some_s[2];
  const int warp = threadIdx.x >> 5, r = TEAM == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int rank = C == 1 ? 0 : (int)cg::this_cluster().block_rank();
  const float c = kLog2e / A.temperature;
  const int64_t step = (int64_t)gridDim.x / C * TEAMS;
  int64_t i = (int64_t)blockIdx.x / C * TEAMS + (TEAM == 32 ? warp : 0);
  V v[NV];
  RowPart P;
  const uint4* sv;
  int nv;                                    // this thread's vectors: q * TEAM < nv
  float one;
  // row i's part and its vectors' place; the loads are issued by the caller
  auto enter = [&](int64_t row) {
    const bool in = row < A.n;
    const T* s = (const T*)A.student + (in ? row : 0) * A.classes;
    P = RowPart::of<T, V::N>(s, A.classes, rank, C, r);
    P.has = P.has && in;
    sv = reinterpret_cast<const uint4*>(s + P.head) + P.v0 + r;
    nv = in ? P.v1 - P.v0 - r : 0;
    one = P.has ? elem_to_f<T>(s[P.single]) : -INFINITY;
  };
  // a vector past the part holds -inf: it adds nothing to the statistics, which
  // are then free of conditions
  auto take = [&](int q) {
    v[q].fill(kNegInf<T>);
    if (q * TEAM < nv) v[q].load(sv, q * TEAM);
  };
  if (C > 1) cg::this_cluster().sync();      // every CTA runs before one writes to another
  Teacher R, next;
  if (AHEAD) {
    if (warp == 0) next = teacher_load<T>(A, i);
    enter(i);
#pragma unroll
    for (int q = 0; q < NV; ++q) take(q);
  }
  for (int turn = 0; i < A.n; i += step, turn ^= 1) {
    const T* s = (const T*)A.student + i * A.classes;
    T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
    if (!AHEAD) {
      enter(i);
#pragma unroll
      for (int q = 0; q < NV; ++q) take(q);
    }
    const int set = (TEAM == 32 ? warp : turn) * DISTILL_MAX_K;
    float* probs = probs_s + set;
    int32_t* ids = ids_s + set;
    if (TEAM == 32 || warp == 0) {
      R = AHEAD ? next : teacher_load<T>(A, i);
      teacher_solve(A, i, R, probs, ids);
      if (TEAM != 32 && r == 0) some_s[turn] = R.some;
    }
    // four maxima and four sums side by side: one chain would wait for itself
    float mp[4] = {one, one, one, one};
    // The passes go over groups of four vectors, each behind a condition that the
    // whole team shares: unused groups are skipped, and a row of 16-bit elements is
    // never unpacked as a whole, which would not fit the registers.
    const int used = (P.v1 - P.v0 + TEAM - 1) / TEAM;
#pragma unroll
    for (int q0 = 0; q0 < NV; q0 += 4)
      if (q0 < used)
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q)
#pragma unroll
          for (int e = 0; e < V::N; ++e) mp[e & 3] = max_nan(mp[e & 3], v[q].get(e));
    float m = max_nan(max_nan(mp[0], mp[1]), max_nan(mp[2], mp[3]));
    if (TEAM == 32) m = warp_max(m);
    const float shift = TEAM != 32 && m == -INFINITY ? 0.0f : m;
    float zp[4] = {exp2_fast((one - shift) * c), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q0 = 0; q0 < NV; q0 += 4)
      if (q0 < used)
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q)
#pragma unroll
          for (int e = 0; e < V::N; ++e) zp[e & 3] += exp2_fast((v[q].get(e) - shift) * c);
    float z = (zp[0] + zp[1]) + (zp[2] + zp[3]);
    bool some = R.some;
    if (TEAM == 32) {
      z = warp_sum(z);
      __syncwarp();
    } else {
      float2 all = cta_join<256>(make_float2(m, z), c, red[turn]);
      if (C > 1) all = cluster_join(all, c, stat[turn], rank, C);
      m = all.x;
      z = all.y;
      some = some_s[turn];
    }
    const RowPart now = P;
    const int nv_now = nv;
    const float one_now = one;
    const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f), aiz = a / z;
    uint4* gv = reinterpret_cast<uint4*>(g + now.head) + now.v0 + r;
    if (AHEAD) {
      if (warp == 0) next = teacher_load<T>(A, i + step);
      enter(i + step);
    }
#pragma unroll
    for (int q0 = 0; q0 < NV; q0 += 4) {
      if (g && some && q0 < used) {
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q) {
          float f[V::N];
#pragma unroll
          for (int e = 0; e < V::N; ++e) f[e] = exp2_fast((v[q].get(e) - m) * c) * aiz;
          V o;
          o.pack(f);
          if (q * TEAM < nv_now) o.store(gv, q * TEAM);
        }
      } else if (g && q0 < used) {
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q)
          if (q * TEAM < nv_now) gv[q * TEAM] = make_uint4(0, 0, 0, 0);
      }
      if (AHEAD) {
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q) take(q);
      }
    }
    if (g && now.has) g[now.single] = elem_from_f<T>(some ? exp2_fast((one_now - m) * c) * aiz : 0.0f);
    if ((TEAM == 32 || warp == 0) && rank == 0) write_loss<T>(A, i, s, m, z, probs, ids, R);
    if (g) {
      // the kept classes after all others; a CTA's next row uses the other sets,
      // and its barrier there holds this row's readers together
      if (TEAM == 32) __syncwarp(); else __syncthreads();
      if (some) {
        if (TEAM == 32 && A.k <= 32) kept_gradients_warp<T>(R, g, m, c, a, aiz, probs);
        else kept_gradients<T>(A.k, r, TEAM, s, g, m, c, a, aiz, probs, ids, now.lo, now.hi);
      }
    }
    if (TEAM == 32) __syncwarp();            // the next row's probabilities overwrite these
  }
  if (C > 1) cg::this_cluster().sync();      // no CTA ends while another reads its statistics
}

// Long rows, or rows whose gradient is aligned unlike them (BYTES = one
// element), streamed by clusters of CTAs, each a part of the row.
constexpr int DW_T = 512;
template <typename T, int BYTES>
__global__ void __launch_bounds__(DW_T, 2)
distill_wide_kernel(DistillArgs A, int C) {
  using V = Vec<T, BYTES>;
  __shared__ float2 red[2][DW_T / 32], stat[2][8];
  __shared__ float probs_s[2][DISTILL_MAX_K];
  __shared__ int32_t ids_s[2][DISTILL_MAX_K];
  __shared__ int some_s[2];
  const int rank = C == 1 ? 0 : (int)cg::this_cluster().block_rank(), t = threadIdx.x, warp = t >> 5;
  const float c = kLog2e / A.temperature;
  if (C > 1) cg::this_cluster().sync();      // every CTA runs before one writes to another
  int turn = 0;
  for (int64_t i = blockIdx.x / C; i < A.n; i += gridDim.x / C, turn ^= 1) {
    const T* s = (const T*)A.student + i * A.classes;
    T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
    const RowPart P = RowPart::of<T, V::N>(s, A.classes, rank, C, t);
    const T* sv = s + P.head;
    float* probs = probs_s[turn];
    int32_t* ids = ids_s[turn];
    Teacher R;
    if (warp == 0) {
      R = teacher_load<T>(A, i);
      teacher_solve(A, i, R, probs, ids);
      if (t == 0) some_s[turn] = R.some;
    }
    // running maximum and sum: the sum is rescaled once per four vectors
    float m = P.has ? elem_to_f<T>(s[P.single]) : -INFINITY, z = P.has && m != -INFINITY ? 1.0f : 0.0f;
    for (int q0 = P.v0 + t; q0 < P.v1; q0 += 4 * DW_T) {
      V v[4];
      float top = m;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < P.v1) v[u].load(sv, q0 + u * DW_T);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < P.v1)
#pragma unroll
          for (int e = 0; e < V::N; ++e) top = max_nan(top, v[u].get(e));
      const float shift = top == -INFINITY ? 0.0f : top;
      z *= m == -INFINITY ? 0.0f : exp2_fast((m - shift) * c);
      m = top;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u * DW_T < P.v1)
#pragma unroll
          for (int e = 0; e < V::N; ++e) z += exp2_fast((v[u].get(e) - shift) * c);
    }
    float2 all = cta_join<DW_T>(make_float2(m, z), c, red[turn]);
    if (C > 1) all = cluster_join(all, c, stat[turn], rank, C);
    m = all.x;
    z = all.y;
    const bool some = some_s[turn];
    if (warp == 0 && rank == 0) write_loss<T>(A, i, s, m, z, probs, ids, R);
    if (g) {
      const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f), aiz = a / z;
      T* gv = g + P.head;
      for (int q0 = P.v0 + t; q0 < P.v1; q0 += 4 * DW_T) {
        V v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q0 + u * DW_T < P.v1) v[u].load(sv, q0 + u * DW_T);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q0 + u * DW_T < P.v1) {
            float f[V::N];
#pragma unroll
            for (int e = 0; e < V::N; ++e)
              f[e] = some ? exp2_fast((v[u].get(e) - m) * c) * aiz : 0.0f;
            V o;
            o.pack(f);
            o.store(gv, q0 + u * DW_T);
          }
      }
      if (P.has) g[P.single] = elem_from_f<T>(some ? exp2_fast((elem_to_f<T>(s[P.single]) - m) * c) * aiz : 0.0f);
      __syncthreads();
      if (some) kept_gradients<T>(A.k, t, DW_T, s, g, m, c, a, aiz, probs, ids, P.lo, P.hi);
    }
  }
  if (C > 1) cg::this_cluster().sync();
}

// `teams` of C CTAs, but no more than run at the same time: the CTAs of a cluster
// share a GPC, whose SMs a size of eight does not divide, so fewer clusters fit
// than SMs x CTAs / C, and a last few started late would run alone.
template <typename K>
cudaError_t run_clusters(K kernel, const DistillArgs& A, int64_t teams, int threads, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  if (C > 1 && teams > 1) {
    static std::atomic<int> fit[4] = {};     // of this kernel, by log2 C; the same on every device (sm_100a)
    std::atomic<int>& f = fit[C == 2 ? 1 : C == 4 ? 2 : 3];
    int most = f.load(std::memory_order_relaxed);
    if (most == 0) {
      cfg.gridDim = dim3((unsigned)C);
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (most < 1) most = 1;
      f.store(most, std::memory_order_relaxed);
    }
    if (teams > most) teams = most;
  }
  cfg.gridDim = dim3((unsigned)(teams * C));
  return cudaLaunchKernelEx(&cfg, kernel, A, C);
}

template <typename T, int TEAM, int NV>
cudaError_t run_rows(const DistillArgs& A, int C, cudaStream_t st) {
  constexpr int TEAMS = 256 / TEAM;
  const int64_t want = (A.n + TEAMS - 1) / TEAMS, most = 148 * rows_per_sm(TEAM, NV) / C;
  return run_clusters(distill_rows_kernel<T, TEAM, NV>, A, want < most ? want : most, 256, C, st);
}

template <typename T, int BYTES>
cudaError_t run_wide(const DistillArgs& A, cudaStream_t st) {
  // CTAs of a row: eight, which with 296 CTAs at a time keeps 37 rows in flight
  // and their second reading in L2; fewer where a part would be below 32 KB
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  int C = 8;
  while (C > 1 && bytes / C < 32768) C /= 2;
  const int64_t most = 296 / C;
  return run_clusters(distill_wide_kernel<T, BYTES>, A, A.n < most ? A.n : most, DW_T, C, st);
}

template <typename T>
cudaError_t run_t(const DistillArgs& A, cudaStream_t st) {
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  // the vectors of student and gradient rows coincide when both start alike
  if (A.grad && ((uintptr_t)A.grad - (uintptr_t)A.student) % 16) return run_wide<T, (int)sizeof(T)>(A, st);
  if (bytes <= 512) return run_rows<T, 32, 1>(A, 1, st);
  if (bytes <= 1024) return run_rows<T, 32, 2>(A, 1, st);
  if (bytes <= 4096) return run_rows<T, 32, 8>(A, 1, st);
  // a warp a row needs some 1200 rows to fill the SMs
  if (A.n >= 1184 && bytes <= 8192) return run_rows<T, 32, 16>(A, 1, st);
  if (A.n >= 1184 && bytes <= 16384) return run_rows<T, 32, 32>(A, 1, st);
  if (bytes <= 16384) return run_rows<T, 256, 4>(A, 1, st);
  int C = 1;                                 // CTAs of a row: parts of 64 KB at most
  while (bytes > 65536 * (int64_t)C) C *= 2;
  if (C > 8) return run_wide<T, 16>(A, st);
  const int64_t part = (bytes + C - 1) / C + 16;
  if (part <= 32768) return run_rows<T, 256, 8>(A, C, st);
  return run_rows<T, 256, 16>(A, C, st);
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
