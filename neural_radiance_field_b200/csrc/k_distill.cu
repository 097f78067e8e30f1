// Distillation of student logits against a teacher's kept top logits, loss and
// gradient in one launch. With c = log2(e) / T, m the row's largest logit and
// Z = sum_i 2^(c (s_i - m)):  q_i = 2^(c (s_i - m)) / Z  and
// log q_i = (s_i - m) / T - log Z. (The difference is taken first: a row of
// masks of the type's lowest value must not overflow.)
//
// Bound by memory: the logits are read once and the gradient is written once.
// Between its statistics and its gradient a row stays
//   in the registers of a warp: rows up to 16 KB, where there are enough of them
//     to fill the GPU; no barrier anywhere;
//   in the shared memory of a CTA (parts up to 50 KB), or of a cluster of two to
//     eight CTAs that join their statistics through distributed shared memory.
//     Two stages: the next row's part is on its way from the start of this one.
//     (In registers, with the next row's loads issued as the gradient frees them,
//     777 rows of 400 KB took 191 us.)
// Longer rows are streamed twice, the second time from L2, by clusters of eight.
// Warp 0 of a CTA works out the teacher's probabilities beside the statistics. A
// row's 16-byte vectors start wherever its address allows; up to 14 elements
// before and after them go one by one.
//
// 65,536 rows of 4,096 bf16 with gradient: 203 us on the device (212 to 216 call by
// call), 5.3 TB/s (0.83 of the measured copy rate; two exponentials an element keep the
// XU pipe 62 % busy). 777 rows of 100,003 fp32: 149 us (152 call by call), 4.2 TB/s
// (0.65): 33 clusters of eight fit the GPCs, 264 of 296 CTAs, and each row ends in a
// cluster barrier.
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

__device__ __forceinline__ void copy_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

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
// barrier a call is enough. It is barrier BAR of the CTA by its number: a kernel whose
// warps call from two places meets there all the same, which __syncthreads, a call of
// all threads from one place, does not promise.
template <int NT, int BAR>
__device__ __forceinline__ float2 cta_join(float2 v, float c, float2* red) {
  v = warp_join(v, c);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  asm volatile("barrier.sync %0, %1;" ::"n"(BAR), "n"(NT) : "memory");
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

// The row's loss, by the warp that has its teacher:
//   T^2 (sum_j p_j log p_j + log Z) - T sum_j p_j (s_j - m),
// the p_j summing to 1. The gaps s - m meet T, not T^2 / T: a class that the teacher
// keeps and the student masks with its type's lowest value has a finite loss.
template <typename T>
__device__ __forceinline__ void write_loss(const DistillArgs& A, int64_t i, const T* s, float m, float z,
                                           const float* probs, const int32_t* ids, const Teacher& R) {
  const int lane = threadIdx.x & 31;
  const float t = A.temperature, rest = R.some ? t * t * (R.plogp + logf(z)) : 0.0f;
  float l = R.p != 0.0f ? R.p * (R.s - m) : 0.0f;
  for (int j = lane + 32; j < A.k; j += 32)
    if (probs[j] != 0.0f) l += probs[j] * (elem_to_f<T>(s[ids[j]]) - m);
  l = warp_sum(l);
  if (lane == 0) A.loss[i] = fmaf(-t, l, rest);   // nothing kept: both are 0
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
// which no CTA passes before all have read it. The barrier is the form that warps may
// reach from different places.
__device__ __forceinline__ float2 cluster_join(float2 v, float c, float2* stat, int rank, int C) {
  cg::cluster_group cluster = cg::this_cluster();
  if ((int)threadIdx.x < C) cluster.map_shared_rank(stat, threadIdx.x)[rank] = v;
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  const int lane = threadIdx.x & 31;
  return warp_join(lane < C ? stat[lane] : make_float2(-INFINITY, 0.0f), c);
}

constexpr float kLog2e = 1.44269504f;

// The passes over one vector, two elements an instruction where there is one.
// Maximum: into four words of elements.
template <typename T, typename V>
__device__ __forceinline__ void pass_max(const V& v, uint32_t* top) {
#pragma unroll
  for (int w = 0; w < V::W; ++w) top[w & 3] = word_max<T>(top[w & 3], v.words[w]);
}
template <typename T>
__device__ __forceinline__ float whole_max(const uint32_t* top, float one) {
  const uint32_t w = word_max<T>(word_max<T>(top[0], top[1]), word_max<T>(top[2], top[3]));
  return max_nan(one, max_nan(word_elem<T>(w, 0), word_elem<T>(w, 1)));   // an fp32 word has one element, twice
}
// 2^((v - m) c) of elements 2i and 2i + 1; less: -m twice, c2: c twice
template <typename V>
__device__ __forceinline__ void pair_exp(const V& v, int i, F2 less, F2 c2, float& a, float& b) {
  ((v.pair(i) + less) * c2).split(a, b);
  a = exp2_fast(a);
  b = exp2_fast(b);
}
template <typename V>
__device__ __forceinline__ void pass_sum(const V& v, F2 less, F2 c2, F2* z) {
#pragma unroll
  for (int i = 0; i < V::N / 2; ++i) {
    float a, b;
    pair_exp(v, i, less, c2, a, b);
    z[i & 1] = z[i & 1] + F2::of(a, b);
  }
}
__device__ __forceinline__ float whole_sum(const F2* z) {
  float a, b;
  (z[0] + z[1]).split(a, b);
  return a + b;
}
// The vector's gradient, aiz 2^((v - m) c), packed.
template <typename V>
__device__ __forceinline__ V pass_grad(const V& v, F2 less, F2 c2, F2 aiz2) {
  float f[V::N];
#pragma unroll
  for (int i = 0; i < V::N / 2; ++i) {
    float a, b;
    pair_exp(v, i, less, c2, a, b);
    (F2::of(a, b) * aiz2).split(f[2 * i], f[2 * i + 1]);
  }
  V o;
  o.pack(f);
  return o;
}

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

// Rows in registers: a warp a row, NV vectors a lane and one single element.
constexpr int rows_per_sm(int nv) { return nv <= 2 ? 4 : nv <= 8 ? 3 : nv <= 16 ? 2 : 1; }
template <typename T, int NV>
__global__ void __launch_bounds__(256, rows_per_sm(NV))
distill_rows_kernel(DistillArgs A) {
  using V = Vec<T, 16>;
  __shared__ float probs_s[8][DISTILL_MAX_K];
  __shared__ int32_t ids_s[8][DISTILL_MAX_K];
  const int warp = threadIdx.x >> 5, r = threadIdx.x & 31;
  float* probs = probs_s[warp];
  int32_t* ids = ids_s[warp];
  const float c = kLog2e / A.temperature;
  const F2 c2 = F2::of(c, c);
  for (int64_t i = (int64_t)blockIdx.x * 8 + warp; i < A.n; i += (int64_t)gridDim.x * 8) {
    const T* s = (const T*)A.student + i * A.classes;
    T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
    const RowPart P = RowPart::of<T, V::N>(s, A.classes, 0, 1, r);
    const T* sv = s + P.head;
    const int nv = P.v1 - r;                 // this lane's vectors: q * 32 < nv
    // a vector past the row holds -inf and adds nothing to the statistics
    V v[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      v[q].fill(kNegInf<T>);
      if (q * 32 < nv) v[q].load(sv, r + q * 32);
    }
    const float one = P.has ? elem_to_f<T>(s[P.single]) : -INFINITY;
    Teacher R = teacher_load<T>(A, i);
    teacher_solve(A, i, R, probs, ids);
    // The passes go over groups of four vectors, each behind a condition that the
    // warp shares: unused groups are skipped, and a row of 16-bit elements is never
    // unpacked as a whole, which would not fit the registers.
    const int used = (P.v1 + 31) / 32;
    uint32_t top[4] = {kNegInf<T>, kNegInf<T>, kNegInf<T>, kNegInf<T>};
#pragma unroll
    for (int q0 = 0; q0 < NV; q0 += 4)
      if (q0 < used)
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q) pass_max<T>(v[q], top);
    const float m = warp_max(whole_max<T>(top, one));
    const F2 less = F2::of(-m, -m);
    F2 zp[2] = {F2::of(exp2_fast((one - m) * c), 0.0f), F2::of(0.0f, 0.0f)};
#pragma unroll
    for (int q0 = 0; q0 < NV; q0 += 4)
      if (q0 < used)
#pragma unroll
        for (int q = q0; q < q0 + 4 && q < NV; ++q) pass_sum(v[q], less, c2, zp);
    const float z = warp_sum(whole_sum(zp));
    const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f), aiz = a / z;
    if (g) {
      T* gv = g + P.head;
#pragma unroll
      for (int q0 = 0; q0 < NV; q0 += 4) {
        if (R.some && q0 < used) {
#pragma unroll
          for (int q = q0; q < q0 + 4 && q < NV; ++q) {
            const V o = pass_grad(v[q], less, c2, F2::of(aiz, aiz));
            if (q * 32 < nv) o.store(gv, r + q * 32);
          }
        } else if (q0 < used) {
          V o;
          o.fill(0);
#pragma unroll
          for (int q = q0; q < q0 + 4 && q < NV; ++q)
            if (q * 32 < nv) o.store(gv, r + q * 32);
        }
      }
      if (P.has) g[P.single] = elem_from_f<T>(R.some ? exp2_fast((one - m) * c) * aiz : 0.0f);
    }
    write_loss<T>(A, i, s, m, z, probs, ids, R);
    __syncwarp();                            // the kept classes after all others
    if (g && R.some) {
      if (A.k <= 32) kept_gradients_warp<T>(R, g, m, c, a, aiz, probs);
      else kept_gradients<T>(A.k, r, 32, s, g, m, c, a, aiz, probs, ids, 0, A.classes);
    }
    __syncwarp();                            // the next row's probabilities overwrite these
  }
}

// Rows in shared memory: a CTA, or a cluster of C of them, a row. Fifteen warps
// work on the row; a thread copies, reads and rewrites only vectors of its own,
// so the stages need no barrier. The last warp has the teacher: it solves a row's
// probabilities while the others take its statistics, writes the loss, and
// corrects the kept classes once the others have written theirs, for which they
// arrive at a barrier without waiting. (On warp 0 that work, a chain of dependent
// loads, held the CTA up for half of the time: 195 us at 777 rows of 400 KB where this takes 151.)
constexpr int DS_T = 512, DS_M = DS_T - 32;
constexpr int DS_PART = 50 * 1024;           // bytes of a part: two stages for each of two CTAs fit an SM
template <typename T>
__global__ void __launch_bounds__(DS_T, 2)
distill_stage_kernel(DistillArgs A, int C, int stage_vecs) {
  using V = Vec<T, 16>;
  extern __shared__ uint4 stages[];          // [2][stage_vecs]
  __shared__ float2 red[2][DS_T / 32], stat[2][8];
  __shared__ float probs[DISTILL_MAX_K];     // of the last warp alone
  __shared__ int32_t ids[DISTILL_MAX_K];
  __shared__ int some_s[2];
  const int t = threadIdx.x, rank = C == 1 ? 0 : (int)cg::this_cluster().block_rank();
  const bool teacher = t >= DS_M;
  const float c = kLog2e / A.temperature;
  const F2 c2 = F2::of(c, c);
  const int64_t step = gridDim.x / C;
  int64_t i = blockIdx.x / C;
  if (C > 1) cg::this_cluster().sync();      // every CTA runs before one writes to another
  if (teacher) {
    Teacher R = teacher_load<T>(A, i);
    for (int turn = 0; i < A.n; i += step, turn ^= 1) {
      const T* s = (const T*)A.student + i * A.classes;
      T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
      teacher_solve(A, i, R, probs, ids);
      if (t == DS_M) some_s[turn] = R.some;
      __syncwarp();
      float2 all = cta_join<DS_T, 2>(make_float2(-INFINITY, 0.0f), c, red[turn]);
      if (C > 1) all = cluster_join(all, c, stat[turn], rank, C);
      const Teacher now = R;
      R = teacher_load<T>(A, i + step);
      if (rank == 0) write_loss<T>(A, i, s, all.x, all.y, probs, ids, now);
      if (g) {
        asm volatile("bar.sync 1, %0;" ::"n"(DS_T) : "memory");
        const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f);
        const RowPart P = RowPart::of<T, V::N>(s, A.classes, rank, C, 0);
        if (now.some) kept_gradients<T>(A.k, t - DS_M, 32, s, g, all.x, c, a, a / all.y, probs, ids, P.lo, P.hi);
      }
      __syncwarp();                          // the next row's probabilities overwrite these
    }
  } else {
    RowPart P, Pn;
    float one, one_next;
    // starts the copies of row `row` (none past the last) into a stage
    auto fetch = [&](int64_t row, int stage) {
      one_next = -INFINITY;
      if (row < A.n) {
        const T* s = (const T*)A.student + row * A.classes;
        Pn = RowPart::of<T, V::N>(s, A.classes, rank, C, t);
        const uint4* sv = reinterpret_cast<const uint4*>(s + Pn.head) + Pn.v0;
        for (int q = t; q < Pn.v1 - Pn.v0; q += DS_M) copy_async16(&stages[stage * stage_vecs + q], sv + q);
        if (Pn.has) one_next = elem_to_f<T>(s[Pn.single]);
      }
      copy_commit();
    };
    fetch(i, 0);
    for (int turn = 0; i < A.n; i += step, turn ^= 1) {
      P = Pn;
      one = one_next;
      fetch(i + step, turn ^ 1);
      T* g = A.grad ? (T*)A.grad + i * A.classes : nullptr;
      const uint4* v = stages + turn * stage_vecs;
      const int nv = P.v1 - P.v0;
      const float a = A.temperature * (A.scale ? __ldg(A.scale + i) : 1.0f);
      copy_wait<1>();                        // this row's copies; the next row's may still run
      uint32_t mp[4] = {kNegInf<T>, kNegInf<T>, kNegInf<T>, kNegInf<T>};
#pragma unroll 2
      for (int q = t; q < nv; q += DS_M) pass_max<T>(V::of(v[q]), mp);
      const float top = whole_max<T>(mp, one);
      const float shift = top == -INFINITY ? 0.0f : top;
      F2 zp[2] = {F2::of(exp2_fast((one - shift) * c), 0.0f), F2::of(0.0f, 0.0f)};
#pragma unroll 2
      for (int q = t; q < nv; q += DS_M) pass_sum(V::of(v[q]), F2::of(-shift, -shift), c2, zp);
      float2 all = cta_join<DS_T, 2>(make_float2(top, whole_sum(zp)), c, red[turn]);
      if (C > 1) all = cluster_join(all, c, stat[turn], rank, C);
      const float m = all.x, aiz = a / all.y;
      const bool some = some_s[turn];
      if (g) {
        T* gv = g + P.head;
        if (some) {
#pragma unroll 2
          for (int q = t; q < nv; q += DS_M)
            pass_grad(V::of(v[q]), F2::of(-m, -m), c2, F2::of(aiz, aiz)).store(gv, P.v0 + q);
        } else {
          V o;
          o.fill(0);
          for (int q = t; q < nv; q += DS_M) o.store(gv, P.v0 + q);
        }
        if (P.has) g[P.single] = elem_from_f<T>(some ? exp2_fast((one - m) * c) * aiz : 0.0f);
        asm volatile("bar.arrive 1, %0;" ::"n"(DS_T) : "memory");
      }
    }
    copy_wait<0>();
  }
  if (C > 1) cg::this_cluster().sync();      // no CTA ends while another writes to it
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
    float2 all = cta_join<DW_T, 0>(make_float2(m, z), c, red[turn]);
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
template <typename K, typename... Args>
cudaError_t run_clusters(K kernel, int64_t teams, int threads, size_t smem, int C, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)(teams * C));
  if (C > 1 && teams * C > 148) {            // so few all run at once, and asking takes the host 0.3 us
    int most = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (most >= 1 && teams > most) cfg.gridDim = dim3((unsigned)most * C);
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int NV>
cudaError_t run_rows(const DistillArgs& A, cudaStream_t st) {
  const int64_t want = (A.n + 7) / 8, most = 148 * rows_per_sm(NV);
  distill_rows_kernel<T, NV><<<(unsigned)(want < most ? want : most), 256, 0, st>>>(A);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_stage(const DistillArgs& A, int C, cudaStream_t st) {
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  const int vecs = (int)((bytes / 16 + C - 1) / C) + 1;
  const size_t smem = (size_t)vecs * 32;
  const cudaError_t e = cudaFuncSetAttribute(distill_stage_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * DS_PART + 64);
  if (e != cudaSuccess) return e;
  const int64_t most = 296 / C;
  return run_clusters(distill_stage_kernel<T>, A.n < most ? A.n : most, DS_T, smem, C, st, A, C, vecs);
}

template <typename T, int BYTES>
cudaError_t run_wide(const DistillArgs& A, cudaStream_t st) {
  // CTAs of a row: eight for few rows (20 rows of 480 KB: 11 us, two CTAs a row 17),
  // fewer where a part would be below 32 KB (4,096 rows of 16 KB: one CTA 69 us, two
  // 139), and fewer where that leaves rows enough for all 296 CTAs and the rows in
  // flight stay in L2 for their second reading (777 rows of 480 KB: four 194 us, two
  // 202, eight 245; 300 rows of 1.2 MB: eight 261, four 299). Clusters of eight leave
  // a tenth of the SMs idle, so those give way at more bytes (777 rows of 800 KB:
  // four 323 us, eight 361).
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  int C = 8;
  while (C > 1) {
    const int64_t held = 296 / (C / 2) * bytes, limit = int64_t(C == 8 ? 80 : 48) << 20;
    if (bytes / C >= 32768 && (A.n * (C / 2) < 296 || held > limit)) break;
    C /= 2;
  }
  const int64_t most = 296 / C;
  return run_clusters(distill_wide_kernel<T, BYTES>, A.n < most ? A.n : most, DW_T, 0, C, st, A, C);
}

template <typename T>
cudaError_t run_t(const DistillArgs& A, cudaStream_t st) {
  const int64_t bytes = (int64_t)A.classes * sizeof(T);
  // the vectors of student and gradient rows coincide when both start alike
  if (A.grad && ((uintptr_t)A.grad - (uintptr_t)A.student) % 16) return run_wide<T, (int)sizeof(T)>(A, st);
  // Vectors of a lane, as few as hold the row: 65,536 rows of 512 bytes 43 us with one,
  // 45 with two; of 1 KB 47 with two, 61 with eight; of 4 KB 91 with eight, 111 with
  // sixteen (100 such rows 4.3 us, as CTAs of their own 4.0; 592 rows 4.4, 4.5).
  if (bytes <= 512) return run_rows<T, 1>(A, st);
  if (bytes <= 1024) return run_rows<T, 2>(A, st);
  if (bytes <= 4096) return run_rows<T, 8>(A, st);
  // A warp a row from four rows an SM on: of 592 rows of 8 KB it takes 6.3 us against
  // the CTA's 7.9, of 16 KB 9.6 against 9.3 (1,184: 6.5 against 13.4, 10.0 against
  // 16.0); of 148 rows 6.1 against 4.3, 9.4 against 4.9.
  if (A.n >= 592 && bytes <= 8192) return run_rows<T, 16>(A, st);
  if (A.n >= 592 && bytes <= 16384) return run_rows<T, 32>(A, st);
  int C = 1;                                 // CTAs of a row
  while (C <= 8 && bytes > (int64_t)DS_PART * C) C *= 2;
  return C <= 8 ? run_stage<T>(A, C, st) : run_wide<T, 16>(A, st);
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
