// The KiloNeRF cell networks on rows sorted by cell, forward and weight gradient:
//   z1 = W1 gamma(x) + b1, h1 = relu(z1); z2 = W2 h1 + b2, h2 = relu(z2);
//   (r, g, b) = Wc [h2; gamma(d/|d|)] + bc, sigma = ws . h2 + bs.
// Backward, with g = d raw: g2 = (Wc_h^T g_rgb + ws g_sigma) (h2 > 0),
// g1 = (W2^T g2) (h1 > 0), and each weight's gradient the sum over the cell's
// rows of (its output's gradient) x (its input).
//
// The products run as mma.sync m16n8k8 in tf32, three per product of two fp32
// operands (v = hi + lo, hi rounded to tf32: hi*hi + hi*lo + lo*hi), which keeps
// fp32 accuracy. The layers are 32 wide, so what decides is where the
// activations live between them: a warp's fragments stay in its registers from
// the encoding to the heads, the output fragment of one layer being the operand
// fragment of the next under a permutation of the weight columns, and nothing
// of a row passes through shared memory or a barrier. Lane l of a warp is
// (g = l / 4, t = l % 4): operand A (16 x 8) holds rows g, g + 8 and columns t,
// t + 4; B (8 x 8) rows t, t + 4 and column g; C (16 x 8) rows g, g + 8 and
// columns 2t, 2t + 1. An angle's sine and cosine are a pair of fragment columns,
// and the columns are ordered so that a lane that has an even octave has the odd
// one above it too: sin 2a = 2 sin a cos a and cos 2a = 1 - 2 sin^2 a, four
// operations in place of a second evaluation. With base q = 0..14
// (coordinate q / 5, octave 2 (q % 5)), base 15 stands for x, y, z and a constant.
//
// mma.sync and not tcgen05: with operands in shared memory every layer's inputs would
// be split and written there (768 bytes a row forward) behind barriers, as
// kilo_eval_kernel does for the renderer. Operand A can also come from tensor memory,
// to which a thread that owns a row could write its split activations; that form has
// not been built. mma.sync runs at 0.9 TMAC/s an SM in tf32 (measured), 57 us for the
// forward layers of 786,432 rows: a floor of the instruction, not of the card. With
// 786,432 rows over 4,096 cells (2,702 of them with rows) the forward pass with its
// hidden layers takes 137 us on the device (2.1 TB/s of 287 MB, 0.32 of the copy rate;
// tensor pipe 44 % busy, issue slots 52 %, shared memory 52 %), the weight gradient
// 193 us (tensor pipe 45 %, issue slots 56 %, shared memory 51 %): no unit is full,
// both are bound by each warp's chain of encoding, split and product at the 16 or 12
// warps that an SM's registers hold.
#include "nerf_experts.cuh"

namespace nerfb {
namespace {

// parameter offsets inside a cell's blob
constexpr int O_B1 = 32 * 63, O_W2 = O_B1 + 32, O_B2 = O_W2 + 32 * 32, O_WS = O_B2 + 32, O_BS = O_WS + 32,
              O_WC = O_BS + 1, O_BC = O_WC + 3 * 59;
static_assert(O_BC + 3 == CELL_NP, "the blob's parts");

__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// v = hi + lo: hi the nearest tf32 (10 stored bits, ties away from zero), lo exact;
// the tensor core reads lo at tf32 precision. An infinity or NaN has a NaN as one of
// the two, so what is computed from it is NaN.
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(v) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(__fsub_rn(v, __uint_as_float(hi)));
}
// max(v, 0) that keeps a NaN: a row or cell that is no longer finite shows it
__device__ __forceinline__ float relu(float v) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(v));
  return y;
}
// sin and cos of pi v: v = n / 2 + r exactly, |r| <= 1/4, and two polynomials in
// r^2 whose coefficients were fitted to sin(pi r) / r and cos(pi r) on that
// interval by reweighted least squares. Within 1.5 * 2^-24 of the value. A float
// of 2^24 or more is an even number (or infinite, whose difference from itself is
// NaN). Two fifths fewer operations than the library call, and no branch: a call
// in these loops would take registers that they need.
__device__ __forceinline__ void sincos_pi(float v, float* s, float* c) {
  if (!(fabsf(v) < 16777216.0f)) v -= v;
  const float t = rintf(v + v);
  const unsigned n = (unsigned)(int)t;
  const float r = fmaf(t, -0.5f, v), q = r * r;
  const float a = r * fmaf(fmaf(fmaf(-5.890786648e-01f, q, 2.549767256f), q, -5.167707920f), q, 3.141592741f);
  const float b = fmaf(fmaf(fmaf(fmaf(2.314295471e-01f, q, -1.335058451f), q, 4.058707905f), q, -4.934802055f), q, 1.0f);
  const float p = n & 1 ? b : a, o = n & 1 ? a : b;
  *s = __uint_as_float(__float_as_uint(p) ^ ((n << 30) & 0x80000000u));
  *c = __uint_as_float(__float_as_uint(o) ^ (((n + 1) << 30) & 0x80000000u));
}
// The unit direction: each coordinate divided by the rounded norm, after a scale by
// the power of two that brings the largest coordinate's exponent to 0 (at the ends of
// the range it lands within 2^-22 .. 4), so that no square overflows or loses its bits. The scale
// is exact and changes no bit of a direction whose squares did neither.
__device__ __forceinline__ void unit3(float* d) {
  const uint32_t most = __float_as_uint(fmaxf(fmaxf(fabsf(d[0]), fabsf(d[1])), fabsf(d[2]))) & 0x7f800000u;
  const float scale = __uint_as_float(0x7f000000u - min(most, 0x7e800000u));
  d[0] *= scale;
  d[1] *= scale;
  d[2] *= scale;
  const float len = sqrtf(fmaf(d[0], d[0], fmaf(d[1], d[1], d[2] * d[2])));
  d[0] /= len;
  d[1] /= len;
  d[2] /= len;
}
// v = (sin, cos) of octave k of coordinate xc, then of octave k + 1; scale = 2^k
__device__ __forceinline__ void two_octaves(float xc, float scale, float* v) {
  sincos_pi(xc * scale, v, v + 1);
  const float s2 = v[0] + v[0];
  v[2] = s2 * v[1];
  v[3] = fmaf(-s2, v[0], 1.0f);
}
// a lane's base of the position encoding: coordinate and 2^octave
struct Base {
  int c;
  float scale;
  bool last;                                 // base 15: x, y, z, constant
  __device__ __forceinline__ explicit Base(int q) {
    c = (q >= 5) + (q >= 10);
    scale = __int_as_float((127 + 2 * (q - 5 * c)) << 23);
    last = q == 15;
  }
  // (sin, cos) of two octaves of the row x, or x, y, z, one
  __device__ __forceinline__ void encode(const float* x, float one, float* v) const {
    two_octaves(x[c], scale, v);
    if (last) {
      v[0] = x[0];
      v[1] = x[1];
      v[2] = x[2];
      v[3] = one;
    }
  }
};
// column of gamma(x) that entry i (sin, cos, sin, cos) of base q stands for; 63 the constant
__device__ __forceinline__ int position_column(int q, int i) {
  const int c = (q >= 5) + (q >= 10), k = 2 * (q - 5 * c) + (i >> 1);
  return q < 15 ? 3 + 30 * (i & 1) + 10 * c + k : i < 3 ? i : 63;
}

// Asynchronous copies into shared memory; zeros where `in` is false.
__device__ __forceinline__ void copy_async16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async4(void* dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// The work of a cell in units: one for its start (its weights are staged, its
// gradient is written) and one per tile of `rows` rows; none without rows.
// first[c] = units of the cells before c, first[n_cells] = all of them. Each
// thread sums a run of cells, an odd number of them, which keeps its reads of
// shared memory clear of the others' banks. Offsets are taken into 0..n and sums
// kept below 2^30, so no table makes a row index leave its buffer.
constexpr int UNITS_MOST = 1 << 30;
__device__ __forceinline__ int units_of(int a, int b, int rows) { return b > a ? (b - a + rows - 1) / rows + 1 : 0; }
template <int THREADS>
__device__ __forceinline__ void unit_prefix(const int32_t* __restrict__ offset, int64_t n, int n_cells, int rows,
                                            int* first) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int sums[WARPS];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
#pragma unroll 8
  for (int c = t; c <= n_cells; c += THREADS) first[c] = (int)min(max((int64_t)__ldg(offset + c), (int64_t)0), n);
  __syncthreads();
  const int per = ((n_cells + THREADS - 1) / THREADS) | 1;
  const int c0 = min(t * per, n_cells), c1 = min(c0 + per, n_cells);
  const int last = first[c1];
  int sum = 0;
  for (int c = c0; c < c1; ++c) sum = min(sum + units_of(first[c], c + 1 < c1 ? first[c + 1] : last, rows), UNITS_MOST);
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run = min(run + u, UNITS_MOST);
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();                           // and every thread has read the offset behind its run
  int before = max(run - sum, 0);
  for (int w = 0; w < warp; ++w) before = min(before + sums[w], UNITS_MOST);
  for (int c = c0, a = c0 < c1 ? first[c0] : 0; c < c1; ++c) {
    const int b = c + 1 < c1 ? first[c + 1] : last, u = units_of(a, b, rows);
    first[c] = before;
    before = min(before + u, UNITS_MOST);
    a = b;
  }
  if (c1 == n_cells && (c0 < c1 || t == 0)) first[n_cells] = before;
  __syncthreads();
}
// the cell of a unit: first[c] <= unit < first[c + 1]
__device__ __forceinline__ int cell_of(const int* first, int n_cells, int tile) {
  int lo = 0, hi = n_cells;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= tile) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ forward

constexpr int CF_WARPS = 4, CF_THREADS = CF_WARPS * 32;
constexpr int CF_ROWS = CF_WARPS * 32;       // rows of a tile, 32 per warp
constexpr int CF_PER_SM = 4;
// A tile of up to CF_SPREAD rows is shared by all four warps, 16 rows each, else a
// warp takes 32: with few rows to a cell the tile's time is one warp's chain. On the
// device 20,000 rows of 4,096 cells take 34 us (39 without; 36 with 32 rows, 8 to a
// warp), 70,000 41 us (45; 50), 2,000 22.7 (26.2; 22.3), the 192 rows of a ray 9.2 us
// (10.6; 9.5). A row's operations and their order are the same.
constexpr int CF_SPREAD = 64;
// rows of each warp in a tile with `rows` rows left
__device__ __forceinline__ int share_of(int64_t rows) { return rows <= CF_SPREAD ? CF_SPREAD / CF_WARPS : CF_ROWS / CF_WARPS; }
struct CellsForwardShared {
  union {
    struct {
      float4 w1[8 * 4 * 32];  // B fragments of W1: [k step][n tile][lane] = (hi, hi, lo, lo)
      float4 w2[4 * 4 * 32];
    };
    int first[EXPERT_MAX + 1];   // units, until this CTA has found where it begins
  };
  float raw_w[CELL_NP + 3];   // the next cell's weights as they stand in the blob
  float4 wh[32], wd[27], bh;  // heads (r, g, b, sigma) on h2 and (r, g, b, 0) on gamma(d)
  float b1[32], b2[32];
  float rows[CF_WARPS][2][2][96];             // [warp][stage]: x and d of a warp's 32 rows
};

__device__ __forceinline__ float4 b_fragment(float b0, float b1) {
  uint32_t h0, l0, h1, l1;
  split3(b0, h0, l0);
  split3(b1, h1, l1);
  return make_float4(__uint_as_float(h0), __uint_as_float(h1), __uint_as_float(l0), __uint_as_float(l1));
}

// The feature of column n of output tile j. Lane t, whose columns are 2t and
// 2t + 1 of the four tiles, has features 8t .. 8t + 7: a run that it stores at once.
__device__ __forceinline__ int out_feature(int j, int n) { return 8 * (n >> 1) + 2 * j + (n & 1); }
// One k step of a layer: M fragments of 16 rows x 32 outputs (four). The three
// products of an accumulator are 4 M instructions apart. The tensor core truncates when
// it adds to the accumulator: the hidden layers are within 5.3e-7 of their norm. Sums
// of every step, or of every two, added by rounded additions bring that to 1.2e-7 or
// 1.7e-7 (fp32 products: 1.5e-7), at 150 or 143 us for the batch in place of 137.
template <int M>
__device__ __forceinline__ void layer_step(float (&c)[M][4][4], const uint32_t (&ah)[M][4],
                                           const uint32_t (&al)[M][4], const float4* w) {
  uint32_t bh[4][2], bl[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = w[j * 32];
    bh[j][0] = __float_as_uint(v.x), bh[j][1] = __float_as_uint(v.y);
    bl[j][0] = __float_as_uint(v.z), bl[j][1] = __float_as_uint(v.w);
  }
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int m = 0; m < M; ++m)
        mma_tf32(c[m][j], p == 0 ? al[m] : ah[m], p == 1 ? bl[j][0] : bh[j][0], p == 1 ? bl[j][1] : bh[j][1]);
}

// a hidden layer of 8 R rows (h0 its first row's): lane (g, t) has features 8t .. 8t + 7
// of rows g + 8 r
template <int R, int M>
__device__ __forceinline__ void store_hidden(float* __restrict__ h0, const float (&h)[M][4][4], int g, int t, int rows) {
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (g + 8 * r < rows) {
      float4* out = reinterpret_cast<float4*>(h0 + (g + 8 * r) * 64 + 8 * t);
      const int m = r >> 1, i = 2 * (r & 1);
      out[0] = make_float4(h[m][0][i], h[m][0][i + 1], h[m][1][i], h[m][1][i + 1]);
      out[1] = make_float4(h[m][2][i], h[m][2][i + 1], h[m][3][i], h[m][3][i + 1]);
    }
}

// A warp's `rows` rows, at most 8 R: lane (g, t) works on rows g + 8 r, r < R. xs, ds:
// their positions and directions in shared memory.
template <int R>
__device__ __forceinline__ void forward_rows(const CellsForwardShared& S, const float* xs, float* ds, int64_t row0,
                                             int rows, float* __restrict__ raw, float* __restrict__ hidden) {
  constexpr int M = (R + 1) / 2;             // fragments of 16 rows
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float h[M][4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 b = *reinterpret_cast<const float2*>(&S.b1[8 * t + 2 * j]);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      h[m][j][0] = h[m][j][2] = b.x;
      h[m][j][1] = h[m][j][3] = b.y;
    }
  }
  // two k steps at a time: a base octave and the one above it. Not unrolled: the
  // code of a whole tile would overrun the instruction cache.
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    uint32_t ah[2][M][4] = {}, al[2][M][4] = {};
    const Base base(4 * b + t);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[4];
      base.encode(xs + 3 * (g + 8 * r), 0.0f, v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        split3(v[i], ah[i >> 1][r >> 1][2 * (i & 1) + (r & 1)], al[i >> 1][r >> 1][2 * (i & 1) + (r & 1)]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) layer_step(h, ah[s], al[s], &S.w1[(2 * b + s) * 128 + lane]);
  }
  float h2[M][4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 b = *reinterpret_cast<const float2*>(&S.b2[8 * t + 2 * j]);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      h2[m][j][0] = h2[m][j][2] = b.x;
      h2[m][j][1] = h2[m][j][3] = b.y;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[m][j][i] = relu(h[m][j][i]);
    }
  }
  if (hidden) store_hidden<R, M>(hidden + row0 * 64, h, g, t, rows);
  // h1's fragment (row, features 8t + 2s, 8t + 2s + 1) is the operand of k step
  // s with its columns t, t + 4 standing for those two features
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t ah[M][4], al[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) split3(h[m][s][i], ah[m][(i & 1) * 2 + (i >> 1)], al[m][(i & 1) * 2 + (i >> 1)]);
    layer_step(h2, ah, al, &S.w2[s * 128 + lane]);
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) h2[m][j][i] = relu(h2[m][j][i]);
  if (hidden) store_hidden<R, M>(hidden + row0 * 64 + 32, h2, g, t, rows);
  // the heads on the FMA pipe, which the tensor products leave idle: each lane
  // its eight features of h2 and its share of gamma(d), for R rows
  float o[R][4] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 w0 = S.wh[8 * t + 2 * j], w1 = S.wh[8 * t + 2 * j + 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float a = h2[r >> 1][j][2 * (r & 1)], b = h2[r >> 1][j][2 * (r & 1) + 1];
      o[r][0] = fmaf(w0.x, a, fmaf(w1.x, b, o[r][0]));
      o[r][1] = fmaf(w0.y, a, fmaf(w1.y, b, o[r][1]));
      o[r][2] = fmaf(w0.z, a, fmaf(w1.z, b, o[r][2]));
      o[r][3] = fmaf(w0.w, a, fmaf(w1.w, b, o[r][3]));
    }
  }
  // one lane a row makes its direction a unit vector; then lane t < 3 has
  // coordinate t and its four octaves
  unit3(ds + 3 * lane);
  __syncwarp();
  const int tc = min(t, 2);
  const float on = t < 3 ? 1.0f : 0.0f;    // lane 3 adds nothing
#pragma unroll
  for (int half = 0; half < 2; ++half) {   // octaves 0, 1 and 2, 3
    float v[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) two_octaves(ds[3 * (g + 8 * r) + tc], half ? 4.0f : 1.0f, v[r]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = S.wd[3 + 12 * (i & 1) + 4 * tc + 2 * half + (i >> 1)];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float e = v[r][i] * on;
        o[r][0] = fmaf(a.x, e, o[r][0]);
        o[r][1] = fmaf(a.y, e, o[r][1]);
        o[r][2] = fmaf(a.z, e, o[r][2]);
      }
    }
  }
  const float4 wu = S.wd[tc];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float ut = ds[3 * (g + 8 * r) + tc] * on;
    o[r][0] = fmaf(wu.x, ut, o[r][0]);
    o[r][1] = fmaf(wu.y, ut, o[r][1]);
    o[r][2] = fmaf(wu.z, ut, o[r][2]);
  }
  // sum over the four lanes of a row; lane t keeps row g + 8 t
  float4 v;
  float* vp = &v.x;
  const bool up = t & 2, odd = t & 1;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (R == 4) {
      const float k0 = up ? o[2 % R][c] : o[0][c], k1 = up ? o[3 % R][c] : o[1 % R][c];
      const float s0 = up ? o[0][c] : o[2 % R][c], s1 = up ? o[1 % R][c] : o[3 % R][c];
      const float p0 = k0 + __shfl_xor_sync(0xffffffffu, s0, 2);
      const float p1 = k1 + __shfl_xor_sync(0xffffffffu, s1, 2);
      vp[c] = (odd ? p1 : p0) + __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float s = o[r][c] + __shfl_xor_sync(0xffffffffu, o[r][c], 2);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        if (r == 0 || t == r) vp[c] = s;
      }
    }
  }
  const float4 bh = S.bh;
  if (t < R && g + 8 * t < rows)
    reinterpret_cast<float4*>(raw)[row0 + g + 8 * t] =
        make_float4(v.x + bh.x, v.y + bh.y, v.z + bh.z, v.w + bh.w);
}

__global__ void __launch_bounds__(CF_THREADS, CF_PER_SM)
cells_forward_kernel(const float* __restrict__ x, const float* __restrict__ d, int64_t n,
                     const int32_t* __restrict__ offset, int n_cells,
                     const float* __restrict__ cell_w, float* __restrict__ raw,
                     float* __restrict__ hidden) {
  extern __shared__ __align__(16) uint8_t cells_sm[];
  CellsForwardShared& S = *reinterpret_cast<CellsForwardShared*>(cells_sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unit_prefix<CF_THREADS>(offset, n, n_cells, CF_ROWS, S.first);
  // This CTA's units [unit, end), an equal share. A place in them: a cell, its
  // first unit and its rows.
  const int units = S.first[n_cells], per = (units + gridDim.x - 1) / gridDim.x;
  const int begin = (int)min((int64_t)blockIdx.x * per, (int64_t)units), end = min(units, begin + per);
  if (begin >= end) return;
  auto clamped = [&](int c) { return (int)min(max((int64_t)__ldg(offset + c), (int64_t)0), n); };
  struct Place {
    int cell, first;                         // -1: past the end
    int lo, hi;
  };
  Place at;
  at.cell = cell_of(S.first, n_cells, begin);
  at.first = S.first[at.cell];
  at.lo = clamped(at.cell);
  at.hi = clamped(at.cell + 1);
  __syncthreads();                           // the units' memory now holds weights
  // the next cell with rows, found 32 at a time
  auto behind = [&](Place p) {
    const int start = p.first + units_of(p.lo, p.hi, CF_ROWS);
    for (int c0 = p.cell + 1; c0 < n_cells; c0 += 32) {
      const int c = c0 + lane, lo = c < n_cells ? clamped(c) : 0, hi = c < n_cells ? clamped(c + 1) : 0;
      const unsigned some = __ballot_sync(0xffffffffu, hi > lo);
      if (some) {
        const int l = __ffs(some) - 1;
        return Place{c0 + l, start, __shfl_sync(0xffffffffu, lo, l), __shfl_sync(0xffffffffu, hi, l)};
      }
    }
    return Place{-1, end, 0, 0};
  };
  // A tile's positions, directions and, where its cell is another than the last
  // tile's, weights are on their way one tile ahead.
  auto fetch_rows = [&](const Place& p, int unit, int stage) {
    const int64_t tile0 = p.lo + (int64_t)(unit - p.first - 1) * CF_ROWS;
    const int share = share_of(p.hi - tile0);
    const int64_t row0 = tile0 + warp * share;
    const int have = (int)max(min((int64_t)share, p.hi - row0), (int64_t)0) * 3;
    const int64_t from = have > 0 ? row0 * 3 : 0;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int e = 32 * q + lane;
      copy_async4(&S.rows[warp][stage][0][e], x + from + (e < have ? e : 0), e < have);
      copy_async4(&S.rows[warp][stage][1][e], d + from + (e < have ? e : 0), e < have);
    }
  };
  auto fetch_weights = [&](int cell) {
    const float* __restrict__ W = cell_w + (int64_t)cell * CELL_NP;
    for (int q = tid; q < CELL_NP; q += CF_THREADS) copy_async4(&S.raw_w[q], W + q, true);
  };
  int unit = max(begin, at.first + 1), staged = -1;
  fetch_weights(at.cell);
  fetch_rows(at, unit, 0);
  copy_commit();
  for (int stage = 0; unit < end; stage ^= 1) {
    const int cell = at.cell;
    copy_wait<0>();                          // this tile's copies
    __syncwarp();
    if (cell != staged) {
      staged = cell;
      __syncthreads();                       // everyone's part of the weights; the last cell's fragments are done with
      const float* W = S.raw_w;
#pragma unroll 4
      for (int q = tid; q < 8 * 4 * 32; q += CF_THREADS) {
        const int l = q & 31, nn = out_feature((q >> 5) & 3, l >> 2), s = q >> 7;
        const int base = 4 * (s >> 1) + (l & 3), c1 = position_column(base, 2 * (s & 1) + 1);
        S.w1[q] = b_fragment(W[nn * 63 + position_column(base, 2 * (s & 1))], c1 < 63 ? W[nn * 63 + c1] : 0.0f);
      }
#pragma unroll
      for (int q = tid; q < 4 * 4 * 32; q += CF_THREADS) {
        const int l = q & 31, nn = out_feature((q >> 5) & 3, l >> 2), f = 8 * (l & 3) + 2 * (q >> 7);
        S.w2[q] = b_fragment(W[O_W2 + nn * 32 + f], W[O_W2 + nn * 32 + f + 1]);
      }
      if (tid < 32) {
        S.b1[tid] = W[O_B1 + tid];
        S.b2[tid] = W[O_B2 + tid];
      } else if (tid < 64) {
        const int f = tid - 32;
        S.wh[f] = make_float4(W[O_WC + f], W[O_WC + 59 + f], W[O_WC + 118 + f], W[O_WS + f]);
      } else if (tid < 91) {
        const int f = tid - 64 + 32;
        S.wd[tid - 64] = make_float4(W[O_WC + f], W[O_WC + 59 + f], W[O_WC + 118 + f], 0.0f);
      } else if (tid == 91) {
        S.bh = make_float4(W[O_BC], W[O_BC + 1], W[O_BC + 2], W[O_BS]);
      }
      __syncthreads();
    }
    const int64_t tile0 = at.lo + (int64_t)(unit - at.first - 1) * CF_ROWS, tile_rows = at.hi - tile0;
    const int share = share_of(tile_rows);
    const int64_t row0 = tile0 + warp * share;
    const int rows = (int)min((int64_t)share, at.hi - row0);
    if (++unit >= at.first + units_of(at.lo, at.hi, CF_ROWS) && unit < end) {
      at = behind(at);
      unit = at.first + 1;
      if (unit < end) fetch_weights(at.cell);
    }
    if (unit < end) fetch_rows(at, unit, stage ^ 1);
    copy_commit();
    if (rows <= 0) continue;
    const float* xs = S.rows[warp][stage][0];
    float* ds = S.rows[warp][stage][1];
    if (tile_rows <= CF_SPREAD) forward_rows<CF_SPREAD / 32>(S, xs, ds, row0, rows, raw, hidden);
    else forward_rows<4>(S, xs, ds, row0, rows, raw, hidden);
  }
  copy_wait<0>();
}

// ------------------------------------------------------------------ backward

// Two roles share the rows: a warp of the first computes g1 and the gradient of
// W1 and b1 (64 accumulators a lane), one of the second the gradients of W2, b2
// and the heads (48). Together they would take 252 registers and leave eight
// warps to an SM; apart, twelve fit. Each role cuts all tiles of 16 rows into
// one contiguous range per warp.
// The tensor core truncates when it adds to an accumulator, an error that grows
// with the number of additions and all in one direction (2e-6 of the gradient
// at 370 rows a cell); so a tile's products go to a fresh accumulator, which is
// added to the cell's by a rounded addition.
constexpr int CB_A = 7, CB_B = 5;             // warps of each role in a CTA (8 and 4: 210 us, 6 and 6: 206, 7 and 5: 196)
constexpr int CB_THREADS = (CB_A + CB_B) * 32;
constexpr int CB_ROWS = 16;
constexpr int CB_SMS = 148;
constexpr int CB_NA = O_W2, CB_NB = CELL_NP - O_W2;   // parameters of each role
// What a tile's rows need, brought in by asynchronous copies one tile ahead of
// its use. A hidden row takes 68 floats: fragments read rows 2t apart in one
// access, and 8t + g then falls in 32 different banks.
struct BackwardTile {
  float hidden[CB_ROWS][68];
  float4 d_raw[CB_ROWS];
  float v[CB_ROWS * 3];                       // x (first role) or d (second)
};
struct CellsBackwardShared {
  BackwardTile tile[CB_A + CB_B][2];
  // A fragments of W2^T, [m tile][k step][lane], hi and lo; heads (r, g, b, sigma) on h2
  uint4 hi[CB_A][2 * 4 * 32], lo[CB_A][2 * 4 * 32];
  float4 wh[CB_A + CB_B][32];
  int first[EXPERT_MAX + 1];
};

int64_t backward_ctas(int64_t n, int n_cells) {
  const int64_t units = (n + CB_ROWS - 1) / CB_ROWS + 2 * (n_cells < n ? n_cells : n);
  const int64_t ctas = (units + CB_B - 1) / CB_B;
  return ctas < CB_SMS ? ctas : CB_SMS;
}

// c += a b, or c = a b where `first`
__device__ __forceinline__ void mma_from(bool first, float* c, const uint32_t* a, const uint32_t* b) {
  if (first)
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
  else
    mma_tf32(c, a, b[0], b[1]);
}
// one output channel's gradient carried to a feature of h2 by the heads' weights
__device__ __forceinline__ float head_grad(const float4& w, const float4& gr) {
  return fmaf(w.x, gr.x, fmaf(w.y, gr.y, fmaf(w.z, gr.z, w.w * gr.w)));
}

// One group of copies: rows row0 .. row0 + 15; zeros for a row past the cell's
// end, which then has no gradient and no input.
__device__ __forceinline__ void fetch_tile(BackwardTile& T, int lane, const float* __restrict__ hidden,
                                           const float* __restrict__ d_raw, const float* __restrict__ v,
                                           int64_t row0, int64_t cell_end) {
  const int64_t safe = min(row0, cell_end - 1);
  const int rows = (int)min((int64_t)CB_ROWS, cell_end - row0);      // 0 or less: nothing is read
  const float* h = hidden + safe * 64;
  const bool full = rows == CB_ROWS;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int r = 2 * q + (lane >> 4);
    const bool in = full || r < rows;
    copy_async16(&T.hidden[r][(lane & 15) * 4], h + (in ? r * 64 + (lane & 15) * 4 : 0), in);
  }
  if (lane < 16) copy_async16(&T.d_raw[lane], d_raw + (safe + (lane < rows ? lane : 0)) * 4, lane < rows);
  const float* w = v + safe * 3;
  copy_async4(&T.v[lane], w + (lane < 3 * rows ? lane : 0), lane < 3 * rows);
  if (lane < 16) copy_async4(&T.v[32 + lane], w + (lane + 32 < 3 * rows ? lane + 32 : 0), lane + 32 < 3 * rows);
  copy_commit();
}

// c[u][m] = z[m] b[u] for two column pairs u and the two fragments m of 32
// outputs; the three products of an accumulator stand four instructions apart
__device__ __forceinline__ void weight_products(float (&c)[2][2][4], const uint32_t (&zh)[2][4],
                                                const uint32_t (&zl)[2][4], const uint32_t (&bh)[2][2],
                                                const uint32_t (&bl)[2][2]) {
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        mma_from(p == 0, c[u][m], p == 0 ? zl[m] : zh[m], p == 1 ? bl[u] : bh[u]);
}

struct CellsBackwardArgs {
  const float *x, *d;
  int64_t n;
  const int32_t* offset;
  int n_cells;
  const float *cell_w, *hidden, *d_raw;
  float* grad;
  int* first_out;
  float *parts_a, *parts_b;
};

// A role's run over the tiles of one cell: rows begin.., tiles [tile, stop) of it.
__device__ __forceinline__ void backward_w1(const CellsBackwardArgs& P, CellsBackwardShared& S, int warp,
                                            int lane, const float* __restrict__ W, int64_t row0,
                                            int64_t cell_end, int tiles, float* __restrict__ G) {
  const int g = lane >> 2, t = lane & 3;
  const float* __restrict__ hidden = P.hidden;
#pragma unroll
  for (int q = 0; q < 8; ++q) {              // rows of W2^T are h1's features; k step s's columns t, t + 4 are h2's 8t + 2s, + 1
    const int m = 16 * (q >> 2) + g, f = 8 * t + 2 * (q & 3);
    uint32_t hi[4], lo[4];
    split3(__ldg(W + O_W2 + f * 32 + m), hi[0], lo[0]);
    split3(__ldg(W + O_W2 + f * 32 + m + 8), hi[1], lo[1]);
    split3(__ldg(W + O_W2 + (f + 1) * 32 + m), hi[2], lo[2]);
    split3(__ldg(W + O_W2 + (f + 1) * 32 + m + 8), hi[3], lo[3]);
    S.hi[warp][q * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    S.lo[warp][q * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncwarp();
  const Base base0(g), base1(8 + g);
  float acc[2][8][4] = {};
  fetch_tile(S.tile[warp][0], lane, hidden, P.d_raw, P.x, row0, cell_end);
  int stage = 0;
#pragma unroll 1
  for (; tiles > 0; --tiles, row0 += CB_ROWS, stage ^= 1) {
    if (tiles > 1) {
      fetch_tile(S.tile[warp][stage ^ 1], lane, hidden, P.d_raw, P.x, row0 + CB_ROWS, cell_end);
      copy_wait<1>();
    } else {
      copy_wait<0>();
    }
    __syncwarp();
    const BackwardTile& T = S.tile[warp][stage];
    // Eight rows at a time, in a loop that is not unrolled: with sixteen in
    // straight line the two roles' code overran the instruction cache.
#pragma unroll 1
    for (int q = 0; q < CB_ROWS; q += 8) {
      asm volatile("" ::: "memory");         // the weights' fragments are read anew, not held in registers
      // g2 as operand B: features 8t .. 8t + 7 of row g; then g1 = (W2^T g2) (h1 > 0)
      const float4 gr = T.d_raw[q + g];
      const float4 m0 = *reinterpret_cast<const float4*>(&T.hidden[q + g][32 + 8 * t]);
      const float4 m1 = *reinterpret_cast<const float4*>(&T.hidden[q + g][36 + 8 * t]);
      const float mask[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
      float dz[2][2][4];                     // [k steps 0, 2 and 1, 3][m tile]
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          split3(mask[2 * s + i] > 0.0f ? head_grad(S.wh[warp][8 * t + 2 * s + i], gr) : 0.0f, bh[i], bl[i]);
        uint32_t wh[2][4], wl[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint4 hi = S.hi[warp][(m * 4 + s) * 32 + lane], lo = S.lo[warp][(m * 4 + s) * 32 + lane];
          wh[m][0] = hi.x, wh[m][1] = hi.y, wh[m][2] = hi.z, wh[m][3] = hi.w;
          wl[m][0] = lo.x, wl[m][1] = lo.y, wl[m][2] = lo.z, wl[m][3] = lo.w;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            mma_from(s < 2 && p == 0, dz[s & 1][m], p == 0 ? wl[m] : wh[m], p == 1 ? bl : bh);
      }
      // C's (g, 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1) are A's (g, t), (g, t+4), (g+8, t), (g+8, t+4)
      uint32_t zh[2][4], zl[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          split3(T.hidden[q + 2 * t + (i & 1)][16 * m + 8 * (i >> 1) + g] > 0.0f ? dz[0][m][i] + dz[1][m][i] : 0.0f,
                 zh[m][(i & 1) * 2 + (i >> 1)], zl[m][(i & 1) * 2 + (i >> 1)]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float e[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) (j ? base1 : base0).encode(&T.v[3 * (q + 2 * t + i)], 1.0f, e[i]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t bh[2][2], bl[2][2];         // [column pair][row]
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            split3(e[0][i + u], bh[u][0], bl[u][0]);
            split3(e[1][i + u], bh[u][1], bl[u][1]);
          }
          float c[2][2][4];
          weight_products(c, zh, zl, bh, bl);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[m][4 * j + i + u][k] += c[u][m][k];
        }
      }
    }
    __syncwarp();                            // this stage may be overwritten
  }
  int tt = t, gg = g;                        // the places below are worked out here, not carried through the loop
  asm volatile("" : "+r"(tt), "+r"(gg));
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int nn = 16 * m + gg + 8 * (k >> 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = position_column(8 * (i >> 2) + 2 * tt + (k & 1), i & 3);
        G[c < 63 ? nn * 63 + c : O_B1 + nn] = acc[m][i][k];
      }
    }
}

__device__ __forceinline__ void backward_w2(const CellsBackwardArgs& P, CellsBackwardShared& S, int warp,
                                            int lane, int64_t row0, int64_t cell_end, int tiles,
                                            float* __restrict__ G) {
  const int g = lane >> 2, t = lane & 3;
  const float* __restrict__ hidden = P.hidden;
  float acc[2][4][4] = {}, ah[4][4] = {}, sb2[4] = {};
  fetch_tile(S.tile[warp][0], lane, hidden, P.d_raw, P.d, row0, cell_end);
  int stage = 0;
#pragma unroll 1
  for (; tiles > 0; --tiles, row0 += CB_ROWS, stage ^= 1) {
    if (tiles > 1) {
      fetch_tile(S.tile[warp][stage ^ 1], lane, hidden, P.d_raw, P.d, row0 + CB_ROWS, cell_end);
      copy_wait<1>();
    } else {
      copy_wait<0>();
    }
    __syncwarp();
    BackwardTile& T = S.tile[warp][stage];
    if (lane < CB_ROWS && row0 + lane < cell_end) unit3(&T.v[3 * lane]);
    __syncwarp();
#pragma unroll 1
    for (int q = 0; q < CB_ROWS; q += 8) {
      asm volatile("" ::: "memory");         // the weights' fragments are read anew, not held in registers
      const int r = q + 2 * t;               // this lane's rows r, r + 1
      float h2[4][2];
      uint32_t zh[2][4], zl[2][4];
      {
        const float4 g0 = T.d_raw[r], g1 = T.d_raw[r + 1];
        // g2 as operand A: features g + 8 j of the two rows
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = S.wh[warp][8 * j + g];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            h2[j][i] = T.hidden[r + i][32 + 8 * j + g];
            const float z = h2[j][i] > 0.0f ? head_grad(w, i ? g1 : g0) : 0.0f;
            sb2[j] += z;
            split3(z, zh[j >> 1][(j & 1) + 2 * i], zl[j >> 1][(j & 1) + 2 * i]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uint32_t bh[2][2], bl[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) split3(T.hidden[r + i][8 * (j + u) + g], bh[u][i], bl[u][i]);
        float c[2][2][4];
        weight_products(c, zh, zl, bh, bl);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[m][j + u][k] += c[u][m][k];
      }
      // the heads: rows of A are features of [h2 | gamma(d)], columns of B the
      // channels. Direction base g < 6 (coordinate g / 2, octave 2 (g % 2)): tile 2
      // its sine and cosine, tile 3 those of the octave above; rows 6 and 7 hold
      // u0, u1, u2 and 1.
      uint32_t gh[2], gl[2];
      float v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        split3(g < 4 ? reinterpret_cast<const float*>(&T.d_raw[r + i])[g & 3] : 0.0f, gh[i], gl[i]);
        const float* e = &T.v[3 * (r + i)];
        two_octaves(e[g < 6 ? g >> 1 : g - 6], g & 1 ? 4.0f : 1.0f, v[i]);
        if (g >= 6) {
          v[i][0] = e[g - 6];
          v[i][2] = g == 6 ? e[2] : 1.0f;
          v[i][1] = v[i][3] = 0.0f;
        }
      }
#pragma unroll
      for (int m0 = 0; m0 < 4; m0 += 2) {
        uint32_t fh[2][4], fl[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              split3(m0 == 0 ? h2[2 * m + k][i] : v[i][2 * m + k], fh[m][2 * i + k], fl[m][2 * i + k]);
        float c[2][4];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int m = 0; m < 2; ++m) mma_from(p == 0, c[m], p == 0 ? fl[m] : fh[m], p == 1 ? gl : gh);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) ah[m0 + m][k] += c[m][k];
      }
    }
    __syncwarp();                            // this stage may be overwritten
  }
  G -= O_W2;                                 // by the blob's offsets below
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        G[O_W2 + (16 * m + g + 8 * (k >> 1)) * 32 + 8 * j + 2 * t + (k & 1)] = acc[m][j][k];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float s = sb2[j];
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (t == 0) G[O_B2 + 8 * j + g] = s;
  }
  if (t < 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = 2 * t + (k & 1), half = k >> 1;         // channel; row g or g + 8 of the tile
#pragma unroll
      for (int m = 0; m < 2; ++m)
        G[ch < 3 ? O_WC + ch * 59 + 16 * m + 8 * half + g : O_WS + 16 * m + 8 * half + g] = ah[m][k];
      const int col = O_WC + ch * 59 + 32;
      if (ch < 3 && g < 6) {
        G[col + 3 + 12 * half + 4 * (g >> 1) + 2 * (g & 1)] = ah[2][k];
        G[col + 3 + 12 * half + 4 * (g >> 1) + 2 * (g & 1) + 1] = ah[3][k];
      } else if (half == 0) {
        if (ch < 3 && g >= 6) G[col + g - 6] = ah[2][k];
        if (ch < 3 && g == 6) G[col + 2] = ah[3][k];
        if (g == 7) G[ch < 3 ? O_BC + ch : O_BS] = ah[3][k];
      }
    }
  }
}

// A cell whose tiles all lie in one warp's range is written by that warp; the
// parts of a cell that spans ranges go to the workspace (slot 0 of a warp: the
// part at its range's start, slot 1: one that begins inside) and are summed in
// warp order by cells_join_kernel, so no result depends on timing.
__global__ void __launch_bounds__(CB_THREADS, 1) cells_backward_kernel(CellsBackwardArgs P) {
  extern __shared__ __align__(16) uint8_t cells_sm[];
  CellsBackwardShared& S = *reinterpret_cast<CellsBackwardShared*>(cells_sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cudaTriggerProgrammaticLaunchCompletion();
  unit_prefix<CB_THREADS>(P.offset, P.n, P.n_cells, CB_ROWS, S.first);
  if (blockIdx.x == 0)
    for (int c = tid; c <= P.n_cells; c += CB_THREADS) P.first_out[c] = S.first[c];
  const bool role_a = warp < CB_A;
  const int W = gridDim.x * (role_a ? CB_A : CB_B);
  const int w = role_a ? blockIdx.x * CB_A + warp : blockIdx.x * CB_B + warp - CB_A;
  const int units = S.first[P.n_cells], per = (units + W - 1) / W;
  const int begin = (int)min((int64_t)w * per, (int64_t)units), end = min(units, begin + per);
  for (int unit = begin; unit < end;) {
    const int cell = cell_of(S.first, P.n_cells, unit);
    const int u0 = S.first[cell] + 1, u1 = S.first[cell + 1], stop = min(end, max(u1, unit + 1));   // its tiles: [u0, u1)
    unit = max(unit, u0);
    const int64_t cell_begin = min(max((int64_t)P.offset[cell], (int64_t)0), P.n);
    const int64_t cell_end = min(max((int64_t)P.offset[cell + 1], (int64_t)0), P.n);
    const int64_t row0 = cell_begin + (int64_t)(unit - u0) * CB_ROWS;
    if (unit < stop && row0 < cell_end) {
      const float* __restrict__ W2 = P.cell_w + (int64_t)cell * CELL_NP;
      __syncwarp();                          // the previous cell's fragments are no longer read
      S.wh[warp][lane] = make_float4(__ldg(W2 + O_WC + lane), __ldg(W2 + O_WC + 59 + lane),
                                     __ldg(W2 + O_WC + 118 + lane), __ldg(W2 + O_WS + lane));
      __syncwarp();
      const bool whole = u0 >= begin && u1 <= end;
      const int64_t slot = (int64_t)w * 2 + (u0 > begin ? 1 : 0);
      if (role_a)
        backward_w1(P, S, warp, lane, W2, row0, cell_end, stop - unit,
                    whole ? P.grad + (int64_t)cell * CELL_NP : P.parts_a + slot * CB_NA);
      else
        backward_w2(P, S, warp, lane, row0, cell_end, stop - unit,
                    whole ? P.grad + (int64_t)cell * CELL_NP + O_W2 : P.parts_b + slot * CB_NB);
    }
    unit = stop;
  }
}

// One CTA per cell: nothing where one warp wrote it, zeros where it has no rows,
// the sum of its parts in warp order where several did; for each role. `first` and
// the parts are written while this kernel may already run: no non-coherent loads.
template <int N, int WARPS>
__device__ __forceinline__ void join_parts(int u0, int u1, int units, int ctas, const float* parts,
                                           float* __restrict__ out) {
  const int per = (units + ctas * WARPS - 1) / (ctas * WARPS), w0 = u0 / per, w1 = (u1 - 1) / per;
  if (w0 == w1) return;
  constexpr int Q = (N + 255) / 256;
  const float* p = parts + ((int64_t)w0 * 2 + (u0 > w0 * per ? 1 : 0)) * N + threadIdx.x;
  if (gridDim.y > 1) {
    for (int i = blockIdx.y; i < Q; i += gridDim.y) {
      if (256 * i + (int)threadIdx.x >= N) break;
      float s = __ldcs(p + 256 * i);
      const float* q = parts + (int64_t)(w0 + 1) * 2 * N + threadIdx.x + 256 * i;
#pragma unroll 8
      for (int w = w0 + 1; w <= w1; ++w, q += 2 * N) s += __ldcs(q);
      out[256 * i + threadIdx.x] = s;
    }
    return;
  }
  float s[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) s[i] = 256 * i + (int)threadIdx.x < N ? __ldcs(p + 256 * i) : 0.0f;
#pragma unroll 2
  for (int w = w0 + 1; w <= w1; ++w) {
    p = parts + (int64_t)w * 2 * N + threadIdx.x;
#pragma unroll
    for (int i = 0; i < Q; ++i) s[i] += 256 * i + (int)threadIdx.x < N ? __ldcs(p + 256 * i) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (256 * i + (int)threadIdx.x < N) out[256 * i + threadIdx.x] = s[i];
}
__global__ void __launch_bounds__(256)
cells_join_kernel(const int32_t* __restrict__ offset, int64_t n, const int* first, int n_cells, int ctas,
                  const float* parts_a, const float* parts_b, float* __restrict__ grad) {
  const int cell = blockIdx.x;
  float* __restrict__ G = grad + (int64_t)cell * CELL_NP;
  const int64_t lo = min(max((int64_t)offset[cell], (int64_t)0), n), hi = min(max((int64_t)offset[cell + 1], (int64_t)0), n);
  if (hi <= lo && blockIdx.y == 0) {         // a blob starts at any float: 16-byte stores from its first 16-byte boundary
    const int head = (int)((0 - (uintptr_t)G) % 16 / 4), vecs = (CELL_NP - head) / 4;
    for (int q = threadIdx.x; q < vecs; q += 256)
      reinterpret_cast<float4*>(G + head)[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int rest = CELL_NP - 4 * vecs;     // before the vectors and after them
    if ((int)threadIdx.x < rest) G[(int)threadIdx.x < head ? threadIdx.x : threadIdx.x + 4 * vecs] = 0.0f;
  }
  cudaGridDependencySynchronize();           // the gradients and their parts; the zeros did not need them
  if (hi <= lo) return;
  const int u0 = __ldcg(first + cell) + 1, u1 = __ldcg(first + cell + 1), units = __ldcg(first + n_cells);
  if (u0 >= u1) return;
  join_parts<CB_NA, CB_A>(u0, u1, units, ctas, parts_a, G);
  join_parts<CB_NB, CB_B>(u0, u1, units, ctas, parts_b, G + O_W2);
}

}  // namespace

cudaError_t launch_cells_forward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                 int n_cells, const float* cell_w, float* raw, float* hidden,
                                 cudaStream_t st) {
  const size_t sm = sizeof(CellsForwardShared);
  cudaError_t e = cudaFuncSetAttribute(cells_forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (n + CF_ROWS - 1) / CF_ROWS + 2 * (n_cells < n ? n_cells : n);   // units at most
  constexpr int64_t most = 148 * CF_PER_SM;
  const unsigned grid = (unsigned)(tiles < most ? tiles : most);
  cells_forward_kernel<<<grid, CF_THREADS, sm, st>>>(x, d, n, offset, n_cells, cell_w, raw, hidden);
  return cudaGetLastError();
}

// [first EXPERT_MAX + 1 ints, padded][ctas * CB_A][2][CB_NA], [ctas * CB_B][2][CB_NB] floats
constexpr int64_t CB_FIRST_BYTES = (EXPERT_MAX + 1 + 3) / 4 * 16;
int64_t cells_backward_workspace(int64_t n, int n_cells) {
  return CB_FIRST_BYTES + (backward_ctas(n, n_cells) * 2 * (CB_A * CB_NA + CB_B * CB_NB) * 4 + 15) / 16 * 16;
}

cudaError_t launch_cells_backward(const float* x, const float* d, int64_t n, const int32_t* offset,
                                  int n_cells, const float* cell_w, const float* hidden,
                                  const float* d_raw, float* grad, void* work, cudaStream_t st) {
  const size_t sm = sizeof(CellsBackwardShared);
  cudaError_t e = cudaFuncSetAttribute(cells_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  const int ctas = (int)backward_ctas(n, n_cells);
  int* first = (int*)work;
  float* parts_a = (float*)((char*)work + CB_FIRST_BYTES);
  float* parts_b = parts_a + (int64_t)ctas * CB_A * 2 * CB_NA;
  const CellsBackwardArgs P{x, d, n, offset, n_cells, cell_w, hidden, d_raw, grad, first, parts_a, parts_b};
  cells_backward_kernel<<<ctas, CB_THREADS, sm, st>>>(P);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Few cells have many parts each: their sums are cut into up to eight slices of
  // parameters (20,000 rows of 64 cells: 26 us, 35 without).
  constexpr int CB_SLICES = (CB_NA + 255) / 256;
  const int slices = n_cells >= 592 ? 1 : 592 / n_cells < CB_SLICES ? 592 / n_cells : CB_SLICES;
  return launch_early(cells_join_kernel, dim3(n_cells, slices), 256, 0, st, offset, n, (const int*)first, n_cells, ctas,
                      (const float*)parts_a, (const float*)parts_b, grad);
}

}  // namespace nerfb
