// The residual norm: a block's result is normed, gated, scaled and added to the residual stream, and the sum is
// normed for the next block, forward and backward.
//
//   u = N(f; w1, b1) (or f),  t = act(gate) u,  z' = z + scale t,  y = N(z'; w2, b2)
//   N(x; w, b) = xh w + b,  xh = (x - mu) rstd,  rstd = (mean((x - mu)^2) + eps)^(-1/2)       (rms: mu = 0)
//   D = dz' + N'(dy w2; zh)                     the gradient of z', and of z
//   dgate = D scale u act'(gate),  du = D scale act(gate),  df = N'(du w1; fh) (or du)
//   N'(d; xh) = rstd (d - mean d - xh mean(d xh))                                             (rms: without mean d)
//   dscale = sum D t,  dw1 = sum du fh,  db1 = sum du,  dw2 = sum dy zh,  db2 = sum dy         over the rows
//
// Bound by memory, and by instructions where rows are narrow: five arrays of rows forward, eight backward, each once.  The
// backward call forms z' again from f, z and
// the gate (as many bytes as reading z' would cost, and not rounded).  A row lies in the registers of `tpr` threads (a power
// of two: part of a warp, a warp, or the block), C columns each, in vectors of V.  The parameters stand in shared memory in
// float32, in the order in which the threads read them (read from L1 in their own type and converted again for every row they
// made up a third of the instructions).  A mean of squares is taken of differences from the mean, in a
// second sweep over the registers.  The next rows are asked for while the present ones are worked on.  The five sums over the
// rows stay in registers, then go through the block in a fixed order, then over the blocks in a second kernel: no
// atomics.
//
// Widths that no vector divides: row r starts (r ld) mod V elements behind a 16-byte boundary, which repeats every `classes`
// rows.  A block takes the rows of one class, so that its threads keep their columns: vector i of a row starts `shift`
// columns before column i V.  The first and last vector reach into the neighbouring rows: they are read whole (but for the first
// and last rows of all) and what is not the row's is dropped when its values are needed, not at the load, which would
// wait for memory there and then (backward, 5003 x 1001: 64 us a call with elements loaded one by one), and are written
// element by element.  Arrays whose
// rows do not all start at the same place behind a boundary are moved element by element throughout (V = 1: neighbouring threads
// have neighbouring columns), and rows of more than kWidest columns take the *_any kernels, which read a row several times.
//
// Measured, forward and backward together, against the copy rate of 6.8 TB/s: 1,000,000 x 64 bfloat16 with a gate 350 us (0.70;
// forward 101, 0.93; backward bound by its 140 instructions a vector and row at 16 warps a multiprocessor, whose registers hold the sums),
// 5003 x 1001 float16 62 us (0.31: a few rows a group, one sum after another).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "sla_act.cuh"
#include "sla_common.cuh"
#include "sla_host.h"
#include "sla_net.cuh"

namespace sla {

constexpr int kNormBlock = 256;    // threads of a block while a row takes no more
constexpr int kNormThreads = 512;  // of a block that shares one row
constexpr int kWidest = kNormThreads * 16;
constexpr int kNormSums = 5;       // dscale, dw1, db1, dw2, db2
constexpr int kAnyParts = 16;      // parts of the rows of the *_any column sums

enum GateAct { kNoGate = -1, kGateNone = 0, kGateSigmoid = 1, kGateSilu = 2 };

struct ResNormArgs {
  int64_t rows;
  int64_t width;
  int tpr;
  int rms, post, act;
  int classes, shift, step;    // rows of one class start (shift + class * step) mod V behind a vector's boundary
  float eps;
  const void *f, *z, *gate;    // T [rows][ld]
  int64_t ldf, ldz, ldg;
  const void *scale, *w1, *b1, *w2, *b2;  // P [width] or NULL: 1, 1, 0, 1, 0
  void *znew, *y;              // T [rows][width]; y NULL: no second norm
  uint32_t bf, bz, bg, bdz, bdy, bw;  // bytes between the rows of f, z, gate, dz, dy and of the results
  float4 *stats;               // [rows]: mean and rstd of f's norm and of z's, or NULL (forward)
  const void *dz, *dy;         // T [rows][ld] or NULL: zero
  int64_t lddz, lddy;
  void *df, *dz_in, *dgate;    // T [rows][width] or NULL
  float *parts;                // [gridDim.x][kNormSums][width], or NULL
  float *row_sums;             // *_any: [2][rows] means of dy w2 and of dy w2 zh
};

// vec: p.classes, p.shift and p.step say how the rows of all arrays lie; else they are moved element by element.
template <typename T, typename P>
cudaError_t resnorm_forward(ResNormArgs p, bool vec, cudaStream_t st);
// grid: blocks, each of which leaves partial sums (a multiple of the classes).
template <typename T, typename P>
cudaError_t resnorm_backward(ResNormArgs p, bool vec, int grid, cudaStream_t st);

// How a call's rows are laid over threads: columns a thread, threads a row, threads a block.
struct ResNormPlan {
  int columns, tpr, block;  // columns 0: *_any
};

inline ResNormPlan resnorm_plan(int64_t width) {
  const int64_t reach = width % 8 ? width + 7 : width;  // a row that starts behind a boundary reaches into one vector more
  if (reach > kWidest) return {0, kNormThreads, kNormThreads};
  const int columns = reach > kNormThreads * 8 ? 16 : 8;
  int tpr = 1;
  while (tpr * columns < reach) tpr <<= 1;
  return {columns, tpr, std::max(tpr, kNormBlock)};
}

// Blocks that fill the GPU with `threads` a multiprocessor, in whole sets of classes, no more than there are rows for.
inline int resnorm_grid(const ResNormPlan &pl, int64_t rows, int64_t rows_a_turn, int classes, int threads) {
  const int64_t most = (int64_t)sm_count() * std::max(1, threads / pl.block);
  const int64_t need = ((rows + classes - 1) / classes + rows_a_turn - 1) / rows_a_turn;
  return (int)(std::max<int64_t>(1, std::min(most / classes, need)) * classes);
}

// ------------------------------------------------------------------ pieces

// Sums over the tpr threads of a group, the same values in each of them.  `slot` (16 K floats) must not be in
// use by an earlier sum that a thread still reads.  Groups of several warps wait for their own alone.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int tpr, float *slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (tpr > o) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
  if (tpr <= 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp & ~(warps - 1);
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) slot[k * 16 + warp] = v[k];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / tpr), "r"(tpr) : "memory");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? slot[k * 16 + first + lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
}

// A thread's columns: C / V vectors, vector i from column (t + i tpr) V - shift on.  Edge: there are vectors that lie in the row
// in part (rows that start or end behind a boundary).
template <int V, int C, bool Edge>
struct Columns {
  static constexpr int n = C / V;
  int t, tpr, width, shift;
  uint32_t whole, some;  // vectors that lie in the row, or at least reach into it
  __device__ __forceinline__ Columns(int t_, int tpr_, int width_, int shift_) : t(t_), tpr(tpr_), width(width_), shift(shift_) {
    whole = some = 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = first(i);
      whole |= (c >= 0 && c + V <= width ? 1u : 0u) << i;
      some |= (c + V > 0 && c < width ? 1u : 0u) << i;
    }
  }
  __device__ __forceinline__ int first(int i) const { return (t + i * tpr) * V - shift; }
  __device__ __forceinline__ int column(int j) const { return first(j / V) + j % V; }
  __device__ __forceinline__ bool inside(int j) const { return column(j) >= 0 && column(j) < width; }
  __device__ __forceinline__ bool full() const { return whole == (1u << n) - 1; }
  // What lies outside of the row becomes zero.
  __device__ __forceinline__ void mask(float2 (&v)[C / 2]) const {
    if (full()) return;
#pragma unroll
    for (int j = 0; j < C; j += 2) {
      const bool in0 = Edge ? inside(j) : whole >> (j / V) & 1, in1 = Edge ? inside(j + 1) : whole >> ((j + 1) / V) & 1;
      v[j / 2] = make_float2(in0 ? v[j / 2].x : 0.f, in1 ? v[j / 2].y : 0.f);
    }
  }
};

// C columns of a row as loaded.
template <typename T, int V, int C, bool Edge>
struct RowPart {
  static constexpr int n = C / V;
  Pack<T, V> v[n];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i].v[k] = from_f32<T>(0.f);
  }
  // beside: the rows around this one cover what its first and last vectors read of them
  __device__ __forceinline__ void load(const T *row, const Columns<V, C, Edge> &q, bool there, bool beside) {
    const uint32_t may = Edge && beside ? q.some : q.whole;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = q.first(i);
      if (there && (may >> i & 1)) {
        v[i] = *reinterpret_cast<const Pack<T, V> *>(row + c);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i].v[k] = from_f32<T>(0.f);
        if (Edge && there && (q.some >> i & 1)) {
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (c + k >= 0 && c + k < q.width) v[i].v[k] = row[c + k];
        }
      }
    }
  }
  __device__ __forceinline__ void values(float2 (&o)[C / 2], const Columns<V, C, Edge> &q) const {
    unpack(o);
    if (Edge) q.mask(o);
  }
  __device__ __forceinline__ void unpack(float2 (&o)[C / 2]) const {
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
      for (int i = 0; i < n; ++i)
#pragma unroll
        for (int k = 0; k < V; k += 2)
          o[(i * V + k) / 2] = unpair16(*reinterpret_cast<const uint32_t *>(&v[i].v[k]), T{});
    } else {
#pragma unroll
      for (int j = 0; j < C; j += 2) o[j / 2] = f2(to_f32(v[j / V].v[j % V]), to_f32(v[(j + 1) / V].v[(j + 1) % V]));
    }
  }
};

template <typename T, int V, int C, bool Edge>
__device__ __forceinline__ void store_part(T *row, const float2 (&o)[C / 2], const Columns<V, C, Edge> &q) {
#pragma unroll
  for (int i = 0; i < C / V; ++i) {
    const int c = q.first(i);
    if (!((Edge ? q.some : q.whole) >> i & 1)) continue;
    Pack<T, V> w;
    if constexpr (V == 1) {
      w.v[0] = from_f32<T>(i % 2 ? o[i / 2].y : o[i / 2].x);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < V; k += 2)
        *reinterpret_cast<uint32_t *>(&w.v[k]) = pair16(o[(i * V + k) / 2].x, o[(i * V + k) / 2].y, T{});
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 2) w.v[k] = o[(i * V + k) / 2].x, w.v[k + 1] = o[(i * V + k) / 2].y;
    }
    if (!Edge || (q.whole >> i & 1)) {
      *reinterpret_cast<Pack<T, V> *>(row + c) = w;
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c + k >= 0 && c + k < q.width) row[c + k] = w.v[k];
    }
  }
}

// Parameters in shared memory ([K][C / 4][tpr]): four columns of a thread beside those of the next thread, zero outside of the
// row.  Bit k of `ones`: what parameter k is where it is absent.  All K are asked for at once: a single row waits once.
template <typename P, int V, int C, int K>
__device__ __forceinline__ void stage_params(float4 *sm, const void *const (&p)[K], uint32_t ones, int tpr, int width,
                                             int shift) {
  const int each = C / 4 * tpr;
  for (int i = threadIdx.x; i < each; i += blockDim.x) {
    const int t = i & (tpr - 1), h = i / tpr;
    float e[K][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (t + (4 * h + j) / V * tpr) * V + (4 * h + j) % V - shift;
      const bool in = c >= 0 && c < width;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        e[k][j] = in && (ones >> k & 1) ? 1.f : 0.f;
        if (in && p[k]) e[k][j] = to_f32(((const P *)p[k])[c]);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) sm[k * each + i] = make_float4(e[k][0], e[k][1], e[k][2], e[k][3]);
  }
}
template <int C>
__device__ __forceinline__ void param_part(const float4 *sm, int t, int tpr, float2 (&o)[C / 2]) {
#pragma unroll
  for (int h = 0; h < C / 4; ++h) {
    const float4 q = sm[h * tpr + t];
    o[2 * h] = f2(q.x, q.y), o[2 * h + 1] = f2(q.z, q.w);
  }
}

__device__ __forceinline__ float2 both(float v) { return f2(v, v); }

// Row `row` of rows `bytes` apart: one wide multiply-add.
template <typename T>
__device__ __forceinline__ T *row_at(const void *base, uint32_t row, uint32_t bytes) {
  return (T *)((char *)const_cast<void *>(base) + (uint64_t)row * bytes);
}

// act(g) and, if asked for, act'(g).
template <bool Derivative>
__device__ __forceinline__ void gate_act(int act, float2 g, float2 &a, float2 &da) {
  if (act == kGateNone) {
    a = g;
    if (Derivative) da = both(1.f);
    return;
  }
  // e = exp(-g); e s is 1 - s, right relative to itself.  Where e is infinite s is zero, and so is what 1 - s multiplies.
  const float2 m = mul2(g, both(-1.4426950408889634f));
  const float2 e = f2(ex2_approx(m.x), ex2_approx(m.y));
  const float2 d = add2(e, both(1.f)), s = f2(rcp_approx(d.x), rcp_approx(d.y));
  a = act == kGateSigmoid ? s : mul2(g, s);
  if (Derivative) {
    const float2 r = mul2(f2(min_nan(e.x, FLT_MAX), min_nan(e.y, FLT_MAX)), s);  // never infinity times zero
    da = act == kGateSigmoid ? mul2(s, r) : fma2(a, r, s);
  }
}

// The rows of v become (v - mu) rstd.
template <int V, int C, bool Edge, int R>
__device__ __forceinline__ void norm_rows(float2 (&v)[R][C / 2], const Columns<V, C, Edge> &q, bool rms, float inv, float eps,
                                          float *slot0, float *slot1, float (&mu)[R], float (&rstd)[R]) {
  constexpr int H = C / 2;
  float s[R];
  if (!rms) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a = both(0.f);
#pragma unroll
      for (int j = 0; j < H; ++j) a = add2(a, v[r][j]);
      s[r] = a.x + a.y;
    }
    row_sums(s, q.tpr, slot0);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mu[r] = rms ? 0.f : s[r] * inv;
    if (!rms) {
#pragma unroll
      for (int j = 0; j < H; ++j) v[r][j] = add2(v[r][j], both(-mu[r]));
      q.mask(v[r]);
    }
    float2 a = both(0.f);
#pragma unroll
    for (int j = 0; j < H; ++j) a = fma2(v[r][j], v[r][j], a);
    s[r] = a.x + a.y;
  }
  row_sums(s, q.tpr, slot1);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    rstd[r] = rsqrtf(s[r] * inv + eps);  // 2 units in the last place
#pragma unroll
    for (int j = 0; j < H; ++j) v[r][j] = mul2(v[r][j], both(rstd[r]));
  }
}

// Which rows a block's groups take: group g of a block row `row`, `step` rows on in the next turn; `next` between the rows of
// a bundle of R.
struct Turns {
  uint32_t lead, row, step, next;  // (there are less than 2^31 rows)
  template <int R>
  __device__ __forceinline__ static Turns of(const ResNormArgs &p, int groups, std::integral_constant<int, R>) {
    Turns w;
    const int cls = blockIdx.x % p.classes;
    w.next = groups * p.classes;
    w.lead = (blockIdx.x / p.classes) * R * w.next + cls;
    w.row = w.lead + threadIdx.x / p.tpr * p.classes;
    w.step = (gridDim.x / p.classes) * R * w.next;
    return w;
  }
};

// ------------------------------------------------------------------ kernels

// R: rows of a group at a time, whose sums go together and which share what is read of the parameters.
template <typename T, typename P, int V, int C, bool Edge, int R>
__global__ void __launch_bounds__(kNormThreads, 1) resnorm_forward_rows(const __grid_constant__ ResNormArgs p) {
  constexpr int H = C / 2;
  extern __shared__ float4 params[];  // [5][C / 4][tpr]: scale, w1, b1, w2, b2
  __shared__ float slots[2][4][R * 16];
  const int tpr = p.tpr, width = (int)p.width, groups = blockDim.x / tpr;
  const int shift = V > 1 ? (p.shift + (blockIdx.x % p.classes) * p.step) % V : 0;
  const Columns<V, C, Edge> q(threadIdx.x & (tpr - 1), tpr, width, shift);
  const float inv = 1.f / (float)width;
  const int each = C / 4 * tpr;
  const Turns w = Turns::of(p, groups, std::integral_constant<int, R>{});
  RowPart<T, V, C, Edge> rf[R], rz[R], rg[R];
  const uint32_t rows = (uint32_t)p.rows, margin = V / width + 1;
  auto ask = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r, row += w.next) {
      const bool there = row < rows, beside = row >= margin && row + margin < rows;
      rf[r].load(row_at<T>(p.f, row, p.bf), q, there, beside);
      if (p.act != kNoGate) rg[r].load(row_at<T>(p.gate, row, p.bg), q, there, beside);
      rz[r].load(row_at<T>(p.z, row, p.bz), q, there, beside);
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) rg[r].clear();
  ask(w.row);
  const void *const from[5] = {p.scale, p.w1, p.b1, p.w2, p.b2};
  stage_params<P, V, C, 5>(params, from, 0b01011, tpr, width, shift);
  __syncthreads();
  int turn = 0;  // the slots alternate, so a turn's sums never meet the previous one's reads
  // every thread of a block makes the same number of turns (the sums need whole warps and blocks)
  uint32_t row = w.row;
  for (uint32_t lead = w.lead; lead < rows; lead += w.step, row += w.step, turn ^= 1) {
    float2 v[R][H], z[R][H], a[R][H], k[H], k2[H];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rf[r].values(v[r], q);
      rz[r].values(z[r], q);
      if (p.act != kNoGate) rg[r].values(a[r], q);
    }
    if (lead + w.step < rows) ask(row + w.step);
    if (p.act != kNoGate)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < H; ++j) {
          float2 none;
          gate_act<false>(p.act, a[r][j], a[r][j], none);
        }
    float mu1[R] = {}, rs1[R] = {}, mu2[R] = {}, rs2[R] = {};
    if (p.post) {
      norm_rows<V, C, Edge, R>(v, q, p.rms, inv, p.eps, slots[turn][0], slots[turn][1], mu1, rs1);
      param_part<C>(params + each, q.t, tpr, k);
      param_part<C>(params + 2 * each, q.t, tpr, k2);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < H; ++j) v[r][j] = fma2(v[r][j], k[j], k2[j]);
    }
    param_part<C>(params, q.t, tpr, k);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (p.act != kNoGate)
#pragma unroll
        for (int j = 0; j < H; ++j) v[r][j] = mul2(v[r][j], a[r][j]);
#pragma unroll
      for (int j = 0; j < H; ++j) v[r][j] = fma2(v[r][j], k[j], z[r][j]);
      const uint32_t at = row + r * w.next;
      if (at < rows) store_part<T, V, C, Edge>(row_at<T>(p.znew, at, p.bw), v[r], q);
    }
    if (p.y) {
      norm_rows<V, C, Edge, R>(v, q, p.rms, inv, p.eps, slots[turn][2], slots[turn][3], mu2, rs2);
      param_part<C>(params + 3 * each, q.t, tpr, k);
      param_part<C>(params + 4 * each, q.t, tpr, k2);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < H; ++j) v[r][j] = fma2(v[r][j], k[j], k2[j]);
        const uint32_t at = row + r * w.next;
        if (at < rows) store_part<T, V, C, Edge>(row_at<T>(p.y, at, p.bw), v[r], q);
      }
    }
    if (p.stats && q.t == 0)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t at = row + r * w.next;
        if (at >= rows) continue;
        p.stats[at] = make_float4(mu1[r], rs1[r], mu2[r], rs2[r]);
      }
  }
}

template <typename T, typename P, int V, int C, bool Edge>
__global__ void __launch_bounds__(kNormThreads, 1) resnorm_backward_rows(const __grid_constant__ ResNormArgs p) {
  constexpr int H = C / 2;
  extern __shared__ float4 params[];  // [4][C / 4][tpr]: scale, w1, b1, w2; then, with more than one group, [kNormSums][width]
  __shared__ float slots[2][2][32];
  grid_dependency_launch();  // the sums over blocks start as multiprocessors become free, and wait there
  const int tpr = p.tpr, width = (int)p.width, groups = blockDim.x / tpr;
  const int shift = V > 1 ? (p.shift + (blockIdx.x % p.classes) * p.step) % V : 0;
  const Columns<V, C, Edge> q(threadIdx.x & (tpr - 1), tpr, width, shift);
  const float inv = 1.f / (float)width;
  const int each = C / 4 * tpr;
  const Turns w = Turns::of(p, groups, std::integral_constant<int, 1>{});
  float2 sums[kNormSums][H];
#pragma unroll
  for (int k = 0; k < kNormSums; ++k)
#pragma unroll
    for (int j = 0; j < H; ++j) sums[k][j] = both(0.f);
  const uint32_t rows = (uint32_t)p.rows, margin = V / width + 1;  // (below 2^31)
  RowPart<T, V, C, Edge> rf, rz, rg, rdz, rdy;
  float4 st;
  rg.clear();
  rdz.clear();
  rdy.clear();
  auto ask = [&](uint32_t r) {
    const bool there = r < rows, beside = r >= margin && r + margin < rows;
    rf.load(row_at<T>(p.f, r, p.bf), q, there, beside);
    if (p.act != kNoGate) rg.load(row_at<T>(p.gate, r, p.bg), q, there, beside);
    rz.load(row_at<T>(p.z, r, p.bz), q, there, beside);
    if (p.dy) rdy.load(row_at<T>(p.dy, r, p.bdy), q, there, beside);
    if (p.dz) rdz.load(row_at<T>(p.dz, r, p.bdz), q, there, beside);
    st = there ? p.stats[r] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  ask(w.row);
  const void *const from[4] = {p.scale, p.w1, p.b1, p.w2};
  stage_params<P, V, C, 4>(params, from, 0b1011, tpr, width, shift);
  __syncthreads();
  int turn = 0;
  uint32_t row = w.row;
  for (uint32_t lead = w.lead; lead < rows; lead += w.step, row += w.step, turn ^= 1) {
    // t = act(gate) u;  sa = scale act(gate), by which D becomes du;  sg = scale u act'(gate), by which it becomes dgate
    float2 fh[H], t[H], sa[H], sg[H], d[H], k[H];
    const float mu1 = st.x, rs1 = st.y, mu2 = st.z, rs2 = st.w;
    rf.values(fh, q);
    if (p.post) {
#pragma unroll
      for (int j = 0; j < H; ++j) fh[j] = mul2(add2(fh[j], both(-mu1)), both(rs1));
      q.mask(fh);  // where there is no row, (0 - mean) rstd may pass the largest float32
      param_part<C>(params + each, q.t, tpr, k);
      param_part<C>(params + 2 * each, q.t, tpr, t);
#pragma unroll
      for (int j = 0; j < H; ++j) t[j] = fma2(fh[j], k[j], t[j]);
    } else {
#pragma unroll
      for (int j = 0; j < H; ++j) t[j] = fh[j];
    }
    param_part<C>(params, q.t, tpr, k);
    if (p.act != kNoGate) {
      float2 g[H];
      rg.values(g, q);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        float2 a, da;
        gate_act<true>(p.act, g[j], a, da);
        sg[j] = mul2(mul2(k[j], t[j]), da);
        sa[j] = mul2(k[j], a);
        t[j] = mul2(t[j], a);
      }
    } else {
#pragma unroll
      for (int j = 0; j < H; ++j) sg[j] = both(0.f), sa[j] = k[j];
    }
    rdz.values(d, q);
    if (p.dy) {
      float2 zh[H], dy[H];
      rz.values(zh, q);
      rdy.values(dy, q);
#pragma unroll
      for (int j = 0; j < H; ++j) zh[j] = mul2(add2(fma2(t[j], k[j], zh[j]), both(-mu2)), both(rs2));
      q.mask(zh);
      param_part<C>(params + 3 * each, q.t, tpr, k);
      float2 s1 = both(0.f), s2 = s1;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        sums[3][j] = fma2(dy[j], zh[j], sums[3][j]);
        sums[4][j] = add2(sums[4][j], dy[j]);
        dy[j] = mul2(dy[j], k[j]);
        s1 = add2(s1, dy[j]);
        s2 = fma2(dy[j], zh[j], s2);
      }
      if (lead + w.step < rows) ask(row + w.step);
      float s[2] = {s1.x + s1.y, s2.x + s2.y};
      row_sums(s, tpr, slots[turn][0]);
      const float m1 = p.rms ? 0.f : -s[0] * inv, m2 = -s[1] * inv;
#pragma unroll
      for (int j = 0; j < H; ++j)
        d[j] = fma2(fma2(zh[j], both(m2), add2(dy[j], both(m1))), both(rs2), d[j]);
    } else if (lead + w.step < rows) {
      ask(row + w.step);
    }
    const bool live = row < rows;
    if (live && p.dz_in) store_part<T, V, C, Edge>(row_at<T>(p.dz_in, row, p.bw), d, q);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      sums[0][j] = fma2(d[j], t[j], sums[0][j]);
      sg[j] = mul2(sg[j], d[j]);
      d[j] = mul2(d[j], sa[j]);
    }
    if (live && p.dgate) store_part<T, V, C, Edge>(row_at<T>(p.dgate, row, p.bw), sg, q);
    if (p.post) {
      param_part<C>(params + each, q.t, tpr, k);
      float2 s1 = both(0.f), s2 = s1;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        sums[1][j] = fma2(d[j], fh[j], sums[1][j]);
        sums[2][j] = add2(sums[2][j], d[j]);
        d[j] = mul2(d[j], k[j]);
        s1 = add2(s1, d[j]);
        s2 = fma2(d[j], fh[j], s2);
      }
      float s[2] = {s1.x + s1.y, s2.x + s2.y};
      row_sums(s, tpr, slots[turn][1]);
      const float m1 = p.rms ? 0.f : -s[0] * inv, m2 = -s[1] * inv;
#pragma unroll
      for (int j = 0; j < H; ++j) d[j] = mul2(fma2(fh[j], both(m2), add2(d[j], both(m1))), both(rs1));
    }
    if (live && p.df) store_part<T, V, C, Edge>(row_at<T>(p.df, row, p.bw), d, q);
  }
  if (!p.parts) return;
  float *to = p.parts + (int64_t)blockIdx.x * kNormSums * width, *cols = (float *)(params + 4 * each);
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < kNormSums; ++k)
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (q.inside(j)) to[k * width + q.column(j)] = j % 2 ? sums[k][j / 2].y : sums[k][j / 2].x;
    return;
  }
  // the groups of a warp by shuffles, then the warps one after another
  for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < kNormSums; ++k)
#pragma unroll
      for (int j = 0; j < H; ++j) {
        sums[k][j].x += __shfl_xor_sync(0xffffffffu, sums[k][j].x, o);
        sums[k][j].y += __shfl_xor_sync(0xffffffffu, sums[k][j].y, o);
      }
  const int size = tpr < 32 ? 32 : tpr;
  for (int from = 0; from < (int)blockDim.x; from += size) {
    if ((int)threadIdx.x >= from && (int)threadIdx.x < from + tpr)
#pragma unroll
      for (int k = 0; k < kNormSums; ++k)
#pragma unroll
        for (int j = 0; j < C; ++j)
          if (q.inside(j)) {
            const float s = j % 2 ? sums[k][j / 2].y : sums[k][j / 2].x;
            float *c = cols + k * width + q.column(j);
            *c = from ? *c + s : s;
          }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < kNormSums * width; c += blockDim.x) to[c] = cols[c];
}

// ------------------------------------------------------------------ rows of any width: a block a row, element by element

// What a column makes of f, z and the gate.
struct Element {
  float fh, u, a, da, sc, z;
};

template <typename T, typename P>
__device__ __forceinline__ Element element(const ResNormArgs &p, int64_t row, int64_t c, float mu1, float rs1) {
  Element e;
  e.fh = to_f32(((const T *)p.f)[row * p.ldf + c]);
  e.u = e.fh;
  if (p.post) {
    e.fh = (e.fh - mu1) * rs1;
    e.u = e.fh * (p.w1 ? to_f32(((const P *)p.w1)[c]) : 1.f) + (p.b1 ? to_f32(((const P *)p.b1)[c]) : 0.f);
  }
  e.a = 1.f, e.da = 0.f;
  if (p.act != kNoGate) {
    float2 a, da;
    gate_act<true>(p.act, both(to_f32(((const T *)p.gate)[row * p.ldg + c])), a, da);
    e.a = a.x, e.da = da.x;
  }
  e.sc = p.scale ? to_f32(((const P *)p.scale)[c]) : 1.f;
  e.z = to_f32(((const T *)p.z)[row * p.ldz + c]) + e.sc * (e.a * e.u);
  return e;
}

template <typename F>
__device__ __forceinline__ float sum_of_row(int64_t width, float *slot, F &&f) {
  float s[1] = {0.f};
  for (int64_t c = threadIdx.x; c < width; c += kNormThreads) s[0] += f(c);
  row_sums(s, kNormThreads, slot);
  return s[0];
}

template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads) resnorm_forward_any(const __grid_constant__ ResNormArgs p) {
  __shared__ float slots[4][16];
  const float inv = 1.f / (float)p.width;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float mu1 = 0.f, rs1 = 0.f, mu2 = 0.f, rs2 = 0.f;
    const T *f = (const T *)p.f + row * p.ldf;
    if (p.post) {
      if (!p.rms) mu1 = sum_of_row(p.width, slots[0], [&](int64_t c) { return to_f32(f[c]); }) * inv;
      rs1 = rsqrtf(sum_of_row(p.width, slots[1],
                              [&](int64_t c) {
                                const float d = to_f32(f[c]) - mu1;
                                return d * d;
                              }) * inv + p.eps);
    }
    for (int64_t c = threadIdx.x; c < p.width; c += kNormThreads)
      ((T *)p.znew)[row * p.width + c] = from_f32<T>(element<T, P>(p, row, c, mu1, rs1).z);
    if (p.y) {
      if (!p.rms)
        mu2 = sum_of_row(p.width, slots[2], [&](int64_t c) { return element<T, P>(p, row, c, mu1, rs1).z; }) * inv;
      rs2 = rsqrtf(sum_of_row(p.width, slots[3],
                              [&](int64_t c) {
                                const float d = element<T, P>(p, row, c, mu1, rs1).z - mu2;
                                return d * d;
                              }) * inv + p.eps);
      for (int64_t c = threadIdx.x; c < p.width; c += kNormThreads) {
        const float zh = (element<T, P>(p, row, c, mu1, rs1).z - mu2) * rs2;
        ((T *)p.y)[row * p.width + c] = from_f32<T>(zh * (p.w2 ? to_f32(((const P *)p.w2)[c]) : 1.f) +
                                                    (p.b2 ? to_f32(((const P *)p.b2)[c]) : 0.f));
      }
    }
    if (p.stats && threadIdx.x == 0) p.stats[row] = make_float4(mu1, rs1, mu2, rs2);
    __syncthreads();  // the slots are free again
  }
}

// D of a column, from the means m1 and m2 of dy w2 and dy w2 zh over its row; zh and dy too.
template <typename T, typename P>
__device__ __forceinline__ float stream_gradient(const ResNormArgs &p, const Element &e, int64_t row, int64_t c, float mu2,
                                                 float rs2, float m1, float m2, float &zh, float &dy) {
  zh = dy = 0.f;
  float d = p.dz ? to_f32(((const T *)p.dz)[row * p.lddz + c]) : 0.f;
  if (p.dy) {
    zh = (e.z - mu2) * rs2;
    dy = to_f32(((const T *)p.dy)[row * p.lddy + c]);
    d += rs2 * (dy * (p.w2 ? to_f32(((const P *)p.w2)[c]) : 1.f) - m1 - zh * m2);
  }
  return d;
}

template <typename T, typename P>
__global__ void __launch_bounds__(kNormThreads) resnorm_backward_any(const __grid_constant__ ResNormArgs p) {
  __shared__ float slots[4][16];
  const float inv = 1.f / (float)p.width;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float4 st = p.stats[row];
    const float mu1 = st.x, rs1 = st.y, mu2 = st.z, rs2 = st.w;
    float m1 = 0.f, m2 = 0.f, n1 = 0.f, n2 = 0.f, zh, dy;
    auto weighted = [&](int64_t c) {
      return to_f32(((const T *)p.dy)[row * p.lddy + c]) * (p.w2 ? to_f32(((const P *)p.w2)[c]) : 1.f);
    };
    if (p.dy) {
      if (!p.rms) m1 = sum_of_row(p.width, slots[0], weighted) * inv;
      m2 = sum_of_row(p.width, slots[1],
                      [&](int64_t c) { return weighted(c) * (element<T, P>(p, row, c, mu1, rs1).z - mu2) * rs2; }) * inv;
    }
    if (p.row_sums && threadIdx.x == 0) p.row_sums[row] = m1, p.row_sums[p.rows + row] = m2;
    auto inner = [&](const Element &e, int64_t c) {  // du w1
      return stream_gradient<T, P>(p, e, row, c, mu2, rs2, m1, m2, zh, dy) * e.sc * e.a *
             (p.w1 ? to_f32(((const P *)p.w1)[c]) : 1.f);
    };
    if (p.post && p.df) {
      if (!p.rms)
        n1 = sum_of_row(p.width, slots[2], [&](int64_t c) { return inner(element<T, P>(p, row, c, mu1, rs1), c); }) * inv;
      n2 = sum_of_row(p.width, slots[3],
                      [&](int64_t c) {
                        const Element e = element<T, P>(p, row, c, mu1, rs1);
                        return inner(e, c) * e.fh;
                      }) * inv;
    }
    for (int64_t c = threadIdx.x; c < p.width; c += kNormThreads) {
      const Element e = element<T, P>(p, row, c, mu1, rs1);
      const float d = stream_gradient<T, P>(p, e, row, c, mu2, rs2, m1, m2, zh, dy);
      const int64_t at = row * p.width + c;
      if (p.dz_in) ((T *)p.dz_in)[at] = from_f32<T>(d);
      if (p.dgate) ((T *)p.dgate)[at] = from_f32<T>(d * e.sc * e.u * e.da);
      if (p.df)
        ((T *)p.df)[at] = from_f32<T>(p.post ? rs1 * (inner(e, c) - n1 - e.fh * n2) : d * e.sc * e.a);
    }
    __syncthreads();
  }
}

// Partial sums over the rows of any width: block (32 columns, part of the rows).
template <typename T, typename P>
__global__ void __launch_bounds__(1024) resnorm_columns_any(const __grid_constant__ ResNormArgs p) {
  __shared__ float sm[kNormSums][32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * 32ll + lane;
  float s[kNormSums] = {};
  if (c < p.width)
    for (int64_t r = blockIdx.y * 32ll + wy; r < p.rows; r += gridDim.y * 32ll) {
      const float4 st = p.stats[r];
      const Element e = element<T, P>(p, r, c, st.x, st.y);
      float zh, dy;
      const float d = stream_gradient<T, P>(p, e, r, c, st.z, st.w, p.row_sums[r], p.row_sums[p.rows + r], zh, dy);
      const float du = d * e.sc * e.a;
      s[0] += d * (e.a * e.u);
      s[1] += du * e.fh;
      s[2] += du;
      s[3] += dy * zh;
      s[4] += dy;
    }
#pragma unroll
  for (int k = 0; k < kNormSums; ++k) sm[k][wy][lane] = s[k];
  __syncthreads();
  if (wy < kNormSums && c < p.width) {
    float a = 0.f;
    for (int i = 0; i < 32; ++i) a += sm[wy][i][lane];
    p.parts[((int64_t)blockIdx.y * kNormSums + wy) * p.width + c] = a;
  }
}

// ------------------------------------------------------------------ launches

template <typename K>
cudaError_t launch_resnorm(K kernel, const ResNormArgs &p, int grid, int block, size_t smem, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, block, smem, st>>>(p);
  return cudaGetLastError();
}

inline int any_grid(int64_t rows) { return (int)std::min<int64_t>(rows, sm_count() * 16); }

template <typename T, typename P>
cudaError_t resnorm_forward_as(ResNormArgs p, bool vec, cudaStream_t st) {
  const ResNormPlan pl = resnorm_plan(p.width);
  constexpr int V = 16 / sizeof(T);
  p.tpr = pl.tpr;
  if (!pl.columns) return launch_resnorm(resnorm_forward_any<T, P>, p, any_grid(p.rows), pl.block, 0, st);
  if (!vec) p.classes = 1, p.shift = p.step = 0;
  const int R = pl.columns == 8 && vec ? 2 : 1;
  const int grid = resnorm_grid(pl, p.rows, (int64_t)(pl.block / pl.tpr) * R, p.classes, 512);
  const size_t smem = 5 * sizeof(float) * (size_t)pl.tpr * pl.columns;
  const bool edge = vec && (p.shift || p.step || p.width % V);
#define SLA_RESNORM_FWD(V, C, EDGE, R) \
  launch_resnorm(resnorm_forward_rows<T, P, V, C, EDGE, R>, p, grid, pl.block, smem, st)
  if (pl.columns == 8)
    return !vec ? SLA_RESNORM_FWD(1, 8, false, 1) : edge ? SLA_RESNORM_FWD(V, 8, true, 2) : SLA_RESNORM_FWD(V, 8, false, 2);
  return !vec ? SLA_RESNORM_FWD(1, 16, false, 1) : edge ? SLA_RESNORM_FWD(V, 16, true, 1) : SLA_RESNORM_FWD(V, 16, false, 1);
#undef SLA_RESNORM_FWD
}

template <typename T, typename P>
cudaError_t resnorm_backward_as(ResNormArgs p, bool vec, int grid, cudaStream_t st) {
  const ResNormPlan pl = resnorm_plan(p.width);
  constexpr int V = 16 / sizeof(T);
  p.tpr = pl.tpr;
  if (!pl.columns) {
    const cudaError_t e = launch_resnorm(resnorm_backward_any<T, P>, p, any_grid(p.rows), pl.block, 0, st);
    if (e != cudaSuccess || !p.parts) return e;
    resnorm_columns_any<T, P><<<dim3((unsigned)((p.width + 31) / 32), grid), 1024, 0, st>>>(p);
    return cudaGetLastError();
  }
  if (!vec) p.classes = 1, p.shift = p.step = 0;
  const size_t smem = 4 * sizeof(float) * (size_t)pl.tpr * pl.columns +
                      (pl.block > pl.tpr && p.parts ? kNormSums * sizeof(float) * (size_t)p.width : 0);
  const bool edge = vec && (p.shift || p.step || p.width % V);
#define SLA_RESNORM_BWD(V, C, EDGE) launch_resnorm(resnorm_backward_rows<T, P, V, C, EDGE>, p, grid, pl.block, smem, st)
  if (pl.columns == 8)
    return !vec ? SLA_RESNORM_BWD(1, 8, false) : edge ? SLA_RESNORM_BWD(V, 8, true) : SLA_RESNORM_BWD(V, 8, false);
  return !vec ? SLA_RESNORM_BWD(1, 16, false) : edge ? SLA_RESNORM_BWD(V, 16, true) : SLA_RESNORM_BWD(V, 16, false);
#undef SLA_RESNORM_BWD
}

}  // namespace sla
