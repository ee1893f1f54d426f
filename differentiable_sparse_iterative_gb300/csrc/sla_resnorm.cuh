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
// Bound by memory: five arrays of rows forward, eight backward, each once.  The backward call forms z' again from f, z and
// the gate (as many bytes as reading z' would cost, and not rounded).  A row lies in the registers of `tpr` threads (a power
// of two: part of a warp, a warp, or the block), C columns each, in vectors of V; rows that no vector divides, or
// that start at no 16-byte boundary, are moved element by element in the same kernel (V = 1: neighbouring threads have
// neighbouring columns, so a warp's accesses stay whole).  A mean of squares is taken of differences from the mean, in a
// second sweep over the registers.  The next row is asked for while the present one is worked on.  The five sums over the rows
// stay in registers, then go through the block in a fixed order, then over the blocks in a second kernel: no
// atomics.  Rows of more than kWidest columns take the *_any kernels, which read a row several times.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

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
  int pvec;                    // parameters may be read in whole vectors
  float eps;
  const void *f, *z, *gate;    // T [rows][ld]
  int64_t ldf, ldz, ldg;
  const void *scale, *w1, *b1, *w2, *b2;  // P [width] or NULL: 1, 1, 0, 1, 0
  void *znew, *y;              // T [rows][width]; y NULL: no second norm
  float *stats;                // [4][rows]: mean and rstd of f's norm and of z's, or NULL (forward)
  const void *dz, *dy;         // T [rows][ld] or NULL: zero
  int64_t lddz, lddy;
  void *df, *dz_in, *dgate;    // T [rows][width] or NULL
  float *parts;                // [gridDim.x][kNormSums][width], or NULL
  float *row_sums;             // *_any: [2][rows] means of dy w2 and of dy w2 zh
};

template <typename T, typename P>
cudaError_t resnorm_forward(ResNormArgs p, bool vec, cudaStream_t st);
// Blocks whose partial sums there are, and the launch.
template <typename T, typename P>
cudaError_t resnorm_backward(ResNormArgs p, bool vec, int grid, cudaStream_t st);

// How a call's rows are laid over threads: columns a thread, threads a row, threads a block.
struct ResNormPlan {
  int columns, tpr, block;  // columns 0: *_any
};

inline ResNormPlan resnorm_plan(int64_t width) {
  if (width > kWidest) return {0, kNormThreads, kNormThreads};
  const int columns = width > kNormThreads * 8 ? 16 : 8;
  int tpr = 1;
  while (tpr * columns < width) tpr <<= 1;
  return {columns, tpr, std::max(tpr, kNormBlock)};
}

// ------------------------------------------------------------------ pieces

// Sums over the tpr threads of a group, the same values in each of them.  `slot` (16 K floats) must not be in
// use by an earlier sum that a thread still reads; for tpr > 32 every thread of the block takes part.
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
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? slot[k * 16 + first + lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
}

// C columns of a row as loaded, in vectors of V: vector i holds columns (t + i tpr) V and those behind it.
template <typename T, int V, int C>
struct RowPart {
  static constexpr int n = C / V;
  Pack<T, V> v[n];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i].v[k] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void load(const T *row, int t, int tpr, int width, bool there) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = (t + i * tpr) * V;
      if (there && c < width) {
        v[i] = *reinterpret_cast<const Pack<T, V> *>(row + c);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i].v[k] = from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void values(float2 (&o)[C / 2]) const {
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

template <typename T, int V, int C>
__device__ __forceinline__ void store_part(T *row, const float2 (&o)[C / 2], int t, int tpr, int width) {
#pragma unroll
  for (int i = 0; i < C / V; ++i) {
    const int c = (t + i * tpr) * V;
    if (c >= width) continue;
    Pack<T, V> q;
    if constexpr (V == 1) {
      q.v[0] = from_f32<T>(i % 2 ? o[i / 2].y : o[i / 2].x);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < V; k += 2)
        *reinterpret_cast<uint32_t *>(&q.v[k]) = pair16(o[(i * V + k) / 2].x, o[(i * V + k) / 2].y, T{});
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 2) q.v[k] = o[(i * V + k) / 2].x, q.v[k + 1] = o[(i * V + k) / 2].y;
    }
    *reinterpret_cast<Pack<T, V> *>(row + c) = q;
  }
}

// A parameter's values at a thread's columns, `other` where there is none, zero outside of the row.
template <typename P, int V, int C>
__device__ __forceinline__ void param_part(const P *p, float other, int t, int tpr, int width, bool vec,
                                           float2 (&o)[C / 2]) {
  float e[C];
#pragma unroll
  for (int i = 0; i < C / V; ++i) {
    const int c = (t + i * tpr) * V;
    if (V > 1 && vec && p && c < width) {
      float q[V];
      load_f32<P, V>(p + c, q);
#pragma unroll
      for (int k = 0; k < V; ++k) e[i * V + k] = q[k];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) e[i * V + k] = c < width ? (p ? to_f32(p[c + k]) : other) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < C / 2; ++j) o[j] = f2(e[2 * j], e[2 * j + 1]);
}

// Which of a thread's columns there are: one or zero.
template <int V, int C>
__device__ __forceinline__ void inside_part(int t, int tpr, int width, float2 (&o)[C / 2]) {
#pragma unroll
  for (int j = 0; j < C; j += 2)
    o[j / 2] = f2((t + j / V * tpr) * V < width ? 1.f : 0.f, (t + (j + 1) / V * tpr) * V < width ? 1.f : 0.f);
}

__device__ __forceinline__ float2 both(float v) { return f2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return f2(-v.x, -v.y); }

// act(g) and, if asked for, act'(g).
template <bool Derivative>
__device__ __forceinline__ void gate_act(int act, float2 g, float2 &a, float2 &da) {
  if (act == kGateNone) {
    a = g;
    if (Derivative) da = both(1.f);
    return;
  }
  const float2 s = sigmoid2(g);
  const float2 r = sigmoid2(neg2(g));  // 1 - s, right relative to itself
  if (act == kGateSigmoid) {
    a = s;
    if (Derivative) da = mul2(s, r);
  } else {
    a = mul2(g, s);
    if (Derivative) da = fma2(a, r, s);
  }
}

// v becomes (v - mu) rstd; returns mu and rstd.  inside: one where there is a column.
template <int H>
__device__ __forceinline__ void norm_row(float2 (&v)[H], const float2 (&inside)[H], bool rms, float inv, float eps,
                                         int tpr, float *slot0, float *slot1, float &mu, float &rstd) {
  mu = 0.f;
  if (!rms) {
    float2 a = both(0.f);
#pragma unroll
    for (int j = 0; j < H; ++j) a = add2(a, v[j]);
    float s[1] = {a.x + a.y};
    row_sums(s, tpr, slot0);
    mu = s[0] * inv;
#pragma unroll
    for (int j = 0; j < H; ++j) v[j] = mul2(add2(v[j], both(-mu)), inside[j]);
  }
  float2 q = both(0.f);
#pragma unroll
  for (int j = 0; j < H; ++j) q = fma2(v[j], v[j], q);
  float s[1] = {q.x + q.y};
  row_sums(s, tpr, slot1);
  rstd = rsqrtf(s[0] * inv + eps);  // 2 units in the last place
#pragma unroll
  for (int j = 0; j < H; ++j) v[j] = mul2(v[j], both(rstd));
}

// ------------------------------------------------------------------ kernels

template <typename T, typename P, int V, int C>
__global__ void __launch_bounds__(kNormThreads, 1) resnorm_forward_rows(const __grid_constant__ ResNormArgs p) {
  constexpr int H = C / 2;
  __shared__ float slots[2][4][16];
  const int tpr = p.tpr, width = (int)p.width, groups = blockDim.x / tpr;
  const int t = threadIdx.x & (tpr - 1);
  const float inv = 1.f / (float)width;
  float2 inside[H];
  inside_part<V, C>(t, tpr, width, inside);
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t lead = (int64_t)blockIdx.x * groups, row = lead + threadIdx.x / tpr;
  RowPart<T, V, C> rf, rz, rg;
  rg.clear();
  auto ask = [&](int64_t r) {
    const bool there = r < p.rows;
    rf.load((const T *)p.f + r * p.ldf, t, tpr, width, there);
    if (p.act != kNoGate) rg.load((const T *)p.gate + r * p.ldg, t, tpr, width, there);
    rz.load((const T *)p.z + r * p.ldz, t, tpr, width, there);
  };
  ask(row);
  int turn = 0;  // the slots alternate, so a turn's sums never meet the previous one's reads
  // every thread of a block makes the same number of turns (the sums need whole warps and blocks)
  for (; lead < p.rows; lead += step, row += step, turn ^= 1) {
    float2 v[H], z[H], w[H];
    rf.values(v);
    rz.values(z);
    float2 a[H];
    if (p.act != kNoGate) {
      float2 g[H], none;
      rg.values(g);
#pragma unroll
      for (int j = 0; j < H; ++j) gate_act<false>(p.act, g[j], a[j], none);
    }
    if (lead + step < p.rows) ask(row + step);
    float mu1 = 0.f, rs1 = 0.f, mu2 = 0.f, rs2 = 0.f;
    if (p.post) {
      norm_row<H>(v, inside, p.rms, inv, p.eps, tpr, slots[turn][0], slots[turn][1], mu1, rs1);
      param_part<P, V, C>((const P *)p.w1, 1.f, t, tpr, width, p.pvec, w);
#pragma unroll
      for (int j = 0; j < H; ++j) v[j] = mul2(v[j], w[j]);
      if (p.b1) {
        param_part<P, V, C>((const P *)p.b1, 0.f, t, tpr, width, p.pvec, w);
#pragma unroll
        for (int j = 0; j < H; ++j) v[j] = add2(v[j], w[j]);
      }
    }
    if (p.act != kNoGate) {
#pragma unroll
      for (int j = 0; j < H; ++j) v[j] = mul2(v[j], a[j]);
    }
    param_part<P, V, C>((const P *)p.scale, 1.f, t, tpr, width, p.pvec, w);
#pragma unroll
    for (int j = 0; j < H; ++j) v[j] = fma2(v[j], w[j], z[j]);
    if (row < p.rows) store_part<T, V, C>((T *)p.znew + row * width, v, t, tpr, width);
    if (p.y) {
      norm_row<H>(v, inside, p.rms, inv, p.eps, tpr, slots[turn][2], slots[turn][3], mu2, rs2);
      param_part<P, V, C>((const P *)p.w2, 1.f, t, tpr, width, p.pvec, w);
#pragma unroll
      for (int j = 0; j < H; ++j) v[j] = mul2(v[j], w[j]);
      if (p.b2) {
        param_part<P, V, C>((const P *)p.b2, 0.f, t, tpr, width, p.pvec, w);
#pragma unroll
        for (int j = 0; j < H; ++j) v[j] = add2(v[j], w[j]);
      }
      if (row < p.rows) store_part<T, V, C>((T *)p.y + row * width, v, t, tpr, width);
    }
    if (p.stats && t == 0 && row < p.rows) {
      p.stats[row] = mu1, p.stats[p.rows + row] = rs1;
      p.stats[2 * p.rows + row] = mu2, p.stats[3 * p.rows + row] = rs2;
    }
  }
}

template <typename T, typename P, int V, int C>
__global__ void __launch_bounds__(kNormThreads, 1) resnorm_backward_rows(const __grid_constant__ ResNormArgs p) {
  constexpr int H = C / 2;
  extern __shared__ float cols[];  // more than one group: [kNormSums][width]
  __shared__ float slots[2][2][32];
  grid_dependency_launch();  // the sums over blocks start as multiprocessors become free, and wait there
  const int tpr = p.tpr, width = (int)p.width, groups = blockDim.x / tpr;
  const int t = threadIdx.x & (tpr - 1);
  const float inv = 1.f / (float)width;
  float2 inside[H], sums[kNormSums][H];
  inside_part<V, C>(t, tpr, width, inside);
#pragma unroll
  for (int k = 0; k < kNormSums; ++k)
#pragma unroll
    for (int j = 0; j < H; ++j) sums[k][j] = both(0.f);
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t lead = (int64_t)blockIdx.x * groups, row = lead + threadIdx.x / tpr;
  RowPart<T, V, C> rf, rz, rg, rdz, rdy;
  float st[4];
  rg.clear();
  rdz.clear();
  rdy.clear();
  auto ask = [&](int64_t r) {
    const bool there = r < p.rows;
    rf.load((const T *)p.f + r * p.ldf, t, tpr, width, there);
    rz.load((const T *)p.z + r * p.ldz, t, tpr, width, there);
    if (p.act != kNoGate) rg.load((const T *)p.gate + r * p.ldg, t, tpr, width, there);
    if (p.dz) rdz.load((const T *)p.dz + r * p.lddz, t, tpr, width, there);
    if (p.dy) rdy.load((const T *)p.dy + r * p.lddy, t, tpr, width, there);
#pragma unroll
    for (int k = 0; k < 4; ++k) st[k] = there ? p.stats[k * p.rows + r] : 0.f;
  };
  ask(row);
  int turn = 0;
  for (; lead < p.rows; lead += step, row += step, turn ^= 1) {
    float2 fh[H], u[H], a[H], da[H], sc[H], d[H];
    const float mu1 = st[0], rs1 = st[1], mu2 = st[2], rs2 = st[3];
    rf.values(fh);
    if (p.post) {
      float2 w[H];
      // outside of the row everything is zero, as (0 - mean) rstd would not be
#pragma unroll
      for (int j = 0; j < H; ++j) fh[j] = mul2(add2(fh[j], both(-mu1)), mul2(inside[j], both(rs1)));
      param_part<P, V, C>((const P *)p.w1, 1.f, t, tpr, width, p.pvec, w);
#pragma unroll
      for (int j = 0; j < H; ++j) u[j] = mul2(fh[j], w[j]);
      if (p.b1) {
        param_part<P, V, C>((const P *)p.b1, 0.f, t, tpr, width, p.pvec, w);
#pragma unroll
        for (int j = 0; j < H; ++j) u[j] = add2(u[j], w[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < H; ++j) u[j] = fh[j];
    }
#pragma unroll
    for (int j = 0; j < H; ++j) a[j] = both(1.f), da[j] = both(0.f);
    if (p.act != kNoGate) {
      float2 g[H];
      rg.values(g);
#pragma unroll
      for (int j = 0; j < H; ++j) gate_act<true>(p.act, g[j], a[j], da[j]);
    }
    param_part<P, V, C>((const P *)p.scale, 1.f, t, tpr, width, p.pvec, sc);
    rdz.values(d);
    if (p.dy) {
      float2 zh[H], dy[H], w[H];
      rz.values(zh);
      rdy.values(dy);
      param_part<P, V, C>((const P *)p.w2, 1.f, t, tpr, width, p.pvec, w);
      float2 s1 = both(0.f), s2 = s1;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        zh[j] = fma2(mul2(u[j], a[j]), sc[j], zh[j]);
        zh[j] = mul2(add2(zh[j], both(-mu2)), mul2(inside[j], both(rs2)));
        sums[3][j] = fma2(dy[j], zh[j], sums[3][j]);
        sums[4][j] = add2(sums[4][j], dy[j]);
        dy[j] = mul2(dy[j], w[j]);
        s1 = add2(s1, dy[j]);
        s2 = fma2(dy[j], zh[j], s2);
      }
      float s[2] = {s1.x + s1.y, s2.x + s2.y};
      row_sums(s, tpr, slots[turn][0]);
      const float m1 = p.rms ? 0.f : -s[0] * inv, m2 = -s[1] * inv;
#pragma unroll
      for (int j = 0; j < H; ++j)
        d[j] = fma2(fma2(zh[j], both(m2), add2(dy[j], both(m1))), both(rs2), d[j]);
    }
    const int64_t at = row * width, present = row;
    const bool live = row < p.rows;
    if (live && p.dz_in) store_part<T, V, C>((T *)p.dz_in + at, d, t, tpr, width);
#pragma unroll
    for (int j = 0; j < H; ++j) {
      sums[0][j] = fma2(d[j], mul2(a[j], u[j]), sums[0][j]);
      d[j] = mul2(d[j], sc[j]);
      u[j] = mul2(mul2(d[j], u[j]), da[j]);  // dgate
      d[j] = mul2(d[j], a[j]);               // du
    }
    if (live && p.dgate) store_part<T, V, C>((T *)p.dgate + at, u, t, tpr, width);
    if (lead + step < p.rows) ask(present + step);
    if (p.post) {
      float2 w[H];
      param_part<P, V, C>((const P *)p.w1, 1.f, t, tpr, width, p.pvec, w);
      float2 s1 = both(0.f), s2 = s1;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        sums[1][j] = fma2(d[j], fh[j], sums[1][j]);
        sums[2][j] = add2(sums[2][j], d[j]);
        d[j] = mul2(d[j], w[j]);
        s1 = add2(s1, d[j]);
        s2 = fma2(d[j], fh[j], s2);
      }
      float s[2] = {s1.x + s1.y, s2.x + s2.y};
      row_sums(s, tpr, slots[turn][1]);
      const float m1 = p.rms ? 0.f : -s[0] * inv, m2 = -s[1] * inv;
#pragma unroll
      for (int j = 0; j < H; ++j) d[j] = mul2(fma2(fh[j], both(m2), add2(d[j], both(m1))), both(rs1));
    }
    if (live && p.df) store_part<T, V, C>((T *)p.df + at, d, t, tpr, width);
  }
  if (!p.parts) return;
  float *to = p.parts + (int64_t)blockIdx.x * kNormSums * width;
  auto column = [&](int j) { return (t + j / V * tpr) * V + j % V; };
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < kNormSums; ++k)
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (column(j) < width) to[k * width + column(j)] = j % 2 ? sums[k][j / 2].y : sums[k][j / 2].x;
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
          if (column(j) < width) {
            const float s = j % 2 ? sums[k][j / 2].y : sums[k][j / 2].x;
            float *c = cols + k * width + column(j);
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
    if (p.stats && threadIdx.x == 0) {
      p.stats[row] = mu1, p.stats[p.rows + row] = rs1;
      p.stats[2 * p.rows + row] = mu2, p.stats[3 * p.rows + row] = rs2;
    }
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
    const float mu1 = p.stats[row], rs1 = p.stats[p.rows + row];
    const float mu2 = p.stats[2 * p.rows + row], rs2 = p.stats[3 * p.rows + row];
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
      const Element e = element<T, P>(p, r, c, p.stats[r], p.stats[p.rows + r]);
      float zh, dy;
      const float d = stream_gradient<T, P>(p, e, r, c, p.stats[2 * p.rows + r], p.stats[3 * p.rows + r], p.row_sums[r],
                                            p.row_sums[p.rows + r], zh, dy);
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
  const int64_t groups = pl.block / pl.tpr;
  const int grid = (int)std::min<int64_t>((p.rows + groups - 1) / groups, sm_count() * (1024 / pl.block));
  if (pl.columns == 8)
    return vec ? launch_resnorm(resnorm_forward_rows<T, P, V, 8>, p, grid, pl.block, 0, st)
               : launch_resnorm(resnorm_forward_rows<T, P, 1, 8>, p, grid, pl.block, 0, st);
  return vec ? launch_resnorm(resnorm_forward_rows<T, P, V, 16>, p, grid, pl.block, 0, st)
             : launch_resnorm(resnorm_forward_rows<T, P, 1, 16>, p, grid, pl.block, 0, st);
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
  const size_t smem = pl.block > pl.tpr && p.parts ? kNormSums * sizeof(float) * (size_t)p.width : 0;
  if (pl.columns == 8)
    return vec ? launch_resnorm(resnorm_backward_rows<T, P, V, 8>, p, grid, pl.block, smem, st)
               : launch_resnorm(resnorm_backward_rows<T, P, 1, 8>, p, grid, pl.block, smem, st);
  return vec ? launch_resnorm(resnorm_backward_rows<T, P, V, 16>, p, grid, pl.block, smem, st)
             : launch_resnorm(resnorm_backward_rows<T, P, 1, 16>, p, grid, pl.block, smem, st);
}

}  // namespace sla
