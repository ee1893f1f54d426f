// A linear layer of few outputs (a network's head): up to kSkinny, over rows of up to kSkinnyWidth columns.
//
//   y_o = act(sum_c x_c W_oc + b_o) + r_o;   dp_o = dy_o act'(p_o),  dx_c = sum_o dp_o W_oc,  dW_oc = sum dp_o x_c,  db_o = sum dp_o
//
// Bound by reading x (and writing dx): a tensor-core tile would be 64 columns wide for one to eight, float32 would be laid
// out in three sheets first, and odd widths copied.  Here x is read once, in float32 arithmetic, with the weights in shared
// memory; dp is not rounded.  Forward, up to 32 lanes share a row, four rows at a time, and add up by shuffles, in which each
// passes half of its sums on.  Backward, a thread keeps eight columns of every row, so that dW accumulates in its
// registers, then over the block's threads and, in a second kernel, over the blocks, in a fixed order; the next rows are read
// before the present ones are used, as sums of eight outputs leave room for eight warps in an SM (302,053 x 384 -> 5, training
// step: 569 -> 507 us; four columns a thread and sixteen warps: 589).
//
// Measured, float32, training step: 1,000,000 tokens, 64 -> 1 136 us (0.84 of the copy rate), 64 -> 3 with gelu 240 (0.49),
// 302,053 tokens, 384 -> 5 507 (0.41; forward 115, 0.60): with more outputs the loads' latency and the instructions.
#pragma once

#include <cuda_runtime.h>

#include "sla_act.cuh"
#include "sla_net.cuh"

namespace sla {

constexpr int kSkinny = 8, kSkinnyWidth = 2048;
constexpr int kSkinnyRows = 4, kSkinnyBackRows = 2;  // rows of a group at a time, which share what is read of the weights

struct SkinnyArgs {
  int64_t tokens;
  int width, out, act;
  const void *x, *w, *bias, *residual;  // T
  int64_t ldx, ldr;
  void *y;
  float *da;             // act'(p), [tokens][ldda], or NULL
  int64_t ldda;
  const void *dy;
  int64_t lddy;
  void *dx;              // or NULL
  float *parts;          // [gridDim.x][out][width] sums of dW, or NULL
  float *bias_parts;     // [gridDim.x][out] sums of db, or NULL
  int tpr;               // threads of a row
};

// Columns of a thread: V neighbours (V > 1), or one, every `lanes` threads; C of them make a turn.  Weights lie in shared
// memory in float32 as threads read them, so that a warp's words are neighbours: [O][turn][C / 4][lanes][4], or [O][width]
// (C = 1).  Outputs beyond out and columns beyond width are zero.
template <int V, int C>
__device__ __forceinline__ int skinny_column(int turn, int t, int lanes, int k) {
  return turn * lanes * C + (V > 1 ? t * C + k : t + k * lanes);
}

template <typename T, int O, int V, int C>
__device__ __forceinline__ void stage_weights(float *sm, const SkinnyArgs &p, int padded) {
  const int lanes = p.tpr, shift = __ffs(lanes) - 1;
#pragma unroll 2
  for (int slot = threadIdx.x; slot < padded; slot += 256) {
    int c = slot;
    if constexpr (C > 1) {
      const int turn = slot / C >> shift, in = slot & (lanes * C - 1);
      c = skinny_column<V, C>(turn, (in >> 2) & (lanes - 1), lanes, (in >> 2 >> shift) * 4 + (in & 3));
    }
#pragma unroll
    for (int o = 0; o < O; ++o) {
      const float w = to_f32(((const T *)p.w)[min(o, p.out - 1) * p.width + min(c, p.width - 1)]);
      sm[o * padded + slot] = o < p.out && c < p.width ? w : 0.f;
    }
  }
}

template <int C>
__device__ __forceinline__ void staged(const float *sm, int turn, int t, int lanes, float (&w)[C]) {
  if constexpr (C == 1) {
    w[0] = sm[turn * lanes + t];
  } else {
#pragma unroll
    for (int k = 0; k < C; k += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(sm + turn * lanes * C + k * lanes + t * 4);
      w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
    }
  }
}

// Words of an output's staged weights.
inline int skinny_padded(int width, int tpr, int c) { return (width + tpr * c - 1) / (tpr * c) * (tpr * c); }

// V columns of a row, or zeros: read all the same, from the row's first columns, so that no branch holds up the next loads.
template <typename T, int V>
__device__ __forceinline__ void load_columns(const T *row, int c, bool there, float (&v)[V]) {
  load_f32<T, V>(row + (there ? c : 0), v);
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = there ? v[k] : 0.f;
}

// V columns at a time (16 bytes, or one where rows are not aligned to them); tpr <= 32.
template <typename T, int O, int V>
__global__ void __launch_bounds__(256) skinny_forward(const __grid_constant__ SkinnyArgs p) {
  constexpr int R = kSkinnyRows, N = R * O;
  extern __shared__ __align__(16) float sm[];
  const int lanes = p.tpr, j = threadIdx.x & (lanes - 1), groups = 256 / lanes;
  const int turns = (p.width + lanes * V - 1) / (lanes * V), padded = turns * lanes * V;
  stage_weights<T, O, V, V>(sm, p, padded);
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * groups * R;
  // all threads of a block make the same number of turns: the sums take whole warps
  for (int64_t lead = (int64_t)blockIdx.x * groups * R; lead < p.tokens; lead += step) {
    const int64_t first = lead + threadIdx.x / lanes * R;
    float acc[N] = {};  // [R][O]
    const T *rows[R];   // beyond the last, the last again: its sums are not written
#pragma unroll
    for (int r = 0; r < R; ++r) rows[r] = (const T *)p.x + min(first + r, p.tokens - 1) * p.ldx;
#pragma unroll 2
    for (int i = 0; i < turns; ++i) {
      const int c = (i * lanes + j) * V;
      float v[R][V];
#pragma unroll
      for (int r = 0; r < R; ++r) load_columns<T, V>(rows[r], c, c < p.width, v[r]);
#pragma unroll
      for (int o = 0; o < O; ++o) {
        float w[V];
        staged<V>(sm + o * padded, i, j, lanes, w);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r * O + o] = fmaf(v[r][k], w[k], acc[r * O + o]);
      }
    }
    // a lane passes half of its sums on and takes the other half, until each has its own (or, fewer sums than lanes, its share)
    int s = lanes >> 1, held = N, from = 0;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2) {
      if (s == 0) break;
      const bool upper = (j & s) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, upper ? acc[i] : acc[i + n], s);
        acc[i] = (upper ? acc[i + n] : acc[i]) + other;
      }
      from += upper ? n : 0, held = n, s >>= 1;
    }
    const int shared = s ? 2 * s - 1 : 0;  // lanes that differ in these bits hold the same sum
    for (; s > 0; s >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], s);
    if (j & shared) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= held) break;
      const int r = (from + i) / O, o = (from + i) % O;
      const int64_t row = first + r;
      if (row >= p.tokens || o >= p.out) continue;
      float v[1] = {acc[i] + (p.bias ? to_f32(((const T *)p.bias)[o]) : 0.f)};
      if (p.act != SLA_ACT_NONE) {
        float d[1];
        with_activation(p.act, [&](auto act) { activate<act.value, true, 1>(v, d); });
        if (p.da) p.da[row * p.ldda + o] = d[0];
      }
      if (p.residual) v[0] += to_f32(((const T *)p.residual)[row * p.ldr + o]);
      ((T *)p.y)[row * p.out + o] = from_f32<T>(v[0]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_eight(const T *row, int t, int tpr, int width, bool there, float (&v)[8]) {
  if constexpr (V > 1) {
#pragma unroll
    for (int i = 0; i < 8; i += V) {
      float q[V];
      load_columns<T, V>(row, t * 8 + i, there && t * 8 + i < width, q);
#pragma unroll
      for (int k = 0; k < V; ++k) v[i + k] = q[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float q[1];
      load_columns<T, 1>(row, t + k * tpr, there && t + k * tpr < width, q);
      v[k] = q[0];
    }
  }
}

template <typename T, int O, int V>
__global__ void __launch_bounds__(256) skinny_backward(const __grid_constant__ SkinnyArgs p) {
  constexpr int R = kSkinnyBackRows;
  extern __shared__ __align__(16) float sm[];  // weights, then the block's sums in the same places
  grid_dependency_launch();
  const int tpr = p.tpr, t = threadIdx.x & (tpr - 1), groups = 256 / tpr, width = p.width, padded = tpr * 8;
  stage_weights<T, O, V, 8>(sm, p, padded);
  __syncthreads();
  float acc[O][8] = {}, bias[O] = {};
  const int64_t step = (int64_t)gridDim.x * groups * R;
  int64_t first = ((int64_t)blockIdx.x * groups + threadIdx.x / tpr) * R;
  float next_x[R][8] = {}, next_dy[R][O], next_da[R][O];
  auto load = [&](int64_t at) {  // rows beyond the last: the last again
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = min(at + r, p.tokens - 1);
      if (p.parts) load_eight<T, V>((const T *)p.x + row * p.ldx, t, tpr, width, true, next_x[r]);
#pragma unroll
      for (int o = 0; o < O; ++o) next_dy[r][o] = to_f32(((const T *)p.dy)[row * p.lddy + min(o, p.out - 1)]);
      if (p.da) {
#pragma unroll
        for (int o = 0; o < O; ++o) next_da[r][o] = p.da[row * p.ldda + min(o, p.out - 1)];
      }
    }
  };
  load(first);
  for (; first < p.tokens; first += step) {
    float x[R][8], dp[R][O], dx[R][8] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool there = first + r < p.tokens;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[r][k] = there ? next_x[r][k] : 0.f;
#pragma unroll
      for (int o = 0; o < O; ++o) dp[r][o] = there && o < p.out ? next_dy[r][o] * (p.da ? next_da[r][o] : 1.f) : 0.f;
    }
    load(first + step);  // the next rows arrive meanwhile
#pragma unroll
    for (int o = 0; o < O; ++o) {
      float w[8];
      staged<8>(sm + o * padded, 0, t, tpr, w);
#pragma unroll
      for (int r = 0; r < R; ++r) bias[o] += dp[r][o];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          dx[r][k] = fmaf(dp[r][o], w[k], dx[r][k]);
          acc[o][k] = fmaf(dp[r][o], x[r][k], acc[o][k]);
        }
    }
    if (!p.dx) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = first + r;
      if (row >= p.tokens) continue;
      T *to = (T *)p.dx + row * width;
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < 8; i += V) {
          if (t * 8 + i >= width) break;
          float q[V];
#pragma unroll
          for (int k = 0; k < V; ++k) q[k] = dx[r][i + k];
          store_f32<T, V>(to + t * 8 + i, q);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (t + k * tpr < width) to[t + k * tpr] = from_f32<T>(dx[r][k]);
      }
    }
  }
  if (!p.parts && !p.bias_parts) return;
  // the groups of a warp together, then the warps one after another
  for (int s = 16; s >= tpr; s >>= 1)
#pragma unroll
    for (int o = 0; o < O; ++o) {
      bias[o] += __shfl_xor_sync(0xffffffffu, bias[o], s);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[o][k] += __shfl_xor_sync(0xffffffffu, acc[o][k], s);
    }
  __shared__ float bsum[O];
  const int unit = tpr < 32 ? 32 : tpr;
  for (int g = 0; g < 256 / unit; ++g) {
    __syncthreads();  // (the first: the weights have been read)
    if ((int)threadIdx.x / unit != g || (int)threadIdx.x % unit >= tpr) continue;
#pragma unroll
    for (int o = 0; o < O; ++o) {
      if (t == 0) bsum[o] = g ? bsum[o] + bias[o] : bias[o];
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        float4 *at = reinterpret_cast<float4 *>(sm + o * padded + k * tpr + t * 4);
        float4 q = make_float4(acc[o][k], acc[o][k + 1], acc[o][k + 2], acc[o][k + 3]);
        if (g) {
          const float4 e = *at;
          q = make_float4(e.x + q.x, e.y + q.y, e.z + q.z, e.w + q.w);
        }
        *at = q;
      }
    }
  }
  __syncthreads();
  if (p.parts)
    for (int o = 0; o < p.out; ++o)
      for (int c = threadIdx.x; c < width; c += 256) {
        const int at = V > 1 ? c >> 3 : c & (tpr - 1), k = V > 1 ? c & 7 : c / tpr;
        p.parts[((int64_t)blockIdx.x * p.out + o) * width + c] = sm[o * padded + (k >> 2) * tpr * 4 + at * 4 + (k & 3)];
      }
  if (p.bias_parts && (int)threadIdx.x < p.out) p.bias_parts[blockIdx.x * p.out + threadIdx.x] = bsum[threadIdx.x];
}

}  // namespace sla
