// The gated feed-forward block and the linear layer for few tokens (up to kFewTokens), forward.
//
// With a token or a few the weights are read once and little else happens: the floor is their bytes
// over the memory's rate (25 MB at 1024 -> 4096 -> 1024: 3.8 us).  tcgen05 tiles would be 128 rows high
// for one to sixteen tokens, and a GPU's worth of them needs sums across blocks; here the weights are
// the 16 rows of mma.sync m16n8k16 and the tokens its 8 columns, and what matters is that every thread
// has many 16-byte loads on their way.
//
// A block takes 16 hidden units (their g and u rows) or 16 outputs.  Its warps, and the blocks of its
// cluster, share k: 32 values a turn, of which a thread loads 8 neighbours of rows g and g + 8 (g = lane
// / 4).  The mma's own order of k would make that four pieces; since any order of k gives the same
// sum, the thread's 8 values stand in the places (2t, 2t+1, 2t+8, 2t+9) of two mma, for weights and
// tokens alike.  The warps' sums are added in shared memory, the cluster's through distributed shared
// memory, in a fixed order.
//
// The second product is launched while the first runs (programmatic dependent launch): it loads its
// first weights, which do not depend on h, and then waits for h.
//
// Measured (both products): one token 9.9 us at 1024 -> 4096 -> 1024 in bfloat16, where the tiled products take
// 21.1; 16 tokens 11.9 against 19.3, and 17.5 against 18.1 at 256 -> 1024 -> 256 in float32.  In float32 one to eight
// tokens take 27 us at 1024 -> 4096 -> 1024 (floor 7.5): every weight is split into three parts in registers and each 32
// of k takes 12 mma.  A third eight of
// tokens does not pay any more: 18.0 against 19.4 and 27.8 against 18.1 at 24 tokens.
#pragma once

#include "sla_product.cuh"

namespace sla {

constexpr int kFewTokens = 16;
constexpr int kFewWarps = 8;
constexpr int kFewTurns = 4;  // turns of weights a thread has on their way

struct FewArgs {
  int tokens, n, k;        // n: hidden units or outputs
  const void *x;           // tokens: T [tokens][ldx] (x), or operand sheets (h)
  int64_t ldx, x_sheet;
  const void *w;           // T [n or 2 n][k]
  const void *bias;        // T [n or 2 n] or NULL
  int x_vec, w_vec;        // 16-byte loads of 8 values can be used
  int act;
  void *c;                 // T [tokens][n] (out)
  void *g, *u;             // T [tokens][ldg]: u act'(g) and act(g), or NULL (gate)
  uint16_t *h;             // operand sheets (gate)
  int64_t ldg, sheet;
  const void *residual;    // T [tokens][ldr] or NULL (linear; act'(..) goes to g, float [tokens][ldg])
  int64_t ldr;
};

// Gate product (kGate), output product (kStore) or linear layer (kLinear) of few tokens.
template <typename T>
cudaError_t launch_few(Epilogue epi, const FewArgs &p, cudaStream_t st);

template <typename T>
using operand_t = typename std::conditional<sizeof(T) == 4, bf16, T>::type;

// Eight neighbouring values as 16-bit parts, two a word.
template <typename T>
struct Eight {
  static constexpr int S = sizeof(T) == 4 ? 3 : 1;
  uint32_t w[S][4];
};

// As loaded: whole where they may be, else value by value.
template <typename T>
struct RawEight {
  uint4 q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p, int left, bool vec) {
    if (vec && left >= 8) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = reinterpret_cast<const uint4 *>(p)[i];
      return;
    }
    Pack<T, 8> e;
#pragma unroll
    for (int i = 0; i < 8; ++i) e.v[i] = i < left ? p[i] : from_f32<T>(0.f);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = reinterpret_cast<const uint4 *>(&e)[i];
  }
  __device__ __forceinline__ void parts(Eight<T> &o) const {
    if constexpr (sizeof(T) == 2) {
      o.w[0][0] = q[0].x, o.w[0][1] = q[0].y, o.w[0][2] = q[0].z, o.w[0][3] = q[0].w;
    } else {
      const uint32_t f[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t a[3], b[3];
        split3(__uint_as_float(f[2 * i]), a);
        split3(__uint_as_float(f[2 * i + 1]), b);
#pragma unroll
        for (int s = 0; s < 3; ++s) o.w[s][i] = a[s] | ((uint32_t)b[s] << 16);
      }
    }
  }
};

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, bf16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, f16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c += the 16 rows (lo: rows g, hi: rows g + 8) times 8 tokens over 32 values of k; float32's six products, smallest first, the
// five small ones into `small`.
template <typename T>
__device__ __forceinline__ void few_mma(float (&c)[4], float (&small)[4], const Eight<T> &lo, const Eight<T> &hi,
                                        const Eight<T> &x) {
  constexpr int order[6][2] = {{0, 2}, {2, 0}, {1, 1}, {0, 1}, {1, 0}, {0, 0}};
#pragma unroll
  for (int q = sizeof(T) == 4 ? 0 : 5; q < 6; ++q)
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      mma16(q < 5 ? small : c, lo.w[order[q][0]][j], hi.w[order[q][0]][j], lo.w[order[q][0]][j + 1], hi.w[order[q][0]][j + 1],
            x.w[order[q][1]][j], x.w[order[q][1]][j + 1], operand_t<T>{});
}

__device__ __forceinline__ float cluster_read(const float *local, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.f32 %0, [r];\n\t}"
      : "=f"(v)
      : "r"(smem_u32(local)), "r"(rank)
      : "memory");
  return v;
}

// NT: tokens in eights.
template <typename T, Epilogue EPI, int NT>
__global__ void __launch_bounds__(32 * kFewWarps) few_kernel(const FewArgs p, int ranks) {
  constexpr bool Gate = EPI == kGate;
  constexpr int M = Gate ? 2 : 1, S = Eight<T>::S;
  extern __shared__ float sums[];  // [warps][M][16][8 NT], then [M][16][8 NT] of the block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % ranks, r0 = blockIdx.x / ranks * 16;
  const int turns = (p.k + 31) / 32, stride = kFewWarps * ranks;
  const T *w = (const T *)p.w;
  // rows past the end are read from the last one and not stored
  const int row_lo = min(r0 + g, p.n - 1), row_hi = min(r0 + g + 8, p.n - 1);

  RawEight<T> raw[kFewTurns][M][2];
  auto ask = [&](int first) {
#pragma unroll
    for (int i = 0; i < kFewTurns; ++i) {
      const int turn = first + i * stride, k = turn * 32 + t * 8;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int64_t base = m * (int64_t)p.n;
        raw[i][m][0].load(w + (base + row_lo) * p.k + k, turn < turns ? p.k - k : 0, p.w_vec);
        raw[i][m][1].load(w + (base + row_hi) * p.k + k, turn < turns ? p.k - k : 0, p.w_vec);
      }
    }
  };
  int turn = rank * kFewWarps + warp;
  ask(turn);
  if (Gate)
    grid_dependency_launch();
  else if (EPI == kStore)
    grid_dependency_wait();

  // A linear layer in float32: the small products have a sum of their own, and both are added up in float32 every kFewTurns
  // turns, since the tensor core drops up to a unit of a running sum with every product (16 tokens, 4096 -> 1000: relative error
  // 1.6e-6 in one sum).
  constexpr bool apart = EPI == kLinear && sizeof(T) == 4;
  float acc[M][NT][4] = {}, small[apart ? NT : 1][4] = {}, total[apart ? NT : 1][4] = {};
  for (; turn < turns; turn += kFewTurns * stride) {
#pragma unroll
    for (int i = 0; i < kFewTurns; ++i) {
      const int k = (turn + i * stride) * 32 + t * 8, left = turn + i * stride < turns ? p.k - k : 0;
      Eight<T> x[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int token = min(j * 8 + g, p.tokens - 1);
        if constexpr (EPI != kStore) {
          RawEight<T> r;
          r.load((const T *)p.x + token * p.ldx + k, left, p.x_vec);
          r.parts(x[j]);
        } else {
#pragma unroll
          for (int s = 0; s < S; ++s) {
            RawEight<operand_t<T>> r;
            r.load((const operand_t<T> *)p.x + s * p.x_sheet + token * p.ldx + k, left, p.x_vec);
            x[j].w[s][0] = r.q[0].x, x[j].w[s][1] = r.q[0].y, x[j].w[s][2] = r.q[0].z, x[j].w[s][3] = r.q[0].w;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        Eight<T> lo, hi;
        raw[i][m][0].parts(lo);
        raw[i][m][1].parts(hi);
#pragma unroll
        for (int j = 0; j < NT; ++j) few_mma<T>(acc[m][j], apart ? small[j] : acc[m][j], lo, hi, x[j]);
      }
    }
    if (turn + kFewTurns * stride < turns) ask(turn + kFewTurns * stride);
    if constexpr (apart)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[j][e] += acc[0][j][e] + small[j][e];
          acc[0][j][e] = small[j][e] = 0.f;
        }
  }
  if constexpr (apart)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][j][e] = total[j][e];

  constexpr int per = M * 16 * 8 * NT;
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sums[warp * per + (m * 16 + g + (e >> 1) * 8) * 8 * NT + j * 8 + 2 * t + (e & 1)] = acc[m][j][e];
  __syncthreads();
  float *block = sums + kFewWarps * per;
  for (int i = threadIdx.x; i < per; i += 32 * kFewWarps) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) s += sums[q * per + i];
    block[i] = s;
  }
  if (ranks > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // the block's rows are finished by its cluster's ranks in turn
  for (int i = threadIdx.x + rank * 32 * kFewWarps; i < 16 * 8 * NT; i += 32 * kFewWarps * ranks) {
    const int row = i & 15, token = i >> 4, r = r0 + row;
    float v = 0.f, u = 0.f;
    for (int q = 0; q < ranks; ++q) {
      const int at = row * 8 * NT + token;
      v += ranks > 1 ? cluster_read(block + at, q) : block[at];
      if (Gate) u += ranks > 1 ? cluster_read(block + 16 * 8 * NT + at, q) : block[16 * 8 * NT + at];
    }
    if (token >= p.tokens || r >= p.n) continue;
    if (p.bias) {
      v += to_f32(((const T *)p.bias)[r]);
      if (Gate) u += to_f32(((const T *)p.bias)[p.n + r]);
    }
    if (Gate) {
      const int64_t o = token * p.ldg + r;
      float a[1] = {v}, b[1] = {u}, h[1];
      with_activation(p.act, [&](auto act) { gate<act.value, true, 1>(a, b, h); });
      if (p.g) {
        ((T *)p.g)[o] = from_f32<T>(a[0]);
        ((T *)p.u)[o] = from_f32<T>(b[0]);
      }
      store_operand<T, 1>(p.h + o, p.sheet, h, 1, false);
    } else {
      if constexpr (EPI == kLinear) {
        if (p.act != SLA_ACT_NONE) {
          float a[1] = {v}, da[1];
          with_activation(p.act, [&](auto act) { activate<act.value, true, 1>(a, da); });
          v = a[0];
          if (p.g) ((float *)p.g)[token * p.ldg + r] = da[0];
        }
        if (p.residual) v += to_f32(((const T *)p.residual)[token * p.ldr + r]);
      }
      ((T *)p.c)[token * (int64_t)p.n + r] = from_f32<T>(v);
    }
  }
  if (ranks > 1) cluster_sync_all();  // the others may still read this block's sums
}

template <typename T, Epilogue EPI, int NT>
cudaError_t launch_few_ranks(const FewArgs &p, int ranks, cudaStream_t st) {
  constexpr int per = (EPI == kGate ? 2 : 1) * 16 * 8 * NT;
  LaunchConfig cfg(dim3((p.n + 15) / 16 * ranks), 32 * kFewWarps, (kFewWarps + 1) * per * sizeof(float), st, EPI == kStore,
                   ranks);
  return cudaLaunchKernelEx(&cfg.c, few_kernel<T, EPI, NT>, p, ranks);
}

template <typename T, Epilogue EPI>
cudaError_t launch_few_as(const FewArgs &p, cudaStream_t st) {
  // blocks of a cluster share k until there are about as many as multiprocessors
  int ranks = 1;
  const int rows = (p.n + 15) / 16;
  while (ranks < 8 && rows * ranks * 2 <= 192 && p.k >= 32 * kFewWarps * ranks * 2) ranks *= 2;
  return p.tokens <= 8 ? launch_few_ranks<T, EPI, 1>(p, ranks, st) : launch_few_ranks<T, EPI, 2>(p, ranks, st);
}

}  // namespace sla
