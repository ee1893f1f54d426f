// Layer norm over the rows of a matrix, forward and backward.
//
//   y = (x - mu) rstd w + b,   mu = mean(x),  rstd = (mean((x - mu)^2) + eps)^(-1/2)     per row
//   dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),   dxh = dy w,  xh = (x - mu) rstd     per row
//   dw = sum over rows of dy xh,   db = sum over rows of dy                              per column
//
// Both directions are bound by memory (8 and 12 operations an element), so each is one pass: a
// group of `tpr` threads (a power of two: part of a warp, a warp, or the block) keeps a row in
// registers as NI vectors of VEC elements a thread, and reduces with shuffles (and shared memory
// beyond a warp).  The variance is the mean of squared differences from the mean, taken from the
// registers in a second sweep: the one-sweep form mean(x^2) - mu^2 cancels when a row sits far
// from zero.  VEC is 16 bytes of elements; rows that cannot be read that way (width, stride or
// address) take VEC = 1, still coalesced over the threads.  Rows wider than the registers of a
// 512-thread block hold (16,384 16-bit elements) are re-read from L2 by the *_wide kernels.
//
// Backward: a thread sees the same columns in every row of its group, so dw and db accumulate in
// its registers over the block's rows (persistent blocks, rows in strides of the grid), then
// across the block in a fixed order, then over the blocks' partial sums in a second kernel.  No
// atomics: the same call gives the same bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sla_common.cuh"
#include "sla_host.h"
#include "sla_net.cuh"

namespace sla {

int sm_count() {
  static thread_local int cached_dev = -1, cached = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev != cached_dev) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    cached = n;
    cached_dev = dev;
  }
  return cached;
}

namespace {

constexpr int kLnBlock = 256;     // threads of a block while a row takes no more
constexpr int kMaxThreads = 512;  // threads of a block that shares one row
constexpr int kInFlight = 4;      // vectors of a thread on their way at a time: rows are taken in bundles
constexpr int kColTile = 32;      // columns of a block of the column sums
constexpr int kMaxParts = 1216;   // blocks that leave partial column sums (8 a multiprocessor)

// Sum over the tpr threads of a group, the same value in each of them.  For tpr > 32 the block is
// one group; `slot` (32 floats) must not be in use by an earlier sum that a thread still reads.
__device__ __forceinline__ float group_sum(float v, int tpr, float *slot) {
  const int in_warp = tpr < 32 ? tpr : 32;
  for (int o = in_warp >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  const int lane = threadIdx.x & 31, warps = tpr >> 5;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = lane < warps ? slot[lane] : 0.f;
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N> &q, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32(q.v[i]);
}

// Rows of a bundle: as many as keep kInFlight vectors of a thread in flight.
template <int NI>
inline constexpr int kBundle = NI >= kInFlight ? 1 : kInFlight / NI;

template <typename T, typename P, int VEC, int NI>
__global__ void __launch_bounds__(kMaxThreads) ln_forward(int64_t rows, int width, int tpr, const T *__restrict__ x,
                                                          int64_t ldx, const P *__restrict__ w,
                                                          const P *__restrict__ b, float eps, T *__restrict__ y,
                                                          float *__restrict__ mean, float *__restrict__ rstd) {
  constexpr int R = kBundle<NI>;
  __shared__ float slots[2 * R][32];
  const int t = threadIdx.x & (tpr - 1), groups = blockDim.x / tpr;
  const int64_t row0 = blockIdx.x * (int64_t)groups * R + threadIdx.x / tpr;
  Pack<T, VEC> raw[R][NI];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + r * groups;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (row < rows && c < width) {
        raw[r][i] = *reinterpret_cast<const Pack<T, VEC> *>(x + row * ldx + c);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) raw[r][i].v[k] = from_f32<T>(0.f);
      }
    }
  }
  const float inv = 1.f / (float)width;
  float mu[R], rs[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float v[VEC];
      unpack(raw[r][i], v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += v[k];
    }
    mu[r] = group_sum(s, tpr, slots[r]) * inv;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool in = (i * tpr + t) * VEC < width;
      float v[VEC];
      unpack(raw[r][i], v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) q += in ? (v[k] - mu[r]) * (v[k] - mu[r]) : 0.f;
    }
    rs[r] = 1.f / sqrtf(group_sum(q, tpr, slots[R + r]) * inv + eps);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = (i * tpr + t) * VEC;
    if (c >= width) break;
    float wv[VEC], bv[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) wv[k] = 1.f, bv[k] = 0.f;
    if (w) load_f32<P, VEC>(w + c, wv);
    if (b) load_f32<P, VEC>(b + c, bv);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r * groups;
      if (row >= rows) break;
      float v[VEC];
      unpack(raw[r][i], v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = (v[k] - mu[r]) * rs[r] * wv[k] + bv[k];
      store_f32<T, VEC>(y + row * width + c, v);
    }
  }
  if (t == 0 && mean)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r * groups;
      if (row < rows) mean[row] = mu[r], rstd[row] = rs[r];
    }
}

// Rows of any width, one block a row, three sweeps (the second and third hit L2).
template <typename T, typename P>
__global__ void __launch_bounds__(kMaxThreads) ln_forward_wide(int64_t rows, int64_t width, const T *__restrict__ x,
                                                               int64_t ldx, const P *__restrict__ w,
                                                               const P *__restrict__ b, float eps, T *__restrict__ y,
                                                               float *__restrict__ mean, float *__restrict__ rstd) {
  __shared__ float slots[2][32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * ldx;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < width; c += kMaxThreads) s += to_f32(xr[c]);
    const float mu = group_sum(s, kMaxThreads, slots[0]) / (float)width;
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < width; c += kMaxThreads) {
      const float d = to_f32(xr[c]) - mu;
      q += d * d;
    }
    const float rs = 1.f / sqrtf(group_sum(q, kMaxThreads, slots[1]) / (float)width + eps);
    for (int64_t c = threadIdx.x; c < width; c += kMaxThreads) {
      const float xh = (to_f32(xr[c]) - mu) * rs;
      y[row * width + c] = from_f32<T>((w ? xh * to_f32(w[c]) : xh) + (b ? to_f32(b[c]) : 0.f));
    }
    if (threadIdx.x == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    __syncthreads();  // slots[0] is free again
  }
}

// parts: [gridDim.x][2][width] partial sums of dw and db (NULL: dx only).
template <typename T, typename P, int VEC, int NI>
__global__ void __launch_bounds__(kMaxThreads) ln_backward(int64_t rows, int width, int tpr, const T *__restrict__ dy,
                                                           int64_t lddy, const T *__restrict__ x, int64_t ldx,
                                                           const P *__restrict__ w, const float *__restrict__ mean,
                                                           const float *__restrict__ rstd, T *__restrict__ dx,
                                                           float *__restrict__ parts) {
  constexpr int R = kBundle<2 * NI>;  // two vectors, of x and of dy, for each of the forward pass's
  extern __shared__ float cols[];     // more than one group: [2][width]
  __shared__ float slots[2][2 * R][32];
  const int t = threadIdx.x & (tpr - 1), groups = blockDim.x / tpr;
  const int64_t step = (int64_t)gridDim.x * groups * R;
  const float inv = 1.f / (float)width;
  float aw[NI][VEC], ab[NI][VEC];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) aw[i][k] = ab[i][k] = 0.f;
  int turn = 0;  // the slots alternate, so a bundle's sums never meet the previous one's reads
  // every thread of a block makes the same number of turns (the sums need whole warps and blocks)
  for (int64_t base = blockIdx.x * (int64_t)groups * R; base < rows; base += step, turn ^= 1) {
    Pack<T, VEC> rx[R][NI], rg[R][NI];
    float mu[R], rs[R], m1[R], m2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = base + r * groups + threadIdx.x / tpr;
      const bool live = row < rows;
      mu[r] = live ? mean[row] : 0.f;
      rs[r] = live ? rstd[row] : 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (live && c < width) {
          rx[r][i] = *reinterpret_cast<const Pack<T, VEC> *>(x + row * ldx + c);
          rg[r][i] = *reinterpret_cast<const Pack<T, VEC> *>(dy + row * lddy + c);
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) rx[r][i].v[k] = rg[r][i].v[k] = from_f32<T>(0.f);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c >= width) break;
        float wv[VEC], xv[VEC], g[VEC];
        unpack(rx[r][i], xv);
        unpack(rg[r][i], g);
        if (w) load_f32<P, VEC>(w + c, wv);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float xh = (xv[k] - mu[r]) * rs[r];
          aw[i][k] += g[k] * xh;
          ab[i][k] += g[k];
          if (w) g[k] *= wv[k];
          s1 += g[k];
          s2 += g[k] * xh;
        }
      }
      m1[r] = group_sum(s1, tpr, slots[turn][2 * r]) * inv;
      m2[r] = group_sum(s2, tpr, slots[turn][2 * r + 1]) * inv;
    }
    if (!dx) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = base + r * groups + threadIdx.x / tpr;
      if (row >= rows) break;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c >= width) break;
        float wv[VEC], xv[VEC], g[VEC];
        unpack(rx[r][i], xv);
        unpack(rg[r][i], g);
        if (w) load_f32<P, VEC>(w + c, wv);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float xh = (xv[k] - mu[r]) * rs[r];
          g[k] = rs[r] * ((w ? g[k] * wv[k] : g[k]) - m1[r] - xh * m2[r]);
        }
        store_f32<T, VEC>(dx + row * width + c, g);
      }
    }
  }
  if (!parts) return;
  float *pw = parts + (int64_t)blockIdx.x * 2 * width, *pb = pw + width;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = (i * tpr + t) * VEC;
      if (c >= width) break;
      store_f32<float, VEC>(pw + c, aw[i]);
      store_f32<float, VEC>(pb + c, ab[i]);
    }
    return;
  }
  // the groups of a warp by shuffles, then the groups that are left one after another
  for (int o = tpr; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        aw[i][k] += __shfl_xor_sync(0xffffffffu, aw[i][k], o);
        ab[i][k] += __shfl_xor_sync(0xffffffffu, ab[i][k], o);
      }
  }
  const int apart = tpr < 32 ? 32 : tpr;
  for (int turn_of = 0; turn_of < (int)blockDim.x / apart; ++turn_of) {
    if ((int)threadIdx.x / apart == turn_of && (int)threadIdx.x % apart < tpr) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c >= width) break;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          cols[c + k] = turn_of ? cols[c + k] + aw[i][k] : aw[i][k];
          cols[width + c + k] = turn_of ? cols[width + c + k] + ab[i][k] : ab[i][k];
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) pw[c] = cols[c];
}

template <typename T, typename P>
__global__ void __launch_bounds__(kMaxThreads) ln_backward_wide(int64_t rows, int64_t width,
                                                                const T *__restrict__ dy, int64_t lddy,
                                                                const T *__restrict__ x, int64_t ldx,
                                                                const P *__restrict__ w,
                                                                const float *__restrict__ mean,
                                                                const float *__restrict__ rstd, T *__restrict__ dx) {
  __shared__ float slots[2][32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < width; c += kMaxThreads) {
      const float g = to_f32(dy[row * lddy + c]) * (w ? to_f32(w[c]) : 1.f);
      s1 += g;
      s2 += g * (to_f32(x[row * ldx + c]) - mu) * rs;
    }
    const float m1 = group_sum(s1, kMaxThreads, slots[0]) / (float)width;
    const float m2 = group_sum(s2, kMaxThreads, slots[1]) / (float)width;
    for (int64_t c = threadIdx.x; c < width; c += kMaxThreads) {
      const float g = to_f32(dy[row * lddy + c]) * (w ? to_f32(w[c]) : 1.f);
      const float xh = (to_f32(x[row * ldx + c]) - mu) * rs;
      dx[row * width + c] = from_f32<T>(rs * (g - m1 - xh * m2));
    }
    __syncthreads();
  }
}

// Partial column sums of dw and db for rows of any width: block (column tile, part), rows in strides.
template <typename T>
__global__ void __launch_bounds__(1024) ln_columns_wide(int64_t rows, int64_t width, const T *__restrict__ dy,
                                                        int64_t lddy, const T *__restrict__ x, int64_t ldx,
                                                        const float *__restrict__ mean,
                                                        const float *__restrict__ rstd, float *__restrict__ parts) {
  __shared__ float sw[32][kColTile + 1], sb[32][kColTile + 1];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * (int64_t)kColTile + lane;
  float aw = 0.f, ab = 0.f;
  if (c < width)
    for (int64_t r = blockIdx.y * 32ll + wy; r < rows; r += gridDim.y * 32ll) {
      const float g = to_f32(dy[r * lddy + c]);
      aw += g * ((to_f32(x[r * ldx + c]) - mean[r]) * rstd[r]);
      ab += g;
    }
  sw[wy][lane] = aw;
  sb[wy][lane] = ab;
  __syncthreads();
  if (wy < 2 && c < width) {
    float s = 0.f;
    for (int i = 0; i < 32; ++i) s += wy ? sb[i][lane] : sw[i][lane];
    parts[((int64_t)blockIdx.y * 2 + wy) * width + c] = s;
  }
}

// dw and db from the blocks' partial sums, in a fixed order.
template <typename P>
__global__ void __launch_bounds__(1024) ln_reduce_parts(int nparts, int64_t width, const float *__restrict__ parts,
                                                        P *__restrict__ dw, P *__restrict__ db) {
  __shared__ float sm[32][kColTile + 1];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * (int64_t)kColTile + lane;
  const int which = blockIdx.y;
  P *out = which ? db : dw;
  if (!out) return;
  float s = 0.f;
  if (c < width)
    for (int p = wy; p < nparts; p += 32) s += parts[((int64_t)p * 2 + which) * width + c];
  sm[wy][lane] = s;
  __syncthreads();
  if (wy == 0 && c < width) {
    float r = 0.f;
    for (int i = 0; i < 32; ++i) r += sm[i][lane];
    out[c] = from_f32<P>(r);
  }
}

// How the rows of one call are laid over threads.
struct LnPlan {
  int vec, items, tpr, block;  // vec = 0: the wide kernels
};

// Widest vector, then the fewest threads a row that hold it in `few` vectors (8 single elements) each, or
// in four (16) where even kMaxThreads threads cannot.
LnPlan ln_plan(int64_t width, int vec, int few) {
  const int64_t nv = (width + vec - 1) / vec;
  const int most = vec > 1 ? 4 : 16;
  if (nv > (int64_t)kMaxThreads * most) return {0, 0, kMaxThreads, kMaxThreads};
  const int enough = vec > 1 ? few : 8;
  int tpr = 1;
  while (tpr < kMaxThreads && ((int64_t)tpr * enough < nv || (tpr < 32 && tpr < nv))) tpr <<= 1;
  const int need = (int)((nv + tpr - 1) / tpr);
  const int items = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 16;
  return {vec, items, tpr, tpr > 32 ? tpr : kLnBlock};
}

template <typename T, typename P, int VEC, int NI>
void launch_forward(const LnPlan &pl, int64_t rows, int64_t width, const void *x, int64_t ldx, const void *w,
                    const void *b, float eps, void *y, float *mean, float *rstd, cudaStream_t st) {
  const int64_t rpb = pl.block / pl.tpr * kBundle<NI>;
  ln_forward<T, P, VEC, NI><<<(unsigned)((rows + rpb - 1) / rpb), pl.block, 0, st>>>(
      rows, (int)width, pl.tpr, (const T *)x, ldx, (const P *)w, (const P *)b, eps, (T *)y, mean, rstd);
}

template <typename T, typename P>
cudaError_t forward(int64_t rows, int64_t width, bool vec_ok, const void *x, int64_t ldx, const void *w,
                    const void *b, float eps, void *y, float *mean, float *rstd, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const LnPlan pl = ln_plan(width, vec_ok ? V : 1, 4);
#define SLA_LN_FWD(VEC, NI) launch_forward<T, P, VEC, NI>(pl, rows, width, x, ldx, w, b, eps, y, mean, rstd, st)
  if (pl.vec == 0)
    ln_forward_wide<T, P><<<(unsigned)std::min<int64_t>(rows, 152 * 64), kMaxThreads, 0, st>>>(
        rows, width, (const T *)x, ldx, (const P *)w, (const P *)b, eps, (T *)y, mean, rstd);
  else if (pl.vec > 1)
    pl.items == 1 ? SLA_LN_FWD(V, 1) : pl.items == 2 ? SLA_LN_FWD(V, 2) : SLA_LN_FWD(V, 4);
  else
    pl.items <= 2 ? SLA_LN_FWD(1, 2) : pl.items <= 8 ? SLA_LN_FWD(1, 8) : SLA_LN_FWD(1, 16);
#undef SLA_LN_FWD
  return cudaGetLastError();
}

template <typename T, typename P, int VEC, int NI>
int launch_backward(const LnPlan &pl, int64_t rows, int64_t width, const void *dy, int64_t lddy, const void *x,
                    int64_t ldx, const void *w, const float *mean, const float *rstd, void *dx, float *parts,
                    cudaStream_t st) {
  const int groups = pl.block / pl.tpr;
  const int64_t rpb = groups * kBundle<2 * NI>;
  // enough blocks to fill the GPU (1024 threads a multiprocessor), no more than there are bundles
  const int per_sm = std::max(1, 1024 / pl.block);
  const int grid = (int)std::min<int64_t>(std::min(sm_count() * per_sm, kMaxParts), (rows + rpb - 1) / rpb);
  const size_t smem = groups > 1 && parts ? 2 * sizeof(float) * (size_t)width : 0;
  ln_backward<T, P, VEC, NI><<<grid, pl.block, smem, st>>>(rows, (int)width, pl.tpr, (const T *)dy, lddy,
                                                           (const T *)x, ldx, (const P *)w, mean, rstd, (T *)dx, parts);
  return grid;
}

template <typename T, typename P>
cudaError_t backward(int64_t rows, int64_t width, bool vec_ok, const void *dy, int64_t lddy, const void *x,
                     int64_t ldx, const void *w, const float *mean, const float *rstd, void *dx, void *dw, void *db,
                     float *parts, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const LnPlan pl = ln_plan(width, vec_ok ? V : 1, 16 / V);  // 16 elements and their two sums fit the registers
  int nparts = 0;
  const int ctiles = (int)((width + kColTile - 1) / kColTile);
#define SLA_LN_BWD(VEC, NI) \
  launch_backward<T, P, VEC, NI>(pl, rows, width, dy, lddy, x, ldx, w, mean, rstd, dx, parts, st)
  if (pl.vec == 0) {
    if (dx)
      ln_backward_wide<T, P><<<(unsigned)std::min<int64_t>(rows, 152 * 64), kMaxThreads, 0, st>>>(
          rows, width, (const T *)dy, lddy, (const T *)x, ldx, (const P *)w, mean, rstd, (T *)dx);
    if (parts) {
      nparts = (int)std::max<int64_t>(1, std::min<int64_t>(16, (rows + 127) / 128));
      ln_columns_wide<T><<<dim3(ctiles, nparts), 1024, 0, st>>>(rows, width, (const T *)dy, lddy, (const T *)x, ldx,
                                                                mean, rstd, parts);
    }
  } else if (pl.vec > 1) {
    nparts = pl.items == 1 ? SLA_LN_BWD(V, 1) : pl.items == 2 ? SLA_LN_BWD(V, 2) : SLA_LN_BWD(V, 4);
  } else {
    nparts = pl.items <= 2 ? SLA_LN_BWD(1, 2) : pl.items <= 8 ? SLA_LN_BWD(1, 8) : SLA_LN_BWD(1, 16);
  }
#undef SLA_LN_BWD
  if (parts) ln_reduce_parts<P><<<dim3(ctiles, 2), 1024, 0, st>>>(nparts, width, parts, (P *)dw, (P *)db);
  return cudaGetLastError();
}

sla_status check_ln(int64_t rows, int64_t width, int32_t dtype, int32_t param_dtype) {
  if (rows < 0 || width < 1 || width > ((int64_t)1 << 24) || rows > ((int64_t)1 << 31) - 1) return SLA_INVALID_ARG;
  if (!net_dtype(dtype)) return SLA_INVALID_ARG;
  return param_dtype == dtype || param_dtype == SLA_F32 ? SLA_OK : SLA_INVALID_ARG;
}

// A matrix of rows `ld` elements apart: not NULL, aligned to its elements, rows not overlapping.
sla_status check_rows(const void *p, int64_t rows, int64_t width, int64_t ld, int32_t dtype) {
  if (rows == 0) return SLA_OK;
  if (!p || !aligned(p, net_size(dtype))) return SLA_INVALID_ARG;
  return ld >= width || rows == 1 ? SLA_OK : SLA_INVALID_ARG;
}

bool vec_rows(const void *p, int64_t width, int64_t ld, int32_t dtype) {
  const size_t e = net_size(dtype);
  return aligned(p, 16) && (width * e) % 16 == 0 && (ld * (int64_t)e) % 16 == 0;
}

// Calls f with the element and parameter types of a call.
template <typename F>
cudaError_t by_type(int32_t dtype, int32_t param_dtype, F &&f) {
  if (dtype == SLA_F32) return f(float{}, float{});
  if (dtype == SLA_F16) return param_dtype == SLA_F16 ? f(f16{}, f16{}) : f(f16{}, float{});
  return param_dtype == SLA_BF16 ? f(bf16{}, bf16{}) : f(bf16{}, float{});
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API sla_status sla_layernorm(int64_t rows, int64_t width, int32_t dtype, int32_t param_dtype, const void *x,
                                 int64_t ldx, const void *weight, const void *bias, double eps, void *y, float *mean,
                                 float *rstd, void *stream) {
  SLA_CHECK(check_ln(rows, width, dtype, param_dtype));
  if (!(eps >= 0.0) || !std::isfinite(eps)) return SLA_INVALID_ARG;
  SLA_CHECK(check_rows(x, rows, width, ldx, dtype));
  SLA_CHECK(check_rows(y, rows, width, width, dtype));
  const size_t ps = net_size(param_dtype);
  if (!aligned(weight, ps) || !aligned(bias, ps) || !aligned(mean, 4) || !aligned(rstd, 4)) return SLA_INVALID_ARG;
  if (rows == 0) return SLA_OK;
  const bool vec = vec_rows(x, width, ldx, dtype) && vec_rows(y, width, width, dtype) && aligned(weight, 16) &&
                   aligned(bias, 16);
  const cudaError_t e = by_type(dtype, param_dtype, [&](auto t, auto p) {
    return forward<decltype(t), decltype(p)>(rows, width, vec, x, ldx, weight, bias, (float)eps, y, mean, rstd,
                                             (cudaStream_t)stream);
  });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

SLA_API size_t sla_layernorm_backward_workspace_bytes(int64_t rows, int64_t width, int32_t dtype) {
  if (check_ln(rows, width, dtype, dtype) != SLA_OK) return 0;
  // the most blocks that any layout of these rows leaves partial sums from
  const int64_t parts = std::max<int64_t>(16, std::min<int64_t>(kMaxParts, rows));
  return align256((size_t)parts * 2 * (size_t)width * sizeof(float));
}

SLA_API sla_status sla_layernorm_backward(int64_t rows, int64_t width, int32_t dtype, int32_t param_dtype,
                                          const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                          const void *weight, const float *mean, const float *rstd, void *dx,
                                          void *dweight, void *dbias, void *workspace, size_t ws_bytes,
                                          void *stream) {
  SLA_CHECK(check_ln(rows, width, dtype, param_dtype));
  SLA_CHECK(check_rows(dy, rows, width, lddy, dtype));
  SLA_CHECK(check_rows(x, rows, width, ldx, dtype));
  const size_t ps = net_size(param_dtype);
  if (!aligned(weight, ps) || !aligned(dweight, ps) || !aligned(dbias, ps) || !aligned(dx, net_size(dtype)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return SLA_INVALID_ARG;
  if (rows > 0 && (!mean || !rstd)) return SLA_INVALID_ARG;
  const bool sums = dweight || dbias;
  if (sums) {
    if (!workspace || !aligned(workspace, 256)) return SLA_INVALID_ARG;
    if (ws_bytes < sla_layernorm_backward_workspace_bytes(rows, width, dtype)) return SLA_WORKSPACE_TOO_SMALL;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // sums over no rows
    cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, ps * (size_t)width, st) : cudaSuccess;
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, ps * (size_t)width, st);
    return e == cudaSuccess ? SLA_OK : fail(e);
  }
  if (!dx && !sums) return SLA_OK;
  const bool vec = vec_rows(dy, width, lddy, dtype) && vec_rows(x, width, ldx, dtype) &&
                   vec_rows(dx, width, width, dtype) && aligned(weight, 16);
  const cudaError_t e = by_type(dtype, param_dtype, [&](auto t, auto p) {
    return backward<decltype(t), decltype(p)>(rows, width, vec, dy, lddy, x, ldx, weight, mean, rstd, dx, dweight,
                                              dbias, sums ? (float *)workspace : nullptr, st);
  });
  if (e != cudaSuccess) return fail(e);
  count_launches(sums ? 2 : 1);
  return SLA_OK;
}

}  // extern "C"
