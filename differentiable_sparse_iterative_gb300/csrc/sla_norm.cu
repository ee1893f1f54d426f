// Layer norm over the rows of a matrix, forward and backward.
//
//   y = (x - mu) rstd w + b,   mu = mean(x),  rstd = (mean((x - mu)^2) + eps)^(-1/2)     per row
//   dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),   dxh = dy w,  xh = (x - mu) rstd     per row
//   dw = sum over rows of dy xh,   db = sum over rows of dy                              per column
//
// Both directions are bound by memory (8 and 12 operations an element), so each is one pass: a
// group of `tpr` threads (a power of two: part of a warp, a warp, or the block) keeps a row in
// registers as NI vectors of 16 bytes a thread, and reduces with shuffles (and shared memory beyond
// a warp).  The variance is the mean of squared differences from the mean, taken from the registers
// in a second sweep: the one-sweep form mean(x^2) - mu^2 cancels when a row sits far from zero.
//
// Blocks are persistent.  The next rows are loaded while the present ones are worked on, and a thread
// sees the same columns in every row, so it reads the weights once, and dw and db accumulate in its
// registers, then across the block in a fixed order, then over the blocks' partial sums in a second
// kernel.  No atomics: the same call gives the same bits.
//
// Widths that no vector divides: row r starts (r * width) mod VEC elements behind a 16-byte boundary,
// which repeats every `classes` = VEC / gcd(width, VEC) rows.  A block takes the rows of one class, so its
// threads keep their columns: the aligned vectors inside of the row, and one element each of the at
// most VEC - 1 before and after them (Edge).  Arrays whose rows do not start at the same boundary (strided
// or odd views) and rows wider than the registers of a 512-thread block hold take the *_any
// kernels, which read element by element and re-read from L2.
//
// Measured, forward and backward together, against the copy rate of 6.69 TB/s: 1,000,000 x 64 bfloat16 122 us
// (0.78), 65536 x 1024 bfloat16 140 us (0.72), x 1001 152 us (0.64), 300,000 x 100 bfloat16 86 us (0.52), 65536 x 512
// float32 125 us (0.80).  Beyond 256 columns 16-bit rows wait for the two sums of a row, one after the other, across warps
// (stalls on shared memory and barriers; issue 46 to 49 %, DRAM 46 to 51 %).  The *_any kernels: 4096 x 40000 bfloat16 997 us
// (0.25), 65536 x 1024 as a view one element off 729 us (0.14).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

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
constexpr int kColTile = 32;      // columns of a block of the column sums
constexpr int kMaxParts = 1216;   // blocks that leave partial column sums (8 a multiprocessor)

// Sums over the tpr threads of a group, the same values in each of them.  `slot` (16 K floats) must not be in
// use by an earlier sum that a thread still reads; for tpr > 32 every thread of the block takes part.
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int tpr, float *slot) {
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

__device__ __forceinline__ float group_sum(float v, int tpr, float *slot) {
  float a[1] = {v};
  group_sums(a, tpr, slot);
  return a[0];
}

// 16 bytes of a row, as pairs of float32.
template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T), pairs = n / 2;
  uint4 q;
  __device__ __forceinline__ void load(const T *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void values(float2 (&v)[pairs]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
      v[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      v[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = unpair16(w[k], T{});
    }
  }
  static __device__ __forceinline__ void store(T *p, const float2 (&v)[pairs]) {
    uint4 q;
    if constexpr (sizeof(T) == 4)
      q = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    else
      q = make_uint4(pair16(v[0].x, v[0].y, T{}), pair16(v[1].x, v[1].y, T{}), pair16(v[2].x, v[2].y, T{}),
                     pair16(v[3].x, v[3].y, T{}));
    *reinterpret_cast<uint4 *>(p) = q;
  }
};

// Columns [c, c + 2 PAIRS) of a parameter as pairs, `other` where there is none.  vec: they may be read at once.
template <typename P, int PAIRS>
__device__ __forceinline__ void param_pairs(const P *p, int c, bool in, float other, bool vec, float2 (&v)[PAIRS]) {
  float e[2 * PAIRS];
  if (vec && p && in) {
    load_f32<P, 2 * PAIRS>(p + c, e);
  } else {
#pragma unroll
    for (int k = 0; k < 2 * PAIRS; ++k) e[k] = in ? (p ? to_f32(p[c + k]) : other) : 0.f;
  }
#pragma unroll
  for (int k = 0; k < PAIRS; ++k) v[k] = f2(e[2 * k], e[2 * k + 1]);
}

// Which rows and columns a thread works on.
struct Share {
  int t, first;        // thread of the group; column of its first vector
  int end;             // the column that no vector reaches
  int edge;            // column of its single element, or -1
  uint32_t row, step;  // its first row; rows from turn to turn (there are less than 2^31 rows)
  uint32_t next;       // rows between the rows of a bundle
};

template <int VEC, int R>
__device__ __forceinline__ Share share_of(int width, int tpr, int classes, int shift, int64_t shift_step) {
  const int groups = blockDim.x / tpr, cls = blockIdx.x % classes;
  Share s;
  s.t = threadIdx.x & (tpr - 1);
  const int head = min(width, (VEC - (int)((shift + cls * shift_step) % VEC)) % VEC), body = (width - head) / VEC * VEC;
  s.first = head + s.t * VEC;
  s.end = head + body;
  const int e = s.t < head ? s.t : s.t + body;
  s.edge = e < width ? e : -1;
  s.next = groups * classes;
  s.row = ((blockIdx.x / classes) * R * groups + threadIdx.x / tpr) * classes + cls;
  s.step = (gridDim.x / classes) * R * groups * classes;
  return s;
}

// Weights stay in registers while they are not more than 16 columns a thread.
template <typename T, int NI>
inline constexpr bool kKeepParams = NI * Vec<T>::n <= 16;

// shift: elements between a 16-byte boundary and row 0, shift_step: added by each row (mod VEC).
template <typename T, typename P, int NI, int R, bool Edge>
__global__ void __launch_bounds__(NI == 1 ? kLnBlock : kMaxThreads, NI == 1 ? 4 : 1)
    ln_forward(uint32_t rows, int width, int tpr, int classes, int shift, int64_t shift_step, int pvec,
               const T *__restrict__ x, int64_t ldx, const P *__restrict__ w, const P *__restrict__ b, float eps,
               T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
  using V = Vec<T>;
  constexpr int N = V::n, H = V::pairs;
  constexpr bool keep = kKeepParams<T, NI>;
  __shared__ float slots[2][2][R * 16];
  const Share s = share_of<N, R>(width, tpr, classes, shift, shift_step);
  const int apart = tpr * N;
  const float inv = 1.f / (float)width;
  float2 wk[keep ? NI : 1][H], bk[keep ? NI : 1][H];
  if constexpr (keep)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = s.first + i * apart;
      param_pairs<P, H>(w, c, c < s.end, 1.f, pvec, wk[i]);
      param_pairs<P, H>(b, c, c < s.end, 0.f, pvec, bk[i]);
    }
  const bool edge = Edge && s.edge >= 0;
  float we = 1.f, be = 0.f;
  if (edge && w) we = to_f32(w[s.edge]);
  if (edge && b) be = to_f32(b[s.edge]);
  // As loaded: a conversion here would wait for the load.
  V raw[R][NI];
  T raw_e[R];
  const T *px = x + s.row * ldx;  // the row that is asked for next
  T *py = y + s.row * (int64_t)width;
  const int64_t x_next = s.next * ldx, x_step = s.step * ldx;
  const int64_t y_next = s.next * (int64_t)width, y_step = s.step * (int64_t)width;
  auto ask = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row + r * s.next < rows;
      raw_e[r] = from_f32<T>(0.f);
      if (edge && live) raw_e[r] = px[r * x_next + s.edge];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = s.first + i * apart;
        raw[r][i].q = make_uint4(0, 0, 0, 0);
        if (live && c < s.end) raw[r][i].load(px + r * x_next + c);
      }
    }
    px += x_step;
  };
  ask(s.row);
  int turn = 0;  // the slots alternate, so a turn's sums never meet the previous one's reads
  // every thread of a block makes the same number of turns (the sums need whole warps and blocks)
  const uint32_t lead = s.row - threadIdx.x / tpr * classes;
  for (uint32_t ahead = lead, row = s.row; ahead < rows; ahead += s.step, row += s.step, py += y_step, turn ^= 1) {
    float2 v[R][NI][H];
    float sum[R], sq[R], ve[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        raw[r][i].values(v[r][i]);
#pragma unroll
        for (int k = 0; k < H; ++k) a = add2(a, v[r][i][k]);
      }
      ve[r] = Edge ? to_f32(raw_e[r]) : 0.f;
      sum[r] = a.x + a.y + ve[r];
    }
    if (ahead + s.step < rows) ask(row + s.step);
    group_sums<R>(sum, tpr, slots[turn][0]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mu = sum[r] * inv;
      const float2 minus = f2(-mu, -mu);
      sq[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float2 a = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < H; ++k) {
          v[r][i][k] = add2(v[r][i][k], minus);
          a = fma2(v[r][i][k], v[r][i][k], a);
        }
        sq[r] += s.first + i * apart < s.end ? a.x + a.y : 0.f;  // no differences where there is no row
      }
      if (edge) {
        ve[r] -= mu;
        sq[r] += ve[r] * ve[r];
      }
      sum[r] = mu;
    }
    group_sums<R>(sq, tpr, slots[turn][1]);
#pragma unroll
    for (int r = 0; r < R; ++r) sq[r] = rsqrtf(sq[r] * inv + eps);  // 2 units in the last place
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = s.first + i * apart;
      float2 wv[H], bv[H];
      if constexpr (keep) {
#pragma unroll
        for (int k = 0; k < H; ++k) wv[k] = wk[i][k], bv[k] = bk[i][k];
      } else {
        param_pairs<P, H>(w, c, c < s.end, 1.f, pvec, wv);
        param_pairs<P, H>(b, c, c < s.end, 0.f, pvec, bv);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int k = 0; k < H; ++k) v[r][i][k] = fma2(mul2(v[r][i][k], f2(sq[r], sq[r])), wv[k], bv[k]);
        if (row + r * s.next < rows && c < s.end) V::store(py + r * y_next + c, v[r][i]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t at = row + r * s.next;
      if (at >= rows) continue;
      if (edge) py[r * y_next + s.edge] = from_f32<T>(ve[r] * sq[r] * we + be);
      if (s.t == 0 && mean) {
        mean[at] = sum[r];
        rstd[at] = sq[r];
      }
    }
  }
}

// Rows of any width and alignment, one block a row, three sweeps (the second and third hit L2).
template <typename T, typename P>
__global__ void __launch_bounds__(kMaxThreads) ln_forward_any(int64_t rows, int64_t width, const T *__restrict__ x,
                                                              int64_t ldx, const P *__restrict__ w,
                                                              const P *__restrict__ b, float eps, T *__restrict__ y,
                                                              float *__restrict__ mean, float *__restrict__ rstd) {
  __shared__ float slots[2][16];
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
    if (threadIdx.x == 0 && mean) {
      mean[row] = mu;
      rstd[row] = rs;
    }
    __syncthreads();  // the slots are free again
  }
}

// parts: [gridDim.x][2][width] partial sums of dw and db (NULL: dx only).
template <typename T, typename P, int NI, int R, bool Edge>
__global__ void __launch_bounds__(NI == 1 ? kLnBlock : kMaxThreads, NI == 1 ? 3 : 1)
    ln_backward(uint32_t rows, int width, int tpr, int classes, int shift, int64_t shift_step, int pvec,
                const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx, const P *__restrict__ w,
                const float *__restrict__ mean, const float *__restrict__ rstd, T *__restrict__ dx,
                float *__restrict__ parts) {
  using V = Vec<T>;
  constexpr int N = V::n, H = V::pairs;
  constexpr bool keep = kKeepParams<T, NI>;
  extern __shared__ float cols[];  // more than one group: [2][width]
  __shared__ float slots[2][2 * R * 16];
  grid_dependency_launch();  // ln_reduce_parts starts as multiprocessors become free, and waits there
  const Share s = share_of<N, R>(width, tpr, classes, shift, shift_step);
  const int apart = tpr * N, groups = blockDim.x / tpr;
  const float inv = 1.f / (float)width;
  float2 wk[keep ? NI : 1][H], aw[NI][H], ab[NI][H];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = s.first + i * apart;
    if constexpr (keep) param_pairs<P, H>(w, c, c < s.end, 1.f, pvec, wk[i]);
#pragma unroll
    for (int k = 0; k < H; ++k) aw[i][k] = ab[i][k] = f2(0.f, 0.f);
  }
  const bool edge = Edge && s.edge >= 0;
  float we = 1.f, awe = 0.f, abe = 0.f;
  if (edge && w) we = to_f32(w[s.edge]);
  V rx[R][NI], rg[R][NI];
  float rm[R], rr[R];
  T ex[R], eg[R];
  const T *px = x + s.row * ldx, *pg = dy + s.row * lddy;  // the rows that are asked for next
  T *pd = dx + s.row * (int64_t)width;
  const int64_t x_next = s.next * ldx, g_next = s.next * lddy, d_next = s.next * (int64_t)width;
  auto ask = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r, row += s.next) {
      const bool live = row < rows;
      rm[r] = live ? mean[row] : 0.f;
      rr[r] = live ? rstd[row] : 0.f;
      ex[r] = eg[r] = from_f32<T>(0.f);
      if (edge && live) {
        ex[r] = px[r * x_next + s.edge];
        eg[r] = pg[r * g_next + s.edge];
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = s.first + i * apart;
        rx[r][i].q = rg[r][i].q = make_uint4(0, 0, 0, 0);
        if (live && c < s.end) {
          rx[r][i].load(px + r * x_next + c);
          rg[r][i].load(pg + r * g_next + c);
        }
      }
    }
    px += s.step * ldx;
    pg += s.step * lddy;
  };
  ask(s.row);
  int turn = 0;
  const uint32_t lead = s.row - threadIdx.x / tpr * classes;
  for (uint32_t ahead = lead, row = s.row; ahead < rows; ahead += s.step, row += s.step, turn ^= 1) {
    float2 xh[R][NI][H], g[R][NI][H];
    float sums[2 * R], rs[R], xe[R], ge[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rs[r] = rr[r];
      float2 a1 = f2(0.f, 0.f), a2 = a1;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        // Outside of the row dy is 0 and so has to be xh: (0 - mean) rstd may pass the largest float32.
        const float inside = s.first + i * apart < s.end ? rs[r] : 0.f;
        const float2 scale = f2(inside, inside);
        float2 wv[H];
        if constexpr (keep) {
#pragma unroll
          for (int k = 0; k < H; ++k) wv[k] = wk[i][k];
        } else {
          const int c = s.first + i * apart;
          param_pairs<P, H>(w, c, c < s.end, 1.f, pvec, wv);
        }
        rx[r][i].values(xh[r][i]);
        rg[r][i].values(g[r][i]);
#pragma unroll
        for (int k = 0; k < H; ++k) {
          xh[r][i][k] = mul2(add2(xh[r][i][k], f2(-rm[r], -rm[r])), scale);
          aw[i][k] = fma2(g[r][i][k], xh[r][i][k], aw[i][k]);
          ab[i][k] = add2(ab[i][k], g[r][i][k]);
          g[r][i][k] = mul2(g[r][i][k], wv[k]);
          a1 = add2(a1, g[r][i][k]);
          a2 = fma2(g[r][i][k], xh[r][i][k], a2);
        }
      }
      sums[2 * r] = a1.x + a1.y;
      sums[2 * r + 1] = a2.x + a2.y;
      xe[r] = ge[r] = 0.f;
      if (edge) {
        const float g1 = to_f32(eg[r]);
        xe[r] = (to_f32(ex[r]) - rm[r]) * rs[r];
        awe += g1 * xe[r];
        abe += g1;
        ge[r] = g1 * we;
        sums[2 * r] += ge[r];
        sums[2 * r + 1] += ge[r] * xe[r];
      }
    }
    if (ahead + s.step < rows) ask(row + s.step);
    group_sums<2 * R>(sums, tpr, slots[turn]);
    T *out = pd;
    pd += s.step * (int64_t)width;
    if (!dx) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float m1 = -sums[2 * r] * inv, m2 = -sums[2 * r + 1] * inv;
      if (row + r * s.next >= rows) continue;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = s.first + i * apart;
#pragma unroll
        for (int k = 0; k < H; ++k)
          g[r][i][k] = mul2(fma2(xh[r][i][k], f2(m2, m2), add2(g[r][i][k], f2(m1, m1))), f2(rs[r], rs[r]));
        if (c < s.end) V::store(out + r * d_next + c, g[r][i]);
      }
      if (edge) out[r * d_next + s.edge] = from_f32<T>(rs[r] * (ge[r] + m1 + xe[r] * m2));
    }
  }
  if (!parts) return;
  float *pw = parts + (int64_t)blockIdx.x * 2 * width, *pb = pw + width;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = s.first + i * apart;
      if (c >= s.end) break;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        pw[c + 2 * k] = aw[i][k].x, pw[c + 2 * k + 1] = aw[i][k].y;
        pb[c + 2 * k] = ab[i][k].x, pb[c + 2 * k + 1] = ab[i][k].y;
      }
    }
    if (edge) pw[s.edge] = awe, pb[s.edge] = abe;
    return;
  }
  // the groups of a warp by shuffles, then what is left one after another
  for (int o = tpr; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int k = 0; k < H; ++k) {
        aw[i][k].x += __shfl_xor_sync(0xffffffffu, aw[i][k].x, o);
        aw[i][k].y += __shfl_xor_sync(0xffffffffu, aw[i][k].y, o);
        ab[i][k].x += __shfl_xor_sync(0xffffffffu, ab[i][k].x, o);
        ab[i][k].y += __shfl_xor_sync(0xffffffffu, ab[i][k].y, o);
      }
    if (Edge) {
      awe += __shfl_xor_sync(0xffffffffu, awe, o);
      abe += __shfl_xor_sync(0xffffffffu, abe, o);
    }
  }
  const int size = tpr < 32 ? 32 : tpr;
  for (int from = 0; from < (int)blockDim.x; from += size) {
    if ((int)threadIdx.x >= from && (int)threadIdx.x < from + tpr) {
      auto put = [&](int c, float a, float d) {
        cols[c] = from ? cols[c] + a : a;
        cols[width + c] = from ? cols[width + c] + d : d;
      };
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = s.first + i * apart;
        if (c >= s.end) break;
#pragma unroll
        for (int k = 0; k < H; ++k) {
          put(c + 2 * k, aw[i][k].x, ab[i][k].x);
          put(c + 2 * k + 1, aw[i][k].y, ab[i][k].y);
        }
      }
      if (edge) put(s.edge, awe, abe);
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) pw[c] = cols[c];
}

template <typename T, typename P>
__global__ void __launch_bounds__(kMaxThreads) ln_backward_any(int64_t rows, int64_t width, const T *__restrict__ dy,
                                                               int64_t lddy, const T *__restrict__ x, int64_t ldx,
                                                               const P *__restrict__ w,
                                                               const float *__restrict__ mean,
                                                               const float *__restrict__ rstd, T *__restrict__ dx) {
  __shared__ float slots[2][16];
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
__global__ void __launch_bounds__(1024) ln_columns_any(int64_t rows, int64_t width, const T *__restrict__ dy,
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
  grid_dependency_wait();
  if (!out) return;
  float s = 0.f;
  if (c < width)
#pragma unroll 8
    for (int p = wy; p < nparts; p += 32) s += parts[((int64_t)p * 2 + which) * width + c];
  sm[wy][lane] = s;
  __syncthreads();
  if (wy == 0 && c < width) {
    float r = 0.f;
    for (int i = 0; i < 32; ++i) r += sm[i][lane];
    out[c] = from_f32<P>(r);
  }
}

// How the rows of one call are laid over threads; items = 0: the *_any kernels.
struct LnPlan {
  int items, tpr, block, classes, shift;
  int64_t shift_step;
  bool edge;  // rows have elements outside of their aligned vectors
  // whole vectors of a parameter may be read at once
  bool pvec(std::initializer_list<const void *> params) const {
    for (const void *p : params)
      if (!aligned(p, 16)) return false;
    return !edge;
  }
};

struct Rows {
  const void *p;
  int64_t ld;
};

// The fewest threads a row that hold it in two vectors each, or in four where even kMaxThreads threads
// cannot.  The arrays have to start every row at the same place behind a 16-byte boundary.
LnPlan ln_plan(int64_t width, int32_t dtype, std::initializer_list<Rows> arrays) {
  const int e = (int)net_size(dtype), vec = 16 / e;
  LnPlan pl{0, kMaxThreads, kMaxThreads, 1, 0, 0, false};
  pl.shift = (int)((uintptr_t)arrays.begin()->p % 16 / e);
  pl.shift_step = arrays.begin()->ld % vec;
  for (const Rows &a : arrays)
    if (a.p && ((int)((uintptr_t)a.p % 16 / e) != pl.shift || a.ld % vec != pl.shift_step)) return pl;
  while ((pl.classes * pl.shift_step) % vec) pl.classes *= 2;
  pl.edge = pl.shift || pl.shift_step || width % vec;
  const int64_t nv = width / vec;
  if (nv > kMaxThreads * 4) return pl;
  int tpr = pl.edge ? 2 * vec : 1;  // at most 2 (vec - 1) single elements
  // (float32's vectors hold half as much: one each up to 256 threads, 61 -> 47 us forward at 65536 x 512)
  const int alone = e == 4 ? 256 : 32;
  while (tpr < kMaxThreads && (2 * tpr < nv || (tpr < alone && tpr < nv))) tpr <<= 1;
  const int64_t need = (nv + tpr - 1) / tpr;
  pl.items = need <= 1 ? 1 : need <= 2 ? 2 : 4;
  pl.tpr = tpr;
  pl.block = std::max(tpr, kLnBlock);
  return pl;
}

// Blocks that fill the GPU with `threads` a multiprocessor, in whole sets of classes, no more than there are bundles.
int ln_grid(const LnPlan &pl, int64_t rows, int64_t rows_a_turn, int threads) {
  const int64_t most = std::min(sm_count() * std::max(1, threads / pl.block), kMaxParts);
  const int64_t need = ((rows + pl.classes - 1) / pl.classes + rows_a_turn - 1) / rows_a_turn;
  return (int)(std::max<int64_t>(1, std::min<int64_t>(most / pl.classes, need)) * pl.classes);
}

template <typename T, typename P, int NI, int R, bool Edge>
void launch_forward(const LnPlan &pl, int64_t rows, int64_t width, const void *x, int64_t ldx, const void *w,
                    const void *b, float eps, void *y, float *mean, float *rstd, cudaStream_t st) {
  // as many as run at once (beyond one vector a thread registers admit half as many: 11.9 -> 9.7 us at 5003 x 1001)
  const int grid = ln_grid(pl, rows, pl.block / pl.tpr * R, NI == 1 ? 1024 : 512);
  ln_forward<T, P, NI, R, Edge><<<grid, pl.block, 0, st>>>((uint32_t)rows, (int)width, pl.tpr, pl.classes, pl.shift,
                                                           pl.shift_step, pl.pvec({w, b}), (const T *)x, ldx,
                                                           (const P *)w, (const P *)b, eps, (T *)y, mean, rstd);
}

template <typename T, typename P>
cudaError_t forward(int64_t rows, int64_t width, const LnPlan &pl, const void *x, int64_t ldx, const void *w,
                    const void *b, float eps, void *y, float *mean, float *rstd, cudaStream_t st) {
#define SLA_LN_FWD(NI, R)                                                                                       \
  (pl.edge ? launch_forward<T, P, NI, R, true>(pl, rows, width, x, ldx, w, b, eps, y, mean, rstd, st)           \
           : launch_forward<T, P, NI, R, false>(pl, rows, width, x, ldx, w, b, eps, y, mean, rstd, st))
  if (pl.items == 0)
    ln_forward_any<T, P><<<(unsigned)std::min<int64_t>(rows, sm_count() * 64), kMaxThreads, 0, st>>>(
        rows, width, (const T *)x, ldx, (const P *)w, (const P *)b, eps, (T *)y, mean, rstd);
  else
    pl.items == 1 ? SLA_LN_FWD(1, 2) : pl.items == 2 ? SLA_LN_FWD(2, 1) : SLA_LN_FWD(4, 1);
#undef SLA_LN_FWD
  return cudaGetLastError();
}

template <typename T, typename P, int NI, int R, bool Edge>
int launch_backward(const LnPlan &pl, int64_t rows, int64_t width, const void *dy, int64_t lddy, const void *x,
                    int64_t ldx, const void *w, const float *mean, const float *rstd, void *dx, float *parts,
                    cudaStream_t st) {
  const int groups = pl.block / pl.tpr, grid = ln_grid(pl, rows, groups * R, NI == 1 ? 768 : 512);
  const size_t smem = groups > 1 && parts ? 2 * sizeof(float) * (size_t)width : 0;
  ln_backward<T, P, NI, R, Edge><<<grid, pl.block, smem, st>>>((uint32_t)rows, (int)width, pl.tpr, pl.classes, pl.shift,
                                                               pl.shift_step, pl.pvec({w}), (const T *)dy, lddy,
                                                               (const T *)x, ldx, (const P *)w, mean, rstd, (T *)dx,
                                                               parts);
  return grid;
}

template <typename T, typename P>
cudaError_t backward(int64_t rows, int64_t width, const LnPlan &pl, const void *dy, int64_t lddy, const void *x,
                     int64_t ldx, const void *w, const float *mean, const float *rstd, void *dx, void *dw, void *db,
                     float *parts, cudaStream_t st) {
  int nparts = 0;
  const int ctiles = (int)((width + kColTile - 1) / kColTile);
#define SLA_LN_BWD(NI, R)                                                                                           \
  (pl.edge ? launch_backward<T, P, NI, R, true>(pl, rows, width, dy, lddy, x, ldx, w, mean, rstd, dx, parts, st)    \
           : launch_backward<T, P, NI, R, false>(pl, rows, width, dy, lddy, x, ldx, w, mean, rstd, dx, parts, st))
  if (pl.items == 0) {
    if (dx)
      ln_backward_any<T, P><<<(unsigned)std::min<int64_t>(rows, sm_count() * 64), kMaxThreads, 0, st>>>(
          rows, width, (const T *)dy, lddy, (const T *)x, ldx, (const P *)w, mean, rstd, (T *)dx);
    if (parts) {
      nparts = (int)std::max<int64_t>(1, std::min<int64_t>(16, (rows + 127) / 128));
      ln_columns_any<T><<<dim3(ctiles, nparts), 1024, 0, st>>>(rows, width, (const T *)dy, lddy, (const T *)x, ldx,
                                                               mean, rstd, parts);
    }
  } else {
    nparts = pl.items == 1 ? SLA_LN_BWD(1, 1) : pl.items == 2 ? SLA_LN_BWD(2, 1) : SLA_LN_BWD(4, 1);
  }
#undef SLA_LN_BWD
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !parts) return err;
  LaunchConfig cfg(dim3(ctiles, 2), 1024, 0, st, true);
  return cudaLaunchKernelEx(&cfg.c, ln_reduce_parts<P>, nparts, width, (const float *)parts, (P *)dw, (P *)db);
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
  if (!mean != !rstd) return SLA_INVALID_ARG;
  if (rows == 0) return SLA_OK;
  const LnPlan pl = ln_plan(width, dtype, {{x, rows == 1 ? width : ldx}, {y, width}});
  const cudaError_t e = by_type(dtype, param_dtype, [&](auto t, auto p) {
    return forward<decltype(t), decltype(p)>(rows, width, pl, x, ldx, weight, bias, (float)eps, y, mean, rstd,
                                             (cudaStream_t)stream);
  });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

SLA_API size_t sla_layernorm_backward_workspace_bytes(int64_t rows, int64_t width, int32_t dtype) {
  if (check_ln(rows, width, dtype, dtype) != SLA_OK) return 0;
  // the most blocks that any layout of these rows leaves partial sums from (whole sets of up to 8 classes)
  const int64_t parts = std::max<int64_t>(16, std::min<int64_t>(kMaxParts, rows + 7));
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
  const bool one = rows == 1;  // a single row has no distance to the next
  const LnPlan pl = ln_plan(width, dtype, {{x, one ? width : ldx}, {dy, one ? width : lddy}, {dx, width}});
  const cudaError_t e = by_type(dtype, param_dtype, [&](auto t, auto p) {
    return backward<decltype(t), decltype(p)>(rows, width, pl, dy, lddy, x, ldx, weight, mean, rstd, dx, dweight,
                                              dbias, sums ? (float *)workspace : nullptr, st);
  });
  if (e != cudaSuccess) return fail(e);
  count_launches(sums ? 2 : 1);
  return SLA_OK;
}

}  // extern "C"
