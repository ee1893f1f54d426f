// Tensor-core matrix products of the gated feed-forward block and the linear layer, with the elementwise work of both as
// their epilogues.
//
//   C[m][n] = sum over segments s, sum over k of A_s(m, k) B_s(n, k)
//
// Operands are 16-bit and read by TMA from three-dimensional tensors (contiguous dimension, rows,
// sheets).  A segment names a sheet of A and one of B: the sum over both halves of [g u], which lie in
// two sheets, has two.  float32 data is held as three bfloat16 parts x = x0 + x1 + x2 of falling size (8
// bits each, 24 in all), in sheets of their own; the six products x_i y_j with i + j <= 2 give float32's
// accuracy (what is dropped is below 2^-26 of a term).  A stage then holds all parts of its k, so that
// six products share six tiles (two tiles a product left the smaller tile shapes waiting for L2: 1.53 us
// a block of 64 k instead of 1.0), and the five small products have an accumulator of their own: the
// tensor core drops up to a unit of the running sum for every 16 k, which the small products
// would feel five times as often in the large one's.  The large one takes 512 of k at a time (kRun: 512 / 16 *
// 2^-24 * 2/3 = 1.3e-6, a plain float32 product's error; measured 1.0e-6 to 1.5e-6, and 2.8e-6 to 4.1e-6 in runs of
// 2048); the epilogue warps add the runs up in float32, in a scratch of their own that stays in L2, while the next
// run is under way (4,096 tokens, 1024 -> 4096, forward: 395 us, 384 in runs of 2048, 486 with splits in their place).
// Either operand may be k-major (k contiguous) or mn-major (rows or columns contiguous): the tensor
// core reads both from the 128-byte swizzled tiles that TMA writes, so no operand is transposed.
//
// One block (or a pair of blocks on two multiprocessors, CG = 2, each with half of B and its own 128
// rows) keeps a tile of 128 CG x BN in tensor memory, twice: while eight warps (sixteen with the widest 16-bit tiles)
// empty one through the epilogue, one warp feeds the next tile's mma and another its TMA loads.  Blocks are
// persistent and take tiles in bands of kBand tile rows, so that what the running blocks read stays in L2.
//
// Measured at 16,384 tokens, 1024 -> 4096 -> 1024 in bfloat16, where cuBLAS reaches 1,725 to 1,902 TFLOP/s: dx,
// dw_in and dw_out in one launch 1,836 TFLOP/s (tensor cores 96 % busy), out 1,531, gate 1,487 (its three arrays
// are 403 MB), gate backward 769: bound by its loads and stores of 1.07 GB a 32,768 tokens, not by its product.
// With few tiles a block (4,096 tokens) filling, draining and the last epilogue are most of a launch.
#pragma once

#include <atomic>

#include "sla_act.cuh"
#include "sla_net.cuh"
#include "sla_tc.cuh"

namespace sla {

enum Epilogue {
  kStore,     // c = sum (+ bias), or the float32 sums of one split of k
  kGate,      // columns of g and u side by side: h = act(g) u; u act'(g) and act(g) kept for kGateBack
  kGateBack,  // sum = dh: dg = dh (u act'(g)), du = dh act(g)
  kLinear,    // c = act(sum + bias) + residual; act'(sum + bias) kept
  kAdd,       // c = sum + bias + residual: kLinear without an activation, whose registers it does without
};
// Whether an epilogue writes the caller's array straight from the registers.
template <int EPI>
inline constexpr bool kPlainStore = EPI == kStore || EPI == kLinear || EPI == kAdd;
template <int EPI>
inline constexpr bool kLayer = EPI == kLinear || EPI == kAdd;

constexpr int kBand = 8;
constexpr int kMaxSegments = 2;

template <typename T>
inline constexpr int kParts = sizeof(T) == 4 ? 3 : 1;  // sheets that make one value
template <typename T>
inline constexpr int kDepth = sizeof(T) == 4 ? 32 : 64;  // k of a stage
template <typename T>
inline constexpr int kSums = sizeof(T) == 4 ? 2 : 1;  // accumulators of a tile
template <typename T>
inline constexpr int kRun = sizeof(T) == 4 ? 512 / kDepth<T> : 1 << 30;  // stages that one accumulator adds up at most
constexpr int kGroup = 3;       // products of one launch

struct ProductArgs {
  int m, n;                  // rows and columns of one half of C
  int m_halves, n_halves;    // 2: A (B) has sheets for each half of C's rows (columns)
  int m_tiles, n_tiles;      // of one half
  int k_blocks;              // of kDepth, of a segment
  int splits;                // k_blocks are dealt to this many work items, whose sums are added later
  int segments;
  int8_t a_sheet[kMaxSegments], b_sheet[kMaxSegments];
  int a_mn, b_mn;
  int f16;                   // operands are float16 (else bfloat16)
  int act;
  int vec;                   // kStore: rows of c are aligned to 32 bytes
  void *c;                   // kStore: T, or with splits float [splits][..]
  int64_t ldc, c_m_half, c_n_half, c_split;
  const void *bias;          // T, [n] (kStore) or [2 n] (kGate), or NULL
  int bias_vec;              // there is one, and its values from any multiple of 16 columns are aligned to 32 bytes
  void *g, *u;               // T [m][ldg]: u act'(g) and act(g), written by kGate (NULL: not kept), read by kGateBack
  uint16_t *h;               // kGate: sheets of [m][ldg]; kGateBack: dg and du, sheets of [m][ldg]
  int64_t ldg, sheet;        // elements between rows and between sheets of h
  float *sums;               // kGateBack: [m / 32][2][ldg] sums of dg and du over 32 rows, or NULL
  const float *factor;       // kStore, float16: what the sums are multiplied by, or NULL
  const void *residual;      // kLinear, kAdd: T [m][ldr], or NULL; act'(sum + bias) goes to g, float [m][ldg], unless that is NULL
  int64_t ldr;
  int residual_vec;          // rows of the residual are aligned to 32 bytes
};

// Up to three products that do not depend on one another, with one tile shape (kStore; one product else).
struct ProductLaunch {
  CUtensorMap a[kGroup], b[kGroup];
  CUtensorMap out[3];        // kGate, kGateBack: the arrays at g, u and h, or dg and du (one map)
  ProductArgs p[kGroup];
  int first[kGroup + 1];     // work items before each product's
  int count;
  int lead, extra;           // see item_of
  float *runs;               // float32 with more than kRun stages: [blocks][128][BN] sums of the runs so far
  uint32_t *timeouts;
};

// Warps that empty the accumulators: each waits on tensor memory, on global memory and on the special
// function unit in turn, so the widest 16-bit tiles, whose epilogue would else outlast their products, take
// sixteen.  (float32's need the registers of eight, and their products take six times as long.)
// A linear layer's narrow tiles too: with a width of 64 their product is over in a tenth of a microsecond.
template <typename T, int EPI, int BN>
inline constexpr int kEpilogueWarps = (BN == 256 || (kLayer<EPI> && BN == 64)) && sizeof(T) == 2 ? 16 : 8;

// Teams of epilogue warps, which take the tiles in turn: while one waits (for the accumulator, for its
// stores) the other computes.  Elsewhere all warps share a tile: a block often has but one.
template <typename T, int EPI, int BN>
inline constexpr int kTeams = kEpilogueWarps<T, EPI, BN> / 8;

// Columns that one warp of the epilogue takes.
template <typename T, int EPI, int BN>
inline constexpr int kWarpColumns = (EPI == kGate ? BN / 2 : BN) / 2;

// The epilogues that write arrays of this library's own (h, the factors, dg, du) put them together in
// shared memory, in boxes of 32 rows, and store them by TMA: a warp that stores 32 bytes of 32 rows at a
// time keeps the load-store unit busy for 32 cycles (it was at 78 % of its rate with three arrays
// stored so).
//
// Columns of one store: 64 bytes a row, or 16 columns of float32 (64 bytes) and of its sheets (32 bytes).
template <typename T, int EPI, int BN>
inline constexpr int kStoreColumns = sizeof(T) == 4 || kWarpColumns<T, EPI, BN> < 32 ? 16 : 32;

// kStore: columns of a turn (as many as the registers hold: 96 a thread with sixteen warps), and the bytes from
// row to row of the transposing buffer: an odd number of words, so that neither rows nor columns meet bank conflicts.
template <typename T, int EPI, int BN>
inline constexpr int kTurnColumns = kEpilogueWarps<T, EPI, BN> == 16 ? 16 : 32;
template <typename T, int EPI, int BN>
inline constexpr int kRowBytes = kTurnColumns<T, EPI, BN> * sizeof(T) + 4;

// Tile shapes: CG blocks of 128 rows, BN columns, stages that fill what the stores leave of a multiprocessor's
// shared memory.
template <typename T, int EPI, int CG, int BN>
struct ProductShape {
  static constexpr int a_bytes = 128 * kDepth<T> * 2;
  static constexpr int b_bytes = BN / CG * kDepth<T> * 2;
  static constexpr int stage_bytes = kParts<T> * (a_bytes + b_bytes);
  // a warp's boxes: 16-bit data two, which it uses again and again; float32 two of factors and three of h, or
  // three each of dg and du
  static constexpr int box = 32 * kStoreColumns<T, EPI, BN> * 2;
  static constexpr int warp_boxes = kPlainStore<EPI>   ? 32 * kRowBytes<T, EPI, BN>
                                    : sizeof(T) == 2   ? 2 * box
                                    : EPI == kGate     ? 7 * box
                                                       : 6 * box;
  static constexpr int boxes = (kEpilogueWarps<T, EPI, BN> * warp_boxes + 1023) / 1024 * 1024;
  static constexpr int room = (225 * 1024 - boxes) / stage_bytes;
  static constexpr int stages = room > 8 ? 8 : room;
  static constexpr int smem = stages * stage_bytes + boxes + 1024 /* alignment */ + 256 /* barriers */;
  static constexpr int columns = 2 * kSums<T> * BN;  // of tensor memory
  static_assert(stages >= 3 && smem <= 227 * 1024 && columns <= 512, "shared and tensor memory");
};

// Three bfloat16 values whose sum is v to 2^-24: each the rounded rest of the one before.  An
// infinity stays in the first (its rest would be NaN).
__device__ __forceinline__ void split3(float v, uint16_t (&s)[3]) {
  const bf16 a = __float2bfloat16_rn(v);
  const float fa = __bfloat162float(a);
  const float r = isinf(fa) ? 0.f : v - fa;
  const bf16 b = __float2bfloat16_rn(r);
  const bf16 c = __float2bfloat16_rn(r - __bfloat162float(b));
  s[0] = __bfloat16_as_ushort(a);
  s[1] = __bfloat16_as_ushort(b);
  s[2] = __bfloat16_as_ushort(c);
}

__device__ __forceinline__ uint16_t bits16(f16 v) { return __half_as_ushort(v); }
__device__ __forceinline__ uint16_t bits16(bf16 v) { return __bfloat16_as_ushort(v); }

// 32 bytes, a whole sector of L2, in one move (p aligned to them).
struct alignas(32) Sector {
  uint32_t w[8];
};

__device__ __forceinline__ void store_sector(void *p, const Sector &s) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s.w[0]), "r"(s.w[1]),
               "r"(s.w[2]), "r"(s.w[3]), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7])
               : "memory");
}

__device__ __forceinline__ Sector load_sector(const void *p) {
  Sector s;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]), "=r"(s.w[5]), "=r"(s.w[6]),
                 "=r"(s.w[7])
               : "l"(p)
               : "memory");
  return s;
}

// N values of a row as an operand of a later product: one sheet of T, or float32's three.
template <typename T, int N>
__device__ __forceinline__ void store_operand(uint16_t *p, int64_t sheet, const float (&v)[N], int count, bool vec) {
  constexpr int S = sizeof(T) == 4 ? 3 : 1;
  uint16_t w[S][N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (S == 3) {
      uint16_t s[3];
      split3(v[i], s);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][i] = s[q];
    } else {
      w[0][i] = bits16(from_f32<T>(v[i]));
    }
  }
#pragma unroll
  for (int q = 0; q < S; ++q) {
    uint16_t *d = p + q * sheet;
    if (vec && count >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        *reinterpret_cast<Pack<uint16_t, 8> *>(d + i) = *reinterpret_cast<Pack<uint16_t, 8> *>(&w[q][i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < count) d[i] = w[q][i];
    }
  }
}

// N values of a row of T; vec: the row is aligned to 32 bytes.
template <typename T, int N>
__device__ __forceinline__ void store_row(T *p, const float (&v)[N], int count, bool vec) {
  constexpr int V = 32 / sizeof(T);
  if (vec && count >= N) {
#pragma unroll
    for (int i = 0; i < N; i += V) {
      Sector q;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 4)
          q.w[k] = __float_as_uint(v[i + k]);
        else
          q.w[k] = pair16(v[i + 2 * k], v[i + 2 * k + 1], T{});
      }
      store_sector(p + i, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < count) p[i] = from_f32<T>(v[i]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, float (&v)[N], int count, bool vec) {
  constexpr int V = 32 / sizeof(T);
  if (vec && count >= N) {
#pragma unroll
    for (int i = 0; i < N; i += V) {
      const Sector q = load_sector(p + i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 4) {
          v[i + k] = __uint_as_float(q.w[k]);
        } else {
          const float2 f = unpair16(q.w[k], T{});
          v[i + 2 * k] = f.x;
          v[i + 2 * k + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < count ? to_f32(p[i]) : 0.f;
  }
}

template <typename T, int N>
__device__ __forceinline__ void add_bias(float (&v)[N], const T *bias, int count, bool vec) {
  float b[N];
  load_row<T, N>(bias, b, count, vec);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += b[i];
}

// Operands that were scaled to float16's range (by a power of two).
template <typename T, int EPI>
inline constexpr bool kScales = EPI == kStore && NetType<T>::dtype == SLA_F16;
template <int N>
__device__ __forceinline__ void scale_sums(const ProductArgs &p, float (&v)[N]) {
  if (!p.factor) return;
  const float f = *p.factor;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= f;
}

// v = act(v) + r, r the residual's N values of the row; act'(v) is kept in g, whose rows are whole sectors.
template <typename T, int N, bool Activates>
__device__ __forceinline__ void finish_linear(const ProductArgs &p, int64_t row, int col, float (&v)[N], const float (&r)[N],
                                              int count) {
  if (Activates && p.act != SLA_ACT_NONE) {
    float da[N];
    if (p.g) {
      with_activation(p.act, [&](auto act) { activate<act.value, true, N>(v, da); });
      float *to = (float *)p.g + row * p.ldg + col;
      if constexpr (N % 8 == 0) {
        store_row<float, N>(to, da, count, true);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < count) to[i] = da[i];
      }
    } else {
      with_activation(p.act, [&](auto act) { activate<act.value, false, N>(v, da); });
    }
  }
  if (p.residual)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += r[i];
}

// Column sums of a tile of 32 rows (thread = row) and N = 16 or 32 columns: lane c gets column c's (N =
// 16: column c % 16's) sum.  Each step trades half of the columns with the lane that has the other half.
template <int N>
__device__ __forceinline__ float sum_columns(const float (&v)[N], int lane) {
  float w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = v[i];
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = lane & o ? w[i] : w[i + o], keep = lane & o ? w[i + o] : w[i];
      w[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  return N == 16 ? w[0] + __shfl_xor_sync(0xffffffffu, w[0], 16) : w[0];
}

// N values of a row as loaded, so that they can be asked for long before they are used.
template <typename T, int N>
struct RawRow {
  static constexpr int n = N * sizeof(T) / 32;
  Sector s[n];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = load_sector(p + i * (32 / sizeof(T)));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[i].w[k] = 0;
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 4) {
          v[8 * i + k] = __uint_as_float(s[i].w[k]);
        } else {
          const float2 f = unpair16(s[i].w[k], T{});
          v[16 * i + 2 * k] = f.x;
          v[16 * i + 2 * k + 1] = f.y;
        }
      }
  }
};

// The tile (of all halves) and split of a work item.
struct Tile {
  int m_half, m0, n_half, n0, split;
};

template <int EPI, int CG, int BN>
__device__ __forceinline__ Tile tile_of(const ProductArgs &p, int item) {
  const int mt = p.m_halves * p.m_tiles, nt = p.n_halves * p.n_tiles, per = mt * nt;
  Tile t;
  if (nt == 1 && p.m_halves == 1 && p.splits == 1) {  // a narrow layer's tiles are over before the divisions below
    t.split = t.m_half = t.n_half = t.n0 = 0;
    t.m0 = item * 128 * CG;
    return t;
  }
  t.split = item / per;
  int i = item - t.split * per;
  const int band = i / (kBand * nt);
  i -= band * kBand * nt;
  const int rows = min(kBand, mt - band * kBand);
  const int tn = i / rows, tm = band * kBand + i % rows;
  t.m_half = tm / p.m_tiles;
  t.m0 = (tm - t.m_half * p.m_tiles) * 128 * CG;
  t.n_half = tn / p.n_tiles;
  t.n0 = (tn - t.n_half * p.n_tiles) * (EPI == kGate ? BN / 2 : BN);
  return t;
}

// A worker's i-th work item, or -1.  Workers take the items in turn.  Where the items of the last product are
// shorter than those before it (`lead` of them), the workers that got one less of those first take
// `extra` of the short ones, about as long together.
__device__ __forceinline__ int item_of(const ProductLaunch &l, int worker, int workers, int i) {
  int item = worker + i * workers;
  if (l.extra) {
    const int mine = worker < l.lead ? (l.lead - worker - 1) / workers + 1 : 0, over = l.lead % workers;
    if (i < mine) return item;
    i -= mine;
    if (worker >= over) {
      if (i < l.extra) return l.lead + (worker - over) * l.extra + i;
      i -= l.extra;
    }
    item = l.lead + l.extra * (workers - over) + worker + i * workers;
  }
  return item < l.first[l.count] ? item : -1;
}

// The product of a work item, which becomes the item's number among that product's.
__device__ __forceinline__ int product_of(const ProductLaunch &l, int &item) {
  int i = 0;
  while (i + 1 < l.count && item >= l.first[i + 1]) ++i;
  item -= l.first[i];
  return i;
}

__device__ __forceinline__ void split_range(const ProductArgs &p, int split, int &k0, int &k1) {
  k0 = 0, k1 = p.k_blocks;
  if (p.splits == 1) return;  // (no division for a tile of one or two stages)
  k0 = (int)((int64_t)p.k_blocks * split / p.splits);
  k1 = (int)((int64_t)p.k_blocks * (split + 1) / p.splits);
}

// N columns of a tile's sums: loaded, and (after the wait) float32's two added.
template <typename T, int BN, int N>
struct Sums {
  float v[N], small[kSums<T> == 2 ? N : 1];
  __device__ __forceinline__ void load(uint32_t addr) {
    if constexpr (N == 32) {
      tmem_load32(addr, v);
      if constexpr (kSums<T> == 2) tmem_load32(addr + BN, small);
    } else {
      tmem_load16(addr, v);
      if constexpr (kSums<T> == 2) tmem_load16(addr + BN, small);
    }
  }
  __device__ __forceinline__ void wait() {
    tmem_wait(v);
    if constexpr (kSums<T> == 2) {
      tmem_wait(small);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += small[i];
    }
  }
};

// Stages of a work item.
__device__ __forceinline__ int steps_of(const ProductArgs &p, int split) {
  int k0, k1;
  split_range(p, split, k0, k1);
  return p.segments * (k1 - k0);
}

// 16 columns of a thread's row among its block's sums of the runs so far, four at a time beside its warp's
// other rows; only this thread reads what it wrote.
__device__ __forceinline__ void add_run(const float *run, int column, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = *reinterpret_cast<const float4 *>(run + (column / 4 + i) * 128);
    v[4 * i] += a.x, v[4 * i + 1] += a.y, v[4 * i + 2] += a.z, v[4 * i + 3] += a.w;
  }
}
__device__ __forceinline__ void put_run(float *run, int column, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4 *>(run + (column / 4 + i) * 128) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// A warp has read its part of an accumulator.
template <int CG>
__device__ __forceinline__ void release_accumulator(uint64_t *acc_empty, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (CG == 2)
      mbar_arrive_rank(acc_empty, 0);
    else
      mbar_arrive(acc_empty);
  }
}

// All runs of a work item but the last, whose sums are added up in float32: `seq` counts the runs of the block.
// The columns of the warp are [first, first + width) and, for Two, those again BN / 2 further on.  False: a wait expired.
template <typename T, int CG, int BN, bool Two>
__device__ __forceinline__ bool drain_runs(int runs, uint32_t &seq, float *run, uint32_t tmem, int first, int width,
                                           uint64_t *acc_full, uint64_t *acc_empty, int lane) {
  for (int r = 0; r + 1 < runs; ++r, ++seq) {
    const uint32_t acc = seq & 1;
    if (!__all_sync(0xffffffffu, mbar_wait_clocks(acc_full + acc, (seq >> 1) & 1))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < (Two ? 2 : 1) * width; i += 16) {
      const int c = i < width ? first + i : BN / 2 + first + i - width;
      Sums<T, BN, 16> sum;
      sum.load(tmem + acc * kSums<T> * BN + c);
      sum.wait();
      if (r) add_run(run, c, sum.v);
      put_run(run, c, sum.v);
    }
    release_accumulator<CG>(acc_empty + acc, lane);
  }
  return true;
}

// A box of 32 rows in shared memory, thread = row, in TMA's swizzle for rows of `Bytes` bytes: units of 16
// bytes change places within their row, so that writing them meets no bank conflicts.
template <int Bytes>
struct StoreBox {
  static constexpr int units = Bytes / 16;
  uint8_t *sm;
  int lane;
  __device__ __forceinline__ void put(int unit, uint4 q) const {
    reinterpret_cast<uint4 *>(sm)[lane * units + (unit ^ ((lane / (8 / units)) & (units - 1)))] = q;
  }
  // 16 columns of the thread's row: 16 bits from column 16 * part, or float32
  __device__ __forceinline__ void put(int part, const uint32_t (&w)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) put(2 * part + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
  }
  __device__ __forceinline__ void put(const float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      put(i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                        __float_as_uint(v[4 * i + 3])));
  }
};

template <typename T>
__device__ __forceinline__ void pack16(const float (&v)[16], uint32_t (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = pair16(v[2 * k], v[2 * k + 1], T{});
}

// float32's three sheets of 16 columns into boxes `apart` bytes apart.
__device__ __forceinline__ void put_sheets(uint8_t *box, int apart, int lane, const float (&v)[16]) {
  uint32_t w[3][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint16_t a[3], b[3];
    split3(v[2 * k], a);
    split3(v[2 * k + 1], b);
#pragma unroll
    for (int q = 0; q < 3; ++q) w[q][k] = a[q] | ((uint32_t)b[q] << 16);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) StoreBox<32>{box + q * apart, lane}.put(0, w[q]);
}

// kGate and kGateBack: 16 columns at a time, stored in boxes of W.
template <typename T, int EPI, int CG, int BN>
__device__ __forceinline__ void tma_epilogue(const ProductLaunch &l, uint32_t tmem, uint8_t *boxes, uint64_t *acc_full,
                                             uint64_t *acc_empty, volatile uint32_t *dead, int worker, int workers,
                                             uint32_t rank) {
  const ProductArgs &p = l.p[0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, team = (warp - 2) >> 3, side = (warp - 2) >> 2 & 1;
  constexpr int width = kWarpColumns<T, EPI, BN>, W = kStoreColumns<T, EPI, BN>, box = ProductShape<T, EPI, CG, BN>::box;
  constexpr bool f32 = sizeof(T) == 4;
  uint8_t *mine = boxes + (warp - 2) * ProductShape<T, EPI, CG, BN>::warp_boxes;
  const StoreBox<f32 ? 64 : 2 * W> box0{mine, lane}, box1{mine + (f32 ? 2 * box : box), lane};
  uint8_t *sheets = mine + (EPI == kGate ? 4 * box : 0);  // float32: of h, or of dg and then of du
  // boxes 0 and 1 hold what the warp's lanes have put there: to columns x.. of rows y.. of two maps or sheets
  auto store2 = [&](const CUtensorMap *m0, const CUtensorMap *m1, int x, int y, int z1) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store(m0, x, y, 0, box0.sm);
      tma_store_commit();
      tma_store(m1, x, y, z1, box1.sm);
      tma_store_commit();
    }
  };
  float *run = f32 ? l.runs + ((int64_t)blockIdx.x * 4 + quarter) * 32 * BN + lane * 4 : nullptr;
  uint32_t seq = team;  // accumulators before this tile's (16-bit data: one a tile)
  for (int tile = team;; tile += kTeams<T, EPI, BN>, seq += kTeams<T, EPI, BN>) {
    int item = item_of(l, worker, workers, tile);
    if (item < 0) break;
    const Tile t = tile_of<EPI, CG, BN>(p, item);
    const int first = side * width;
    int runs = 1;
    if constexpr (f32) {
      runs = (steps_of(p, t.split) + kRun<T> - 1) / kRun<T>;
      if (!drain_runs<T, CG, BN, EPI == kGate>(runs, seq, run, tmem + ((uint32_t)quarter << 21), first, width, acc_full,
                                               acc_empty, lane)) {
        *dead = 1;
        break;
      }
    }
    const uint32_t acc = seq & 1;
    const int row0 = t.m0 + (int)rank * 128 + quarter * 32, row = row0 + lane;
    const bool live = row < p.m;
    // What the next columns need from memory is on its way while these are worked on, and the first
    // columns' while the product runs.  kGateBack: the factors (rows are padded to whole sectors of 16
    // columns); kGate: the biases.
    RawRow<T, 16> raw_g, raw_u;
    auto ask = [&](int c) {
      if constexpr (EPI == kGate) {
        if (p.bias_vec && t.n0 + c + 16 <= p.n) {
          raw_g.load((const T *)p.bias + t.n0 + c);
          raw_u.load((const T *)p.bias + p.n + t.n0 + c);
        }
      } else if (live && t.n0 + c + 16 <= p.ldg) {
        const int64_t o = row * p.ldg + t.n0 + c;
        raw_g.load((const T *)p.g + o);
        raw_u.load((const T *)p.u + o);
      } else {
        raw_g.clear();
        raw_u.clear();
      }
    };
    ask(first);
    if (!__all_sync(0xffffffffu, mbar_wait_clocks(acc_full + acc, (seq >> 1) & 1))) {
      *dead = 1;
      break;
    }
    tc_fence_after();
    const uint32_t base = tmem + acc * kSums<T> * BN + ((uint32_t)quarter << 21);
#pragma unroll 1
    for (int c = first; c < first + width; c += W) {
      const bool some = row0 < p.m && t.n0 + c < p.n, last = c + W >= first + width;
      uint32_t ph[W / 16][8];
      if (lane == 0) tma_store_read<0>();  // the boxes are free
      __syncwarp();
#pragma unroll
      for (int j = 0; j < W; j += 16) {
        const int count = p.n - t.n0 - c - j;
        Sums<T, BN, 16> sum;
        float(&v)[16] = sum.v;
        sum.load(base + c + j);
        if constexpr (EPI == kGate) {
          Sums<T, BN, 16> sum_u;
          float(&u)[16] = sum_u.v;
          sum_u.load(base + BN / 2 + c + j);
          const RawRow<T, 16> bias_g = raw_g, bias_u = raw_u;
          if (c + j + 16 < first + width) ask(c + j + 16);
          sum.wait();
          sum_u.wait();
          if constexpr (f32)
            if (runs > 1) {
              add_run(run, c + j, v);
              add_run(run, BN / 2 + c + j, u);
            }
          if (p.bias_vec && count >= 16) {
            float bg[16], bu[16];
            bias_g.values(bg);
            bias_u.values(bu);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 a = add2(f2(v[i], v[i + 1]), f2(bg[i], bg[i + 1]));
              const float2 b = add2(f2(u[i], u[i + 1]), f2(bu[i], bu[i + 1]));
              v[i] = a.x, v[i + 1] = a.y, u[i] = b.x, u[i + 1] = b.y;
            }
          } else if (p.bias) {
            add_bias<T, 16>(v, (const T *)p.bias + t.n0 + c + j, count, false);
            add_bias<T, 16>(u, (const T *)p.bias + p.n + t.n0 + c + j, count, false);
          }
          float h[16];
          if (p.g) {
            with_activation(p.act, [&](auto act) { gate<act.value, true, 16>(v, u, h); });
            if constexpr (f32) {
              box0.put(v);
              box1.put(u);
            } else {
              uint32_t w[8];
              pack16<T>(v, w);
              box0.put(j / 16, w);
              pack16<T>(u, w);
              box1.put(j / 16, w);
            }
          } else {
            with_activation(p.act, [&](auto act) { gate<act.value, false, 16>(v, u, h); });
          }
          if constexpr (f32)
            put_sheets(sheets, box, lane, h);
          else
            pack16<T>(h, ph[j / 16]);
        } else {
          float g[16], u[16];
          raw_g.values(g);
          raw_u.values(u);
          if (c + j + 16 < first + width) ask(c + j + 16);
          sum.wait();
          if constexpr (f32)
            if (runs > 1) add_run(run, c + j, v);
          gate_gradients(v, g, u);
          if constexpr (f32) {
            put_sheets(sheets, box, lane, g);
            put_sheets(sheets + 3 * box, box, lane, u);
          } else {
            uint32_t w[8];
            pack16<T>(g, w);
            box0.put(j / 16, w);
            pack16<T>(u, w);
            box1.put(j / 16, w);
          }
          if (p.sums && row0 < p.m) {
            if (!live) {  // not a row: its product is no zero if a weight is infinite
#pragma unroll
              for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.f;
            }
            const float sg = sum_columns(g, lane), su = sum_columns(u, lane);
            if (lane < 16 && lane < count) {
              float *to = p.sums + (int64_t)(row0 >> 5) * 2 * p.ldg + t.n0 + c + j + lane;
              to[0] = sg;
              to[p.ldg] = su;
            }
          }
        }
      }
      if (last) release_accumulator<CG>(acc_empty + acc, lane);
      if (!some) continue;
      if constexpr (f32) {
        if (EPI == kGate && p.g) store2(&l.out[0], &l.out[1], t.n0 + c, row0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {  // all three or six sheets at once
          tma_store(&l.out[EPI == kGate ? 2 : 0], t.n0 + c, row0, 0, sheets);
          tma_store_commit();
        }
      } else if constexpr (EPI == kGate) {
        if (p.g) {
          store2(&l.out[0], &l.out[1], t.n0 + c, row0, 0);
          if (lane == 0) tma_store_read<1>();  // box 0 is free again
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < W / 16; ++j) box0.put(j, ph[j]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store(&l.out[2], t.n0 + c, row0, 0, box0.sm);
          tma_store_commit();
        }
      } else {
        store2(&l.out[0], &l.out[0], t.n0 + c, row0, 1);
      }
    }
  }
  if (lane == 0) tma_store_done();
  __syncwarp();
}

// kStore: straight from the registers, since TMA may not be able to write the caller's arrays.  Rows that are
// not aligned to whole sectors would take a store an element, each to 32 lines: they go through shared
// memory, so that a warp's stores run along the rows (2049 x 131 outputs: 16 -> 10 us).
template <typename T, int EPI, int CG, int BN>
__device__ __forceinline__ void store_epilogue(const ProductLaunch &l, uint32_t tmem, uint8_t *boxes,
                                               uint64_t *acc_full, uint64_t *acc_empty, volatile uint32_t *dead, int worker, int workers,
                                               uint32_t rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, team = (warp - 2) >> 3, side = (warp - 2) >> 2 & 1;
  constexpr int width = kWarpColumns<T, EPI, BN>, N = kTurnColumns<T, EPI, BN>, pitch = kRowBytes<T, EPI, BN>;
  uint8_t *mine = boxes + (warp - 2) * 32 * pitch;
  constexpr bool f32 = sizeof(T) == 4;
  float *run = f32 ? l.runs + ((int64_t)blockIdx.x * 4 + quarter) * 32 * BN + lane * 4 : nullptr;
  // kLinear, kAdd: the residual's columns of the next turn are asked for while the present ones are worked on, those of a tile's
  // first turn while the tile before it is (1,000,000 tokens, 64 -> 64: 107 -> 102 us; the bias's too cost registers: 112)
  RawRow<T, N> raw;
  auto ask = [&](const Tile &t, int c) {
    const ProductArgs &p = l.p[0];
    const int row = t.m0 + (int)rank * 128 + quarter * 32 + lane, col = t.n0 + c;
    if (p.residual && p.residual_vec && row < p.m && p.n - col >= N) raw.load((const T *)p.residual + row * p.ldr + col);
  };
  auto ask_tile = [&](int tile) {
    const int item = item_of(l, worker, workers, tile);
    if (item >= 0) ask(tile_of<EPI, CG, BN>(l.p[0], item), side * width);
  };
  if (kLayer<EPI>) ask_tile(team);
  uint32_t seq = team;  // accumulators before this tile's (16-bit data: one a tile)
  for (int tile = team;; tile += kTeams<T, EPI, BN>, seq += kTeams<T, EPI, BN>) {
    int item = item_of(l, worker, workers, tile);
    if (item < 0) break;
    const ProductArgs &p = l.p[EPI == kStore ? product_of(l, item) : 0];
    const Tile t = tile_of<EPI, CG, BN>(p, item);
    int runs = 1;
    if constexpr (f32) {
      runs = (steps_of(p, t.split) + kRun<T> - 1) / kRun<T>;
      if (!drain_runs<T, CG, BN, false>(runs, seq, run, tmem + ((uint32_t)quarter << 21), side * width, width, acc_full,
                                        acc_empty, lane)) {
        *dead = 1;
        break;
      }
    }
    const uint32_t acc = seq & 1;
    const int row = t.m0 + (int)rank * 128 + quarter * 32 + lane;
    const bool live = row < p.m;
    if (!__all_sync(0xffffffffu, mbar_wait_clocks(acc_full + acc, (seq >> 1) & 1))) {
      *dead = 1;
      break;
    }
    tc_fence_after();
    const uint32_t base = tmem + acc * kSums<T> * BN + ((uint32_t)quarter << 21);
#pragma unroll 1
    for (int c = side * width; c < (side + 1) * width; c += N) {
      const int col = t.n0 + c, count = p.n - col;
      Sums<T, BN, N> sum;
      float(&v)[N] = sum.v;
      sum.load(base + c);
      float r[kLayer<EPI> ? N : 1];
      if constexpr (kLayer<EPI>) {
        if (p.residual && live && count > 0) {
          if (p.residual_vec && count >= N)
            raw.values(r);
          else
            load_row<T, N>((const T *)p.residual + row * p.ldr + col, r, count, p.residual_vec);
        }
        if (c + N < (side + 1) * width)
          ask(t, c + N);
        else
          ask_tile(tile + kTeams<T, EPI, BN>);
      }
      sum.wait();
      if constexpr (f32)
        if (runs > 1) {
#pragma unroll
          for (int i = 0; i < N; i += 16) add_run(run, c + i, *reinterpret_cast<float(*)[16]>(v + i));
        }
      if (c + N >= (side + 1) * width) release_accumulator<CG>(acc_empty + acc, lane);
      if (live && count > 0) {
        const int64_t o = t.m_half * p.c_m_half + t.n_half * p.c_n_half + row * p.ldc + col;
        if (p.splits > 1) {
          store_row<float, N>((float *)p.c + t.split * p.c_split + o, v, count, true);
        } else {
          if constexpr (kScales<T, EPI>) scale_sums(p, v);
          if (p.bias) add_bias<T, N>(v, (const T *)p.bias + col, count, p.bias_vec);
          if constexpr (kLayer<EPI>) finish_linear<T, N, EPI == kLinear>(p, row, col, v, r, count);
          if (p.vec && count >= N) store_row<T, N>((T *)p.c + o, v, count, true);
        }
      }
      if (p.splits == 1 && !(p.vec && count >= N) && count > 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4 / sizeof(T)) {
          uint32_t w;
          if constexpr (sizeof(T) == 4)
            w = __float_as_uint(v[i]);
          else
            w = pair16(v[i], v[i + 1], T{});
          *reinterpret_cast<uint32_t *>(mine + lane * pitch + i * sizeof(T)) = w;
        }
        __syncwarp();
        const int rows = p.m - (row - lane);
        T *out = (T *)p.c + t.m_half * p.c_m_half + t.n_half * p.c_n_half + (row - lane) * p.ldc + col;
#pragma unroll 8
        for (int i = 0; i < N; ++i) {
          const int r = (i * 32 + lane) / N, k = (i * 32 + lane) % N;
          if (r < rows && k < count) out[r * p.ldc + k] = *reinterpret_cast<const T *>(mine + r * pitch + k * sizeof(T));
        }
        __syncwarp();
      }
    }
  }
}

template <typename T, int EPI, int CG, int BN>
__global__ void __launch_bounds__(64 + 32 * kEpilogueWarps<T, EPI, BN>, 1)
    product_kernel(const __grid_constant__ ProductLaunch l) {
  using Shape = ProductShape<T, EPI, CG, BN>;
  constexpr int S = Shape::stages;
  extern __shared__ uint8_t raw[];
  uint8_t *tiles = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t *boxes = tiles + S * Shape::stage_bytes;
  uint64_t *full = (uint64_t *)(boxes + Shape::boxes);
  uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 2, *drained = acc_empty + 2;
  uint32_t *tmem_slot = (uint32_t *)(drained + 1);
  volatile uint32_t *dead = tmem_slot + 1;

  const int warp = threadIdx.x >> 5;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int worker = blockIdx.x / CG, workers = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 8 * CG);
    }
    mbar_init(drained, 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
    tma_prefetch_map(&l.a[0]);
    tma_prefetch_map(&l.b[0]);
  }
  if (warp == 1) tmem_alloc<CG>(tmem_slot, Shape::columns);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // what came before in the stream has written its results; what comes next may be made ready meanwhile
  grid_dependency_wait();
  grid_dependency_launch();

  if (warp == 0) {
    // loads: one stage is kDepth of k of the tile's rows of A and columns of B, all parts
    constexpr uint32_t bytes = CG * Shape::stage_bytes;
    uint32_t n = 0;
    for (int i = 0; !*dead; ++i) {
      int item = item_of(l, worker, workers, i);
      if (item < 0) break;
      const int which = EPI == kStore ? product_of(l, item) : 0;
      const ProductArgs &p = l.p[which];
      const CUtensorMap &ma = l.a[which], &mb = l.b[which];
      const Tile t = tile_of<EPI, CG, BN>(p, item);
      int k0, k1;
      split_range(p, t.split, k0, k1);
      const int am = t.m0 + (int)rank * 128;
      for (int seg = 0; seg < p.segments && !*dead; ++seg) {
        // the parts of a value are neighbouring sheets
        const int az = (p.a_sheet[seg] + t.m_half) * kParts<T>, bz = (p.b_sheet[seg] + t.n_half) * kParts<T>;
        for (int kb = k0; kb < k1; ++kb, ++n) {
          const int s = n % S;
          if (n >= S && !__all_sync(0xffffffffu, mbar_wait_clocks(empty + s, ((n / S) - 1) & 1))) {
            *dead = 1;
            break;
          }
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
            const int k = kb * kDepth<T>;
#pragma unroll
            for (int q = 0; q < kParts<T>; ++q) {
              uint8_t *da = tiles + s * Shape::stage_bytes + q * Shape::a_bytes;
              const int z = az + q;
              if (p.a_mn) {
                tma_load<CG>(da, &ma, am, k, z, full + s);
                tma_load<CG>(da + Shape::a_bytes / 2, &ma, am + 64, k, z, full + s);
              } else {
                tma_load<CG>(da, &ma, k, am, z, full + s);
              }
            }
#pragma unroll
            for (int q = 0; q < kParts<T>; ++q) {
              uint8_t *db = tiles + s * Shape::stage_bytes + kParts<T> * Shape::a_bytes + q * Shape::b_bytes;
              const int z = bz + q;
              if (EPI == kGate) {
                // half of the columns are g's, half u's; in a pair of blocks each loads one of them
                if (CG == 2) {
                  tma_load<CG>(db, &mb, k, t.n0, z + (int)rank * kParts<T>, full + s);
                } else {
                  tma_load<CG>(db, &mb, k, t.n0, z, full + s);
                  tma_load<CG>(db + Shape::b_bytes / 2, &mb, k, t.n0, z + kParts<T>, full + s);
                }
              } else if (p.b_mn) {
#pragma unroll
                for (int j = 0; j < BN / CG / 64; ++j)
                  tma_load<CG>(db + j * kDepth<T> * 128, &mb, t.n0 + (int)rank * (BN / CG) + j * 64, k, z, full + s);
              } else {
                tma_load<CG>(db, &mb, k, t.n0 + (int)rank * (BN / CG), z, full + s);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    // every copy has landed before the block may end (the mma warp waited for all but after a timeout)
    if (rank == 0)
      for (uint32_t i = n > S ? n - S : 0; i < n; ++i)
        if (!mbar_wait_clocks(full + i % S, (i / S) & 1)) *dead = 1;
  } else if (warp == 1 && rank == 0) {
    uint32_t n = 0, seq = 0;  // stages and accumulators so far
    for (int tile = 0; !*dead; ++tile) {
      int item = item_of(l, worker, workers, tile);
      if (item < 0) break;
      const int which = EPI == kStore ? product_of(l, item) : 0;
      const ProductArgs &p = l.p[which];
      const uint32_t idesc = tc_idesc(p.f16, p.a_mn, p.b_mn, 128 * CG, BN);
      const uint32_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
      const uint64_t a0 = tc_desc(tiles, p.a_mn, Shape::a_bytes / 2, kDepth<T>);
      const uint64_t b0 = tc_desc(tiles + kParts<T> * Shape::a_bytes, p.b_mn, kDepth<T> * 128, kDepth<T>);
      const Tile t = tile_of<EPI, CG, BN>(p, item);
      int left = steps_of(p, t.split);
      bool lost = false;
      while (left && !lost) {
        const uint32_t acc = seq & 1, use = seq >> 1;
        if (use > 0 && !__all_sync(0xffffffffu, mbar_wait_clocks(acc_empty + acc, (use - 1) & 1))) {
          lost = true;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * kSums<T> * BN;
        const int steps = min(left, kRun<T>);
        for (int i = 0; i < steps; ++i, ++n) {
          const int s = n % S;
          if (!__all_sync(0xffffffffu, mbar_wait_clocks(full + s, (n / S) & 1))) {
            lost = true;
            break;
          }
          tc_fence_after();
          const uint64_t a = a0 + s * (Shape::stage_bytes >> 4), b = b0 + s * (Shape::stage_bytes >> 4);
          if (elect_one()) {
            if constexpr (kParts<T> == 3) {
              constexpr int pairs[6][2] = {{0, 0}, {0, 1}, {1, 0}, {1, 1}, {0, 2}, {2, 0}};
#pragma unroll
              for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int j = 0; j < kDepth<T> / 16; ++j)
                  tc_mma<CG>(q ? d + BN : d, a + pairs[q][0] * (Shape::a_bytes >> 4) + j * a_step,
                             b + pairs[q][1] * (Shape::b_bytes >> 4) + j * b_step, idesc, i > 0 || j > 0 || q > 1);
            } else {
#pragma unroll
              for (int j = 0; j < kDepth<T> / 16; ++j)
                tc_mma<CG>(d, a + j * a_step, b + j * b_step, idesc, i > 0 || j > 0);
            }
            tc_commit<CG>(empty + s);
            if (i == steps - 1) tc_commit<CG>(acc_full + acc);
          }
          __syncwarp();
        }
        left -= steps;
        ++seq;
      }
      if (lost) {
        *dead = 1;
        break;
      }
    }
    if (*dead) {  // the mma in flight still read shared memory
      if (elect_one()) tc_commit<CG>(drained);
      __syncwarp();
      mbar_wait_clocks(drained, 0);
    }
  } else if (warp >= 2) {
    if constexpr (!kPlainStore<EPI>)
      tma_epilogue<T, EPI, CG, BN>(l, tmem, boxes, acc_full, acc_empty, dead, worker, workers, rank);
    else
      store_epilogue<T, EPI, CG, BN>(l, tmem, boxes, acc_full, acc_empty, dead, worker, workers, rank);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, Shape::columns);
  if (threadIdx.x == 0 && *dead) atomicAdd_system(l.timeouts, 1u);
}

// Tile shapes by index, widest first.  float32's two accumulators, twice, leave no room for the widest.
struct ProductTile {
  int cg, bn;
};
constexpr ProductTile kProductTiles[] = {{2, 256}, {2, 128}, {1, 128}, {1, 64}};
constexpr int kProductTileCount = 4;

// Launches `epi` with tile shape kProductTiles[shape] on `blocks` blocks.  early: the launch may be made
// ready while the kernel before it in the stream, one of this call's own, still runs.
template <typename T>
cudaError_t launch_product(int epi, int shape, int blocks, const ProductLaunch &l, bool early, cudaStream_t st);

template <typename T, int EPI, int CG, int BN>
cudaError_t launch_product_as(int blocks, const ProductLaunch &l, bool early, cudaStream_t st) {
  constexpr int smem = ProductShape<T, EPI, CG, BN>::smem;
  auto kernel = product_kernel<T, EPI, CG, BN>;
  // once per device: the attribute stays with the loaded kernel
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) allowed.fetch_or(1ull << (dev & 63));
  }
  if (e != cudaSuccess) return e;
  LaunchConfig cfg(dim3(blocks), 64 + 32 * kEpilogueWarps<T, EPI, BN>, smem, st, early, CG);
  return cudaLaunchKernelEx(&cfg.c, kernel, l);
}

template <typename T, int EPI>
cudaError_t launch_product_shape(int shape, int blocks, const ProductLaunch &l, bool early, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (shape == 0) return launch_product_as<T, EPI, 2, 256>(blocks, l, early, st);
  switch (shape) {
    case 1: return launch_product_as<T, EPI, 2, 128>(blocks, l, early, st);
    case 2: return launch_product_as<T, EPI, 1, 128>(blocks, l, early, st);
    default: return launch_product_as<T, EPI, 1, 64>(blocks, l, early, st);
  }
}

}  // namespace sla
