// The gated scan: a linear recurrence along the rows of sequences, channel by channel, forward and backward.
//
//   h_t = a_t h_{t-1} + (1 - a_t) x_t,  a = 1 / (1 + e^-g),  h_0 the sequence's state                 (a solve with a
//   l_t = dh_t + a_{t+1} l_{t+1}        the gradient of h_t                                   unit bidiagonal matrix, and
//   dx = (1 - a) l,  dg = l (h_{t-1} - x) a (1 - a),  dstate = a_1 l_1                             with its transpose)
//
// Both are bound by memory: two reads and a write forward, three reads and two writes backward (h is formed
// again from x and g, from float32 states that the forward call leaves every kRows rows: an eighth of what reading h
// in 16 bits would cost, and exact).  To read everything once with the rows in parallel, a block
// takes a tile of rows by kCols channels into registers, kRows rows a warp, two channels a lane, and goes
// over them twice: once for the map (B, H) from the state before the rows to the state behind them,
// s -> (1 - B) s + H, and, when that state is known, once for the results.  In between the maps of the block's warps
// are joined in shared memory, the block's is published, and the state before the tile is put together from
// the maps of the tiles before it, back to the tile in which the sequence starts or the last of the states that
// every kSpan-th tile publishes.  Tiles are handed out in order of time by a counter, so those waited for are
// always at work; which block takes which tile changes no result, and the maps are joined in a fixed order.
//
// A map's two float32 are published as one 64-bit word, so that the word itself says whether it is there (the
// workspace is set to ones, a NaN that no map has): no flag, no fence.
//
// Rounding.  Of a and 1 - a the smaller is kept (with the gate's sign), and a step is written as h + (1 - a)(x - h) or
// x + a (h - x): with a rounded to float32 a constant gate close to 1 would lose 2^-25 / (1 - a) of the result, the same way
// in every step.  For the same reason maps carry B = 1 - (product of a).  A sequence's start is a map with B = kCut, whose
// H replaces what came before, whatever that is: an infinity or a NaN stays within its sequence (and makes NaN of what follows
// it there).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sla_act.cuh"
#include "sla_common.cuh"
#include "sla_host.h"
#include "sla_net.cuh"

namespace sla {
namespace {

constexpr int kRows = 16;     // of a warp; the distance of the saved states
constexpr int kCols = 64;     // channels of a tile, two a lane
constexpr int kSpan = 64;     // tiles between published states
constexpr int kForwardWarps = 16, kBackwardWarps = 8;
constexpr float kCut = 2.f;
constexpr long long kScanClocks = 4000000000ll;  // about two seconds
constexpr uint64_t kAbsent = ~0ull;

struct Sequences {
  int64_t rows;          // of all
  int64_t count, length; // length 0: by offsets
  const void *offsets;
  int wide;              // offsets are 64 bits
  int reverse;
};

struct ScanArgs {
  Sequences q;
  int channels, groups;  // groups of kCols channels
  int outside;           // rows outside of all sequences become zero
  int vec;               // two channels may be moved at once
  const void *x, *g, *dh;
  int64_t ldx, ldg, lddh;
  void *out0, *out1;     // h; or dx and dg
  const float *state;    // [count][channels] or NULL
  const float *dfinal;   // the same, backward
  float *end;            // [count][channels] or NULL: states behind the sequences; or dstate
  float *saved;          // [rows / kRows][channels]: states before those rows
  int tiles;             // of a group
  uint32_t *counter;     // tiles taken so far, less one
  uint64_t *maps, *states;  // [tiles][groups][kCols], [tiles / kSpan][groups][kCols]
  uint32_t *timeouts;
};

// The sequence of a row (in memory order): -1 outside of all.
struct Place {
  int seq;
  int64_t begin, end;
};

__device__ __forceinline__ int64_t offset_at(const Sequences &q, int64_t s) {
  return q.wide ? ((const int64_t *)q.offsets)[s] : ((const int32_t *)q.offsets)[s];
}

__device__ __forceinline__ Place place_of(const Sequences &q, int64_t row) {
  Place p{-1, 0, 0};
  if (row < 0 || row >= q.rows) return p;
  if (q.length) {
    p.seq = (uint32_t)row / (uint32_t)q.length;
    p.begin = p.seq * q.length;
    p.end = p.begin + q.length;
    return p;
  }
  int64_t lo = 0, hi = q.count;  // the last s in [0, count) with offsets[s] <= row
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (offset_at(q, mid) <= row)
      lo = mid + 1;
    else
      hi = mid;
  }
  if (lo == 0) return p;
  // (offsets that are none may lie outside of the rows, or fall: no row is then taken to be in two places)
  p.begin = max(offset_at(q, lo - 1), (int64_t)0), p.end = min(offset_at(q, lo), q.rows);
  if (row >= p.begin && row < p.end) p.seq = (int)(lo - 1);
  return p;
}

// Memory row of the i-th row in the scan's order.
__device__ __forceinline__ int64_t row_of(const Sequences &q, int64_t i) { return q.reverse ? q.rows - 1 - i : i; }

// What a warp knows of its rows: bit r of the masks, and lane r's sequence.
struct RowInfo {
  uint32_t live, first, last;  // in a sequence; the first or last of one, in the scan's order
  int seq;
  int64_t origin;              // lane r: the scan's index of its sequence's first row
  int64_t until;               // ... and of the row behind its last
};

__device__ __forceinline__ RowInfo rows_info(const Sequences &q, int64_t i0, int lane) {
  RowInfo f;
  const int64_t i = i0 + lane, row = row_of(q, i);
  Place p{-1, 0, 0};
  if (lane < kRows && i < q.rows) p = place_of(q, row);
  const bool in = p.seq >= 0, at_begin = in && row == p.begin, at_end = in && row == p.end - 1;
  f.seq = p.seq;
  f.origin = q.reverse ? q.rows - p.end : p.begin;
  f.until = q.reverse ? q.rows - p.begin : p.end;
  f.live = __ballot_sync(0xffffffffu, in);
  f.first = __ballot_sync(0xffffffffu, q.reverse ? at_end : at_begin);
  f.last = __ballot_sync(0xffffffffu, q.reverse ? at_begin : at_end);
  return f;
}

// Two channels of a row.
template <typename T>
struct Two {
  using Raw = typename std::conditional<sizeof(T) == 4, float2, uint32_t>::type;
  static __device__ __forceinline__ Raw zero() {
    if constexpr (sizeof(T) == 4)
      return f2(0.f, 0.f);
    else
      return 0u;
  }
  static __device__ __forceinline__ Raw load(const T *p, int count, bool vec) {
    if (vec) return count > 0 ? *reinterpret_cast<const Raw *>(p) : zero();
    const T none = from_f32<T>(0.f);
    const T a = count > 0 ? p[0] : none, b = count > 1 ? p[1] : none;
    if constexpr (sizeof(T) == 4)
      return f2(a, b);
    else
      return *reinterpret_cast<const uint16_t *>(&a) | ((uint32_t) * reinterpret_cast<const uint16_t *>(&b) << 16);
  }
  static __device__ __forceinline__ float2 values(Raw r) {
    if constexpr (sizeof(T) == 4)
      return r;
    else
      return unpair16(r, T{});
  }
  static __device__ __forceinline__ void store(T *p, float2 v, int count, bool vec) {
    if (vec) {
      if (count <= 0) return;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2 *>(p) = v;
      else
        *reinterpret_cast<uint32_t *>(p) = pair16(v.x, v.y, T{});
    } else {
      if (count > 0) p[0] = from_f32<T>(v.x);
      if (count > 1) p[1] = from_f32<T>(v.y);
    }
  }
};

__device__ __forceinline__ bool below(float s) { return __float_as_int(s) < 0; }

// The smaller of a and 1 - a, with the gate's sign: positive where it is 1 - a.
template <bool Exact>
__device__ __forceinline__ float small_side(float g) {
  const float m = fabsf(g) * -1.4426950408889634f;
  float e = ex2_approx(m);
  // the rounding of the exponent, which the exponential multiplies (log2 e = 1.44269502... + 1.92596303e-8)
  if constexpr (Exact) {
    const float rest = fmaf(fabsf(g), -1.4426950408889634f, -m) + fabsf(g) * -1.92596303e-8f;
    e = fmaf(e * 0.6931471805599453f, rest, e);
    e = fabsf(g) > 88.f ? 0.f : e;  // an infinity's rest is no number
  }
  return copysignf(e * rcp_approx(1.f + e), g);
}

// One step of h, and of B (which is h for x = 1 from 0).
__device__ __forceinline__ float step(float h, float x, float s) { return fmaf(s, x - h, below(s) ? x : h); }
__device__ __forceinline__ float2 step(float2 h, float2 x, float2 s) {
  const float2 d = add2(x, f2(-h.x, -h.y));
  return fma2(s, d, f2(below(s.x) ? x.x : h.x, below(s.y) ? x.y : h.y));
}
// One step of the gradient's message a l.
__device__ __forceinline__ float2 message(float2 l, float2 s) {
  return fma2(f2(-s.x, -s.y), l, f2(below(s.x) ? 0.f : l.x, below(s.y) ? 0.f : l.y));
}

// s -> (1 - b) s + h of two channels; b = kCut: s -> h.
struct Map {
  float2 b, h;
};

__device__ __forceinline__ float apply(float b, float h, float s) { return b == kCut ? h : fmaf(-b, s, s) + h; }
__device__ __forceinline__ float2 apply(const Map &m, float2 s) {
  return f2(apply(m.b.x, m.h.x, s.x), apply(m.b.y, m.h.y, s.y));
}
__device__ __forceinline__ void join(float &b, float &h, float b2, float h2) {  // (b, h) first
  h = apply(b2, h2, h);
  b = b2 == kCut || b == kCut ? kCut : fmaf(b2, 1.f - b, b);
}
__device__ __forceinline__ void join(Map &m, const Map &n) {
  join(m.b.x, m.h.x, n.b.x, n.h.x);
  join(m.b.y, m.h.y, n.b.y, n.h.y);
}

__device__ __forceinline__ uint64_t word_of(float b, float h) {
  const uint64_t w = (uint64_t)__float_as_uint(h) << 32 | __float_as_uint(b);
  return w == kAbsent ? 0x7fffffff7fffffffull : w;  // both are NaN: another one
}
__device__ __forceinline__ void publish(uint64_t *p, const Map &m) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(word_of(m.b.x, m.h.x)),
               "l"(word_of(m.b.y, m.h.y))
               : "memory");
}
__device__ __forceinline__ bool look(const uint64_t *p, Map &m) {
  uint64_t a, b;
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
  m.b = f2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)b));
  m.h = f2(__uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)(b >> 32)));
  return a != kAbsent && b != kAbsent;
}

// Waits until all lanes' words are there.  False: they never came.
__device__ __forceinline__ bool wait_for(const uint64_t *p, Map &m) {
  if (__all_sync(0xffffffffu, look(p, m))) return true;
  const long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, look(p, m))) return true;
    if (__any_sync(0xffffffffu, clock64() - t0 > kScanClocks)) return false;
  }
}

__device__ __forceinline__ void copy_async(void *dst, const void *src, bool eight) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if (eight)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

// Asks for the rows of `from` ([count][channels] float32) that belong to the sequences of the marked rows: to lane's
// two places of row r of `to` ([kRows][kCols]), from where the lane itself reads them.
__device__ __forceinline__ void ask_states(float *to, const float *from, uint32_t marks, int seq, int channels, int c,
                                           int lane) {
  const bool both = channels % 2 == 0 && ((uintptr_t)from & 7) == 0;
  for (uint32_t m = marks; m; m &= m - 1) {
    const int r = __ffs(m) - 1;
    const int64_t s = __shfl_sync(0xffffffffu, seq, r);
    const float *p = from + s * channels + c;
    float *d = to + r * kCols + 2 * lane;
    if (both) {
      if (c < channels) copy_async(d, p, true);
    } else {
      if (c < channels) copy_async(d, p, false);
      if (c + 1 < channels) copy_async(d + 1, p + 1, false);
    }
  }
}

__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void put_state(float *to, int64_t s, int channels, int c, float2 v) {
  if (c < channels) to[s * channels + c] = v.x;
  if (c + 1 < channels) to[s * channels + c + 1] = v.y;
}

// The tile a block works on, and the maps of its warps.
template <int Warps>
struct TileMemory {
  Map maps[Warps][32];      // of the warps
  Map carry[Warps][32];     // parts of the way from the known state to the tile
  int64_t origin;           // the scan's index of the first row that the tile's first row depends on
  uint32_t next;
};

// The state before the tile: what comes from the tiles before it, in the order of time.  `first` is the
// tile where the present sequence starts.  All warps take part; afterwards (and a barrier) carry holds maps of which the
// first `parts` are joined in order.
template <int Warps>
__device__ __forceinline__ int look_back(const ScanArgs &p, TileMemory<Warps> &sm, int tile, int group, int first,
                                         int warp, int lane) {
  const int base = tile / kSpan * kSpan, lo = max(first, base);
  const bool known = first < base;  // the state before `base` is needed
  const int count = tile - lo, per = (count + Warps - 1) / Warps;
  const int from = lo + warp * per, to = min(tile, from + per);
  bool ok = true;
  Map m{f2(0.f, 0.f), f2(0.f, 0.f)};
  if (warp == 0 && known)
    ok = wait_for(p.states + ((int64_t)(base / kSpan - 1) * p.groups + group) * kCols + 2 * lane, m);
  for (int i = from; i < to; ++i) {
    Map n;
    ok = wait_for(p.maps + ((int64_t)i * p.groups + group) * kCols + 2 * lane, n) && ok;
    join(m, n);
  }
  sm.carry[warp][lane] = m;
  if (!ok && lane == 0) atomicAdd_system(p.timeouts, 1u);
  return per ? (count + per - 1) / per : 1;
}

// Joins the maps of the block's warps up to `warps`.
template <int Warps>
__device__ __forceinline__ Map joined(const TileMemory<Warps> &sm, int warps, int lane) {
  Map m = sm.maps[0][lane];
  for (int w = 1; w < warps; ++w) join(m, sm.maps[w][lane]);
  return m;
}

// Publishes the tile's map, finds the state before it, publishes the state behind it where others look for it, and
// returns the state before this warp's rows.  maps are in place (and a barrier behind them).
template <int Warps, bool Chain>
__device__ __forceinline__ float2 state_before(const ScanArgs &p, TileMemory<Warps> &sm, int tile, int group, int64_t i0,
                                               int warp, int lane) {
  float2 s = f2(0.f, 0.f);
  if constexpr (Chain) {
    const int64_t origin = sm.origin;  // i0: nothing before the tile matters
    const bool needed = origin < i0;
    Map own;
    if (warp == Warps - 1) {
      own = joined<Warps>(sm, Warps, lane);
      publish(p.maps + ((int64_t)tile * p.groups + group) * kCols + 2 * lane, own);
    }
    int parts = 0;
    if (needed) parts = look_back<Warps>(p, sm, tile, group, (int)(origin / (Warps * kRows)), warp, lane);
    __syncthreads();
    for (int w = 0; w < parts; ++w) s = apply(sm.carry[w][lane], s);
    if (warp == Warps - 1 && (tile + 1) % kSpan == 0) {
      const Map behind{f2(kCut, kCut), apply(own, s)};
      publish(p.states + ((int64_t)(tile / kSpan) * p.groups + group) * kCols + 2 * lane, behind);
    }
  }
  for (int w = 0; w < warp; ++w) s = apply(sm.maps[w][lane], s);
  return s;
}

// The next tile of the launch (of all groups), for all threads of the block.
template <int Warps, bool Chain>
__device__ __forceinline__ uint32_t first_tile(const ScanArgs &p, TileMemory<Warps> &sm) {
  if constexpr (!Chain) return blockIdx.x;
  if (threadIdx.x == 0) sm.next = atomicAdd(p.counter, 1u) + 1u;
  __syncthreads();
  return sm.next;
}

template <typename T, bool Chain>
__global__ void __launch_bounds__(32 * kForwardWarps, sizeof(T) == 2 ? 2 : 1) scan_forward(const __grid_constant__ ScanArgs p) {
  constexpr int W = kForwardWarps;
  using Raw = typename Two<T>::Raw;
  extern __shared__ float dynamic[];  // [W][kRows][kCols] states of the sequences that start in the tile
  __shared__ TileMemory<W> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *starts = dynamic + warp * kRows * kCols;
  const uint32_t all = (uint32_t)p.tiles * (uint32_t)p.groups;
  uint32_t id = first_tile<W, Chain>(p, sm);
  while (id < all) {
    const int tile = id / (uint32_t)p.groups, group = id - tile * p.groups;
    const int64_t t0 = (int64_t)tile * W * kRows, i0 = t0 + warp * kRows;
    const int c = group * kCols + 2 * lane, count = p.channels - c;
    const int64_t row0 = row_of(p.q, i0), dir = p.q.reverse ? -1 : 1;
    uint32_t ahead = 0;
    if (Chain && threadIdx.x == 0) ahead = atomicAdd(p.counter, 1u) + 1u;
    Raw xr[kRows], gr[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      xr[r] = gr[r] = Two<T>::zero();
      if (i0 + r < p.q.rows) {
        const int64_t row = row0 + r * dir;
        gr[r] = Two<T>::load((const T *)p.g + row * p.ldg + c, count, p.vec);
        xr[r] = Two<T>::load((const T *)p.x + row * p.ldx + c, count, p.vec);
      }
    }
    const RowInfo f = rows_info(p.q, i0, lane);
    if (Chain && threadIdx.x == 0) sm.origin = f.live & 1 ? f.origin : t0;
    if (p.state) {
      ask_states(starts, p.state, f.first, f.seq, p.channels, c, lane);
    }
    float2 s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float2 g = Two<T>::values(gr[r]);
      s[r] = f2(small_side<sizeof(T) == 4>(g.x), small_side<sizeof(T) == 4>(g.y));
    }
    copies_done();
    Map m{f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (f.first >> r & 1) m.h = p.state ? *reinterpret_cast<float2 *>(starts + r * kCols + 2 * lane) : f2(0.f, 0.f);
      m.h = step(m.h, Two<T>::values(xr[r]), s[r]);
      m.b = step(m.b, f2(1.f, 1.f), s[r]);
    }
    if (f.first) m.b = f2(kCut, kCut);
    sm.maps[warp][lane] = m;
    __syncthreads();
    float2 h = state_before<W, Chain>(p, sm, tile, group, t0, warp, lane);
    if (p.saved && i0 < p.q.rows) put_state(p.saved, i0 / kRows, p.channels, c, h);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (f.first >> r & 1) h = p.state ? *reinterpret_cast<float2 *>(starts + r * kCols + 2 * lane) : f2(0.f, 0.f);
      h = step(h, Two<T>::values(xr[r]), s[r]);
      const bool live = f.live >> r & 1;
      if (live || (p.outside && i0 + r < p.q.rows))
        Two<T>::store((T *)p.out0 + (row0 + r * dir) * p.channels + c, live ? h : f2(0.f, 0.f), count,
                      p.vec);
      if (p.end && (f.last >> r & 1)) put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, c, h);
    }
    if (Chain && threadIdx.x == 0) sm.next = ahead;
    __syncthreads();  // everything in shared memory has been read
    id = Chain ? sm.next : id + gridDim.x;
  }
}

template <typename T, bool Chain>
__global__ void __launch_bounds__(32 * kBackwardWarps, 2) scan_backward(const __grid_constant__ ScanArgs p) {
  constexpr int W = kBackwardWarps;
  using Raw = typename Two<T>::Raw;
  extern __shared__ float dynamic[];  // [W][2][kRows][kCols]: states where sequences start, dfinal where they end
  __shared__ TileMemory<W> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *starts = dynamic + warp * 2 * kRows * kCols, *ends = starts + kRows * kCols;
  const uint32_t all = (uint32_t)p.tiles * (uint32_t)p.groups;
  uint32_t id = first_tile<W, Chain>(p, sm);
  while (id < all) {
    // time runs backwards: tile 0 holds the last rows and warp 0 the last of a tile
    const int tile = id / (uint32_t)p.groups, group = id - tile * p.groups;
    const int64_t i0 = ((int64_t)(p.tiles - 1 - tile) * W + (W - 1 - warp)) * kRows;
    const int c = group * kCols + 2 * lane, count = p.channels - c;
    const int64_t row0 = row_of(p.q, i0), dir = p.q.reverse ? -1 : 1;
    uint32_t ahead = 0;
    if (Chain && threadIdx.x == 0) ahead = atomicAdd(p.counter, 1u) + 1u;
    Raw xr[kRows], gr[kRows], dr[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      xr[r] = gr[r] = dr[r] = Two<T>::zero();
      if (i0 + r < p.q.rows) {
        const int64_t row = row0 + r * dir;
        gr[r] = Two<T>::load((const T *)p.g + row * p.ldg + c, count, p.vec);
        xr[r] = Two<T>::load((const T *)p.x + row * p.ldx + c, count, p.vec);
        if (p.dh) dr[r] = Two<T>::load((const T *)p.dh + row * p.lddh + c, count, p.vec);
      }
    }
    float2 h = f2(0.f, 0.f);
    if (i0 < p.q.rows) {
      const float *from = p.saved + i0 / kRows * p.channels + c;
      if (count > 0) h.x = from[0];
      if (count > 1) h.y = from[1];
    }
    const RowInfo f = rows_info(p.q, i0, lane);
    if (p.state) ask_states(starts, p.state, f.first, f.seq, p.channels, c, lane);
    if (p.dfinal) ask_states(ends, p.dfinal, f.last, f.seq, p.channels, c, lane);
    if (Chain) {
      // the row behind which the present sequence ends, counted backwards from the end of the last tile
      const int64_t span = (int64_t)p.tiles * W * kRows;
      const int64_t until = __shfl_sync(0xffffffffu, f.until, kRows - 1);
      if (threadIdx.x == 0) sm.origin = f.live >> (kRows - 1) & 1 ? span - until : (int64_t)tile * W * kRows;
    }
    float2 s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float2 g = Two<T>::values(gr[r]);
      s[r] = f2(small_side<sizeof(T) == 4>(g.x), small_side<sizeof(T) == 4>(g.y));
    }
    copies_done();
    float2 e[kRows];  // h_{t-1} - x_t
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (f.first >> r & 1) h = p.state ? *reinterpret_cast<float2 *>(starts + r * kCols + 2 * lane) : f2(0.f, 0.f);
      const float2 x = Two<T>::values(xr[r]);
      e[r] = add2(h, f2(-x.x, -x.y));
      h = fma2(f2(-s[r].x, -s[r].y), e[r], f2(below(s[r].x) ? x.x : h.x, below(s[r].y) ? x.y : h.y));
    }
    Map m{f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int r = kRows - 1; r >= 0; --r) {
      if (f.last >> r & 1) m.h = p.dfinal ? *reinterpret_cast<float2 *>(ends + r * kCols + 2 * lane) : f2(0.f, 0.f);
      m.h = message(add2(Two<T>::values(dr[r]), m.h), s[r]);
      m.b = step(m.b, f2(1.f, 1.f), s[r]);
    }
    if (f.last) m.b = f2(kCut, kCut);
    sm.maps[warp][lane] = m;
    __syncthreads();
    float2 carry = state_before<W, Chain>(p, sm, tile, group, (int64_t)tile * W * kRows, warp, lane);
#pragma unroll
    for (int r = kRows - 1; r >= 0; --r) {
      if (f.last >> r & 1) carry = p.dfinal ? *reinterpret_cast<float2 *>(ends + r * kCols + 2 * lane) : f2(0.f, 0.f);
      const float2 l = add2(Two<T>::values(dr[r]), carry);
      carry = message(l, s[r]);
      const bool live = f.live >> r & 1;
      if (i0 + r < p.q.rows) {
        const float2 a = f2(fabsf(s[r].x), fabsf(s[r].y)), b = add2(f2(1.f, 1.f), f2(-a.x, -a.y));
        const float2 in = f2(below(s[r].x) ? b.x : a.x, below(s[r].y) ? b.y : a.y);  // 1 - a
        const int64_t at = (row0 + r * dir) * p.channels + c;
        const float2 none = f2(0.f, 0.f);
        if (p.out0) Two<T>::store((T *)p.out0 + at, live ? mul2(in, l) : none, count, p.vec);
        if (p.out1) Two<T>::store((T *)p.out1 + at, live ? mul2(mul2(l, e[r]), mul2(a, b)) : none, count, p.vec);
      }
      if (p.end && (f.first >> r & 1)) put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, c, carry);
    }
    if (Chain && threadIdx.x == 0) sm.next = ahead;
    __syncthreads();
    id = Chain ? sm.next : id + gridDim.x;
  }
}

// Sequences of one row: nothing to scan.  Two channels a thread.
template <typename T>
__global__ void __launch_bounds__(256) scan_single(const __grid_constant__ ScanArgs p) {
  const int64_t pairs = (p.channels + 1) / 2, total = p.q.rows * pairs;
  const bool both = p.channels % 2 == 0 && ((uintptr_t)p.state & 7) == 0 && ((uintptr_t)p.end & 7) == 0;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t row = i / pairs;
    const int c = (int)(i - row * pairs) * 2, count = p.channels - c;
    const float2 g = Two<T>::values(Two<T>::load((const T *)p.g + row * p.ldg + c, count, p.vec));
    const float2 x = Two<T>::values(Two<T>::load((const T *)p.x + row * p.ldx + c, count, p.vec));
    const int64_t at = row * p.channels + c;
    float2 h = f2(0.f, 0.f);
    if (p.state) h = Two<float>::load(p.state + at, count, both);
    h = step(h, x, f2(small_side<sizeof(T) == 4>(g.x), small_side<sizeof(T) == 4>(g.y)));
    Two<T>::store((T *)p.out0 + at, h, count, p.vec);
    if (p.end) Two<float>::store(p.end + at, h, count, both);
  }
}

// ------------------------------------------------------------------ the calls

int64_t tiles_of(int64_t rows, int warps) { return (rows + warps * kRows - 1) / (warps * kRows); }

// Whether no sequence leaves a tile: whole sequences in every one, or a single tile.
bool closed_tiles(const sla_scan *s, int warps) {
  const int64_t tile = warps * kRows;
  if (s->rows <= tile) return true;
  if (s->offsets || s->sequences < 1) return false;
  return tile % (s->rows / s->sequences) == 0;
}

size_t chain_bytes(const sla_scan *s, int warps) {
  if (closed_tiles(s, warps)) return 0;
  const size_t groups = (size_t)((s->channels + kCols - 1) / kCols), tiles = (size_t)tiles_of(s->rows, warps);
  return align256(256 + (tiles + tiles / kSpan) * groups * kCols * sizeof(uint64_t));
}

size_t saved_bytes(const sla_scan *s) {
  return align256((size_t)((s->rows + kRows - 1) / kRows) * (size_t)s->channels * sizeof(float));
}

sla_status check_scan(const sla_scan *s) {
  if (!s) return SLA_INVALID_ARG;
  const int64_t most = ((int64_t)1 << 31) - 1;
  if (s->rows < 0 || s->rows > most || s->channels < 1 || s->channels > (int64_t)1 << 24) return SLA_INVALID_ARG;
  if (s->sequences < 0 || s->sequences > most || !net_dtype(s->dtype)) return SLA_INVALID_ARG;
  if (s->reverse != 0 && s->reverse != 1) return SLA_INVALID_ARG;
  if (s->outside != 0 && s->outside != 1) return SLA_INVALID_ARG;
  if (s->offsets) {
    if (s->offsets_type != SLA_I32 && s->offsets_type != SLA_I64) return SLA_INVALID_ARG;
    if (!aligned(s->offsets, s->offsets_type == SLA_I64 ? 8 : 4)) return SLA_INVALID_ARG;
  } else if (s->sequences ? s->rows % s->sequences != 0 : s->rows != 0) {
    return SLA_INVALID_ARG;
  }
  // tiles of all groups are counted in 32 bits
  const int64_t groups = (s->channels + kCols - 1) / kCols;
  return tiles_of(s->rows, kBackwardWarps) * groups < most ? SLA_OK : SLA_INVALID_ARG;
}

sla_status check_rows(const void *p, const sla_scan *s, int64_t ld) {
  if (s->rows == 0) return SLA_OK;
  if (!p || !aligned(p, net_size(s->dtype))) return SLA_INVALID_ARG;
  return ld >= s->channels || s->rows == 1 ? SLA_OK : SLA_INVALID_ARG;
}

sla_status check_buffer(const void *p, size_t bytes, size_t need) {
  if (need == 0) return SLA_OK;
  if (!p || !aligned(p, 256)) return SLA_INVALID_ARG;
  return bytes < need ? SLA_WORKSPACE_TOO_SMALL : SLA_OK;
}

ScanArgs scan_args(const sla_scan *s, int warps, void *ws) {
  ScanArgs p{};
  p.q = {s->rows, s->sequences, s->offsets || !s->sequences ? 0 : s->rows / s->sequences, s->offsets,
         s->offsets_type == SLA_I64, s->reverse};
  p.channels = (int)s->channels, p.groups = (int)((s->channels + kCols - 1) / kCols);
  p.outside = s->outside;
  p.tiles = (int)tiles_of(s->rows, warps);
  p.counter = (uint32_t *)ws;
  p.maps = (uint64_t *)((char *)ws + 256);
  p.states = p.maps + (int64_t)p.tiles * p.groups * kCols;
  return p;
}

// Whether two neighbouring channels of every row may be moved at once.
bool pairs_aligned(const sla_scan *s, const void *p, int64_t ld) {
  return aligned(p, 2 * net_size(s->dtype)) && (s->rows == 1 || ld % 2 == 0);
}

template <typename K>
cudaError_t launch(K kernel, const ScanArgs &p, int block, size_t smem, int resident, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.tiles * p.groups;
  kernel<<<(unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * resident), block, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_forward(const ScanArgs &p, bool chain, cudaStream_t st) {
  const size_t smem = p.state ? kForwardWarps * kRows * kCols * sizeof(float) : 0;
  constexpr int resident = sizeof(T) == 2 ? 2 : 1;
  return chain ? launch(scan_forward<T, true>, p, 32 * kForwardWarps, smem, resident, st)
               : launch(scan_forward<T, false>, p, 32 * kForwardWarps, smem, resident, st);
}

template <typename T>
cudaError_t run_backward(const ScanArgs &p, bool chain, cudaStream_t st) {
  const size_t smem = p.state || p.dfinal ? kBackwardWarps * 2 * kRows * kCols * sizeof(float) : 0;
  return chain ? launch(scan_backward<T, true>, p, 32 * kBackwardWarps, smem, 2, st)
               : launch(scan_backward<T, false>, p, 32 * kBackwardWarps, smem, 2, st);
}

// `to` = `from`, or zero: what sequences without rows have.
cudaError_t copy_states(float *to, const float *from, const sla_scan *s, cudaStream_t st) {
  const size_t bytes = (size_t)s->sequences * (size_t)s->channels * sizeof(float);
  if (!to || to == from || !bytes) return cudaSuccess;
  return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API size_t sla_gated_scan_saved_bytes(const sla_scan *s) { return check_scan(s) == SLA_OK ? saved_bytes(s) : 0; }

SLA_API size_t sla_gated_scan_workspace_bytes(const sla_scan *s) {
  return check_scan(s) == SLA_OK ? std::max(chain_bytes(s, kForwardWarps), chain_bytes(s, kBackwardWarps)) : 0;
}

SLA_API sla_status sla_gated_scan(const sla_scan *s, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                                  const float *state, void *h, float *final_state, void *saved, size_t saved_size,
                                  void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_scan(s));
  SLA_CHECK(check_rows(x, s, ldx));
  SLA_CHECK(check_rows(gate, s, ldg));
  SLA_CHECK(check_rows(h, s, s->channels));
  if (!aligned(state, 4) || !aligned(final_state, 4)) return SLA_INVALID_ARG;
  if (saved) SLA_CHECK(check_buffer(saved, saved_size, saved_bytes(s)));
  const size_t need = chain_bytes(s, kForwardWarps);
  SLA_CHECK(check_buffer(workspace, ws_bytes, need));
  cudaStream_t st = (cudaStream_t)stream;
  if (s->offsets || s->rows == 0) {
    const cudaError_t e = copy_states(final_state, state, s, st);
    if (e != cudaSuccess) return fail(e);
  }
  if (s->rows == 0) return SLA_OK;
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  ScanArgs p = scan_args(s, kForwardWarps, workspace);
  p.x = x, p.ldx = ldx, p.g = gate, p.ldg = ldg, p.state = state, p.out0 = h, p.end = final_state;
  p.saved = (float *)saved, p.timeouts = earlier.count;
  p.vec = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
          pairs_aligned(s, h, s->channels);
  const bool chain = need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  if (p.q.length == 1 && !saved) {
    const int64_t pairs = p.q.rows * ((p.channels + 1) / 2);
    const unsigned grid = (unsigned)std::min<int64_t>((pairs + 255) / 256, sm_count() * 8);
    if (s->dtype == SLA_F32)
      scan_single<float><<<grid, 256, 0, st>>>(p);
    else if (s->dtype == SLA_F16)
      scan_single<f16><<<grid, 256, 0, st>>>(p);
    else
      scan_single<bf16><<<grid, 256, 0, st>>>(p);
    e = cudaGetLastError();
  } else {
    e = s->dtype == SLA_F32   ? run_forward<float>(p, chain, st)
        : s->dtype == SLA_F16 ? run_forward<f16>(p, chain, st)
                              : run_forward<bf16>(p, chain, st);
  }
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

SLA_API sla_status sla_gated_scan_backward(const sla_scan *s, const void *dh, int64_t lddh, const float *dfinal,
                                           const void *x, int64_t ldx, const void *gate, int64_t ldg,
                                           const float *state, const void *saved, size_t saved_size, void *dx,
                                           void *dgate, float *dstate, void *workspace, size_t ws_bytes,
                                           void *stream) {
  SLA_CHECK(check_scan(s));
  if (dh) SLA_CHECK(check_rows(dh, s, lddh));
  SLA_CHECK(check_rows(x, s, ldx));
  SLA_CHECK(check_rows(gate, s, ldg));
  const size_t e0 = net_size(s->dtype);
  if (!aligned(state, 4) || !aligned(dfinal, 4) || !aligned(dstate, 4) || !aligned(dx, e0) || !aligned(dgate, e0))
    return SLA_INVALID_ARG;
  SLA_CHECK(check_buffer(saved, saved_size, saved_bytes(s)));
  const size_t need = chain_bytes(s, kBackwardWarps);
  SLA_CHECK(check_buffer(workspace, ws_bytes, need));
  cudaStream_t st = (cudaStream_t)stream;
  if (s->offsets || s->rows == 0) {
    const cudaError_t e = copy_states(dstate, dfinal, s, st);
    if (e != cudaSuccess) return fail(e);
  }
  if (s->rows == 0 || (!dx && !dgate && !dstate)) return SLA_OK;
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  ScanArgs p = scan_args(s, kBackwardWarps, workspace);
  p.dh = dh, p.lddh = lddh, p.x = x, p.ldx = ldx, p.g = gate, p.ldg = ldg, p.state = state, p.dfinal = dfinal;
  p.out0 = dx, p.out1 = dgate, p.end = dstate, p.saved = (float *)const_cast<void *>(saved);
  p.timeouts = earlier.count;
  p.vec = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
          (!dh || pairs_aligned(s, dh, lddh)) && pairs_aligned(s, dx, s->channels) &&
          pairs_aligned(s, dgate, s->channels);
  const bool chain = need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  e = s->dtype == SLA_F32   ? run_backward<float>(p, chain, st)
      : s->dtype == SLA_F16 ? run_backward<f16>(p, chain, st)
                            : run_backward<bf16>(p, chain, st);
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

}  // extern "C"
