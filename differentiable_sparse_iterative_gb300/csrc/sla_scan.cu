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
// over them twice: once for the map (A, H) from the state before the rows to the state behind them,
// s -> A s + H, and, when that state is known, once for the results.  In between the maps of the block's warps
// are joined in shared memory, the block's is published, and the state before the tile is put together from
// the maps of the tiles before it, back to the tile in which the sequence starts or the last of the states that
// every kSpan-th tile publishes.  Tiles are handed out in order of time by a counter, so those waited for are
// always at work; which block takes which tile changes no result, and the maps are joined in a fixed order.
//
// A map's two float32 are published as one 64-bit word, so that the word itself says whether it is there (the
// workspace is set to ones, a NaN that no map has): no flag, no fence.
//
// A step is h' = x + a (h - x), so that a's rounding never makes a and 1 - a sum up to something else than one; where
// 1 - a itself is a factor of a result it is e a with e = exp(-g), right relative to itself.  A sequence's start is a map
// with A = kCut, whose H replaces what came before, whatever that is: an infinity or a NaN stays within its sequence.
//
// What costs is instructions as much as bytes (two special functions an element and some twenty other
// instructions), so rows are walked with running pointers, and warps whose rows hold no sequence's start or end, nearly
// all where sequences are long, take a copy of the loops without those checks.
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
constexpr float kCut = -1.f;
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

// A lane's two channels: neighbours where every row's pairs are aligned (Pair), else 32 apart, so that a warp's
// accesses stay whole.
template <typename T, bool Pair>
struct Lane {
  using Raw = typename std::conditional<sizeof(T) == 4, float2, uint32_t>::type;
  static constexpr int apart = Pair ? 1 : 32;
  int c;          // the first channel
  bool on0, on1;  // whether there are such channels
  __device__ __forceinline__ Lane(int group, int lane, int channels)
      : c(group * kCols + (Pair ? 2 * lane : lane)), on0(c < channels), on1(c + apart < channels) {}
  static __device__ __forceinline__ Raw none() {
    if constexpr (sizeof(T) == 4)
      return f2(0.f, 0.f);
    else
      return 0u;
  }
  // p: the first channel's place
  __device__ __forceinline__ Raw load(const T *p) const {
    if constexpr (Pair) {
      return on0 ? *reinterpret_cast<const Raw *>(p) : none();
    } else {
      const T zero = from_f32<T>(0.f);
      const T a = on0 ? p[0] : zero, b = on1 ? p[apart] : zero;
      if constexpr (sizeof(T) == 4)
        return f2(a, b);
      else
        return *reinterpret_cast<const uint16_t *>(&a) | ((uint32_t) * reinterpret_cast<const uint16_t *>(&b) << 16);
    }
  }
  static __device__ __forceinline__ float2 values(Raw r) {
    if constexpr (sizeof(T) == 4)
      return r;
    else
      return unpair16(r, T{});
  }
  __device__ __forceinline__ void store(T *p, float2 v) const {
    if constexpr (Pair) {
      if (!on0) return;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2 *>(p) = v;
      else
        *reinterpret_cast<uint32_t *>(p) = pair16(v.x, v.y, T{});
    } else {
      if (on0) p[0] = from_f32<T>(v.x);
      if (on1) p[apart] = from_f32<T>(v.y);
    }
  }
  // float32 states, [rows][channels]
  __device__ __forceinline__ float2 state(const float *p, int64_t row, int channels) const {
    p += row * channels + c;
    return f2(on0 ? p[0] : 0.f, on1 ? p[apart] : 0.f);
  }
  __device__ __forceinline__ void put_state(float *p, int64_t row, int channels, float2 v) const {
    p += row * channels + c;
    if (on0) p[0] = v.x;
    if (on1) p[apart] = v.y;
  }
};

// The smaller of two, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// e = exp(-g) (at most 2^126, so that nothing below is infinite) and a = 1 / (1 + e).
__device__ __forceinline__ float2 exp_minus(float2 g) {
  const float2 m = mul2(g, f2(-1.4426950408889634f, -1.4426950408889634f));
  return f2(ex2_approx(min_nan(m.x, 126.f)), ex2_approx(min_nan(m.y, 126.f)));
}
__device__ __forceinline__ float2 keep_of(float2 e) {
  const float2 d = add2(e, f2(1.f, 1.f));
  return f2(rcp_approx(d.x), rcp_approx(d.y));
}

// One step of h.
__device__ __forceinline__ float2 step(float2 h, float2 x, float2 a) { return fma2(a, add2(h, f2(-x.x, -x.y)), x); }

// s -> a s + h of two channels; a = kCut: s -> h.
struct Map {
  float2 a, h;
};

__device__ __forceinline__ float2 apply(const Map &m, float2 s) {
  const float2 r = fma2(m.a, s, m.h);
  return m.a.x == kCut ? m.h : r;
}
__device__ __forceinline__ void join(Map &m, const Map &n) {  // m first
  m.h = apply(n, m.h);
  const float2 a = mul2(m.a, n.a);
  const bool cut = m.a.x == kCut || n.a.x == kCut;
  m.a = cut ? f2(kCut, kCut) : a;
}

__device__ __forceinline__ uint64_t word_of(float a, float h) {
  const uint64_t w = (uint64_t)__float_as_uint(h) << 32 | __float_as_uint(a);
  return w == kAbsent ? 0x7fffffff7fffffffull : w;  // both are NaN: another one
}
__device__ __forceinline__ void publish(uint64_t *p, const Map &m) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(word_of(m.a.x, m.h.x)),
               "l"(word_of(m.a.y, m.h.y))
               : "memory");
}
__device__ __forceinline__ bool look(const uint64_t *p, Map &m) {
  uint64_t a, b;
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
  m.a = f2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)b));
  m.h = f2(__uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)(b >> 32)));
  return a != kAbsent && b != kAbsent;
}

// Looks until all lanes' words are there (`there`: what a first look found).  False: they never came.
__device__ __forceinline__ bool wait_for(const uint64_t *p, Map &m, bool there) {
  if (__all_sync(0xffffffffu, there)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, look(p, m))) return true;
    if (__any_sync(0xffffffffu, clock64() - t0 > kScanClocks)) return false;
  }
}

__device__ __forceinline__ void copy_async(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Asks for the rows of `from` ([count][channels] float32) that belong to the sequences of the marked rows: to the lane's
// two places of row r of `to` ([kRows][32] pairs), which the lane itself reads.
template <typename L>
__device__ __forceinline__ void ask_states(float2 *to, const float *from, uint32_t marks, int seq, int channels, const L &l,
                                           int lane) {
  for (uint32_t m = marks; m; m &= m - 1) {
    const int r = __ffs(m) - 1;
    const int64_t s = __shfl_sync(0xffffffffu, seq, r);
    const float *p = from + s * channels + l.c;
    float *d = &to[r * 32 + lane].x;
    if (l.on0) copy_async(d, p);
    if (l.on1) copy_async(d + 1, p + L::apart);
  }
}

// The tile a block works on, and the maps of its warps.
template <int Warps>
struct TileMemory {
  Map maps[Warps][32];      // of the warps
  Map carry[Warps][32];     // parts of the way from the known state to the tile
  int64_t origin;           // the scan's index of the first row that the tile's first row depends on
  uint32_t next;
};

// The state before this warp's rows.  maps are in place (and a barrier behind them); `own` is this warp's; i0: the scan's
// index of the tile's first row.  On the way the tile's map is published, the state before the tile found, back from the
// tile where the present sequence starts or the last published state, in the order of time, and the state
// behind the tile published where others look for it.
template <int Warps, bool Chain>
__device__ __forceinline__ float2 state_before(const ScanArgs &p, TileMemory<Warps> &sm, int tile, int group, int64_t i0,
                                               Map own, int warp, int lane) {
  float2 s = f2(0.f, 0.f);
  Map before{f2(1.f, 1.f), f2(0.f, 0.f)};  // of the warps before this one
  if constexpr (!Chain) {
#pragma unroll 4
    for (int w = 0; w < warp; ++w) join(before, sm.maps[w][lane]);
    return apply(before, s);
  } else {
    const int64_t origin = sm.origin;  // i0: nothing before the tile matters
    const bool needed = origin < i0;
    const int first = (int)(origin / (Warps * kRows)), base = tile / kSpan * kSpan, lo = max(first, base);
    const bool known = first < base;  // the state before `base` is needed
    const int count = needed ? tile - lo : 0, per = (count + Warps - 1) / Warps;
    const int from = lo + warp * per, to = min(lo + count, from + per);
    const int64_t apart = (int64_t)p.groups * kCols;
    const uint64_t *at = p.maps + from * apart + group * kCols + 2 * lane;
    Map n;
    bool there = true;  // the first look is under way while the maps of the block are joined
    if (from < to) there = look(at, n);
#pragma unroll 4
    for (int w = 0; w < warp; ++w) join(before, sm.maps[w][lane]);
    if (warp == Warps - 1) {
      Map all = before;
      join(all, own);
      publish(p.maps + tile * apart + group * kCols + 2 * lane, all);
      own = all;
    }
    if (needed) {
      Map m{f2(1.f, 1.f), f2(0.f, 0.f)};
      bool ok = true;
      if (warp == 0 && known) {
        Map k;
        const uint64_t *q = p.states + (base / kSpan - 1) * apart + group * kCols + 2 * lane;
        ok = wait_for(q, k, look(q, k));
        m = k;
      }
      for (int i = from; i < to; ++i, at += apart) {
        if (i > from) there = look(at, n);
        ok = wait_for(at, n, there) && ok;
        join(m, n);
      }
      sm.carry[warp][lane] = m;
      if (!ok && lane == 0) atomicAdd_system(p.timeouts, 1u);
      __syncthreads();
      const int parts = per ? (count + per - 1) / per : 1;
#pragma unroll 4
      for (int w = 0; w < parts; ++w) s = apply(sm.carry[w][lane], s);
    }
    if (warp == Warps - 1 && (tile + 1) % kSpan == 0) {
      const Map behind{f2(kCut, kCut), apply(own, s)};
      publish(p.states + (tile / kSpan) * apart + group * kCols + 2 * lane, behind);
    }
    return apply(before, s);
  }
}

// The block's first tile of the launch (of all groups), for all its threads.
template <int Warps, bool Chain>
__device__ __forceinline__ uint32_t first_tile(const ScanArgs &p, TileMemory<Warps> &sm) {
  if constexpr (!Chain) return blockIdx.x;
  if (threadIdx.x == 0) sm.next = atomicAdd(p.counter, 1u) + 1u;
  __syncthreads();
  return sm.next;
}

template <typename T, bool Chain, bool Pair>
__global__ void __launch_bounds__(32 * kForwardWarps, sizeof(T) == 2 ? 2 : 1) scan_forward(const __grid_constant__ ScanArgs p) {
  constexpr int W = kForwardWarps;
  using L = Lane<T, Pair>;
  extern __shared__ float2 dynamic[];  // [W][kRows][32] states of the sequences that start in the tile
  __shared__ TileMemory<W> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 *starts = dynamic + warp * kRows * 32;
  const uint32_t all = (uint32_t)p.tiles * (uint32_t)p.groups;
  const int64_t dir = p.q.reverse ? -1 : 1;
  uint32_t id = first_tile<W, Chain>(p, sm);
  while (id < all) {
    const int tile = id / (uint32_t)p.groups, group = id - tile * p.groups;
    const int64_t t0 = (int64_t)tile * W * kRows, i0 = t0 + warp * kRows;
    const L l(group, lane, p.channels);
    const int64_t row0 = row_of(p.q, i0);
    const int left = (int)min((int64_t)kRows, p.q.rows - i0);
    typename L::Raw xr[kRows], gr[kRows];
    {
      const T *px = (const T *)p.x + row0 * p.ldx + l.c, *pg = (const T *)p.g + row0 * p.ldg + l.c;
      const int64_t sx = dir * p.ldx, sg = dir * p.ldg;
#pragma unroll
      for (int r = 0; r < kRows; ++r, px += sx, pg += sg) {
        xr[r] = gr[r] = L::none();
        if (r < left) {
          gr[r] = l.load(pg);
          xr[r] = l.load(px);
        }
      }
    }
    const RowInfo f = rows_info(p.q, i0, lane);
    const bool inner = f.live == (1u << kRows) - 1 && !f.first && !f.last;
    if (Chain && threadIdx.x == 0) sm.origin = f.live & 1 ? f.origin : t0;
    if (p.state && f.first) ask_states(starts, p.state, f.first, f.seq, p.channels, l, lane);
    float2 a[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) a[r] = keep_of(exp_minus(L::values(gr[r])));
    Map m{f2(1.f, 1.f), f2(0.f, 0.f)};
    auto start = [&](int r) { return p.state ? starts[r * 32 + lane] : f2(0.f, 0.f); };
    if (inner) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        m.h = step(m.h, L::values(xr[r]), a[r]);
        m.a = mul2(m.a, a[r]);
      }
    } else {
      copies_done();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (f.first >> r & 1) m.h = start(r);
        m.h = step(m.h, L::values(xr[r]), a[r]);
        m.a = mul2(m.a, a[r]);
      }
      if (f.first) m.a = f2(kCut, kCut);
    }
    sm.maps[warp][lane] = m;
    __syncthreads();
    float2 h = state_before<W, Chain>(p, sm, tile, group, t0, m, warp, lane);
    // (taken no sooner: a tile that waits for its block's present one keeps all later ones waiting)
    uint32_t ahead = 0;
    if (Chain && threadIdx.x == 0) ahead = atomicAdd(p.counter, 1u) + 1u;
    if (p.saved && left > 0) l.put_state(p.saved, i0 / kRows, p.channels, h);
    T *po = (T *)p.out0 + row0 * p.channels + l.c;
    const int64_t so = dir * p.channels;
    if (inner) {
#pragma unroll
      for (int r = 0; r < kRows; ++r, po += so) {
        h = step(h, L::values(xr[r]), a[r]);
        l.store(po, h);
      }
    } else {
#pragma unroll
      for (int r = 0; r < kRows; ++r, po += so) {
        if (f.first >> r & 1) h = start(r);
        h = step(h, L::values(xr[r]), a[r]);
        const bool live = f.live >> r & 1;
        if (live || (p.outside && r < left)) l.store(po, live ? h : f2(0.f, 0.f));
        if (p.end && (f.last >> r & 1)) l.put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, h);
      }
    }
    if (Chain && threadIdx.x == 0) sm.next = ahead;
    __syncthreads();  // everything in shared memory has been read
    id = Chain ? sm.next : id + gridDim.x;
  }
}

template <typename T, bool Chain, bool Pair>
__global__ void __launch_bounds__(32 * kBackwardWarps, 2) scan_backward(const __grid_constant__ ScanArgs p) {
  constexpr int W = kBackwardWarps;
  using L = Lane<T, Pair>;
  extern __shared__ float2 dynamic[];  // [W][2][kRows][32]: states where sequences start, dfinal where they end
  __shared__ TileMemory<W> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 *starts = dynamic + warp * 2 * kRows * 32, *ends = starts + kRows * 32;
  const uint32_t all = (uint32_t)p.tiles * (uint32_t)p.groups;
  const int64_t dir = p.q.reverse ? -1 : 1;
  uint32_t id = first_tile<W, Chain>(p, sm);
  while (id < all) {
    // time runs backwards: tile 0 holds the last rows and warp 0 the last of a tile
    const int tile = id / (uint32_t)p.groups, group = id - tile * p.groups;
    const int64_t t0 = (int64_t)tile * W * kRows;
    const int64_t i0 = ((int64_t)(p.tiles - 1 - tile) * W + (W - 1 - warp)) * kRows;
    const L l(group, lane, p.channels);
    const int64_t row0 = row_of(p.q, i0);
    const int left = (int)max(min((int64_t)kRows, p.q.rows - i0), (int64_t)0);
    typename L::Raw xr[kRows], gr[kRows], dr[kRows];
    {
      const T *px = (const T *)p.x + row0 * p.ldx + l.c, *pg = (const T *)p.g + row0 * p.ldg + l.c;
      const T *pd = (const T *)p.dh + row0 * p.lddh + l.c;
      const int64_t sx = dir * p.ldx, sg = dir * p.ldg, sd = dir * p.lddh;
#pragma unroll
      for (int r = 0; r < kRows; ++r, px += sx, pg += sg, pd += sd) {
        xr[r] = gr[r] = dr[r] = L::none();
        if (r < left) {
          gr[r] = l.load(pg);
          xr[r] = l.load(px);
          if (p.dh) dr[r] = l.load(pd);
        }
      }
    }
    float2 h = left > 0 ? l.state(p.saved, i0 / kRows, p.channels) : f2(0.f, 0.f);
    const RowInfo f = rows_info(p.q, i0, lane);
    const bool inner = f.live == (1u << kRows) - 1 && !f.first && !f.last;
    if (p.state && f.first) ask_states(starts, p.state, f.first, f.seq, p.channels, l, lane);
    if (p.dfinal && f.last) ask_states(ends, p.dfinal, f.last, f.seq, p.channels, l, lane);
    if (Chain) {
      // the row behind which the present sequence ends, counted backwards from the end of the last tile
      const int64_t span = (int64_t)p.tiles * W * kRows;
      const int64_t until = __shfl_sync(0xffffffffu, f.until, kRows - 1);
      if (threadIdx.x == 0) sm.origin = f.live >> (kRows - 1) & 1 ? span - until : t0;
    }
    float2 a[kRows], e[kRows];  // e: h_{t-1} - x_t
#pragma unroll
    for (int r = 0; r < kRows; ++r) a[r] = keep_of(exp_minus(L::values(gr[r])));
    auto start = [&](int r) { return p.state ? starts[r * 32 + lane] : f2(0.f, 0.f); };
    auto end = [&](int r) { return p.dfinal ? ends[r * 32 + lane] : f2(0.f, 0.f); };
    Map m{f2(1.f, 1.f), f2(0.f, 0.f)};
    if (inner) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float2 x = L::values(xr[r]);
        e[r] = add2(h, f2(-x.x, -x.y));
        h = fma2(a[r], e[r], x);
      }
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r) {
        m.h = mul2(a[r], add2(L::values(dr[r]), m.h));
        m.a = mul2(m.a, a[r]);
      }
    } else {
      copies_done();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (f.first >> r & 1) h = start(r);
        const float2 x = L::values(xr[r]);
        e[r] = add2(h, f2(-x.x, -x.y));
        h = fma2(a[r], e[r], x);
      }
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r) {
        if (f.last >> r & 1) m.h = end(r);
        m.h = mul2(a[r], add2(L::values(dr[r]), m.h));
        m.a = mul2(m.a, a[r]);
      }
      if (f.last) m.a = f2(kCut, kCut);
    }
    sm.maps[warp][lane] = m;
    __syncthreads();
    float2 carry = state_before<W, Chain>(p, sm, tile, group, t0, m, warp, lane);
    uint32_t ahead = 0;
    if (Chain && threadIdx.x == 0) ahead = atomicAdd(p.counter, 1u) + 1u;
    const int64_t so = dir * p.channels, o = (row0 + (kRows - 1) * dir) * p.channels + l.c;
    T *px = (T *)p.out0 + o, *pg = (T *)p.out1 + o;
    auto results = [&](int r, float2 lam, bool live) {
      const float2 b = mul2(exp_minus(L::values(gr[r])), a[r]);  // 1 - a
      const float2 none = f2(0.f, 0.f);
      if (p.out0) l.store(px, live ? mul2(b, lam) : none);
      if (p.out1) l.store(pg, live ? mul2(mul2(lam, e[r]), mul2(a[r], b)) : none);
    };
    if (inner) {
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r, px -= so, pg -= so) {
        const float2 lam = add2(L::values(dr[r]), carry);
        carry = mul2(a[r], lam);
        results(r, lam, true);
      }
    } else {
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r, px -= so, pg -= so) {
        if (f.last >> r & 1) carry = end(r);
        const float2 lam = add2(L::values(dr[r]), carry);
        carry = mul2(a[r], lam);
        if (r < left) results(r, lam, f.live >> r & 1);
        if (p.end && (f.first >> r & 1)) l.put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, carry);
      }
    }
    if (Chain && threadIdx.x == 0) sm.next = ahead;
    __syncthreads();
    id = Chain ? sm.next : id + gridDim.x;
  }
}

// Sequences of one row: nothing to scan.  Two channels a thread.
template <typename T, bool Pair>
__global__ void __launch_bounds__(256) scan_single(const __grid_constant__ ScanArgs p) {
  using L = Lane<T, Pair>;
  const int64_t total = p.q.rows * p.groups * 32;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t rg = i >> 5, row = rg / p.groups;
    const L l((int)(rg - row * p.groups), (int)(i & 31), p.channels);
    const float2 g = L::values(l.load((const T *)p.g + row * p.ldg + l.c));
    const float2 x = L::values(l.load((const T *)p.x + row * p.ldx + l.c));
    float2 h = p.state ? l.state(p.state, row, p.channels) : f2(0.f, 0.f);
    h = step(h, x, keep_of(exp_minus(g)));
    l.store((T *)p.out0 + row * p.channels + l.c, h);
    if (p.end) l.put_state(p.end, row, p.channels, h);
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

// Whether every row's pairs of channels may be moved at once.
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

template <typename T, bool Pair>
cudaError_t run_forward(const ScanArgs &p, bool chain, cudaStream_t st) {
  if (p.q.length == 1 && !p.saved) {
    const int64_t threads = p.q.rows * p.groups * 32;
    scan_single<T, Pair><<<(unsigned)std::min<int64_t>((threads + 255) / 256, sm_count() * 8), 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  const size_t smem = p.state ? kForwardWarps * kRows * kCols * sizeof(float) : 0;
  constexpr int resident = sizeof(T) == 2 ? 2 : 1;
  return chain ? launch(scan_forward<T, true, Pair>, p, 32 * kForwardWarps, smem, resident, st)
               : launch(scan_forward<T, false, Pair>, p, 32 * kForwardWarps, smem, resident, st);
}

template <typename T, bool Pair>
cudaError_t run_backward(const ScanArgs &p, bool chain, cudaStream_t st) {
  const size_t smem = p.state || p.dfinal ? kBackwardWarps * 2 * kRows * kCols * sizeof(float) : 0;
  return chain ? launch(scan_backward<T, true, Pair>, p, 32 * kBackwardWarps, smem, 2, st)
               : launch(scan_backward<T, false, Pair>, p, 32 * kBackwardWarps, smem, 2, st);
}

// Calls f with the element type and whether channels go in pairs.
template <typename F>
cudaError_t by_type(int32_t dtype, bool pairs, F &&f) {
  using std::false_type;
  using std::true_type;
  if (dtype == SLA_F32) return pairs ? f(float{}, true_type{}) : f(float{}, false_type{});
  if (dtype == SLA_F16) return pairs ? f(f16{}, true_type{}) : f(f16{}, false_type{});
  return pairs ? f(bf16{}, true_type{}) : f(bf16{}, false_type{});
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
  const bool pairs = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
                     pairs_aligned(s, h, s->channels);
  const bool chain = need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  e = by_type(s->dtype, pairs, [&](auto t, auto pair) { return run_forward<decltype(t), decltype(pair)::value>(p, chain, st); });
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
  const bool pairs = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
                     (!dh || pairs_aligned(s, dh, lddh)) && pairs_aligned(s, dx, s->channels) &&
                     pairs_aligned(s, dgate, s->channels);
  const bool chain = need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  e = by_type(s->dtype, pairs, [&](auto t, auto pair) { return run_backward<decltype(t), decltype(pair)::value>(p, chain, st); });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

}  // extern "C"
