// The gated scan: a linear recurrence along the rows of sequences, channel by channel, forward and backward.
//
//   h_t = a_t h_{t-1} + (1 - a_t) x_t,  a = 1 / (1 + e^-g),  h_0 the sequence's state                 (a solve with a
//   l_t = dh_t + a_{t+1} l_{t+1}        the gradient of h_t                                   unit bidiagonal matrix, and
//   dx = (1 - a) l,  dg = l (h_{t-1} - x) a (1 - a),  dstate = a_1 l_1                             with its transpose)
//
// Both are bound by memory: two reads and a write forward, three reads and two writes backward (h is formed
// again from x and g, from float32 states that the forward call leaves every kSaved rows: an eighth of what reading h
// would cost, and exact).  To read everything once with the rows in parallel, a block
// takes a tile of rows by kCols channels into registers, kRows rows a warp, two channels a lane, and goes
// over them twice: once for the map (A, H) from the state before the rows to the state behind them,
// s -> A s + H, and, when that state is known, once for the results.  In between the maps of the block's warps
// are joined in shared memory, the block's is published, and the state before the tile is put together from
// the maps of the tiles before it, back to the tile in which the sequence starts or the last of the states that
// every kSpan-th tile publishes; every kFold-th tile publishes the map of its kFold tiles, so that at most 15 tiles, 31 folds
// and a state are looked at.  (One path of 1,000,000 rows waits from state to state, 3 us each, so they are far apart.)
//
// Tiles are handed out in order of time by a counter, so those waited for are
// always at work; which block takes which tile changes no result, and the maps are joined in a fixed order.  A block takes its
// next tile only when the present one's state is known: a tile that waits for its block keeps all later ones waiting (taken
// while the present one still waited, one path of 1,000,000 rows took 454 us, 1000 lines of 1000 a training step of 1023).
//
// A map's two float32 are published as one 64-bit word, so that the word itself says whether it is there (the
// workspace is set to ones, a NaN that no map has): no flag, no fence.
//
// A gate is held as the smaller of a and 1 - a, right relative to itself (next to one, float32's a has lost what 1 - a is: from a
// gate of 17 on nothing of x would be left, at 10 one part in 1,700 of what x adds to a state of zero would be wrong), and a step is
// h' = h + (1 - a) (x - h) where the gate is open, x + a (h - x) where it is closed: a and 1 - a sum up to one in both.  What a map
// takes from the state is held in the same way: a gate of 14 keeps a state over a path of a million rows, each of which takes less
// than two parts in a million (as a product of float32's a it was off by 0.5 % at the end).  A state is rounded once a row, so
// that n rows may move it by n 2^-25 of itself; a walk's (below) by all of its rows, a tile's by its 128 and the maps before it.  A
// sequence's start is a map with A = kCut, whose H replaces what came before, whatever that is: an infinity or a NaN stays
// within its sequence.
//
// What costs is instructions as much as bytes (two special functions an element and some thirty other
// instructions), so an address is one multiply-add, and warps whose rows hold no sequence's start or end, nearly
// all where sequences are long, take a copy of the loops without those checks.
//
// Measured by tiles, against the copy rate of 6.8 TB/s: one sequence of 1,000,000 x 64 float32 209 us (0.54), in bfloat16 181
// (0.31) and 434 a training step (0.35); 57 packed sequences, 60,001 x 333 float16, backwards, a training step 185 us (0.25).
// By walks (below): 1000 sequences of 1000 x 64 bfloat16, a training step 286 us (0.53), in float32 352 (0.86).  (With maps of
// float32's a and 1 - a taken from that: 181, 153 and 384; 173; 263 and 328.)
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "sla_act.cuh"
#include "sla_common.cuh"
#include "sla_host.h"
#include "sla_net.cuh"

namespace sla {
namespace {

// Rows of a warp: as many as the registers hold, backward with h_{t-1} - x_t beside the rest.
template <typename T, bool Backward>
inline constexpr int kRows = Backward && sizeof(T) == 4 ? 8 : 16;
template <typename T>
inline constexpr int kSaved = kRows<T, true>;  // rows between the saved states
constexpr int kCols = 64;     // channels of a tile, two a lane
constexpr int kWarps = 8;     // of a block
constexpr int kFold = 16;     // tiles whose maps the last of them joins to one
constexpr int kSpan = 512;    // tiles between published states
constexpr int kWalkRows = 64, kWalks = 5;  // see walks_pay
constexpr float kCut = -1.f;
constexpr long long kScanClocks = 4000000000ll;  // about two seconds
constexpr uint64_t kAbsent = ~0ull;

// Of the next launches (sla_test_set_scan_wait; normally 0 and kScanClocks).
std::atomic<int> withheld{0};
std::atomic<int64_t> wait_clocks{kScanClocks};

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
  int bx, bg, bdh, bo;   // bytes from a row to the next in the scan's order; bo: of the results
  void *out0, *out1;     // h; or dx and dg
  const float *state;    // [count][channels] or NULL
  const float *dfinal;   // the same, backward
  float *end;            // [count][channels] or NULL: states behind the sequences; or dstate
  float *saved;          // [rows / kSaved][channels]: states before those rows
  int tiles;             // of a group
  uint32_t *counter;     // tiles taken so far, less one
  // [tiles][groups][kCols], and of every kFold-th and every kSpan-th tile
  uint64_t *maps, *folds, *states;
  uint32_t *timeouts;
  long long clocks;      // of a wait
  int withheld;          // tiles before this one publish no map: 0
};

// The sequence of a row (in memory order): -1 outside of all.
struct Place {
  int seq;
  int64_t begin, end;
};

__device__ __forceinline__ int64_t offset_at(const Sequences &q, int64_t s) {
  return q.wide ? ((const int64_t *)q.offsets)[s] : ((const int32_t *)q.offsets)[s];
}

// The sequence of every lane's row; all lanes take part.  With offsets: the last s with
// offsets[s] <= the smallest row, by 33 parts at a time, and from there on through the next 31 offsets, and by halves where
// they do not reach (many sequences without rows).
__device__ __forceinline__ Place place_of(const Sequences &q, int64_t row, int lane) {
  Place p{-1, 0, 0};
  const bool there = row >= 0 && row < q.rows;
  if (q.length) {
    if (!there) return p;
    p.seq = (uint32_t)row / (uint32_t)q.length;
    p.begin = p.seq * q.length;
    p.end = p.begin + q.length;
    return p;
  }
  int64_t least = there ? row : q.rows;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) least = min(least, (int64_t)__shfl_xor_sync(0xffffffffu, least, o));
  int64_t lo = 0, hi = q.count;  // how many s in [0, count) have offsets[s] <= least: in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 32) / 33, at = lo + (lane + 1) * step - 1;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && offset_at(q, at) <= least));
    hi = min(hi, lo + (n + 1) * step - 1);
    lo = lo + n * step;
  }
  // offsets[lo - 1] is the last; lane k has offsets[lo + k]
  const int64_t next = lo + lane <= q.count ? offset_at(q, lo + lane) : INT64_MAX;
  int n = 0;
  for (int k = 0; k < 32; ++k) {
    const int64_t v = __shfl_sync(0xffffffffu, next, k);
    if (__all_sync(0xffffffffu, v > row || !there)) break;
    n += v <= row && lo + k < q.count;
  }
  int64_t s = lo + n;
  if (n == 32) {
    int64_t top = q.count;
    while (s < top) {
      const int64_t mid = (s + top) >> 1;
      if (offset_at(q, mid) <= row)
        s = mid + 1;
      else
        top = mid;
    }
  }
  if (s == 0 || !there) return p;
  // (offsets that are none may lie outside of the rows, or fall: no row is then taken to be in two places)
  p.begin = max(offset_at(q, s - 1), (int64_t)0), p.end = min(offset_at(q, s), q.rows);
  if (row >= p.begin && row < p.end) p.seq = (int)(s - 1);
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

template <int N>
__device__ __forceinline__ RowInfo rows_info(const Sequences &q, int64_t i0, int lane) {
  RowInfo f;
  const int64_t i = i0 + lane, row = row_of(q, i);
  const Place p = place_of(q, lane < N && i < q.rows ? row : -1, lane);
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
  int c;          // the first channel; a lane without one reads the row's first
  int more;       // to the second, or to the first again
  bool on0, on1;  // whether there are such channels
  __device__ __forceinline__ Lane(int group, int lane, int channels) {
    c = group * kCols + (Pair ? 2 * lane : lane);
    on0 = c < channels, on1 = c + apart < channels;
    if (!on0) c = 0;
    more = on1 ? apart : 0;
  }
  static __device__ __forceinline__ Raw none() {
    if constexpr (sizeof(T) == 4)
      return f2(0.f, 0.f);
    else
      return 0u;
  }
  // p: the first channel's place
  __device__ __forceinline__ Raw load(const T *p) const {
    if constexpr (Pair) {
      return *reinterpret_cast<const Raw *>(p);
    } else {
      const T a = p[0], b = p[more];
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

// A gate is held as the smaller of its two factors, m = e^-|g| / (1 + e^-|g|), which is right relative to itself, with a sign that
// says which it is: c = -m where the gate is open (m = 1 - a), c = m where it is closed (m = a).
// An open gate's value, or a closed one's: by masks, so that no row takes a branch (a select may become one).
__device__ __forceinline__ float choose(float c, float open, float closed) {
  const int m = __float_as_int(c) >> 31;
  return __int_as_float((__float_as_int(open) & m) | (__float_as_int(closed) & ~m));
}
__device__ __forceinline__ float2 choose(float2 c, float2 open, float2 closed) {
  return f2(choose(c.x, open.x, closed.x), choose(c.y, open.y, closed.y));
}

// v's magnitude with the sign bit of `of`.  (A zero's sign is set by its bits, and not left to sums and products.)
__device__ __forceinline__ float with_sign(float v, int of) {
  return __int_as_float((__float_as_int(v) & INT32_MAX) | (of & INT32_MIN));
}

// e^-t for t >= 0.
template <typename T>
__device__ __forceinline__ float2 exp_of_minus(float2 t) {
  if constexpr (sizeof(T) == 2) {
    // the exponent's rounding is off by 2^-24 of t, beside the rounding of 16-bit data
    return f2(ex2_approx(t.x * -1.4426950408889634f), ex2_approx(t.y * -1.4426950408889634f));
  } else {
    // what the product and log2(e) lose to rounding follows as a factor 1 + rest (beyond 128 the exponential is zero)
    t = f2(min_nan(t.x, 128.f), min_nan(t.y, 128.f));
    constexpr float L = 1.4426950408889634f, L2 = (float)(1.4426950408889634074 - (double)L), ln2 = 0.6931471805599453f;
    const float2 n = mul2(t, f2(-L, -L));
    const float2 rest = fma2(t, f2(-L2 * ln2, -L2 * ln2), mul2(fma2(t, f2(-L, -L), f2(-n.x, -n.y)), f2(ln2, ln2)));
    const float2 e = f2(ex2_approx(n.x), ex2_approx(n.y));
    return mul2(e, add2(rest, f2(1.f, 1.f)));
  }
}

template <typename T>
__device__ __forceinline__ float2 gate_of(float2 g) {
  const float2 e = exp_of_minus<T>(f2(fabsf(g.x), fabsf(g.y))), d = add2(e, f2(1.f, 1.f));
  const float2 m = mul2(e, f2(rcp_approx(d.x), rcp_approx(d.y)));
  auto sign = [](float v, float of) { return __int_as_float(__float_as_int(v) | (~__float_as_int(of) & INT32_MIN)); };
  return f2(sign(m.x, g.x), sign(m.y, g.y));
}

// (1 - a) v, and a (1 - a).
__device__ __forceinline__ float2 drop(float2 v, float2 c) {
  return fma2(f2(-c.x, -c.y), v, choose(c, f2(0.f, 0.f), v));
}
__device__ __forceinline__ float2 keep_drop(float2 c) {
  return f2(fmaf(-c.x, c.x, fabsf(c.x)), fmaf(-c.y, c.y, fabsf(c.y)));
}

// a v: v - m v where the gate is open, so that a is not rounded.
__device__ __forceinline__ float2 keep(float2 v, float2 c) {
  return fma2(c, v, choose(c, v, f2(0.f, 0.f)));
}

// d + a v: the gradient of a row's h from that of the next one's.  (An open gate's v + d first, then less m v: two steps in a
// chain of rows, where keep makes three.)
__device__ __forceinline__ float2 back(float2 d, float2 v, float2 c) {
  return fma2(c, v, fma2(choose(c, f2(1.f, 1.f), f2(0.f, 0.f)), v, d));
}

// One step of h, a h + (1 - a) x: h + m (x - h) where the gate is open, x + m (h - x) where it is closed (c h and c x apart: the
// difference of h and x may pass the largest float32).
__device__ __forceinline__ float2 step(float2 h, float2 x, float2 c) {
  const float2 t = mul2(c, x), u = fma2(c, h, f2(-t.x, -t.y));
  return add2(choose(c, h, x), u);
}

// s -> A s + h of two channels.  A is held as a gate's factors are: a = A, or, next to one, a = A - 1 (with the sign bit, -0 is one),
// so that what a state loses over many open rows is right relative to itself.  a = kCut: s -> h.
struct Map {
  float2 a, h;
};

__device__ __forceinline__ float2 apply(const Map &m, float2 s) {
  const float2 r = add2(choose(m.a, s, f2(0.f, 0.f)), fma2(m.a, s, m.h));
  return m.a.x == kCut ? m.h : r;
}
__device__ __forceinline__ void join(Map &m, const Map &n) {  // m first
  m.h = apply(n, m.h);
  const bool cut = m.a.x == kCut || n.a.x == kCut;
  const float2 A = add2(choose(m.a, f2(1.f, 1.f), f2(0.f, 0.f)), m.a), v = fma2(n.a, A, choose(n.a, m.a, f2(0.f, 0.f)));
  // (two factors next to one make one that is not positive, whatever the sign of a zero)
  auto factor = [](float v, float a, float b) {
    return v < -0.5f ? 1.f + v : with_sign(v, __float_as_int(a) & __float_as_int(b));
  };
  m.a = cut ? f2(kCut, kCut) : f2(factor(v.x, m.a.x, n.a.x), factor(v.y, m.a.y, n.a.y));
}

// The factor of a map over rows, taken row after row, as A and as A - 1.
struct Factor {
  float2 all = f2(1.f, 1.f), less = f2(-0.f, -0.f);
  __device__ __forceinline__ void row(float2 c) {
    all = keep(all, c);
    less = fma2(c, add2(less, f2(1.f, 1.f)), choose(c, less, f2(-1.f, -1.f)));
  }
  __device__ __forceinline__ float2 a() const {
    auto one = [](float less, float all) { return less >= -0.5f ? __int_as_float(__float_as_int(less) | INT32_MIN) : all; };
    return f2(one(less.x, all.x), one(less.y, all.y));
  }
};

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
__device__ __forceinline__ bool wait_for(const uint64_t *p, Map &m, bool there, long long clocks) {
  if (__all_sync(0xffffffffu, there)) return true;
  const long long t0 = clock64();
  for (;;) {
    __nanosleep(100);  // many wait for the same words
    if (__all_sync(0xffffffffu, look(p, m))) return true;
    if (__any_sync(0xffffffffu, clock64() - t0 > clocks)) return false;
  }
}

__device__ __forceinline__ void copy_async(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Asks for the rows of `from` ([count][channels] float32) that belong to the sequences of the marked rows: to the lane's
// two places of row r of `to` ([..][32] pairs), which the lane itself reads.
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

struct TileMemory {
  Map maps[kWarps][32];   // of the block's warps
  Map carry[kWarps][32];  // parts of the way from the known state to the tile: folds, then tiles
  int64_t origin;         // the scan's index of the first row that the tile's first row depends on
  uint32_t next;
  volatile uint32_t dead; // a wait of this block has expired: it waits no more, so that the launch ends
};

__device__ __forceinline__ Map no_rows() { return {f2(-0.f, -0.f), f2(0.f, 0.f)}; }

__device__ __forceinline__ Map joined(const Map (*maps)[32], int from, int to, int lane) {
  Map m = no_rows();
#pragma unroll 4
  for (int w = from; w < to; ++w) join(m, maps[w][lane]);
  return m;
}

// This warp's part of the way from the start of the tile's sequence, in tile `first`, or the state before its span, to the tile.
__device__ __forceinline__ Map look_back(const ScanArgs &p, TileMemory &sm, int tile, int first, int64_t mine, int64_t apart,
                                         int warp, int lane) {
  Map m = no_rows();
  if (__any_sync(0xffffffffu, sm.dead)) return m;
  const int base = tile / kSpan * kSpan, fold = tile / kFold * kFold;
  // half of the warps take the folds before the present one, half the tiles of the present one
  constexpr int H = kWarps / 2;
  const bool tiles = warp >= H;
  const int lo = tiles ? max(first, fold) : max(first, base) / kFold, hi = tiles ? tile : fold / kFold;
  const int per = (max(hi - lo, 0) + H - 1) / H, from = lo + (tiles ? warp - H : warp) * per, to = min(hi, from + per);
  const uint64_t *at = (tiles ? p.maps : p.folds) + from * apart + mine;
  bool ok = true;
  if (warp == 0 && first < base) {
    const uint64_t *q = p.states + (int64_t)(base / kSpan - 1) * apart + mine;
    ok = wait_for(q, m, look(q, m), p.clocks);
  }
  for (int i = from; i < to && ok; i += 2, at += 2 * apart) {
    Map n, n2;
    const bool two = i + 1 < to;
    const bool there = look(at, n), there2 = !two || look(at + apart, n2);
    ok = wait_for(at, n, there, p.clocks);
    join(m, n);
    if (two && ok) {
      ok = wait_for(at + apart, n2, there2, p.clocks);
      join(m, n2);
    }
  }
  if (!ok && lane == 0) {
    sm.dead = 1;
    atomicAdd_system(p.timeouts, 1u);
  }
  return m;
}

// Where a warp's rows of a tile lie.  Backward, tile 0 holds the last rows and warp 0 the last of a tile.
template <typename T, bool Pair, bool Backward>
struct Rows {
  static constexpr int n = kRows<T, Backward>, tile_rows = kWarps * n;
  Lane<T, Pair> l;
  int tile, group, left;  // rows that there are
  int64_t t0, i0, row0;   // the tile's first row in the order of the tiles; the scan's index of the warp's first row, and its row
  __device__ __forceinline__ Rows(const ScanArgs &p, uint32_t id, int warp, int lane)
      : l(id % (uint32_t)p.groups, lane, p.channels), tile(id / (uint32_t)p.groups), group(id % (uint32_t)p.groups) {
    t0 = (int64_t)tile * tile_rows;
    i0 = Backward ? ((int64_t)(p.tiles - 1 - tile) * kWarps + (kWarps - 1 - warp)) * n : t0 + warp * n;
    left = (int)max(min((int64_t)n, p.q.rows - i0), (int64_t)0);
    row0 = row_of(p.q, i0);
  }
  // The first channel of the first row.
  __device__ __forceinline__ char *at(const void *base, int64_t ld) const {
    return (char *)const_cast<void *>(base) + (row0 * ld + l.c) * (int64_t)sizeof(T);
  }
  // Loads the rows, `step` bytes apart (one wide multiply-add an address).
  __device__ __forceinline__ void ask(const void *base, int64_t ld, int step, typename Lane<T, Pair>::Raw (&raw)[n]) const {
    const char *p = at(base, ld);
    if (left == n) {
#pragma unroll
      for (int r = 0; r < n; ++r) raw[r] = l.load((const T *)(p + (int64_t)step * r));
    } else {
#pragma unroll
      for (int r = 0; r < n; ++r) {
        raw[r] = Lane<T, Pair>::none();
        if (r < left) raw[r] = l.load((const T *)(p + (int64_t)step * r));
      }
    }
  }
};

// The state before this warp's rows.  All maps are in place (and a barrier behind them).  On the way the tile's map is
// published, the state before the tile found, and what others look for published.
template <bool Chain, typename R>
__device__ __forceinline__ float2 state_before(const ScanArgs &p, TileMemory &sm, const R &t, int warp, int lane) {
  float2 s = f2(0.f, 0.f);
  if constexpr (!Chain) return apply(joined(sm.maps, 0, warp, lane), s);
  const int64_t apart = (int64_t)p.groups * kCols, mine = t.group * kCols + 2 * lane, origin = sm.origin;
  const bool needed = origin < t.t0;
  const Map before = joined(sm.maps, 0, warp, lane);
  Map own;
  if (warp == kWarps - 1) {
    own = before;
    join(own, sm.maps[warp][lane]);
    if (t.tile >= p.withheld) publish(p.maps + t.tile * apart + mine, own);
  }
  sm.carry[warp][lane] = needed ? look_back(p, sm, t.tile, (int)(origin / R::tile_rows), mine, apart, warp, lane) : no_rows();
  if ((t.tile + 1) % kFold == 0 && warp >= kWarps / 2) {
    // as soon as the tiles' half is through, not waiting for the states that the others may wait for
    asm volatile("bar.sync 1, %0;" ::"n"(32 * (kWarps - kWarps / 2)) : "memory");
    if (warp == kWarps - 1) {
      Map f = joined(sm.carry, kWarps / 2, kWarps, lane);
      join(f, own);
      publish(p.folds + (int64_t)(t.tile / kFold) * apart + mine, f);
    }
  }
  __syncthreads();
  if (needed)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = apply(sm.carry[w][lane], s);
  if (warp == kWarps - 1 && (t.tile + 1) % kSpan == 0)
    publish(p.states + (int64_t)(t.tile / kSpan) * apart + mine, Map{f2(kCut, kCut), apply(own, s)});
  return apply(before, s);
}

template <typename T, bool Chain, bool Pair>
__device__ __forceinline__ void tile_forward(const ScanArgs &p, TileMemory &sm, uint32_t id, float2 *starts, int warp, int lane) {
  using L = Lane<T, Pair>;
  constexpr int N = kRows<T, false>;
  const Rows<T, Pair, false> t(p, id, warp, lane);
  typename L::Raw xr[N], gr[N];
  t.ask(p.g, p.ldg, p.bg, gr);
  t.ask(p.x, p.ldx, p.bx, xr);
  const RowInfo f = rows_info<N>(p.q, t.i0, lane);
  const bool inner = f.live == (1u << N) - 1 && !f.first && !f.last;  // no row is the first or last of a sequence, or in none
  if (Chain && threadIdx.x == 0) sm.origin = f.live & 1 ? f.origin : t.t0;
  if (p.state && f.first) ask_states(starts, p.state, f.first, f.seq, p.channels, t.l, lane);
  auto start = [&](int r) { return p.state ? starts[r * 32 + lane] : f2(0.f, 0.f); };
  float2 c[N];
#pragma unroll
  for (int r = 0; r < N; ++r) c[r] = gate_of<T>(L::values(gr[r]));
  Map m = no_rows();
  Factor factor;
  if (inner) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      m.h = step(m.h, L::values(xr[r]), c[r]);
      factor.row(c[r]);
    }
    m.a = factor.a();
  } else {
    copies_done();
#pragma unroll
    for (int r = 0; r < N; ++r) {
      if (f.first >> r & 1) m.h = start(r);
      m.h = step(m.h, L::values(xr[r]), c[r]);
      factor.row(c[r]);
    }
    m.a = f.first ? f2(kCut, kCut) : factor.a();
  }
  sm.maps[warp][lane] = m;
  __syncthreads();
  float2 h = state_before<Chain>(p, sm, t, warp, lane);
  // (taken no sooner, see above)
  if (Chain && threadIdx.x == 0) sm.next = atomicAdd(p.counter, 1u) + 1u;
  char *to = t.at(p.out0, p.channels);
  auto save = [&](int r) {
    if (r % kSaved<T> == 0 && p.saved && r < t.left) t.l.put_state(p.saved, (t.i0 + r) / kSaved<T>, p.channels, h);
  };
  if (inner) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      save(r);
      h = step(h, L::values(xr[r]), c[r]);
      t.l.store((T *)(to + (int64_t)p.bo * r), h);
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < N; ++r) {
    save(r);
    if (f.first >> r & 1) h = start(r);
    h = step(h, L::values(xr[r]), c[r]);
    const bool live = f.live >> r & 1;
    if (live || (p.outside && r < t.left)) t.l.store((T *)(to + (int64_t)p.bo * r), live ? h : f2(0.f, 0.f));
    if (p.end && (f.last >> r & 1)) t.l.put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, h);
  }
}

template <typename T, bool Chain, bool Pair>
__device__ __forceinline__ void tile_backward(const ScanArgs &p, TileMemory &sm, uint32_t id, float2 *starts, int warp, int lane) {
  using L = Lane<T, Pair>;
  constexpr int N = kRows<T, true>;
  const Rows<T, Pair, true> t(p, id, warp, lane);
  float2 *ends = starts + N * 32;
  typename L::Raw xr[N], gr[N], dr[N];
  t.ask(p.g, p.ldg, p.bg, gr);
  t.ask(p.x, p.ldx, p.bx, xr);
  if (p.dh) {
    t.ask(p.dh, p.lddh, p.bdh, dr);
  } else {
#pragma unroll
    for (int r = 0; r < N; ++r) dr[r] = L::none();
  }
  float2 h = t.left > 0 ? t.l.state(p.saved, t.i0 / N, p.channels) : f2(0.f, 0.f);
  const RowInfo f = rows_info<N>(p.q, t.i0, lane);
  const bool inner = f.live == (1u << N) - 1 && !f.first && !f.last;
  if (p.state && f.first) ask_states(starts, p.state, f.first, f.seq, p.channels, t.l, lane);
  if (p.dfinal && f.last) ask_states(ends, p.dfinal, f.last, f.seq, p.channels, t.l, lane);
  if (Chain) {
    // the row behind which the present sequence ends, counted backwards from the end of the last tile
    const int64_t span = (int64_t)p.tiles * t.tile_rows, until = __shfl_sync(0xffffffffu, f.until, N - 1);
    if (threadIdx.x == 0) sm.origin = f.live >> (N - 1) & 1 ? span - until : t.t0;
  }
  auto start = [&](int r) { return p.state ? starts[r * 32 + lane] : f2(0.f, 0.f); };
  auto end = [&](int r) { return p.dfinal ? ends[r * 32 + lane] : f2(0.f, 0.f); };
  float2 c[N], e[N];  // e: h_{t-1} - x_t
#pragma unroll
  for (int r = 0; r < N; ++r) c[r] = gate_of<T>(L::values(gr[r]));
  Map m = no_rows();
  Factor factor;
  auto form = [&](int r) {
    const float2 x = L::values(xr[r]);
    e[r] = f2(h.x - x.x, h.y - x.y);
    h = step(h, x, c[r]);
  };
  auto pass = [&](int r) {
    m.h = keep(add2(L::values(dr[r]), m.h), c[r]);
    factor.row(c[r]);
  };
  if (inner) {
#pragma unroll
    for (int r = 0; r < N; ++r) form(r);
#pragma unroll
    for (int r = N - 1; r >= 0; --r) {
      const float2 d = L::values(dr[r]);
      m.h = r == N - 1 ? d : back(d, m.h, c[r + 1 < N ? r + 1 : r]);
      factor.row(c[r]);
    }
    m.h = keep(m.h, c[0]);
    m.a = factor.a();
  } else {
    copies_done();
#pragma unroll
    for (int r = 0; r < N; ++r) {
      if (f.first >> r & 1) h = start(r);
      form(r);
    }
#pragma unroll
    for (int r = N - 1; r >= 0; --r) {
      if (f.last >> r & 1) m.h = end(r);
      pass(r);
    }
    m.a = f.last ? f2(kCut, kCut) : factor.a();
  }
  sm.maps[warp][lane] = m;
  __syncthreads();
  float2 carry = state_before<Chain>(p, sm, t, warp, lane);
  if (Chain && threadIdx.x == 0) sm.next = atomicAdd(p.counter, 1u) + 1u;
  char *tx = t.at(p.out0, p.channels), *tg = t.at(p.out1, p.channels);
  auto results = [&](int r, float2 lam, bool live) {
    const float2 none = f2(0.f, 0.f);
    if (p.out0) t.l.store((T *)(tx + (int64_t)p.bo * r), live ? drop(lam, c[r]) : none);
    if (p.out1) t.l.store((T *)(tg + (int64_t)p.bo * r), live ? mul2(mul2(lam, e[r]), keep_drop(c[r])) : none);
  };
  if (inner) {
#pragma unroll
    for (int r = N - 1; r >= 0; --r) {
      const float2 d = L::values(dr[r]);
      carry = r == N - 1 ? add2(d, carry) : back(d, carry, c[r + 1 < N ? r + 1 : r]);  // the row's l
      results(r, carry, true);
    }
    return;
  }
#pragma unroll
  for (int r = N - 1; r >= 0; --r) {
    if (f.last >> r & 1) carry = end(r);
    const float2 lam = add2(L::values(dr[r]), carry);
    carry = keep(lam, c[r]);
    if (r < t.left) results(r, lam, f.live >> r & 1);
    if (p.end && (f.first >> r & 1)) t.l.put_state(p.end, __shfl_sync(0xffffffffu, f.seq, r), p.channels, carry);
  }
}

// Blocks of a multiprocessor: as many as the registers of a tile's rows admit.
template <typename T, bool Backward>
inline constexpr int kResident = !Backward && sizeof(T) == 2 ? 3 : 2;

template <typename T, bool Chain, bool Pair, bool Backward>
__global__ void __launch_bounds__(32 * kWarps, kResident<T, Backward>) scan_kernel(const __grid_constant__ ScanArgs p) {
  // [kWarps][kRows][32], backward twice: states of the sequences that start (and end) in the tile
  extern __shared__ float2 dynamic[];
  __shared__ TileMemory sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 *starts = dynamic + warp * (Backward ? 2 : 1) * kRows<T, Backward> * 32;
  const uint32_t all = (uint32_t)p.tiles * (uint32_t)p.groups;
  uint32_t id = blockIdx.x;
  if (Chain) {
    if (threadIdx.x == 0) {
      sm.dead = 0;
      sm.next = atomicAdd(p.counter, 1u) + 1u;
    }
    __syncthreads();
    id = sm.next;
  }
  while (id < all) {
    if constexpr (Backward)
      tile_backward<T, Chain, Pair>(p, sm, id, starts, warp, lane);
    else
      tile_forward<T, Chain, Pair>(p, sm, id, starts, warp, lane);
    __syncthreads();  // everything in shared memory has been read
    id = Chain ? sm.next : id + gridDim.x;
  }
}

// ------------------------------------------------------------------ many sequences of one length: a warp walks along each

// With a sequence and kCols channels for every warp that there is room for, nothing has to be joined: a warp walks from row to
// row with the state in its registers, one pass, and what counts is that enough rows are on their way: kAhead forward,
// a chunk of kSaved rows backward while the one behind it is worked on.  Rows in the middle are worked on without a branch, so
// that their gates are formed side by side (with a test a row: 443 us in place of 81), four rows' at a time: a barrier of the warp
// every four rows keeps the compiler from forming all rows' first, for which it spills (203 us in place of 88).
template <typename T>
inline constexpr int kAhead = sizeof(T) == 2 ? 32 : 16;

template <typename T>
__global__ void __launch_bounds__(32) walk_forward(const __grid_constant__ ScanArgs p) {
  using L = Lane<T, true>;
  constexpr int D = kAhead<T>;
  const int lane = threadIdx.x, seq = blockIdx.x / (uint32_t)p.groups;
  const L l(blockIdx.x % (uint32_t)p.groups, lane, p.channels);
  const int n = (int)p.q.length;
  const int64_t row0 = p.q.reverse ? (seq + 1) * p.q.length - 1 : seq * p.q.length;
  const int64_t i0 = p.q.reverse ? p.q.rows - (seq + 1) * p.q.length : row0;  // the scan's index of the first row
  const char *px = (const char *)((const T *)p.x + row0 * p.ldx + l.c), *pg = (const char *)((const T *)p.g + row0 * p.ldg + l.c);
  char *po = (char *)((T *)p.out0 + row0 * p.channels + l.c);
  typename L::Raw xr[D], gr[D];
#pragma unroll
  for (int r = 0; r < D; ++r) {
    gr[r] = xr[r] = L::none();
    if (r < n) {
      gr[r] = l.load((const T *)(pg + (int64_t)p.bg * r));
      xr[r] = l.load((const T *)(px + (int64_t)p.bx * r));
    }
  }
  float2 h = p.state ? l.state(p.state, seq, p.channels) : f2(0.f, 0.f);
  const int phase = (int)(i0 % kSaved<T>);
  float *saved = p.saved ? p.saved + i0 / kSaved<T> * p.channels + l.c : nullptr;
  auto row = [&](int t, int r) {
    const float2 c = gate_of<T>(L::values(gr[r]));
    if (saved && (phase + t + r) % kSaved<T> == 0) {
      float *to = saved + (int64_t)((phase + t + r) / kSaved<T>) * p.channels;
      if (l.on0) to[0] = h.x;
      if (l.on1) to[L::apart] = h.y;
    }
    h = step(h, L::values(xr[r]), c);
    l.store((T *)(po + (int64_t)p.bo * r), h);
  };
  int t = 0;
  for (; t + 2 * D <= n; t += D) {
    px += (int64_t)p.bx * D, pg += (int64_t)p.bg * D;
#pragma unroll
    for (int r = 0; r < D; ++r) {
      if (r % 4 == 0) __syncwarp();
      row(t, r);
      gr[r] = l.load((const T *)(pg + (int64_t)p.bg * r));
      xr[r] = l.load((const T *)(px + (int64_t)p.bx * r));
    }
    po += (int64_t)p.bo * D;
  }
  for (; t < n; t += D) {
    px += (int64_t)p.bx * D, pg += (int64_t)p.bg * D;
#pragma unroll
    for (int r = 0; r < D; ++r)
      if (t + r < n) {
        row(t, r);
        if (t + r + D < n) {
          gr[r] = l.load((const T *)(pg + (int64_t)p.bg * r));
          xr[r] = l.load((const T *)(px + (int64_t)p.bx * r));
        }
      }
    po += (int64_t)p.bo * D;
  }
  if (p.end) l.put_state(p.end, seq, p.channels, h);
}

template <typename T>
struct WalkRows {
  typename Lane<T, true>::Raw x[kSaved<T>], g[kSaved<T>], d[kSaved<T>];
  float2 h;  // the state before them
};

template <typename T>
__global__ void __launch_bounds__(32) walk_backward(const __grid_constant__ ScanArgs p) {
  using L = Lane<T, true>;
  constexpr int N = kSaved<T>;
  const int lane = threadIdx.x, seq = blockIdx.x / (uint32_t)p.groups;
  const L l(blockIdx.x % (uint32_t)p.groups, lane, p.channels);
  const int64_t n = p.q.length;
  const int64_t row0 = p.q.reverse ? (seq + 1) * n - 1 : seq * n, i0 = p.q.reverse ? p.q.rows - (seq + 1) * n : row0;
  const int dir = p.q.reverse ? -1 : 1;
  // chunk k: the scan's rows from k N on, of which those of the sequence count
  const int64_t first = i0 / N, last = (i0 + n - 1) / N;
  auto at = [&](const void *base, int64_t ld, int64_t k) {
    return (char *)const_cast<void *>(base) + ((row0 + dir * (k * N - i0)) * ld + l.c) * (int64_t)sizeof(T);
  };
  auto ask = [&](WalkRows<T> &w, int64_t k) {
    if (k < first) return;
    const char *px = at(p.x, p.ldx, k), *pg = at(p.g, p.ldg, k), *pd = at(p.dh, p.lddh, k);
    const int lo = (int)max(i0 - k * N, (int64_t)0), hi = (int)min(i0 + n - k * N, (int64_t)N);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      w.g[r] = w.x[r] = w.d[r] = L::none();
      if (r >= lo && r < hi) {
        w.g[r] = l.load((const T *)(pg + (int64_t)p.bg * r));
        w.x[r] = l.load((const T *)(px + (int64_t)p.bx * r));
        if (p.dh) w.d[r] = l.load((const T *)(pd + (int64_t)p.bdh * r));
      }
    }
    if (k * N > i0)
      w.h = l.state(p.saved, k, p.channels);
    else
      w.h = p.state ? l.state(p.state, seq, p.channels) : f2(0.f, 0.f);
  };
  float2 carry = p.dfinal ? l.state(p.dfinal, seq, p.channels) : f2(0.f, 0.f);
  auto work = [&](const WalkRows<T> &w, int64_t k) {
    const int lo = (int)max(i0 - k * N, (int64_t)0), hi = (int)min(i0 + n - k * N, (int64_t)N);
    char *tx = at(p.out0, p.channels, k), *tg = at(p.out1, p.channels, k);
    float2 c[N], e[N], h = w.h;
    auto form = [&](int r) {
      const float2 x = L::values(w.x[r]);
      e[r] = f2(h.x - x.x, h.y - x.y);
      h = step(h, x, c[r]);
    };
    float2 lam;
    auto results = [&](int r, bool first) {
      const float2 d = L::values(w.d[r]);
      lam = first ? add2(d, carry) : back(d, lam, c[r + 1 < N ? r + 1 : r]);
      if (p.out0) l.store((T *)(tx + (int64_t)p.bo * r), drop(lam, c[r]));
      if (p.out1) l.store((T *)(tg + (int64_t)p.bo * r), mul2(mul2(lam, e[r]), keep_drop(c[r])));
    };
#pragma unroll
    for (int r = 0; r < N; ++r) c[r] = gate_of<T>(L::values(w.g[r]));
    if (lo == 0 && hi == N) {
#pragma unroll
      for (int r = 0; r < N; ++r) form(r);
#pragma unroll
      for (int r = N - 1; r >= 0; --r) results(r, r == N - 1);
      carry = keep(lam, c[0]);
      return;
    }
#pragma unroll
    for (int r = 0; r < N; ++r)
      if (r >= lo) form(r);  // (rows behind the last one change what nothing reads)
#pragma unroll
    for (int r = N - 1; r >= 0; --r)
      if (r >= lo && r < hi) {
        results(r, true);
        carry = keep(lam, c[r]);
      }
  };
  WalkRows<T> even, odd;
  ask(even, last);
  for (int64_t k = last; k >= first; k -= 2) {
    ask(odd, k - 1);
    work(even, k);
    if (k - 1 < first) break;
    ask(even, k - 2);
    work(odd, k - 1);
  }
  if (p.end) l.put_state(p.end, seq, p.channels, carry);
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
    h = step(h, x, gate_of<T>(g));
    l.store((T *)p.out0 + row * p.channels + l.c, h);
    if (p.end) l.put_state(p.end, row, p.channels, h);
  }
}

// ------------------------------------------------------------------ the calls

int tile_rows(const sla_scan *s, bool backward) {
  return kWarps * (s->dtype != SLA_F32 ? kRows<f16, true> : backward ? kRows<float, true> : kRows<float, false>);
}

int64_t tiles_of(const sla_scan *s, bool backward) {
  const int n = tile_rows(s, backward);
  return (s->rows + n - 1) / n;
}

// Whether no sequence leaves a tile: whole sequences in every one, or a single tile.
bool closed_tiles(const sla_scan *s, bool backward) {
  const int n = tile_rows(s, backward);
  if (s->rows <= n) return true;
  if (s->offsets || s->sequences < 1) return false;
  return n % (s->rows / s->sequences) == 0;
}

// Whether a warp for each sequence and kCols channels pays, where channels go in pairs: sequences long enough for rows on their
// way, and enough of them to keep the memory busy.  A training step in bfloat16, walks against tiles: 1000 sequences of 1000 x 64
// 292 us and 373 (float32 353 and 495), 16,000 of 64 x 64 253 and 365, 300 of 1000 x 130 288 and 335, 760 of 1000 x 64 280 and 290;
// but 500 of 1000 x 64 234 and 198, 16 of 2048 x 2048 467 and 368.  (Single channels 32 apart were three times the tiles' time.)
bool walks_pay(const sla_scan *s, bool pairs) {
  if (!pairs || s->offsets || s->sequences < 1 || s->rows / s->sequences < kWalkRows) return false;
  const int64_t strands = s->sequences * ((s->channels + kCols - 1) / kCols);
  return strands >= (int64_t)kWalks * sm_count() && strands < ((int64_t)1 << 31);
}

size_t chain_bytes(const sla_scan *s, bool backward) {
  if (closed_tiles(s, backward)) return 0;
  const size_t groups = (size_t)((s->channels + kCols - 1) / kCols), tiles = (size_t)tiles_of(s, backward);
  return align256(256 + (tiles + tiles / kFold + tiles / kSpan) * groups * kCols * sizeof(uint64_t));
}

size_t saved_bytes(const sla_scan *s) {
  const int64_t apart = s->dtype == SLA_F32 ? kSaved<float> : kSaved<f16>;
  return align256((size_t)((s->rows + apart - 1) / apart) * (size_t)s->channels * sizeof(float));
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
  return tiles_of(s, true) * groups < most ? SLA_OK : SLA_INVALID_ARG;
}

sla_status check_rows(const void *p, const sla_scan *s, int64_t ld) {
  if (s->rows == 0) return SLA_OK;
  if (!p || !aligned(p, net_size(s->dtype))) return SLA_INVALID_ARG;
  // (the kernels count a row's bytes in 32 bits)
  return s->rows == 1 || (ld >= s->channels && ld < (int64_t)1 << 28) ? SLA_OK : SLA_INVALID_ARG;
}

sla_status check_buffer(const void *p, size_t bytes, size_t need) {
  if (need == 0) return SLA_OK;
  if (!p || !aligned(p, 256)) return SLA_INVALID_ARG;
  return bytes < need ? SLA_WORKSPACE_TOO_SMALL : SLA_OK;
}

// Bytes from a row to the next in the scan's order.
int row_bytes(const sla_scan *s, int64_t ld) {
  return (int)((s->reverse ? -ld : ld) * (int64_t)net_size(s->dtype));
}

ScanArgs scan_args(const sla_scan *s, bool backward, void *ws) {
  ScanArgs p{};
  p.q = {s->rows, s->sequences, s->offsets || !s->sequences ? 0 : s->rows / s->sequences, s->offsets,
         s->offsets_type == SLA_I64, s->reverse};
  p.channels = (int)s->channels, p.groups = (int)((s->channels + kCols - 1) / kCols);
  p.outside = s->outside;
  p.tiles = (int)tiles_of(s, backward);
  p.bo = row_bytes(s, s->channels);
  p.counter = (uint32_t *)ws;
  p.maps = (uint64_t *)((char *)ws + 256);
  p.folds = p.maps + (int64_t)p.tiles * p.groups * kCols;
  p.states = p.folds + (int64_t)(p.tiles / kFold) * p.groups * kCols;
  p.clocks = wait_clocks.load(), p.withheld = withheld.load();
  return p;
}

// Whether every row's pairs of channels may be moved at once.
bool pairs_aligned(const sla_scan *s, const void *p, int64_t ld) {
  return aligned(p, 2 * net_size(s->dtype)) && (s->rows == 1 || ld % 2 == 0);
}

template <typename T, bool Backward, typename K>
cudaError_t launch(K kernel, const ScanArgs &p, size_t smem, cudaStream_t st) {
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = (int64_t)p.tiles * p.groups;
  kernel<<<(unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * kResident<T, Backward>), 32 * kWarps, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T, bool Pair>
cudaError_t run_forward(const ScanArgs &p, bool walk, bool chain, cudaStream_t st) {
  if (Pair && walk) {
    walk_forward<T><<<(unsigned)(p.q.count * p.groups), 32, 0, st>>>(p);
    return cudaGetLastError();
  }
  if (p.q.length == 1 && !p.saved) {
    const int64_t threads = p.q.rows * p.groups * 32;
    scan_single<T, Pair><<<(unsigned)std::min<int64_t>((threads + 255) / 256, sm_count() * 8), 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  const size_t smem = p.state ? kWarps * kRows<T, false> * kCols * sizeof(float) : 0;
  return chain ? launch<T, false>(scan_kernel<T, true, Pair, false>, p, smem, st)
               : launch<T, false>(scan_kernel<T, false, Pair, false>, p, smem, st);
}

template <typename T, bool Pair>
cudaError_t run_backward(const ScanArgs &p, bool walk, bool chain, cudaStream_t st) {
  if (Pair && walk) {
    walk_backward<T><<<(unsigned)(p.q.count * p.groups), 32, 0, st>>>(p);
    return cudaGetLastError();
  }
  const size_t smem = p.state || p.dfinal ? kWarps * 2 * kRows<T, true> * kCols * sizeof(float) : 0;
  return chain ? launch<T, true>(scan_kernel<T, true, Pair, true>, p, smem, st)
               : launch<T, true>(scan_kernel<T, false, Pair, true>, p, smem, st);
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
  return check_scan(s) == SLA_OK ? std::max(chain_bytes(s, false), chain_bytes(s, true)) : 0;
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
  const size_t need = chain_bytes(s, false);
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
  ScanArgs p = scan_args(s, false, workspace);
  p.x = x, p.ldx = ldx, p.g = gate, p.ldg = ldg, p.state = state, p.out0 = h, p.end = final_state;
  p.bx = row_bytes(s, ldx), p.bg = row_bytes(s, ldg);
  p.saved = (float *)saved, p.timeouts = earlier.count;
  const bool pairs = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
                     pairs_aligned(s, h, s->channels);
  const bool walk = walks_pay(s, pairs), chain = !walk && need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  e = by_type(s->dtype, pairs, [&](auto t, auto pair) { return run_forward<decltype(t), decltype(pair)::value>(p, walk, chain, st); });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

SLA_API sla_status sla_test_set_scan_wait(int32_t withhold, int64_t clocks) {
  if (withhold < 0 || withhold > 1 || clocks < 0 || clocks > kScanClocks) return SLA_INVALID_ARG;
  withheld.store(withhold);
  wait_clocks.store(clocks ? clocks : kScanClocks);
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
  const size_t need = chain_bytes(s, true);
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
  ScanArgs p = scan_args(s, true, workspace);
  p.dh = dh, p.lddh = lddh, p.x = x, p.ldx = ldx, p.g = gate, p.ldg = ldg, p.state = state, p.dfinal = dfinal;
  p.bx = row_bytes(s, ldx), p.bg = row_bytes(s, ldg), p.bdh = row_bytes(s, lddh);
  p.out0 = dx, p.out1 = dgate, p.end = dstate, p.saved = (float *)const_cast<void *>(saved);
  p.timeouts = earlier.count;
  const bool pairs = s->channels % 2 == 0 && pairs_aligned(s, x, ldx) && pairs_aligned(s, gate, ldg) &&
                     (!dh || pairs_aligned(s, dh, lddh)) && pairs_aligned(s, dx, s->channels) &&
                     pairs_aligned(s, dgate, s->channels);
  const bool walk = walks_pay(s, pairs), chain = !walk && need > 0;
  cudaError_t e = chain ? cudaMemsetAsync(workspace, 0xff, need, st) : cudaSuccess;
  if (e != cudaSuccess) return fail(e);
  e = by_type(s->dtype, pairs, [&](auto t, auto pair) { return run_backward<decltype(t), decltype(pair)::value>(p, walk, chain, st); });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

}  // extern "C"
