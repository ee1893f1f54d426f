// The gated feed-forward block, forward and backward.
//
//   [g u] = x w_in^T + b_in,  h = act(g) u,  y = h w_out^T + b_out
//   dh = dy w_out,  dg = dh u act'(g),  du = dh act(g)
//   dx = [dg du] w_in,  dw_in = [dg du]^T x,  dw_out = dy^T h,  db_in = sum [dg du],  db_out = sum dy
//
// Six tensor-core products (sla_product.cuh); the activation, the product with u and their
// derivatives are the epilogues of the two that make g, u and dh.  This file lays out the operands,
// picks each product's tile shape and split, and adds what is split.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "sla_common.cuh"
#include "sla_few.cuh"
#include "sla_host.h"
#include "sla_narrow.cuh"
#include "sla_net.cuh"
#include "sla_product.cuh"

namespace sla {
namespace {

// ------------------------------------------------------------------ expired waits

constexpr int kDevices = 64;

// A device's count of blocks of products that gave up a wait, since the process started.  It lies in host memory that the
// kernels add to, so that a call sees without waiting for the GPU whether an earlier one was cut short.  It only
// grows: what a thread has been told of is its own number, so that no thread takes another's report.
struct Expired {
  uint32_t *count = nullptr;
  int dev = 0;
  cudaError_t err = cudaSuccess;
};

std::mutex expired_mutex;
std::atomic<uint32_t *> expired_count[kDevices];
thread_local bool expired_met[kDevices];  // this thread has been here
thread_local uint32_t expired_told[kDevices];

uint32_t read_count(const Expired &x) { return *(const volatile uint32_t *)x.count; }

// The current device's.  A thread is told of what expires after its first time here.
Expired expired() {
  Expired x;
  x.err = cudaGetDevice(&x.dev);
  if (x.err == cudaSuccess && x.dev >= kDevices) x.err = cudaErrorInvalidDevice;
  if (x.err != cudaSuccess) return x;
  x.count = expired_count[x.dev].load();
  if (!x.count) {
    std::lock_guard<std::mutex> lock(expired_mutex);
    x.count = expired_count[x.dev].load();
    if (!x.count) {
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // another thread's capture has nothing to do with this
      cudaThreadExchangeStreamCaptureMode(&mode);
      x.err = cudaHostAlloc((void **)&x.count, sizeof(uint32_t), cudaHostAllocPortable | cudaHostAllocMapped);
      cudaThreadExchangeStreamCaptureMode(&mode);
      if (x.err != cudaSuccess) return x;
      *x.count = 0;
      expired_count[x.dev].store(x.count);
    }
  }
  if (!expired_met[x.dev]) {
    expired_met[x.dev] = true;
    expired_told[x.dev] = read_count(x);
  }
  return x;
}

// SLA_TIMEOUT if waits have expired that this thread has not been told of.
sla_status report_expired(const Expired &x) {
  const uint32_t n = read_count(x);
  if (n == expired_told[x.dev]) return SLA_OK;
  expired_told[x.dev] = n;
  return SLA_TIMEOUT;
}

// A wait that nothing ends, of a quarter of a millisecond, counted as the products' kernels count theirs.
__global__ void __launch_bounds__(32) expire_wait(uint32_t *timeouts) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) mbar_init(&bar, 1);
  __syncwarp();
  if (!mbar_wait_clocks(&bar, 0, 500000) && threadIdx.x == 0) atomicAdd_system(timeouts, 1u);
}

// ------------------------------------------------------------------ operands

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// A 16-bit matrix that TMA can read: [sheets][rows][cols], cols contiguous.
struct Operand {
  const void *p;
  int64_t cols, rows, sheets, ld, sheet;
};

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// Map of boxes of box_cols columns by box_rows rows (and some sheets), zeros outside; the swizzle is as many bytes as a row
// of the box has (128, 64 or 32).
cudaError_t encode(CUtensorMap *map, const Operand &o, int box_cols, int box_rows, int32_t dtype, int box_sheets = 1) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const size_t e = net_size(dtype);
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.sheets};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * e, (cuuint64_t)o.sheet * e};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, (cuuint32_t)box_sheets}, step[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == SLA_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == SLA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const size_t row = box_cols * e;
  const CUtensorMapSwizzle swizzle = row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_32B;
  const CUresult r = fn(map, type, 3, const_cast<void *>(o.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Up to four matrices laid out for TMA in one launch: rows padded to ld (zeros), float32 split into three
// sheets.  Halves of src lie src_half apart; part q of half i becomes sheet 3 i + q.
struct PackJob {
  const void *src;
  uint16_t *dst;
  int64_t rows, cols, src_ld, src_half, ld;
  int halves, vec, first, blocks;  // its blocks of the grid
};

struct PackJobs {
  PackJob job[4];
  int count = 0, blocks = 0;
};

// A thread moves eight columns at a time.
template <typename T>
__global__ void __launch_bounds__(256) pack_operands(const __grid_constant__ PackJobs jobs) {
  grid_dependency_wait();
  grid_dependency_launch();
  int which = 0;
  while (which + 1 < jobs.count && (int)blockIdx.x >= jobs.job[which + 1].first) ++which;
  const PackJob &j = jobs.job[which];
  const int64_t chunks = j.ld / 8, total = j.halves * j.rows * chunks, sheet = j.rows * j.ld;
  for (int64_t i = (blockIdx.x - j.first) * 256ll + threadIdx.x; i < total; i += j.blocks * 256ll) {
    const int64_t c = i % chunks * 8, hr = i / chunks;
    const int64_t half = hr / j.rows, r = hr - half * j.rows;
    float v[8];
    const T *s = (const T *)j.src + half * j.src_half + r * j.src_ld + c;
    const int count = (int)(j.cols - c < 8 ? j.cols - c : 8);
    if (j.vec && count == 8) {
      load_f32<T, 8>(s, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < count ? to_f32(s[k]) : 0.f;
    }
    store_operand<T, 8>(j.dst + half * kParts<T> * sheet + r * j.ld + c, sheet, v, 8, true);
  }
}

bool tma_ready(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

template <typename T>
constexpr int sheets_of() {
  return sizeof(T) == 4 ? 3 : 1;
}

size_t packed_bytes(int64_t rows, int64_t cols, int32_t dtype) {
  return align256((size_t)rows * (size_t)round_up(cols, 8) * 2 * (dtype == SLA_F32 ? 3 : 1));
}

// Scratch handed out front to back.
struct Arena {
  char *base;
  size_t used = 0;
  void *take(size_t bytes) {
    void *p = base ? base + used : nullptr;
    used += align256(bytes);
    return p;
  }
};

struct Call {
  cudaStream_t st;
  cudaError_t err = cudaSuccess;
  uint64_t launches = 0;
  uint32_t *timeouts = nullptr;
  // the kernels after a call's first may be made ready while the one before them runs
  bool early() const { return launches > 0; }
  template <typename... P, typename... A>
  void launch(void (*kernel)(P...), dim3 grid, int block, A &&...args) {
    if (err != cudaSuccess) return;
    LaunchConfig cfg(grid, block, 0, st, early());
    launched(cudaLaunchKernelEx(&cfg.c, kernel, P(args)...));
  }
  void launched(cudaError_t e) {
    ++launches;
    if (err == cudaSuccess) err = e;
  }
};

// Where a call finds an operand laid out for TMA.
enum Copy {
  kOwn,   // in place where TMA can read it, else packed by and for this call alone
  kLeft,  // packed whatever its layout: a later call reads the copy
  kKept,  // an earlier call's copy
};

// The matrix as an operand: in place, or from `to` with, unless it is there already, a job to pack it.
template <typename T>
Operand as_operand(PackJobs &jobs, const T *src, int64_t rows, int64_t cols, int64_t ld, int halves, void *to,
                   Copy copy = kOwn) {
  const int64_t half = rows * ld;                        // between the halves of src
  if (rows == 1 && halves == 1) ld = round_up(cols, 8);  // a single row has no distance to the next
  if (copy == kOwn && sizeof(T) == 2 && tma_ready(src, ld) && (halves == 1 || half % 8 == 0))
    return {src, cols, rows, halves, ld, rows * ld};
  const int64_t pitch = round_up(cols, 8);
  if (copy != kKept) {
    PackJob &j = jobs.job[jobs.count++];
    j.src = src, j.dst = (uint16_t *)to, j.rows = rows, j.cols = cols, j.src_ld = ld, j.src_half = half, j.ld = pitch;
    j.halves = halves, j.vec = aligned(src, 16) && ld * sizeof(T) % 16 == 0;
    j.first = jobs.blocks;
    j.blocks = (int)std::min<int64_t>((halves * rows * (pitch / 8) + 255) / 256, sm_count() * 16);
    jobs.blocks += j.blocks;
  }
  return {to, cols, rows, (int64_t)sheets_of<T>() * halves, pitch, rows * pitch};
}

template <typename T>
void run_packs(Call &c, const PackJobs &jobs) {
  if (jobs.count) c.launch(pack_operands<T>, dim3(jobs.blocks), 256, jobs);
}

// ------------------------------------------------------------------ plans

constexpr int kPlanDepth = 64;  // k of the blocks that plans are made in

struct ProductSize {
  int64_t m, n, k;           // of one half, of one segment
  int m_halves, n_halves, k_halves;
};

// Tile shape and splits of the products of one launch.
struct ProductPlan {
  int shape;
  int splits[kGroup];
  size_t partial[kGroup + 1];  // where each product's split sums start, and their end
};

// The tile shape and splits with the least predicted time.  Workers (multiprocessors, or pairs) take the
// items in turn, each of which costs its k blocks or its epilogue, whichever is longer; splits cost writing
// and reading their sums and a launch.  Measured: a k block (64 deep) 0.27 us with the 256 x 256 tile, where
// the tensor core is the limit, and 0.22 to 0.26 us with the smaller ones, where it is the 64 bytes a clock
// that a multiprocessor takes in from L2; pairs of blocks start 2 us later than single ones.
ProductPlan plan_products(Epilogue epi, const ProductSize *s, int count, int sheets) {
  static const double blocks_us[2][kProductTileCount] = {{0.27, 0.225, 0.255, 0.245}, {0, 0.81, 1.0, 0.84}};
  const auto &block_us = blocks_us[sheets == 3];
  static const double start_us[kProductTileCount] = {5.0, 5.0, 3.0, 3.0};
  static const double epilogues_us[2][3][kProductTileCount] = {
      {{2.1, 1.25, 1.25, 0.8}, {3.0, 1.8, 1.8, 1.15}, {10.0, 5.5, 5.5, 3.0}},   // kStore, kGate, kGateBack
      {{0, 1.6, 1.6, 0.9}, {0, 4.5, 4.5, 2.3}, {0, 6.0, 6.0, 3.0}}};            // float32
  const auto &epilogue_us = epilogues_us[sheets == 3];
  const int sms = sm_count();
  ProductPlan best{};
  double best_us = 1e30;
  for (int i = sheets == 3 ? 1 : 0; i < kProductTileCount; ++i) {
    const int64_t bm = 128 * kProductTiles[i].cg, bn = kProductTiles[i].bn, workers = sms / kProductTiles[i].cg;
    int64_t tiles[kGroup], kb[kGroup];
    double per[kGroup], blocks = 0;
    for (int j = 0; j < count; ++j) {
      kb[j] = (s[j].k + kPlanDepth - 1) / kPlanDepth;
      per[j] = s[j].k_halves;
      // columns of g and of u make separate tiles when their product is split
      tiles[j] = s[j].m_halves * ((s[j].m + bm - 1) / bm) * (epi == kGate ? 2 : s[j].n_halves) * ((s[j].n + bn - 1) / bn);
      blocks += tiles[j] * kb[j] * per[j];
    }
    for (int fill = 0; fill < 6; ++fill) {  // whole; as many items as workers, up to five times
      ProductPlan plan{i, {}, {}};
      double busy = 0, us = start_us[i], longest = 0;
      bool split = false;
      int64_t items = 0;
      size_t partial = 0;
      for (int j = 0; j < count; ++j) {
        int64_t t = tiles[j];
        int64_t n = std::max<int64_t>(1, (int64_t)(kb[j] * per[j] * fill * workers / std::max(1.0, blocks)));
        n = std::min(n, kb[j]);
        if (epi == kGate && n == 1)
          t = s[j].m_halves * ((s[j].m + bm - 1) / bm) * ((s[j].n + bn / 2 - 1) / (bn / 2));
        const double main = (kb[j] + n - 1) / n * per[j] * block_us[i], end = epilogue_us[n > 1 ? kStore : epi][i];
        plan.splits[j] = (int)n;
        plan.partial[j] = partial;
        if (n > 1) {
          const int halves = epi == kGate ? 2 : s[j].n_halves;
          partial += align256(4 * (size_t)(s[j].m * s[j].m_halves) * (size_t)(round_up(s[j].n, 16) * halves) * n);
          split = true;
        }
        // rounds of this product's items, a partial round shared with the next product's
        const double rounds = count > 1 ? (double)(t * n) / workers : (double)((t * n + workers - 1) / workers);
        busy += rounds * std::max(main, end);
        longest = std::max(longest, std::max(main, end));
        us += j == 0 ? std::min(main, end) : 0;
        items += t * n;
      }
      plan.partial[count] = partial;
      us += count > 1 ? std::max(longest, busy + (items > workers ? 0.5 * longest : 0)) : busy;
      if (split) us += 4.0 + 1.0 * partial / 5e6;
      if (us < best_us) {
        best_us = us;
        best = plan;
      }
    }
  }
  return best;
}

// ------------------------------------------------------------------ sums of splits

struct SplitSums {
  ProductArgs p[kGroup];  // c: the result; ldc, c_n_half, c_split: of the sums
  const float *parts[kGroup];
  int64_t rows[kGroup];
};

// The epilogue of products whose k was split (blockIdx.y: which): adds the parts in order, four columns a thread.
template <typename T, int EPI>
__global__ void __launch_bounds__(256) finish_splits(const __grid_constant__ SplitSums f) {
  grid_dependency_wait();
  grid_dependency_launch();
  const ProductArgs &p = f.p[blockIdx.y];
  const int64_t chunks = (p.n + 3) / 4, total = f.rows[blockIdx.y] * chunks;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t row = i / chunks;
    const int col = (int)(i - row * chunks) * 4, count = p.n - col;
    const float *src = f.parts[blockIdx.y] + row * p.ldc + col;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      float t[4];
      load_f32<float, 4>(src + s * p.c_split, t);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += t[k];
      if (EPI == kGate) {
        load_f32<float, 4>(src + s * p.c_split + p.c_n_half, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] += t[k];
      }
    }
    if (EPI == kStore) {
      T *out = (T *)p.c + row * (int64_t)p.n + col;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p.bias && k < count) v[k] += to_f32(((const T *)p.bias)[col + k]);
      if (p.vec && count >= 4) {
        store_f32<T, 4>(out, v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < count) out[k] = from_f32<T>(v[k]);
      }
      continue;
    }
    const int64_t o = row * p.ldg + col;
    if (EPI == kGate) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= count) break;
        if (p.bias) {
          v[k] += to_f32(((const T *)p.bias)[col + k]);
          u[k] += to_f32(((const T *)p.bias)[p.n + col + k]);
        }
      }
      float h[4];
      with_activation(p.act, [&](auto act) { gate<act.value, true, 4>(v, u, h); });
      if (p.g)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < count) {
            ((T *)p.g)[o + k] = from_f32<T>(v[k]);
            ((T *)p.u)[o + k] = from_f32<T>(u[k]);
          }
      store_operand<T, 4>(p.h + o, p.sheet, h, count, false);
    } else {
      float g[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[k] = k < count ? to_f32(((const T *)p.g)[o + k]) : 0.f;
        u[k] = k < count ? to_f32(((const T *)p.u)[o + k]) : 0.f;
      }
      gate_gradients(v, g, u);
      store_operand<T, 4>(p.h + o, p.sheet, g, count, false);
      store_operand<T, 4>(p.h + kParts<T> * p.sheet + o, p.sheet, u, count, false);
    }
  }
}

// One product: A(m, k) and B(n, k) with their majors, and the epilogue's arrays in `p`.
struct ProductJob {
  ProductSize s;
  Operand a;
  bool a_mn;
  Operand b;
  bool b_mn;
  ProductArgs p;
  bool wanted;
};

// Runs the wanted ones of up to kGroup products with the plan made for all of them (whose split sums `parts` holds).
template <typename T>
void run_products(Call &c, Epilogue epi, const ProductJob *jobs, int count, const ProductPlan &plan, float *parts,
                  float *runs) {
  if (c.err != cudaSuccess) return;
  constexpr int S = sheets_of<T>(), D = kDepth<T>;
  constexpr int32_t part = S == 3 ? SLA_BF16 : NetType<T>::dtype;  // type of the operands
  const ProductTile tile = kProductTiles[plan.shape];
  const int bm = 128 * tile.cg, bn = tile.bn;
  // items with the most k blocks first, so that the last round is one of short ones
  int order[kGroup] = {0, 1, 2};
  auto depth = [&](int j) {
    return (double)jobs[j].s.k * jobs[j].s.k_halves / plan.splits[j];
  };
  std::stable_sort(order, order + count, [&](int x, int y) { return depth(x) > depth(y); });
  ProductLaunch l;
  l.count = 0;
  l.first[0] = 0;
  l.timeouts = c.timeouts;
  l.runs = runs;
  SplitSums f;
  int nsplit = 0;
  int64_t items = 0, finish = 0;
  for (int oi = 0; oi < count; ++oi) {
    const int j = order[oi];
    if (!jobs[j].wanted) continue;
    const ProductSize &s = jobs[j].s;
    const Operand &a = jobs[j].a, &b = jobs[j].b;
    const bool split = plan.splits[j] > 1, gate = epi == kGate && !split;
    ProductArgs &p = l.p[l.count];
    p = jobs[j].p;
    p.m = (int)s.m, p.n = (int)s.n;
    p.m_halves = s.m_halves, p.n_halves = epi == kGate && split ? 2 : s.n_halves;
    const int cols = gate ? bn / 2 : bn;
    p.m_tiles = (int)((s.m + bm - 1) / bm), p.n_tiles = (int)((s.n + cols - 1) / cols);
    p.k_blocks = (int)((s.k + D - 1) / D);
    p.splits = plan.splits[j];
    p.a_mn = jobs[j].a_mn, p.b_mn = jobs[j].b_mn, p.f16 = sizeof(T) == 2 && NetType<T>::dtype == SLA_F16;
    p.segments = s.k_halves;
    for (int h = 0; h < s.k_halves; ++h) p.a_sheet[h] = p.b_sheet[h] = (int8_t)h;
    cudaError_t e = encode(&l.a[l.count], a, p.a_mn ? 64 : D, p.a_mn ? D : 128, part);
    if (e == cudaSuccess) e = encode(&l.b[l.count], b, p.b_mn ? 64 : D, p.b_mn ? D : gate ? bn / 2 : bn / tile.cg, part);
    if (epi != kStore && !split) {
      // the epilogue's own arrays (see tma_epilogue); a warp's columns of the 64-wide gate tile are 16
      const int box = S == 3 || (gate && bn == 64) ? 16 : 32;
      const Operand h{p.h, s.n, s.m, S * (epi == kGate ? 1 : 2), p.ldg, p.sheet};
      Operand g = h, u = h;
      g.sheets = u.sheets = 1;
      g.p = p.g, u.p = p.u;
      if (epi == kGate && p.g) {
        if (e == cudaSuccess) e = encode(&l.out[0], g, box, 32, NetType<T>::dtype);
        if (e == cudaSuccess) e = encode(&l.out[1], u, box, 32, NetType<T>::dtype);
      }
      if (e == cudaSuccess) e = encode(&l.out[epi == kGate ? 2 : 0], h, box, 32, part, S == 3 ? (int)h.sheets : 1);
    }
    if (e != cudaSuccess) {
      c.err = e;
      return;
    }
    if (split) {
      const int64_t ncols = round_up(s.n, 16) * p.n_halves, rows = s.m * s.m_halves;
      float *to = parts + plan.partial[j] / sizeof(float);
      ProductArgs &q = f.p[nsplit];
      q = p;
      q.ldc = p.ldc = ncols;
      q.c_n_half = p.c_n_half = round_up(s.n, 16);
      q.c_split = p.c_split = rows * ncols;
      p.c_m_half = s.m * ncols;
      p.c = to;
      f.parts[nsplit] = to;
      f.rows[nsplit++] = rows;
      finish = std::max(finish, rows * ((s.n + 3) / 4));
    }
    items += (int64_t)p.m_halves * p.m_tiles * p.n_halves * p.n_tiles * p.splits;
    l.first[++l.count] = (int)std::min<int64_t>(items, INT32_MAX);
  }
  if (items > INT32_MAX) {  // more tiles than a launch counts
    c.err = cudaErrorInvalidConfiguration;
    return;
  }
  if (!l.count) return;
  // The items before the last product's are the longer ones; the workers that get one of them less make up
  // for it with short ones.
  const int64_t workers = std::min<int64_t>(items, sm_count() / tile.cg);
  l.lead = l.first[l.count - 1], l.extra = 0;
  if (l.count > 1 && l.lead % workers) {
    auto blocks_of = [](const ProductArgs &p) { return (double)p.k_blocks / p.splits * p.segments; };
    const int64_t shorter = workers - l.lead % workers, shorts = l.first[l.count] - l.lead;
    l.extra = (int)std::min<int64_t>((int64_t)(blocks_of(l.p[l.count - 2]) / blocks_of(l.p[l.count - 1])), shorts / shorter);
  }
  // a split gate or gate-back product leaves plain sums
  const int as = nsplit ? kStore : epi;
  const int blocks = (int)workers * tile.cg;
  c.launched(launch_product<T>(as, plan.shape, blocks, l, c.early(), c.st));
  if (!nsplit) return;
  const dim3 grid((unsigned)std::min<int64_t>((finish + 255) / 256, sm_count() * 16), nsplit);
  if (epi == kStore)
    c.launch(finish_splits<T, kStore>, grid, 256, f);
  else if (epi == kGate)
    c.launch(finish_splits<T, kGate>, grid, 256, f);
  else
    c.launch(finish_splits<T, kGateBack>, grid, 256, f);
}

// ------------------------------------------------------------------ column sums (bias gradients)

constexpr int kSumParts = 512;    // parts of the rows at most
constexpr int kDirectRows = 1024; // rows that are added up without parts

// parts[part][cols]: sums over a part of the rows, VEC columns a thread; the block's threads cover
// 256 / tpr rows at a time.  S sheets `sheet` apart are parts of one value.
template <typename E, int S, int VEC>
__global__ void __launch_bounds__(256) column_parts(int64_t rows, int64_t cols, const E *__restrict__ a, int64_t lda,
                                                    int64_t sheet, int tpr, int64_t per, float *__restrict__ parts) {
  __shared__ float sm[256 * VEC];
  grid_dependency_wait();
  grid_dependency_launch();
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = 256 / tpr;
  const int64_t c = (blockIdx.x * (int64_t)tpr + t) * VEC;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  float s[VEC] = {};
  if (c < cols)
#pragma unroll 4
    for (int64_t r = r0 + group; r < r1; r += groups) {
#pragma unroll
      for (int q = S - 1; q >= 0; --q) {
        float v[VEC];
        load_f32<E, VEC>(a + q * sheet + r * lda + c, v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] += v[k];
      }
    }
#pragma unroll
  for (int k = 0; k < VEC; ++k) sm[threadIdx.x * VEC + k] = s[k];
  __syncthreads();
  for (int i = threadIdx.x; i < tpr * VEC; i += 256) {
    const int64_t col = blockIdx.x * (int64_t)tpr * VEC + i;
    float sum = 0.f;
    for (int g = 0; g < groups; ++g) sum += sm[g * tpr * VEC + i];
    if (col < cols) parts[blockIdx.y * cols + col] = sum;
  }
}

// Rows of float32 to be added up, in order; column c of half h of `pitch` columns goes to out[h * n + c].
struct AddJob {
  const float *rows;
  void *out;
  int64_t cols, pitch, n;
  int count, first;  // rows; its first block
};

struct AddJobs {
  AddJob job[3];
  int jobs = 0, blocks = 0;
};

template <typename T>
__global__ void __launch_bounds__(1024) add_rows(const __grid_constant__ AddJobs jobs) {
  __shared__ float sm[32][33];
  grid_dependency_wait();
  grid_dependency_launch();
  int which = 0;
  while (which + 1 < jobs.jobs && (int)blockIdx.x >= jobs.job[which + 1].first) ++which;
  const AddJob &j = jobs.job[which];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t c = (blockIdx.x - j.first) * 32ll + lane;
  float s = 0.f;
  if (c < j.cols)
#pragma unroll 8
    for (int p = wy; p < j.count; p += 32) s += j.rows[p * j.cols + c];
  sm[wy][lane] = s;
  __syncthreads();
  const int64_t half = c / j.pitch, i = c - half * j.pitch;
  if (wy == 0 && c < j.cols && i < j.n) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += sm[k][lane];
    ((T *)j.out)[half * j.n + i] = from_f32<T>(t);
  }
}

// Column sums of up to three matrices: each in two steps, of which the second is one launch for all.
struct ColumnSums {
  Call &c;
  float *parts;  // scratch for kSumParts rows of every matrix
  AddJobs jobs;
  void add(const float *rows, int count, int64_t cols, int64_t pitch, int64_t n, void *out) {
    jobs.job[jobs.jobs++] = {rows, out, cols, pitch, n, count, jobs.blocks};
    jobs.blocks += (int)((cols + 31) / 32);
  }
  // out = column sums of [rows][cols] (in halves of `pitch` columns, the first n of each wanted)
  template <typename E, int S>
  void of(int64_t rows, int64_t cols, const E *a, int64_t lda, int64_t sheet, int64_t pitch, int64_t n, void *out) {
    if (sizeof(E) == 4 && S == 1 && lda == cols && rows <= kDirectRows) {
      add((const float *)a, (int)rows, cols, pitch, n, out);
      return;
    }
    constexpr int V = 16 / sizeof(E);
    const bool vec = aligned(a, 16) && lda % V == 0 && cols % V == 0 && sheet % V == 0;
    const int64_t chunks = vec ? cols / V : cols;
    int tpr = 1;
    while (tpr < 32 && tpr < chunks) tpr <<= 1;
    const int64_t tiles = (chunks + tpr - 1) / tpr;
    // enough blocks to fill the GPU, each with at least eight turns of its threads
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kSumParts, sm_count() * 8 / tiles));
    const int64_t per = std::max<int64_t>(8 * (256 / tpr), (rows + most - 1) / most);
    const int nparts = (int)((rows + per - 1) / per);
    c.launch(vec ? column_parts<E, S, V> : column_parts<E, S, 1>, dim3((unsigned)tiles, nparts), 256, rows, cols, a, lda,
             sheet, tpr, per, parts);
    add(parts, nparts, cols, pitch, n, out);
    parts += kSumParts * cols;
  }
  template <typename T>
  void finish() {
    if (jobs.jobs) c.launch(add_rows<T>, dim3(jobs.blocks), 1024, jobs);
  }
};

// ------------------------------------------------------------------ buffers

int64_t hidden_pitch(const sla_ffn *f) { return round_up(f->hidden, 16); }

// Whether a forward call leaves a packed copy of a matrix with this many columns to the backward call: where
// TMA cannot read a dense original.  The sizes alone decide, so that both calls and the layout of what is saved
// agree: a view with wider rows, or a single row, is packed too, though TMA could read it where it is.  (A
// matrix that is only misaligned is packed by each call.)
bool keeps_packed(const sla_ffn *f, int64_t cols) {
  return f->tokens > kFewTokens && (f->dtype == SLA_F32 || cols % 8 != 0);
}

// u act'(g), act(g) (dtype) and h (operand sheets), rows hidden_pitch apart, then packed copies of x, w_in and w_out.
struct SavedLayout {
  size_t u, h, x, w_in, w_out, total;
};

SavedLayout saved_layout(const sla_ffn *f) {
  const size_t n = (size_t)f->tokens * (size_t)hidden_pitch(f);
  SavedLayout L;
  L.u = align256(n * net_size(f->dtype));
  L.h = 2 * L.u;
  L.x = L.h + align256(n * 2 * (f->dtype == SLA_F32 ? 3 : 1));
  L.w_in = L.x + (keeps_packed(f, f->width) ? packed_bytes(f->tokens, f->width, f->dtype) : 0);
  L.w_out = L.w_in + (keeps_packed(f, f->width) ? packed_bytes(2 * f->hidden, f->width, f->dtype) : 0);
  L.total = L.w_out + (keeps_packed(f, f->hidden) ? packed_bytes(f->out, f->hidden, f->dtype) : 0);
  return L;
}

ProductSize gate_size(const sla_ffn *f) { return {f->tokens, f->hidden, f->width, 1, 1, 1}; }
ProductSize out_size(const sla_ffn *f) { return {f->tokens, f->out, f->hidden, 1, 1, 1}; }
ProductSize dh_size(const sla_ffn *f) { return {f->tokens, f->hidden, f->out, 1, 1, 1}; }
ProductSize dx_size(const sla_ffn *f) { return {f->tokens, f->width, f->hidden, 1, 1, 2}; }
ProductSize dw_in_size(const sla_ffn *f) { return {f->hidden, f->width, f->tokens, 2, 1, 1}; }
ProductSize dw_out_size(const sla_ffn *f) { return {f->out, f->hidden, f->tokens, 1, 1, 1}; }

// Sums of the runs so far of every block's tile (float32's tiles have 128 columns at most).
size_t run_bytes(const sla_ffn *f) { return f->dtype == SLA_F32 ? (size_t)sm_count() * 128 * 128 * sizeof(float) : 0; }

struct ForwardScratch {
  void *x, *w_in, *w_out, *h;
  float *parts, *runs;
  size_t total;
  ProductPlan gate, y;
};

ForwardScratch forward_scratch(const sla_ffn *f, char *base) {
  const int S = f->dtype == SLA_F32 ? 3 : 1;
  Arena a{base};
  ForwardScratch w{};
  w.h = a.take(saved_layout(f).x - saved_layout(f).h);
  w.total = a.used;
  if (f->tokens <= kFewTokens) return w;
  w.x = a.take(packed_bytes(f->tokens, f->width, f->dtype));
  w.w_in = a.take(packed_bytes(2 * f->hidden, f->width, f->dtype));
  w.w_out = a.take(packed_bytes(f->out, f->hidden, f->dtype));
  const ProductSize gate = gate_size(f), out = out_size(f);
  w.gate = plan_products(kGate, &gate, 1, S);
  w.y = plan_products(kStore, &out, 1, S);
  w.parts = (float *)a.take(std::max(w.gate.partial[1], w.y.partial[1]));
  w.runs = (float *)a.take(run_bytes(f));
  w.total = a.used;
  return w;
}

struct BackwardScratch {
  void *dy, *x, *w_in, *w_out, *dgu;
  float *sums, *columns, *parts, *runs;
  size_t total;
  ProductPlan dh, rest;
};

BackwardScratch backward_scratch(const sla_ffn *f, char *base) {
  const int S = f->dtype == SLA_F32 ? 3 : 1;
  Arena a{base};
  BackwardScratch w;
  w.dy = a.take(packed_bytes(f->tokens, f->out, f->dtype));
  w.x = a.take(packed_bytes(f->tokens, f->width, f->dtype));
  w.w_in = a.take(packed_bytes(2 * f->hidden, f->width, f->dtype));
  w.w_out = a.take(packed_bytes(f->out, f->hidden, f->dtype));
  w.dgu = a.take((size_t)f->tokens * (size_t)hidden_pitch(f) * 2 * 2 * S);
  w.sums = (float *)a.take((size_t)((f->tokens + 31) / 32) * 2 * (size_t)hidden_pitch(f) * sizeof(float));
  w.columns = (float *)a.take(kSumParts * sizeof(float) * (size_t)(2 * hidden_pitch(f) + f->out));
  const ProductSize dh = dh_size(f), rest[kGroup] = {dx_size(f), dw_in_size(f), dw_out_size(f)};
  w.dh = plan_products(kGateBack, &dh, 1, S);
  w.rest = plan_products(kStore, rest, kGroup, S);
  w.parts = (float *)a.take(std::max(w.dh.partial[1], w.rest.partial[kGroup]));
  w.runs = (float *)a.take(run_bytes(f));
  w.total = a.used;
  return w;
}

// ------------------------------------------------------------------ narrow blocks

template <typename T>
bool vec_out(const T *p, int64_t ld) {
  return aligned(p, 32) && ld * sizeof(T) % 32 == 0;
}

// Tiles of x that the fused kernel of a narrow block keeps on their way (4 to 2), or 0 where its weights and
// they do not fit a multiprocessor's shared memory.
int narrow_stages(const sla_ffn *f) {
  if (f->dtype == SLA_F32 || f->width > kNarrowMost || f->out > kNarrowMost || f->hidden > 64 * kNarrowChunk) return 0;
  for (int s = 4; s >= 2; --s)
    if (narrow_bytes((f->width + 63) / 64, (f->hidden + kNarrowChunk - 1) / kNarrowChunk, round_up(f->out, 16), s) <=
        227 * 1024)
      return s;
  return 0;
}

template <typename T>
void run_narrow(Call &c, const sla_ffn *f, int stages, const Operand &x, const Operand &w_in, const T *b_in,
                const Operand &w_out, const T *b_out, T *y) {
  if constexpr (sizeof(T) == 2) {
    if (c.err != cudaSuccess) return;
    NarrowArgs p;
    p.tokens = (int)f->tokens, p.hidden = (int)f->hidden, p.out = (int)f->out;
    p.k_blocks = (int)((f->width + 63) / 64), p.chunks = (int)((f->hidden + kNarrowChunk - 1) / kNarrowChunk);
    p.out_pad = (int)round_up(f->out, 16), p.stages = stages;
    p.f16 = f->dtype == SLA_F16, p.act = f->activation;
    p.b_in = b_in;
    p.b_out = b_out, p.b_out_vec = aligned(b_out, 32);
    p.y = y, p.y_vec = vec_out(y, f->out), p.timeouts = c.timeouts;
    cudaError_t e = encode(&p.x, x, 64, 128, f->dtype);
    if (e == cudaSuccess) e = encode(&p.w_in, w_in, 64, 64, f->dtype);
    if (e == cudaSuccess) e = encode(&p.w_out, w_out, 64, p.out_pad, f->dtype);
    if (e == cudaSuccess) {
      const int blocks = (int)std::min<int64_t>((f->tokens + 127) / 128, sm_count());
      c.launched(launch_narrow<T>(p, blocks, c.early(), c.st));
    } else {
      c.err = e;
    }
  }
}

// ------------------------------------------------------------------ the two calls

sla_status finish(const Call &c) {
  count_launches(c.launches);
  return c.err == cudaSuccess ? SLA_OK : fail(c.err);
}

template <typename T>
sla_status forward(const sla_ffn *f, const T *x, int64_t ldx, const T *w_in, const T *b_in, const T *w_out,
                   const T *b_out, T *y, char *saved, const ForwardScratch &w, cudaStream_t st) {
  Call c{st};
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  c.timeouts = earlier.count;
  const SavedLayout L = saved_layout(f);
  const int64_t ldg = hidden_pitch(f);
  void *h = saved ? saved + L.h : w.h;
  if (f->tokens <= kFewTokens) {
    FewArgs p{};
    p.tokens = (int)f->tokens, p.n = (int)f->hidden, p.k = (int)f->width, p.act = f->activation;
    p.x = x, p.ldx = ldx, p.w = w_in, p.bias = b_in;
    p.x_vec = aligned(x, 16) && (f->tokens == 1 || ldx % 8 == 0), p.w_vec = aligned(w_in, 16) && f->width % 8 == 0;
    p.g = saved, p.u = saved ? saved + L.u : nullptr, p.h = (uint16_t *)h, p.ldg = ldg, p.sheet = f->tokens * ldg;
    c.launched(launch_few<T>(kGate, p, st));
    FewArgs q{};
    q.tokens = (int)f->tokens, q.n = (int)f->out, q.k = (int)f->hidden;
    q.x = h, q.ldx = ldg, q.x_sheet = p.sheet, q.x_vec = 1, q.w = w_out, q.bias = b_out;
    q.w_vec = aligned(w_out, 16) && f->hidden % 8 == 0, q.c = y;
    c.launched(launch_few<T>(kStore, q, st));
    return finish(c);
  }
  PackJobs packs;
  const Copy copy_x = saved && keeps_packed(f, f->width) ? kLeft : kOwn;
  const Copy copy_o = saved && keeps_packed(f, f->hidden) ? kLeft : kOwn;
  const Operand ox = as_operand(packs, x, f->tokens, f->width, ldx, 1, copy_x ? saved + L.x : w.x, copy_x);
  const Operand oi = as_operand(packs, w_in, f->hidden, f->width, f->width, 2, copy_x ? saved + L.w_in : w.w_in, copy_x);
  const Operand oo = as_operand(packs, w_out, f->out, f->hidden, f->hidden, 1, copy_o ? saved + L.w_out : w.w_out, copy_o);
  run_packs<T>(c, packs);
  if (const int stages = saved ? 0 : narrow_stages(f)) {
    run_narrow<T>(c, f, stages, ox, oi, b_in, oo, b_out, y);
    return finish(c);
  }
  const Operand oh{h, f->hidden, f->tokens, sheets_of<T>(), ldg, f->tokens * ldg};
  ProductJob gate{gate_size(f), ox, false, oi, false, {}, true};
  gate.p.act = f->activation;
  gate.p.bias = b_in, gate.p.bias_vec = b_in && aligned(b_in, 32) && f->hidden % 16 == 0;
  gate.p.g = saved, gate.p.u = saved ? saved + L.u : nullptr;
  gate.p.h = (uint16_t *)h, gate.p.ldg = ldg, gate.p.sheet = f->tokens * ldg;
  run_products<T>(c, kGate, &gate, 1, w.gate, w.parts, w.runs);
  ProductJob out{out_size(f), oh, false, oo, false, {}, true};
  out.p.bias = b_out, out.p.bias_vec = aligned(b_out, 32);
  out.p.c = y, out.p.ldc = f->out, out.p.vec = vec_out(y, f->out);
  run_products<T>(c, kStore, &out, 1, w.y, w.parts, w.runs);
  return finish(c);
}

template <typename T>
sla_status backward(const sla_ffn *f, const T *dy, int64_t lddy, const T *x, int64_t ldx, const T *w_in,
                    const T *w_out, const char *saved, T *dx, T *dw_in, T *dw_out, T *db_in, T *db_out,
                    const BackwardScratch &w, cudaStream_t st) {
  using E = typename std::conditional<sizeof(T) == 4, bf16, T>::type;  // type of the operand sheets
  constexpr int S = sheets_of<T>();
  Call c{st};
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  c.timeouts = earlier.count;
  const SavedLayout L = saved_layout(f);
  const int64_t ldg = hidden_pitch(f), sheet = f->tokens * ldg;
  const bool inner = dx || dw_in || db_in;
  const Copy copy_x = keeps_packed(f, f->width) ? kKept : kOwn, copy_o = keeps_packed(f, f->hidden) ? kKept : kOwn;
  char *sv = const_cast<char *>(saved);
  PackJobs packs;
  Operand ody{}, ox{}, oi{}, oo{};
  if (inner || dw_out) ody = as_operand(packs, dy, f->tokens, f->out, lddy, 1, w.dy);
  if (dw_in) ox = as_operand(packs, x, f->tokens, f->width, ldx, 1, copy_x ? sv + L.x : w.x, copy_x);
  if (dx) oi = as_operand(packs, w_in, f->hidden, f->width, f->width, 2, copy_x ? sv + L.w_in : w.w_in, copy_x);
  if (inner) oo = as_operand(packs, w_out, f->out, f->hidden, f->hidden, 1, copy_o ? sv + L.w_out : w.w_out, copy_o);
  run_packs<T>(c, packs);
  const Operand odgu{w.dgu, f->hidden, f->tokens, 2 * S, ldg, sheet};
  const Operand oh{saved + L.h, f->hidden, f->tokens, S, ldg, sheet};
  ColumnSums columns{c, w.columns, {}};
  if (inner) {
    ProductJob dh{dh_size(f), ody, false, oo, true, {}, true};
    dh.p.g = sv, dh.p.u = sv + L.u;
    dh.p.h = (uint16_t *)w.dgu, dh.p.ldg = ldg, dh.p.sheet = sheet;
    // the epilogue sums dg and du over 32 rows on its way, unless the product is split
    if (db_in && w.dh.splits[0] == 1) dh.p.sums = w.sums;
    run_products<T>(c, kGateBack, &dh, 1, w.dh, w.parts, w.runs);
    if (dh.p.sums)
      columns.of<float, 1>((f->tokens + 31) / 32, 2 * ldg, w.sums, 2 * ldg, 0, ldg, f->hidden, db_in);
    else if (db_in)
      for (int half = 0; half < 2; ++half)
        columns.of<E, S>(f->tokens, f->hidden, (const E *)w.dgu + half * S * sheet, ldg, sheet, f->hidden, f->hidden,
                         db_in + half * f->hidden);
  }
  if (db_out) columns.of<T, 1>(f->tokens, f->out, dy, lddy, 0, f->out, f->out, db_out);
  columns.finish<T>();
  auto job = [&](const ProductSize &s, const Operand &a, bool a_mn, const Operand &b, T *out) {
    ProductJob j{s, a, a_mn, b, true, {}, out != nullptr};
    j.p.c = out, j.p.ldc = s.n, j.p.c_m_half = s.m * s.n, j.p.vec = vec_out(out, s.n);
    return j;
  };
  const ProductJob rest[kGroup] = {job(dx_size(f), odgu, false, oi, dx), job(dw_in_size(f), odgu, true, ox, dw_in),
                                   job(dw_out_size(f), ody, true, oh, dw_out)};
  run_products<T>(c, kStore, rest, kGroup, w.rest, w.parts, w.runs);
  return finish(c);
}

// ------------------------------------------------------------------ argument checks

sla_status check_ffn(const sla_ffn *f) {
  if (!f) return SLA_INVALID_ARG;
  const int64_t most = (int64_t)1 << 24;
  if (f->tokens < 0 || f->tokens > (int64_t)1 << 30) return SLA_INVALID_ARG;
  if (f->width < 1 || f->width > most || f->hidden < 1 || f->hidden > most || f->out < 1 || f->out > most)
    return SLA_INVALID_ARG;
  if (!net_dtype(f->dtype) || f->activation < SLA_ACT_SILU || f->activation > SLA_ACT_RELU) return SLA_INVALID_ARG;
  return SLA_OK;
}

sla_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  if (rows == 0) return SLA_OK;
  if (!p || !aligned(p, net_size(dtype))) return SLA_INVALID_ARG;
  return ld >= cols || rows == 1 ? SLA_OK : SLA_INVALID_ARG;
}

sla_status check_scratch(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return SLA_OK;
  if (!ws || !aligned(ws, 256)) return SLA_INVALID_ARG;
  return bytes < need ? SLA_WORKSPACE_TOO_SMALL : SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API size_t sla_gated_ffn_saved_bytes(const sla_ffn *f) {
  return check_ffn(f) == SLA_OK ? saved_layout(f).total : 0;
}

SLA_API size_t sla_gated_ffn_workspace_bytes(const sla_ffn *f) {
  return check_ffn(f) == SLA_OK ? forward_scratch(f, nullptr).total : 0;
}

SLA_API size_t sla_gated_ffn_backward_workspace_bytes(const sla_ffn *f) {
  return check_ffn(f) == SLA_OK ? backward_scratch(f, nullptr).total : 0;
}

SLA_API sla_status sla_gated_ffn(const sla_ffn *f, const void *x, int64_t ldx, const void *w_in, const void *b_in,
                                 const void *w_out, const void *b_out, void *y, void *saved, size_t saved_bytes,
                                 void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_ffn(f));
  SLA_CHECK(check_matrix(x, f->tokens, f->width, ldx, f->dtype));
  SLA_CHECK(check_matrix(y, f->tokens, f->out, f->out, f->dtype));
  SLA_CHECK(check_matrix(w_in, 2 * f->hidden, f->width, f->width, f->dtype));
  SLA_CHECK(check_matrix(w_out, f->out, f->hidden, f->hidden, f->dtype));
  const size_t e = net_size(f->dtype);
  if (!aligned(b_in, e) || !aligned(b_out, e)) return SLA_INVALID_ARG;
  if (saved) SLA_CHECK(check_scratch(saved, saved_bytes, saved_layout(f).total));
  const ForwardScratch w = forward_scratch(f, (char *)workspace);
  SLA_CHECK(check_scratch(workspace, ws_bytes, w.total));
  if (f->tokens == 0) return SLA_OK;
#define SLA_FFN_FWD(T)                                                                                             \
  forward<T>(f, (const T *)x, ldx, (const T *)w_in, (const T *)b_in, (const T *)w_out, (const T *)b_out, (T *)y, \
             (char *)saved, w, (cudaStream_t)stream)
  return f->dtype == SLA_F32 ? SLA_FFN_FWD(float) : f->dtype == SLA_F16 ? SLA_FFN_FWD(f16) : SLA_FFN_FWD(bf16);
#undef SLA_FFN_FWD
}

SLA_API sla_status sla_gated_ffn_backward(const sla_ffn *f, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                          const void *w_in, const void *w_out, const void *saved, size_t saved_bytes,
                                          void *dx, void *dw_in, void *dw_out, void *db_in, void *db_out,
                                          void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_ffn(f));
  SLA_CHECK(check_matrix(dy, f->tokens, f->out, lddy, f->dtype));
  SLA_CHECK(check_matrix(x, f->tokens, f->width, ldx, f->dtype));
  SLA_CHECK(check_matrix(w_in, 2 * f->hidden, f->width, f->width, f->dtype));
  SLA_CHECK(check_matrix(w_out, f->out, f->hidden, f->hidden, f->dtype));
  const size_t e = net_size(f->dtype);
  for (const void *p : {(const void *)dx, (const void *)dw_in, (const void *)dw_out, (const void *)db_in,
                        (const void *)db_out})
    if (!aligned(p, e)) return SLA_INVALID_ARG;
  SLA_CHECK(check_scratch(saved, saved_bytes, saved_layout(f).total));
  const BackwardScratch w = backward_scratch(f, (char *)workspace);
  SLA_CHECK(check_scratch(workspace, ws_bytes, w.total));
  cudaStream_t st = (cudaStream_t)stream;
  if (f->tokens == 0) {  // sums over no tokens
    const struct {
      void *p;
      int64_t n;
    } out[] = {{dw_in, 2 * f->hidden * f->width}, {dw_out, f->out * f->hidden}, {db_in, 2 * f->hidden}, {db_out, f->out}};
    for (const auto &o : out)
      if (o.p) {
        const cudaError_t err = cudaMemsetAsync(o.p, 0, e * (size_t)o.n, st);
        if (err != cudaSuccess) return fail(err);
      }
    return SLA_OK;
  }
#define SLA_FFN_BWD(T)                                                                                               \
  backward<T>(f, (const T *)dy, lddy, (const T *)x, ldx, (const T *)w_in, (const T *)w_out, (const char *)saved,    \
              (T *)dx, (T *)dw_in, (T *)dw_out, (T *)db_in, (T *)db_out, w, st)
  return f->dtype == SLA_F32 ? SLA_FFN_BWD(float) : f->dtype == SLA_F16 ? SLA_FFN_BWD(f16) : SLA_FFN_BWD(bf16);
#undef SLA_FFN_BWD
}

SLA_API sla_status sla_gated_ffn_check(void *stream) {
  const Expired x = expired();
  if (x.err != cudaSuccess) return fail(x.err);
  const cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  return e == cudaSuccess ? report_expired(x) : fail(e);
}

SLA_API sla_status sla_test_expire_wait(void *stream) {
  const Expired x = expired();
  if (x.err != cudaSuccess) return fail(x.err);
  expire_wait<<<1, 32, 0, (cudaStream_t)stream>>>(x.count);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

}  // extern "C"
