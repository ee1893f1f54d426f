// The whole gated feed-forward block of a narrow network in one kernel (16-bit data, forward, nothing kept).
//
// Between the two products of a narrow block h is the largest array by far: at 64 -> 256 -> 64 it is four
// times x, and a million tokens write and read 1 GB of it for 0.25 GB of x and y.  Here it never leaves
// the multiprocessor.  A block keeps both weight matrices in shared memory for its lifetime and takes
// tiles of 128 tokens; of the hidden units it takes 64 at a time:
//
//   S = X [Wg; Wu]^T   128 x 128 in tensor memory, three times (two with more than 64 outputs)   (mma)
//   H = act(g) u       128 x 64 in shared memory, twice      (sixteen warps, in two teams)
//   Y += H Wo^T        128 x out in tensor memory, twice     (mma)
//
// One warp issues the first products, as far ahead as there is room for, and another the second ones.  H is
// written as TMA would have put it there: 128-byte rows of 64 hidden units, 16-byte units swizzled by the row.
//
// Measured at 1,000,000 tokens: 168 us at 64 -> 256 -> 64 in bfloat16 where the two tiled products take 323, 82 against
// 189 at 32 -> 128 -> 32 and 137 against 242 at 128 -> 96 -> 128; 64 tokens 8.4 us against 8.6.  Bound by the
// load-store pipe (66 % busy: sums out of tensor memory, H into shared memory, biases); special functions 34 %, tensor
// cores 25 %, DRAM 16 %.
#pragma once

#include "sla_product.cuh"

namespace sla {

constexpr int kNarrowMost = 128;    // columns of x and of y at most
constexpr int kNarrowChunk = 64;    // hidden units at a time
constexpr int kNarrowTile = 16384;  // bytes of 128 rows of 64 values
constexpr int kNarrowThreads = 19 * 32;

struct NarrowArgs {
  CUtensorMap x, w_in, w_out;  // boxes of 64 columns by 128, 64 and out_pad rows
  int tokens, hidden, out;
  int k_blocks, chunks, out_pad, stages;
  int f16, act;
  const void *b_in, *b_out;    // T or NULL
  int b_out_vec, y_vec;
  void *y;                     // T [tokens][out]
  uint32_t *timeouts;
};

// Bytes of shared memory with `stages` tiles of x: weights, x, H, the biases of g and u in float32 and the barriers.
inline int64_t narrow_bytes(int64_t k_blocks, int64_t chunks, int64_t out_pad, int stages) {
  return chunks * (k_blocks * kNarrowTile + out_pad * 128 + 2 * kNarrowChunk * 4) + stages * k_blocks * kNarrowTile +
         2 * kNarrowTile + 1024 + 256;
}

template <typename T>
cudaError_t launch_narrow(const NarrowArgs &p, int blocks, bool early, cudaStream_t st);

// Ragged: the last chunk has hidden units past the last one.  Their products are zero only where x is finite, so h is
// set to it.  (A kernel of its own: a branch on it costs the others 2 to 7 us of 160 to 212 at a million tokens.)
template <typename T, int Act, bool Ragged>
__global__ void __launch_bounds__(kNarrowThreads, 1) narrow_kernel(const __grid_constant__ NarrowArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t *w_in = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t *w_out = w_in + p.chunks * p.k_blocks * kNarrowTile;
  uint8_t *xs = w_out + p.chunks * p.out_pad * 128;
  uint8_t *hs = xs + p.stages * p.k_blocks * kNarrowTile;
  float *bias = (float *)(hs + 2 * kNarrowTile);  // of a chunk: 64 of g, then 64 of u
  uint64_t *w_full = (uint64_t *)(bias + p.chunks * 2 * kNarrowChunk);
  uint64_t *s_full = w_full + 1, *s_empty = s_full + 3, *h_full = s_empty + 3, *h_empty = h_full + 2,
           *y_full = h_empty + 2, *y_empty = y_full + 2, *drained = y_empty + 2, *x_full = drained + 2,
           *x_empty = x_full + 4;
  uint32_t *tmem_slot = (uint32_t *)(x_empty + 4);
  volatile uint32_t *dead = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (p.tokens + 127) / 128, mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;

  if (threadIdx.x == 0) {
    mbar_init(w_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(h_full + i, 8);
      mbar_init(h_empty + i, 1);
      mbar_init(y_full + i, 1);
      mbar_init(y_empty + i, 8);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(x_full + i, 1);
      mbar_init(x_empty + i, 1);
    }
    mbar_init(drained, 1);
    mbar_init(drained + 1, 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
    tma_prefetch_map(&p.x);
    tma_prefetch_map(&p.w_in);
    tma_prefetch_map(&p.w_out);
  }
  if (warp == 1) tmem_alloc<1>(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int y_columns = p.out_pad <= 64 ? 64 : 128, sums = (512 - 2 * y_columns) / 128;
  const uint32_t tmem_y = tmem + 512 - 2 * y_columns;
  grid_dependency_wait();
  grid_dependency_launch();

  if (warp == 0) {
    if (elect_one()) {
      mbar_arrive_expect_tx(w_full, p.chunks * (p.k_blocks * kNarrowTile + p.out_pad * 128));
      for (int c = 0; c < p.chunks; ++c) {
        for (int k = 0; k < p.k_blocks; ++k) {
          uint8_t *to = w_in + (c * p.k_blocks + k) * kNarrowTile;  // 64 rows of Wg, then of Wu
          tma_load<1>(to, &p.w_in, k * 64, c * kNarrowChunk, 0, w_full);
          tma_load<1>(to + kNarrowTile / 2, &p.w_in, k * 64, c * kNarrowChunk, 1, w_full);
        }
        tma_load<1>(w_out + c * p.out_pad * 128, &p.w_out, c * kNarrowChunk, 0, 0, w_full);
      }
    }
    __syncwarp();
    int n = 0;
    for (; n < mine && !*dead; ++n) {
      const int s = n % p.stages;
      if (n >= p.stages && !__all_sync(0xffffffffu, mbar_wait_clocks(x_empty + s, (n / p.stages - 1) & 1))) {
        *dead = 1;
        break;
      }
      if (elect_one()) {
        mbar_arrive_expect_tx(x_full + s, p.k_blocks * kNarrowTile);
        const int row = (blockIdx.x + n * gridDim.x) * 128;
        for (int k = 0; k < p.k_blocks; ++k)
          tma_load<1>(xs + (s * p.k_blocks + k) * kNarrowTile, &p.x, k * 64, row, 0, x_full + s);
      }
      __syncwarp();
    }
    // every copy has landed before the block may end
    if (!mbar_wait_clocks(w_full, 0)) *dead = 1;
    for (int i = n > p.stages ? n - p.stages : 0; i < n; ++i)
      if (!mbar_wait_clocks(x_full + i % p.stages, (i / p.stages) & 1)) *dead = 1;
  } else if (warp == 1) {
    // Buffers and phases are counted along: with the divisions that find them from a chunk's number, and both
    // products in one warp, issuing them took 2,000 clocks a chunk and was what the others waited for.  A wait
    // for a fresh barrier's phase before its first is over at once.
    const uint32_t idesc = tc_idesc(p.f16, false, false, 128, 128);
    const uint64_t dx = tc_desc(xs, false, 0, 64), dw = tc_desc(w_in, false, 0, 64);
    bool lost = !__all_sync(0xffffffffu, mbar_wait_clocks(w_full, 0));
    int s = 0, b = 0;
    uint32_t x_phase = 0, s_phase = 1;
    for (int n = 0; n < mine && !lost; ++n) {
      lost = !__all_sync(0xffffffffu, mbar_wait_clocks(x_full + s, x_phase));
      for (int c = 0; c < p.chunks && !lost; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait_clocks(s_empty + b, s_phase))) {
          lost = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          uint64_t da = dx + s * p.k_blocks * (kNarrowTile >> 4), db = dw + c * p.k_blocks * (kNarrowTile >> 4);
          for (int k = 0; k < p.k_blocks; ++k, da += kNarrowTile >> 4, db += kNarrowTile >> 4)
#pragma unroll
            for (int q = 0; q < 4; ++q) tc_mma<1>(tmem + b * 128, da + q * 2, db + q * 2, idesc, k > 0 || q > 0);
          tc_commit<1>(s_full + b);
          if (c == p.chunks - 1) tc_commit<1>(x_empty + s);
        }
        __syncwarp();
        if (++b == sums) b = 0, s_phase ^= 1;
      }
      if (++s == p.stages) s = 0, x_phase ^= 1;
    }
    if (lost) {
      *dead = 1;
      if (elect_one()) tc_commit<1>(drained);  // the mma in flight still read shared memory
      __syncwarp();
      mbar_wait_clocks(drained, 0);
    }
  } else if (warp == 18) {
    const uint32_t idesc = tc_idesc(p.f16, false, false, 128, p.out_pad);
    const uint64_t dh = tc_desc(hs, false, 0, 64), dw = tc_desc(w_out, false, 0, 64);
    bool lost = !__all_sync(0xffffffffu, mbar_wait_clocks(w_full, 0));
    uint32_t b = 0, y = 0, h_phase = 0, y_phase = 3;  // y_phase: a bit for each of the two
    for (int n = 0; n < mine && !lost; ++n) {
      lost = !__all_sync(0xffffffffu, mbar_wait_clocks(y_empty + y, (y_phase >> y) & 1));
      y_phase ^= 1u << y;
      for (int c = 0; c < p.chunks && !lost; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait_clocks(h_full + b, h_phase))) {
          lost = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = dh + b * (kNarrowTile >> 4), db = dw + c * (p.out_pad * 128 >> 4);
#pragma unroll
          for (int q = 0; q < 4; ++q) tc_mma<1>(tmem_y + y * y_columns, da + q * 2, db + q * 2, idesc, c > 0 || q > 0);
          tc_commit<1>(h_empty + b);
          if (c == p.chunks - 1) tc_commit<1>(y_full + y);
        }
        __syncwarp();
        h_phase ^= b;
        b ^= 1;
      }
      y ^= 1;
    }
    if (lost) {
      *dead = 1;
      if (elect_one()) tc_commit<1>(drained + 1);
      __syncwarp();
      mbar_wait_clocks(drained + 1, 0);
    }
  } else {
    const int quarter = warp & 3, team = (warp - 2) >> 3, side = (warp - 2) >> 2 & 1;
    const int row = quarter * 32 + lane;  // of the tile
    const uint32_t lanes = (uint32_t)quarter << 21;
    if (p.b_in) {
      for (int i = threadIdx.x - 64; i < p.chunks * 2 * kNarrowChunk; i += 512) {
        const int f = i / (2 * kNarrowChunk) * kNarrowChunk + i % kNarrowChunk;
        const bool up = i / kNarrowChunk & 1;
        bias[i] = f < p.hidden ? to_f32(((const T *)p.b_in)[f + (up ? p.hidden : 0)]) : 0.f;
      }
      asm volatile("bar.sync 1, 512;" ::: "memory");  // the epilogue warps
    }
    // y of one tile: 16 columns at a time, the team's halves in turn
    auto finish = [&](int tile) {
      if (!__all_sync(0xffffffffu, mbar_wait_clocks(y_full + (tile & 1), (tile >> 1) & 1))) return false;
      tc_fence_after();
      const int64_t token = (blockIdx.x + (int64_t)tile * gridDim.x) * 128 + row;
      for (int c = side * 16; c < p.out_pad; c += 32) {
        float v[16];
        tmem_load16(tmem_y + lanes + (tile & 1) * y_columns + c, v);
        tmem_wait(v);
        const int count = p.out - c;
        if (token < p.tokens && count > 0) {
          if (p.b_out) add_bias<T, 16>(v, (const T *)p.b_out + c, count, p.b_out_vec);
          store_row<T, 16>((T *)p.y + token * p.out + c, v, count, p.y_vec);
        }
      }
      release_accumulator<1>(y_empty + (tile & 1), lane);
      return true;
    };
    int pending = -1;  // a tile whose y this team has to store, once the next tile's chunks are under way
    bool lost = false;
    const int total = mine * p.chunks;
    int tile = 0, c = team, b = team;  // chunk j is chunk c of its tile, its sums are in b
    uint32_t s_phase = 0, h_phase = 1;
    while (c >= p.chunks) c -= p.chunks, ++tile;
    for (int j = team; j < total && !lost; j += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait_clocks(s_full + b, s_phase))) {
        lost = true;
        break;
      }
      tc_fence_after();
      uint32_t ph[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float g[16], u[16], h[16];
        tmem_load16(tmem + lanes + b * 128 + side * 32 + q * 16, g);
        tmem_load16(tmem + lanes + b * 128 + 64 + side * 32 + q * 16, u);
        tmem_wait(g);
        tmem_wait(u);
        if (p.b_in) {
          const float4 *bg = (const float4 *)(bias + c * 2 * kNarrowChunk + side * 32 + q * 16);
          const float4 *bu = bg + kNarrowChunk / 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 a = bg[i], d = bu[i];
            const float2 g0 = add2(f2(g[4 * i], g[4 * i + 1]), f2(a.x, a.y)), g1 = add2(f2(g[4 * i + 2], g[4 * i + 3]), f2(a.z, a.w));
            const float2 u0 = add2(f2(u[4 * i], u[4 * i + 1]), f2(d.x, d.y)), u1 = add2(f2(u[4 * i + 2], u[4 * i + 3]), f2(d.z, d.w));
            g[4 * i] = g0.x, g[4 * i + 1] = g0.y, g[4 * i + 2] = g1.x, g[4 * i + 3] = g1.y;
            u[4 * i] = u0.x, u[4 * i + 1] = u0.y, u[4 * i + 2] = u1.x, u[4 * i + 3] = u1.y;
          }
        }
        if (q == 1) release_accumulator<1>(s_empty + b, lane);
        gate<Act, false, 16>(g, u, h);
        pack16<T>(h, ph[q]);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_clocks(h_empty + team, h_phase))) {
        lost = true;
        break;
      }
      h_phase ^= 1;
      if constexpr (Ragged)
        if (c == p.chunks - 1) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int unit = c * kNarrowChunk + side * 32 + q * 16 + 2 * i;
              ph[q][i] &= unit + 1 < p.hidden ? 0xFFFFFFFFu : unit < p.hidden ? 0xFFFFu : 0u;
            }
        }
      const StoreBox<128> box{hs + team * kNarrowTile + quarter * 4096, lane};
#pragma unroll
      for (int q = 0; q < 2; ++q) box.put(2 * side + q, ph[q]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(h_full + team);
      if (pending >= 0 && tile > pending) {
        lost = !finish(pending);
        pending = -1;
      }
      if ((tile & 1) == team && pending < 0) pending = tile;
      b += 2;
      if (b >= sums) b -= sums, s_phase ^= 1;
      c += 2;
      while (c >= p.chunks) c -= p.chunks, ++tile;
    }
    // tiles whose y is left: those of this team's parity that no later chunk of the team made it store
    if (!lost && pending >= 0) lost = !finish(pending);
    if (lost) *dead = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  tc_fence_after();
  if (warp == 1) tmem_free<1>(tmem, 512);
  if (threadIdx.x == 0 && *dead) atomicAdd_system(p.timeouts, 1u);
}

template <typename T, int Act, bool Ragged>
cudaError_t launch_narrow_act(const NarrowArgs &p, int blocks, bool early, cudaStream_t st) {
  const int smem = (int)narrow_bytes(p.k_blocks, p.chunks, p.out_pad, p.stages);
  auto kernel = narrow_kernel<T, Act, Ragged>;
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess) allowed.fetch_or(1ull << (dev & 63));
  }
  if (e != cudaSuccess) return e;
  LaunchConfig cfg(dim3(blocks), kNarrowThreads, smem, st, early);
  return cudaLaunchKernelEx(&cfg.c, kernel, p);
}

template <typename T, bool Ragged>
cudaError_t launch_narrow_ragged(const NarrowArgs &p, int blocks, bool early, cudaStream_t st) {
  switch (p.act) {
    case SLA_ACT_SILU: return launch_narrow_act<T, SLA_ACT_SILU, Ragged>(p, blocks, early, st);
    case SLA_ACT_GELU: return launch_narrow_act<T, SLA_ACT_GELU, Ragged>(p, blocks, early, st);
    case SLA_ACT_GELU_TANH: return launch_narrow_act<T, SLA_ACT_GELU_TANH, Ragged>(p, blocks, early, st);
    default: return launch_narrow_act<T, SLA_ACT_RELU, Ragged>(p, blocks, early, st);
  }
}

template <typename T>
cudaError_t launch_narrow_as(const NarrowArgs &p, int blocks, bool early, cudaStream_t st) {
  return p.hidden % kNarrowChunk ? launch_narrow_ragged<T, true>(p, blocks, early, st)
                                 : launch_narrow_ragged<T, false>(p, blocks, early, st);
}

}  // namespace sla
