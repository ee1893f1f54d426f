// The linear layer, forward and backward.
//
//   p = x W^T + b,  y = act(p) + r
//   dp = dy act'(p),  dx = dp W,  dW = dp^T x,  db = sum dp
//
// Three tensor-core products (sla_product.cuh): the forward one with activation, derivative and residual as its
// epilogue, the two of the backward pass in one launch.  Between them stands dp, which both read as an operand: without an
// activation it is dy itself, in place where TMA can read it; else a kernel forms it from dy and the kept act'(p), lays
// it out, and sums its columns on the way.  Up to kFewTokens tokens the forward product is sla_few.cuh's; layers of a few
// outputs are sla_skinny.cuh's (skinny).
//
// act'(p) is kept in float32.  16-bit tensor-core operands have to be 16 bits: dp = dy act'(p) is rounded once, beside the
// result's own rounding (0.0024 in relative L2 in bfloat16, 0.0003 in float16, where one rounding makes 0.0017 and 0.00021;
// act'(p) kept in 16 bits made it 0.0004, for two bytes a value less), unless the products are small (kTwoParts): then dp
// is two 16-bit parts, which the products take one after the other, and the result's rounding is the only one.  db is
// summed from dp before its rounding.
//
// Measured: 32,768 tokens, 1024 -> 2048 bfloat16, forward 88 us (1,560 TFLOP/s; tensor cores 74 % busy), dx and dW 161 (1,710;
// 87 %), the bias's sums 25 us between them (DRAM 70 %); 1,000,000 tokens, 64 -> 64 with a residual 87 us (0.65 of the copy
// rate: the epilogue's instructions); one token, 1024 -> 4096, 6 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "sla_dense.cuh"
#include "sla_few.cuh"
#include "sla_skinny.cuh"

namespace sla {
namespace {

int64_t out_pitch(const sla_layer *f) { return round_up(f->out, 16); }
bool activates(const sla_layer *f) { return f->activation != SLA_ACT_NONE; }

// Few outputs take sla_skinny.cuh's kernels.  Training step, there against here: float32, 302,053 tokens, 384 -> 5 507 us
// against 710, 1,000,000, 64 -> 1 136 against 645; 16 bits, 300,000 tokens, 384 -> 2 224 against 331, 384 -> 4 490 against 332
// (the arithmetic outweighs the copies of float32 data in parts), 1,000,000, 128 -> 4 423 against 477, 128 -> 8 550 against 498.
// The rule has no term for the tokens: float32, 2048 -> 8, whose weights are the most, 100 tokens 28 against 30, 608 36 against 38,
// 5000 64 against 86, 100,000 712 against 1147; 512 -> 4, 608 tokens 19 against 25; 64 -> 1, 608 tokens 13 against 19.
bool skinny(const sla_layer *f) {
  if (f->out > kSkinny || f->width > kSkinnyWidth) return false;
  return f->dtype == SLA_F32 || f->out <= 2 || f->out * f->width <= 512;
}

// Forward, 16-bit rows of some length, or of no alignment, are the tensor cores' all the same (384 -> 1: 55 us against 69; 63 -> 4:
// 122 against 155; 128 -> 2: 85 against 66), and up to kFewTokens tokens sla_few.cuh's.
bool skinny_y(const sla_layer *f) {
  return skinny(f) && (f->dtype == SLA_F32 || (f->width <= 128 && f->width % 8 == 0));
}

// Whether a forward call leaves packed copies of x and the weight: where TMA cannot read dense originals (the sizes alone
// decide, so that both calls and the layout of what is saved agree).
bool keeps_packed(const sla_layer *f) {
  return !skinny(f) && f->tokens > kFewTokens && (f->dtype == SLA_F32 || f->width % 8 != 0);
}

// act'(p) in float32, rows out_pitch apart, then packed copies of x and the weight.
struct SavedLayout {
  size_t x, w, total;
};

SavedLayout saved_layout(const sla_layer *f) {
  SavedLayout L;
  L.x = activates(f) ? align256((size_t)f->tokens * (size_t)out_pitch(f) * sizeof(float)) : 0;
  L.w = L.x + (keeps_packed(f) ? packed_bytes(f->tokens, f->width, f->dtype) : 0);
  L.total = L.w + (keeps_packed(f) ? packed_bytes(f->out, f->width, f->dtype) : 0);
  return L;
}

// Up to this many multiply-adds of each product of the backward pass dp has two parts: the second costs 4.3 GFLOP a product at
// most, and a gradient of few rows or columns does not average its roundings out (its error may be several times the result's
// rounding by chance).  Beyond, it would double the products' time.  relu's dp, dy or zero, is exact in one.
constexpr int64_t kTwoParts = (int64_t)1 << 31;

bool two_parts(const sla_layer *f) {
  if (!activates(f) || f->activation == SLA_ACT_RELU || f->dtype == SLA_F32 || skinny(f)) return false;
  const int64_t plane = f->width * f->out;  // at most 2^48
  return plane <= kTwoParts && f->tokens <= kTwoParts / plane;
}

// float16 gradients are as small as the loss makes them, and below 6e-5 float16 loses their digits (at 2e-6 dx and dW were 1.3 %
// off, in one part or two); act' of more than one may make them infinite.  So float16's dp is scaled by the power of two that takes the
// largest of dy to 2^14, and the products' sums by its inverse.  That reads dy once more: 32,768 tokens, 1024 -> 2048, silu, backward 265 -> 308 us,
// 2049 tokens, 250 -> 131 17 -> 23.
bool scales(const sla_layer *f) {
  return f->dtype == SLA_F16 && activates(f) && f->activation != SLA_ACT_RELU && !skinny(f);
}
constexpr int kLargestBlocks = 1024;

int sheets(const sla_layer *f) { return f->dtype == SLA_F32 ? 3 : 1; }

// What the tensor core drops of a running sum (2^-24 of it for every 16 products, on average over a sum that grows as its root
// 2/3 of that) grows with the sum's length: dW over 250,000 tokens, 2048 -> 2048, was too small by 1.3e-4 of itself in one
// sum, beside float16's rounding of 2.1e-4.  So 16-bit sums over tokens end after 2^14 products (4.1e-5 by that formula), and the parts
// are added in float32; their bytes are out / 2^13 of x's (that case's backward call: 2,480 us as before).  Sums over a row, which do not
// grow with the batch and whose parts are as many as the results, end after 2^16 (1.6e-4), float32's all after 512 (kRun).
int64_t longest(const sla_layer *f, int bits) { return f->dtype == SLA_F32 ? 0 : (int64_t)1 << bits; }
ProductSize y_size(const sla_layer *f) { return {f->tokens, f->out, f->width, 1, 1, 1, longest(f, 16)}; }
ProductSize dx_size(const sla_layer *f) { return {f->tokens, f->width, f->out, 1, 1, two_parts(f) ? 2 : 1, longest(f, 16)}; }
ProductSize dw_size(const sla_layer *f) { return {f->out, f->width, f->tokens, 1, 1, two_parts(f) ? 2 : 1, longest(f, 14)}; }

struct ForwardScratch {
  void *x, *w;
  float *parts, *runs;
  size_t total;
  ProductPlan plan;
};

ForwardScratch forward_scratch(const sla_layer *f, char *base) {
  Arena a{base};
  ForwardScratch s{};
  if (f->tokens <= kFewTokens || skinny_y(f)) return s;
  s.x = a.take(packed_bytes(f->tokens, f->width, f->dtype));
  s.w = a.take(packed_bytes(f->out, f->width, f->dtype));
  const ProductSize y = y_size(f);
  s.plan = plan_products(activates(f) ? kLinear : kAdd, &y, 1, sheets(f));
  s.parts = (float *)a.take(s.plan.partial[1]);
  s.runs = (float *)a.take(run_bytes(f->dtype));
  s.total = a.used;
  return s;
}

struct BackwardScratch {
  void *dp, *x, *w;
  float *columns, *parts, *runs;
  uint32_t *largest;  // of dy, block by block
  float *factor;
  size_t total;
  ProductPlan plan;
};

// Blocks of the backward kernel for few outputs, each of which leaves partial sums.
int skinny_blocks(const sla_layer *f) {
  int tpr = 1;
  while (tpr * 8 < f->width) tpr <<= 1;
  const int64_t rows = (int64_t)(256 / tpr) * kSkinnyBackRows;  // of a block's turn
  return (int)std::min<int64_t>(sm_count() * 2, (f->tokens + rows - 1) / rows);
}

BackwardScratch backward_scratch(const sla_layer *f, char *base) {
  Arena a{base};
  BackwardScratch s{};
  if (skinny(f)) {
    const size_t blocks = (size_t)skinny_blocks(f);
    s.parts = (float *)a.take(blocks * (size_t)(f->out * f->width) * sizeof(float));
    s.columns = (float *)a.take(blocks * (size_t)f->out * sizeof(float));
    s.total = a.used;
    return s;
  }
  s.dp = a.take((two_parts(f) ? 2 : 1) * packed_bytes(f->tokens, f->out, f->dtype));
  s.x = a.take(packed_bytes(f->tokens, f->width, f->dtype));
  s.w = a.take(packed_bytes(f->out, f->width, f->dtype));
  s.columns = (float *)a.take(kSumParts * sizeof(float) * (size_t)f->out);
  const ProductSize two[2] = {dx_size(f), dw_size(f)};
  s.plan = plan_products(kStore, two, 2, sheets(f));
  s.parts = (float *)a.take(s.plan.partial[2]);
  s.runs = (float *)a.take(run_bytes(f->dtype));
  if (scales(f)) {
    s.largest = (uint32_t *)a.take((kLargestBlocks + 1) * sizeof(uint32_t));
    s.factor = (float *)(s.largest + kLargestBlocks);
  }
  s.total = a.used;
  return s;
}

// The largest finite magnitude of the block's part of a float16 matrix, as its bits; eight columns of `tpr` threads a row.
__global__ void __launch_bounds__(256) largest_f16(int64_t rows, int64_t cols, const f16 *__restrict__ a, int64_t lda, int vec,
                                                   int tpr, uint32_t *__restrict__ largest) {
  __shared__ uint32_t sm[8];
  grid_dependency_wait();
  grid_dependency_launch();
  const int t = threadIdx.x & (tpr - 1), groups = 256 / tpr;
  const int64_t step = (int64_t)gridDim.x * groups;
  uint32_t most = 0;
  for (int64_t c = t * 8; c < cols; c += tpr * 8) {
    const int count = (int)(cols - c < 8 ? cols - c : 8);
#pragma unroll 8
    for (int64_t r = (int64_t)blockIdx.x * groups + threadIdx.x / tpr; r < rows; r += step) {
      const uint16_t *p = reinterpret_cast<const uint16_t *>(a) + r * lda + c;
      Pack<uint16_t, 8> q{};
      if (vec && count == 8) {
        q = *reinterpret_cast<const Pack<uint16_t, 8> *>(p);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < count) q.v[k] = p[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t bits = q.v[k] & 0x7fffu;
        most = max(most, bits < 0x7c00u ? bits : 0u);
      }
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x < 8) most = __reduce_max_sync(0xffu, sm[threadIdx.x]);
  if (threadIdx.x == 0) largest[blockIdx.x] = most;
}

// The power of two that takes the largest of all blocks to 2^14 .. 2^15.  `sm`: eight words.
__device__ __forceinline__ float scale_of(const uint32_t *largest, int count, uint32_t *sm) {
  uint32_t most = 0;
  for (int i = threadIdx.x; i < count; i += 256) most = max(most, largest[i]);
  most = __reduce_max_sync(0xffffffffu, most);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, sm[i]);
  if (most == 0) return 1.f;
  const int exponent = __float_as_int(to_f32(__ushort_as_half((unsigned short)most))) >> 23;  // with float32's bias of 127
  return __int_as_float((127 + 127 + 14 - exponent) << 23);
}

// dp = dy act'(p) as an operand (rows `pitch` apart, float32 in three sheets; two: 16 bits in two), eight columns a thread; a block covers 256 / tpr
// rows at a time, from row blockIdx.y * per, and leaves the column sums of its rows (parts: [gridDim.y][cols], or NULL).  float16: dp is
// scaled (scales), and `factor` becomes the scale's inverse.
template <typename T>
__global__ void __launch_bounds__(256) form_dp(int64_t rows, int64_t cols, const T *__restrict__ dy, int64_t lddy, int vec,
                                               const float *__restrict__ da, int64_t ldda, uint16_t *__restrict__ dp,
                                               int64_t pitch, int two, int tpr, int64_t per, float *__restrict__ parts,
                                               const uint32_t *__restrict__ largest, int blocks, float *__restrict__ factor) {
  __shared__ float sm[256 * 8];
  grid_dependency_wait();
  grid_dependency_launch();
  float scale = 1.f;
  if constexpr (std::is_same<T, f16>::value) {
    __shared__ uint32_t words[8];
    if (largest) {
      scale = scale_of(largest, blocks, words);
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *factor = 1.f / scale;
    }
  }
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = 256 / tpr;
  const int64_t c = (blockIdx.x * (int64_t)tpr + t) * 8;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
  const int count = (int)(cols - c < 8 ? cols - c : 8);
  float s[8] = {};
  if (c < cols)
#pragma unroll 2
    for (int64_t r = r0 + group; r < r1; r += groups) {
      float v[8], d[8];
      load_f32<float, 8>(da + r * ldda + c, d);
      if (vec && count == 8) {
        load_f32<T, 8>(dy + r * lddy + c, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < count ? to_f32(dy[r * lddy + c + k]) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = k < count ? v[k] * d[k] : 0.f;
        s[k] += v[k];
        if constexpr (std::is_same<T, f16>::value) v[k] *= scale;
      }
      store_operand<T, 8>(dp + r * pitch + c, rows * pitch, v, 8, true);
      if constexpr (sizeof(T) == 2)
        if (two) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float rest = v[k] - to_f32(from_f32<T>(v[k]));
            v[k] = isfinite(rest) ? rest : 0.f;  // an infinity or NaN stays in the first part
          }
          store_operand<T, 8>(dp + (rows + r) * pitch + c, rows * pitch, v, 8, true);
        }
    }
  if (!parts) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sm[threadIdx.x * 8 + k] = s[k];
  __syncthreads();
  for (int i = threadIdx.x; i < tpr * 8; i += 256) {
    const int64_t col = blockIdx.x * (int64_t)tpr * 8 + i;
    float sum = 0.f;
    for (int g = 0; g < groups; ++g) sum += sm[g * tpr * 8 + i];
    if (col < cols) parts[blockIdx.y * cols + col] = sum;
  }
}

// Calls run with O = 1, 2, 4 or 8, no fewer than the outputs.
template <typename F>
cudaError_t by_outputs(int64_t out, F &&run) {
  if (out <= 1) return run(std::integral_constant<int, 1>{});
  if (out <= 2) return run(std::integral_constant<int, 2>{});
  return out <= 4 ? run(std::integral_constant<int, 4>{}) : run(std::integral_constant<int, 8>{});
}

template <typename K>
cudaError_t launch_skinny(K kernel, const SkinnyArgs &p, int blocks, size_t smem, cudaStream_t st) {
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<blocks, 256, smem, st>>>(p);
  return cudaGetLastError();
}

// Whether rows of x (and dx) may be read in vectors of 16 bytes.
template <typename T>
bool skinny_vec(const SkinnyArgs &p) {
  constexpr int V = 16 / sizeof(T);
  return p.width % V == 0 && aligned(p.x, 16) && (p.tokens == 1 || p.ldx % V == 0) && aligned(p.dx, 16);
}

template <typename T>
cudaError_t run_skinny_forward(SkinnyArgs p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = skinny_vec<T>(p);
  p.tpr = 1;
  while (p.tpr < 32 && p.tpr * (vec ? V : 1) < p.width) p.tpr <<= 1;
  const int64_t rows = (int64_t)(256 / p.tpr) * kSkinnyRows;
  const int blocks = (int)std::min<int64_t>((p.tokens + rows - 1) / rows, sm_count() * 6);
  return by_outputs(p.out, [&](auto o) {
    constexpr int O = decltype(o)::value;
    const size_t smem = O * sizeof(float) * (size_t)skinny_padded(p.width, p.tpr, vec ? V : 1);
    return vec ? launch_skinny(skinny_forward<T, O, V>, p, blocks, smem, st)
               : launch_skinny(skinny_forward<T, O, 1>, p, blocks, smem, st);
  });
}

template <typename T>
cudaError_t run_skinny_backward(SkinnyArgs p, int blocks, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = skinny_vec<T>(p);
  p.tpr = 1;
  while (p.tpr * 8 < p.width) p.tpr <<= 1;
  return by_outputs(p.out, [&](auto o) {
    constexpr int O = decltype(o)::value;
    const size_t smem = O * sizeof(float) * (size_t)p.tpr * 8;
    return vec ? launch_skinny(skinny_backward<T, O, V>, p, blocks, smem, st)
               : launch_skinny(skinny_backward<T, O, 1>, p, blocks, smem, st);
  });
}

template <typename T>
sla_status forward(const sla_layer *f, const T *x, int64_t ldx, const T *w, const T *bias, const T *residual, int64_t ldr,
                   T *y, char *saved, const ForwardScratch &s, cudaStream_t st) {
  Call c{st};
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  c.timeouts = earlier.count;
  const SavedLayout L = saved_layout(f);
  float *da = saved && activates(f) ? (float *)saved : nullptr;
  if (f->tokens <= kFewTokens) {
    FewArgs p{};
    p.tokens = (int)f->tokens, p.n = (int)f->out, p.k = (int)f->width, p.act = f->activation;
    p.x = x, p.ldx = ldx, p.w = w, p.bias = bias;
    p.x_vec = aligned(x, 16) && (f->tokens == 1 || ldx % 8 == 0), p.w_vec = aligned(w, 16) && f->width % 8 == 0;
    p.c = y, p.g = da, p.ldg = out_pitch(f), p.residual = residual, p.ldr = ldr;
    c.launched(launch_few<T>(kLinear, p, st));
    return finish(c);
  }
  if (skinny_y(f)) {
    SkinnyArgs p{};
    p.tokens = f->tokens, p.width = (int)f->width, p.out = (int)f->out, p.act = f->activation;
    p.x = x, p.ldx = ldx, p.w = w, p.bias = bias, p.residual = residual, p.ldr = ldr, p.y = y;
    p.da = da, p.ldda = out_pitch(f);
    c.launched(run_skinny_forward<T>(p, st));
    return finish(c);
  }
  PackJobs packs;
  const Copy copy = saved && keeps_packed(f) ? kLeft : kOwn;
  const Operand ox = as_operand(packs, x, f->tokens, f->width, ldx, 1, copy ? saved + L.x : s.x, copy);
  const Operand ow = as_operand(packs, w, f->out, f->width, f->width, 1, copy ? saved + L.w : s.w, copy);
  run_packs<T>(c, packs);
  ProductJob job{y_size(f), ox, false, ow, false, {}, true};
  job.p.bias = bias, job.p.bias_vec = aligned(bias, 32);
  job.p.c = y, job.p.ldc = f->out, job.p.vec = vec_out(y, f->out);
  job.p.act = f->activation, job.p.g = da, job.p.ldg = out_pitch(f);
  job.p.residual = residual, job.p.ldr = ldr, job.p.residual_vec = vec_out(residual, ldr);
  // with nothing to add, the wide tiles' plain epilogue (32,768 tokens, 1024 -> 2048: 97 -> 90 us); on the narrow ones the
  // linear layer's has twice the warps
  const bool plain = !residual && kProductTiles[s.plan.shape].bn > 64;
  run_products<T>(c, activates(f) ? kLinear : plain ? kStore : kAdd, &job, 1, s.plan, s.parts, s.runs);
  return finish(c);
}

template <typename T>
sla_status backward(const sla_layer *f, const T *dy, int64_t lddy, const T *x, int64_t ldx, const T *w, const char *saved,
                    T *dx, T *dw, T *db, const BackwardScratch &s, cudaStream_t st) {
  Call c{st};
  const Expired earlier = expired();
  if (earlier.err != cudaSuccess) return fail(earlier.err);
  SLA_CHECK(report_expired(earlier));
  c.timeouts = earlier.count;
  if (skinny(f)) {
    const int blocks = skinny_blocks(f);
    SkinnyArgs p{};
    p.tokens = f->tokens, p.width = (int)f->width, p.out = (int)f->out;
    p.x = x, p.ldx = ldx, p.w = w, p.da = activates(f) ? (float *)const_cast<char *>(saved) : nullptr, p.ldda = out_pitch(f);
    p.dy = dy, p.lddy = lddy, p.dx = dx, p.parts = dw ? s.parts : nullptr, p.bias_parts = db ? s.columns : nullptr;
    c.launched(run_skinny_backward<T>(p, blocks, st));
    ColumnSums sums{c, nullptr, {}};
    if (dw) sums.add(s.parts, blocks, f->out * f->width, f->out * f->width, f->out * f->width, dw);
    if (db) sums.add(s.columns, blocks, f->out, f->out, f->out, db);
    sums.finish<T>();
    return finish(c);
  }
  const SavedLayout L = saved_layout(f);
  const Copy copy = keeps_packed(f) ? kKept : kOwn;
  char *sv = const_cast<char *>(saved);
  const bool products = dx || dw;
  PackJobs packs;
  Operand odp{}, ox{}, ow{};
  ColumnSums columns{c, s.columns, {}};
  if (products && !activates(f)) odp = as_operand(packs, dy, f->tokens, f->out, lddy, 1, s.dp);
  if (dw) ox = as_operand(packs, x, f->tokens, f->width, ldx, 1, copy ? sv + L.x : s.x, copy);
  if (dx) ow = as_operand(packs, w, f->out, f->width, f->width, 1, copy ? sv + L.w : s.w, copy);
  run_packs<T>(c, packs);
  if (activates(f)) {
    const int64_t pitch = round_up(f->out, 8), chunks = pitch / 8;
    int tpr = 1;
    while (tpr < 32 && tpr < chunks) tpr <<= 1;
    const int64_t tiles = (chunks + tpr - 1) / tpr;
    // enough blocks to fill the GPU, each with at least four turns of its threads
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kSumParts, sm_count() * 8 / tiles));
    const int64_t per = std::max<int64_t>(4 * (256 / tpr), (f->tokens + most - 1) / most);
    const int nparts = (int)((f->tokens + per - 1) / per);
    const int vec = aligned(dy, 16) && (f->tokens == 1 || lddy * sizeof(T) % 16 == 0);
    int blocks = 0;
    if constexpr (std::is_same<T, f16>::value)
      if (scales(f)) {
        int row = tpr;
        while (row < 256 && row < chunks) row <<= 1;
        blocks = (int)std::min<int64_t>(kLargestBlocks, (f->tokens + 256 / row - 1) / (256 / row));
        c.launch(largest_f16, dim3(blocks), 256, f->tokens, f->out, dy, lddy, vec, row, s.largest);
      }
    c.launch(form_dp<T>, dim3((unsigned)tiles, nparts), 256, f->tokens, f->out, dy, lddy, vec, (const float *)saved,
             out_pitch(f), (uint16_t *)s.dp, pitch, (int)two_parts(f), tpr, per, db ? s.columns : nullptr,
             (const uint32_t *)s.largest, blocks, s.factor);
    if (db) columns.add(s.columns, nparts, f->out, f->out, f->out, db);
    odp = {s.dp, f->out, f->tokens, two_parts(f) ? 2 : sheets_of<T>(), pitch, f->tokens * pitch};
  } else if (db) {
    columns.of<T, 1>(f->tokens, f->out, dy, lddy, 0, f->out, f->out, db);
  }
  columns.finish<T>();
  if (products) {
    auto job = [&](const ProductSize &size, bool a_mn, const Operand &b, T *out) {
      ProductJob j{size, odp, a_mn, b, true, {}, out != nullptr};
      j.p.c = out, j.p.ldc = size.n, j.p.vec = vec_out(out, size.n);
      j.same_b = two_parts(f);
      j.p.factor = s.factor;
      return j;
    };
    const ProductJob two[2] = {job(dx_size(f), false, ow, dx), job(dw_size(f), true, ox, dw)};
    run_products<T>(c, kStore, two, 2, s.plan, s.parts, s.runs);
  }
  return finish(c);
}

sla_status check_layer(const sla_layer *f) {
  if (!f) return SLA_INVALID_ARG;
  const int64_t most = (int64_t)1 << 24;
  if (f->tokens < 0 || f->tokens > (int64_t)1 << 30) return SLA_INVALID_ARG;
  if (f->width < 1 || f->width > most || f->out < 1 || f->out > most) return SLA_INVALID_ARG;
  if (!net_dtype(f->dtype) || f->activation < SLA_ACT_SILU || f->activation > SLA_ACT_NONE) return SLA_INVALID_ARG;
  return SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API size_t sla_linear_saved_bytes(const sla_layer *f) { return check_layer(f) == SLA_OK ? saved_layout(f).total : 0; }

SLA_API size_t sla_linear_workspace_bytes(const sla_layer *f) {
  return check_layer(f) == SLA_OK ? forward_scratch(f, nullptr).total : 0;
}

SLA_API size_t sla_linear_backward_workspace_bytes(const sla_layer *f) {
  return check_layer(f) == SLA_OK ? backward_scratch(f, nullptr).total : 0;
}

SLA_API sla_status sla_linear(const sla_layer *f, const void *x, int64_t ldx, const void *weight, const void *bias,
                              const void *residual, int64_t ldr, void *y, void *saved, size_t saved_bytes,
                              void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_layer(f));
  SLA_CHECK(check_matrix(x, f->tokens, f->width, ldx, f->dtype));
  SLA_CHECK(check_matrix(y, f->tokens, f->out, f->out, f->dtype));
  SLA_CHECK(check_matrix(weight, f->out, f->width, f->width, f->dtype));
  if (residual) SLA_CHECK(check_matrix(residual, f->tokens, f->out, ldr, f->dtype));
  if (!aligned(bias, net_size(f->dtype))) return SLA_INVALID_ARG;
  if (saved) SLA_CHECK(check_scratch(saved, saved_bytes, saved_layout(f).total));
  const ForwardScratch s = forward_scratch(f, (char *)workspace);
  SLA_CHECK(check_scratch(workspace, ws_bytes, s.total));
  if (f->tokens == 0) return SLA_OK;
#define SLA_LINEAR_FWD(T)                                                                                       \
  forward<T>(f, (const T *)x, ldx, (const T *)weight, (const T *)bias, (const T *)residual, ldr, (T *)y, \
             (char *)saved, s, (cudaStream_t)stream)
  return f->dtype == SLA_F32 ? SLA_LINEAR_FWD(float) : f->dtype == SLA_F16 ? SLA_LINEAR_FWD(f16) : SLA_LINEAR_FWD(bf16);
#undef SLA_LINEAR_FWD
}

SLA_API sla_status sla_linear_backward(const sla_layer *f, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                       const void *weight, const void *saved, size_t saved_bytes, void *dx,
                                       void *dweight, void *dbias, void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_layer(f));
  SLA_CHECK(check_matrix(dy, f->tokens, f->out, lddy, f->dtype));
  SLA_CHECK(check_matrix(x, f->tokens, f->width, ldx, f->dtype));
  SLA_CHECK(check_matrix(weight, f->out, f->width, f->width, f->dtype));
  const size_t e = net_size(f->dtype);
  for (const void *p : {(const void *)dx, (const void *)dweight, (const void *)dbias})
    if (!aligned(p, e)) return SLA_INVALID_ARG;
  SLA_CHECK(check_scratch(saved, saved_bytes, saved_layout(f).total));
  const BackwardScratch s = backward_scratch(f, (char *)workspace);
  SLA_CHECK(check_scratch(workspace, ws_bytes, s.total));
  cudaStream_t st = (cudaStream_t)stream;
  if (f->tokens == 0) {  // sums over no tokens
    cudaError_t err = dweight ? cudaMemsetAsync(dweight, 0, e * (size_t)(f->out * f->width), st) : cudaSuccess;
    if (err == cudaSuccess && dbias) err = cudaMemsetAsync(dbias, 0, e * (size_t)f->out, st);
    return err == cudaSuccess ? SLA_OK : fail(err);
  }
  if (!dx && !dweight && !dbias) return SLA_OK;
#define SLA_LINEAR_BWD(T)                                                                                             \
  backward<T>(f, (const T *)dy, lddy, (const T *)x, ldx, (const T *)weight, (const char *)saved, (T *)dx, (T *)dweight, \
              (T *)dbias, s, st)
  return f->dtype == SLA_F32 ? SLA_LINEAR_BWD(float) : f->dtype == SLA_F16 ? SLA_LINEAR_BWD(f16) : SLA_LINEAR_BWD(bf16);
#undef SLA_LINEAR_BWD
}

}  // extern "C"
