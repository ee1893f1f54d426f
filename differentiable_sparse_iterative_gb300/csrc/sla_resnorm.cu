// The residual norm's C entries, and its sums over the rows (kernels: sla_resnorm.cuh).
#include "sla_resnorm.cuh"

#include <cmath>
#include <initializer_list>

namespace sla {
namespace {

struct SumTargets {
  void *p[kNormSums];
};

// The five sums from the blocks' partial sums, in a fixed order.
template <typename P>
__global__ void __launch_bounds__(1024) resnorm_reduce(int nparts, int64_t width, const float *__restrict__ parts,
                                                       const __grid_constant__ SumTargets to) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5, which = blockIdx.y;
  const int64_t c = blockIdx.x * 32ll + lane;
  P *out = (P *)to.p[which];
  grid_dependency_wait();
  if (!out) return;
  float s = 0.f;
  if (c < width)
#pragma unroll 8
    for (int p = wy; p < nparts; p += 32) s += parts[((int64_t)p * kNormSums + which) * width + c];
  sm[wy][lane] = s;
  __syncthreads();
  if (wy == 0 && c < width) {
    float r = 0.f;
    for (int i = 0; i < 32; ++i) r += sm[i][lane];
    out[c] = from_f32<P>(r);
  }
}

constexpr int kMostClasses = 8;

// Blocks of the backward kernel, each of which leaves partial sums.
int backward_grid(int64_t rows, int64_t width, int classes) {
  const ResNormPlan pl = resnorm_plan(width);
  if (!pl.columns) return (int)std::max<int64_t>(1, std::min<int64_t>(kAnyParts, (rows + 127) / 128));
  return resnorm_grid(pl, rows, pl.block / pl.tpr, classes, 512);
}

size_t row_sum_bytes(int64_t rows, int64_t width) {
  return resnorm_plan(width).columns ? 0 : align256(2 * (size_t)rows * sizeof(float));
}

size_t backward_bytes(int64_t rows, int64_t width) {
  int blocks = 0;  // the most that any layout of these rows takes
  for (int classes = 1; classes <= kMostClasses; classes *= 2) blocks = std::max(blocks, backward_grid(rows, width, classes));
  return row_sum_bytes(rows, width) + align256((size_t)blocks * kNormSums * (size_t)width * sizeof(float));
}

sla_status check_resnorm(const sla_resnorm *n) {
  if (!n) return SLA_INVALID_ARG;
  if (n->rows < 0 || n->rows > ((int64_t)1 << 31) - 1 || n->width < 1 || n->width > (int64_t)1 << 24)
    return SLA_INVALID_ARG;
  if (!net_dtype(n->dtype) || (n->param_dtype != n->dtype && n->param_dtype != SLA_F32)) return SLA_INVALID_ARG;
  if (n->reserved != 0) return SLA_INVALID_ARG;
  if (n->norm != SLA_NORM_LAYER && n->norm != SLA_NORM_RMS) return SLA_INVALID_ARG;
  if (n->post_norm != 0 && n->post_norm != 1) return SLA_INVALID_ARG;
  if (n->gate_act < SLA_GATE_NONE || n->gate_act > SLA_GATE_SILU) return SLA_INVALID_ARG;
  return n->eps >= 0.0 && std::isfinite(n->eps) ? SLA_OK : SLA_INVALID_ARG;
}

// A matrix of rows `ld` elements apart, which may be absent.
sla_status check_rows(const void *p, const sla_resnorm *n, int64_t ld, bool needed) {
  if (n->rows == 0 || (!p && !needed)) return SLA_OK;
  if (!p || !aligned(p, net_size(n->dtype))) return SLA_INVALID_ARG;
  // (the kernels count a row's bytes in 32 bits)
  return n->rows == 1 || (ld >= n->width && ld < (int64_t)1 << 29) ? SLA_OK : SLA_INVALID_ARG;
}

ResNormArgs resnorm_args(const sla_resnorm *n, const void *gate) {
  ResNormArgs p{};
  p.rows = n->rows, p.width = n->width;
  p.rms = n->norm == SLA_NORM_RMS, p.post = n->post_norm, p.eps = (float)n->eps;
  p.act = !gate ? kNoGate : n->gate_act == SLA_GATE_SILU ? kGateSilu : n->gate_act == SLA_GATE_SIGMOID ? kGateSigmoid : kGateNone;
  return p;
}

uint32_t row_bytes(const sla_resnorm *n, int64_t ld) { return n->rows == 1 ? 0 : (uint32_t)((size_t)ld * net_size(n->dtype)); }

// How the rows of a call's arrays lie behind 16-byte boundaries, and whether they all lie alike.
struct RowLayout {
  const sla_resnorm *n;
  int vec, shift = 0, step = 0;
  bool met = false, alike = true;
  explicit RowLayout(const sla_resnorm *n_) : n(n_), vec((int)(16 / net_size(n_->dtype))) {}
  RowLayout &with(const void *p, int64_t ld) {
    if (!p) return *this;
    const int s = (int)((uintptr_t)p % 16 / net_size(n->dtype)), d = n->rows == 1 ? 0 : (int)(ld % vec);
    if (!met) shift = s, step = d, met = true;
    alike = alike && s == shift && d == step;
    return *this;
  }
  // Rows r, r + classes, ... start at the same place behind a boundary.  (The plan leaves room for a row that starts behind one
  // only where the width says that rows may.)
  bool put(ResNormArgs &p) const {
    p.shift = shift, p.step = step, p.classes = 1;
    while (p.classes * step % vec) p.classes *= 2;
    return alike && (n->width % 8 != 0 || (shift == 0 && step == 0));
  }
};

template <typename F>
cudaError_t by_type(const sla_resnorm *n, F &&f) {
  if (n->dtype == SLA_F32) return f(float{}, float{});
  if (n->dtype == SLA_F16) return n->param_dtype == SLA_F16 ? f(f16{}, f16{}) : f(f16{}, float{});
  return n->param_dtype == SLA_BF16 ? f(bf16{}, bf16{}) : f(bf16{}, float{});
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API sla_status sla_residual_norm(const sla_resnorm *n, const void *block, int64_t ldblock, const void *z, int64_t ldz,
                                     const void *gate, int64_t ldgate, const void *scale, const void *post_weight,
                                     const void *post_bias, const void *weight, const void *bias, void *z_out, void *y,
                                     float *stats, void *stream) {
  SLA_CHECK(check_resnorm(n));
  SLA_CHECK(check_rows(block, n, ldblock, true));
  SLA_CHECK(check_rows(z, n, ldz, true));
  SLA_CHECK(check_rows(gate, n, ldgate, false));
  SLA_CHECK(check_rows(z_out, n, n->width, true));
  SLA_CHECK(check_rows(y, n, n->width, false));
  const size_t ps = net_size(n->param_dtype);
  for (const void *p : {scale, post_weight, post_bias, weight, bias})
    if (!aligned(p, ps)) return SLA_INVALID_ARG;
  if (!aligned(stats, 16)) return SLA_INVALID_ARG;
  if (n->rows == 0) return SLA_OK;
  ResNormArgs p = resnorm_args(n, gate);
  p.f = block, p.ldf = ldblock, p.z = z, p.ldz = ldz, p.gate = gate, p.ldg = ldgate;
  p.scale = scale, p.w1 = post_weight, p.b1 = post_bias, p.w2 = weight, p.b2 = bias;
  p.znew = z_out, p.y = y, p.stats = (float4 *)stats;
  p.bf = row_bytes(n, ldblock), p.bz = row_bytes(n, ldz), p.bg = row_bytes(n, ldgate), p.bw = row_bytes(n, n->width);
  const bool vec = RowLayout(n).with(block, ldblock).with(z, ldz).with(gate, ldgate).with(z_out, n->width).with(y, n->width).put(p);
  const cudaError_t e = by_type(n, [&](auto t, auto q) {
    return resnorm_forward<decltype(t), decltype(q)>(p, vec, (cudaStream_t)stream);
  });
  if (e != cudaSuccess) return fail(e);
  count_launches(1);
  return SLA_OK;
}

SLA_API size_t sla_residual_norm_backward_workspace_bytes(const sla_resnorm *n) {
  return check_resnorm(n) == SLA_OK ? backward_bytes(n->rows, n->width) : 0;
}

SLA_API sla_status sla_residual_norm_backward(const sla_resnorm *n, const void *dz_out, int64_t lddz, const void *dy,
                                              int64_t lddy, const void *block, int64_t ldblock, const void *z, int64_t ldz,
                                              const void *gate, int64_t ldgate, const void *scale,
                                              const void *post_weight, const void *post_bias, const void *weight,
                                              const float *stats, void *dblock, void *dz, void *dgate, void *dscale,
                                              void *dpost_weight, void *dpost_bias, void *dweight, void *dbias,
                                              void *workspace, size_t ws_bytes, void *stream) {
  SLA_CHECK(check_resnorm(n));
  SLA_CHECK(check_rows(dz_out, n, lddz, false));
  SLA_CHECK(check_rows(dy, n, lddy, false));
  SLA_CHECK(check_rows(block, n, ldblock, true));
  SLA_CHECK(check_rows(z, n, ldz, true));
  SLA_CHECK(check_rows(gate, n, ldgate, false));
  for (const void *p : {(const void *)dblock, (const void *)dz, (const void *)dgate})
    if (!aligned(p, net_size(n->dtype))) return SLA_INVALID_ARG;
  const size_t ps = net_size(n->param_dtype);
  for (const void *p : {scale, post_weight, post_bias, weight, (const void *)dscale, (const void *)dpost_weight,
                        (const void *)dpost_bias, (const void *)dweight, (const void *)dbias})
    if (!aligned(p, ps)) return SLA_INVALID_ARG;
  if (!aligned(stats, 16) || (n->rows > 0 && !stats) || (dgate && !gate && n->rows > 0)) return SLA_INVALID_ARG;
  const SumTargets to{{dscale, dpost_weight, dpost_bias, dweight, dbias}};
  const bool sums = dscale || dpost_weight || dpost_bias || dweight || dbias;
  // (a workspace is only needed for sums)
  if (sums) {
    if (!workspace || !aligned(workspace, 256)) return SLA_INVALID_ARG;
    if (ws_bytes < backward_bytes(n->rows, n->width)) return SLA_WORKSPACE_TOO_SMALL;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (n->rows == 0) {  // sums over no rows
    for (void *p : to.p)
      if (p) {
        const cudaError_t e = cudaMemsetAsync(p, 0, ps * (size_t)n->width, st);
        if (e != cudaSuccess) return fail(e);
      }
    return SLA_OK;
  }
  if (!sums && !dblock && !dz && !dgate) return SLA_OK;
  ResNormArgs p = resnorm_args(n, gate);
  p.f = block, p.ldf = ldblock, p.z = z, p.ldz = ldz, p.gate = gate, p.ldg = ldgate;
  p.scale = scale, p.w1 = post_weight, p.b1 = post_bias, p.w2 = weight;
  p.stats = (float4 *)const_cast<float *>(stats), p.dz = dz_out, p.lddz = lddz, p.dy = dy, p.lddy = lddy;
  p.df = dblock, p.dz_in = dz, p.dgate = dgate;
  p.bf = row_bytes(n, ldblock), p.bz = row_bytes(n, ldz), p.bg = row_bytes(n, ldgate), p.bw = row_bytes(n, n->width);
  p.bdz = row_bytes(n, lddz), p.bdy = row_bytes(n, lddy);
  if (sums) {
    const size_t first = row_sum_bytes(n->rows, n->width);
    p.row_sums = first ? (float *)workspace : nullptr;
    p.parts = (float *)((char *)workspace + first);
  }
  const bool vec = RowLayout(n).with(dz_out, lddz).with(dy, lddy).with(block, ldblock).with(z, ldz).with(gate, ldgate)
                       .with(dblock, n->width).with(dz, n->width).with(dgate, n->width).put(p);
  const int grid = backward_grid(n->rows, n->width, vec ? p.classes : 1);
  cudaError_t e = by_type(n, [&](auto t, auto q) {
    return resnorm_backward<decltype(t), decltype(q)>(p, vec, grid, st);
  });
  uint64_t launches = 1;
  if (e == cudaSuccess && sums) {
    LaunchConfig cfg(dim3((unsigned)((n->width + 31) / 32), kNormSums), 1024, 0, st, true);
    e = by_type(n, [&](auto, auto q) {
      return cudaLaunchKernelEx(&cfg.c, resnorm_reduce<decltype(q)>, grid, n->width, (const float *)p.parts, to);
    });
    launches += resnorm_plan(n->width).columns ? 1 : 2;
  }
  if (e != cudaSuccess) return fail(e);
  count_launches(launches);
  return SLA_OK;
}

}  // extern "C"
