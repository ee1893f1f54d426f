// The gated feed-forward block, forward and backward.
//
//   [g u] = x w_in^T + b_in,  h = act(g) u,  y = h w_out^T + b_out
//   dh = dy w_out,  dg = dh u act'(g),  du = dh act(g)
//   dx = [dg du] w_in,  dw_in = [dg du]^T x,  dw_out = dy^T h,  db_in = sum [dg du],  db_out = sum dy
//
// Six matrix products; the activation, the product with u and their derivatives are the epilogues
// of the two products that make g, u and dh.
#include <cuda_runtime.h>

#include <algorithm>

#include "sla_act.cuh"
#include "sla_common.cuh"
#include "sla_host.h"
#include "sla_net.cuh"

namespace sla {
namespace {

constexpr int kTile = 64, kDepth = 16;

enum Epilogue { kStore, kGate, kGateBack };

// One product C = A B^T of matrices given by their strides, with its epilogue.
template <typename T>
struct Product {
  int64_t m, n, k;
  const T *a;
  int64_t a_row, a_col;  // A(i, k) = a[i * a_row + k * a_col]
  const T *b;
  int64_t b_row, b_col;
  int64_t b_up;     // kGate: offset of the up projection's rows in b
  const T *bias;    // kStore: [n]; kGate: [2 n]; NULL: none
  T *c;             // kStore: C; kGate: h
  int64_t ldc;
  T *gu;            // kGate: [m][ldgu], g and u (NULL: not kept); kGateBack: read
  int64_t ldgu;
  T *dgu;           // kGateBack: [m][ldgu]
  int act;
};

template <typename T, int EPI>
__global__ void __launch_bounds__(256) product_tile(Product<T> p) {
  constexpr int NB = EPI == kGate ? 2 : 1;
  __shared__ float sa[kDepth][kTile + 1], sb[NB][kDepth][kTile + 1];
  const int64_t m0 = blockIdx.y * (int64_t)kTile, n0 = blockIdx.x * (int64_t)kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[NB][4][4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
      const int r = i / kDepth, kk = i % kDepth;
      const bool kin = k0 + kk < p.k;
      sa[kk][r] = kin && m0 + r < p.m ? to_f32(p.a[(m0 + r) * p.a_row + (k0 + kk) * p.a_col]) : 0.f;
#pragma unroll
      for (int q = 0; q < NB; ++q)
        sb[q][kk][r] =
            kin && n0 + r < p.n ? to_f32(p.b[q * p.b_up + (n0 + r) * p.b_row + (k0 + kk) * p.b_col]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < NB; ++q)
            acc[q][i][j] = fmaf(sa[kk][ty + 16 * i], sb[q][kk][tx + 16 * j], acc[q][i][j]);
    __syncthreads();
  }
  constexpr bool fast = sizeof(T) == 2;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
      if (r >= p.m || c >= p.n) continue;
      if (EPI == kStore) {
        p.c[r * p.ldc + c] = from_f32<T>(acc[0][i][j] + (p.bias ? to_f32(p.bias[c]) : 0.f));
      } else if (EPI == kGate) {
        const float g = acc[0][i][j] + (p.bias ? to_f32(p.bias[c]) : 0.f);
        const float u = acc[NB - 1][i][j] + (p.bias ? to_f32(p.bias[p.n + c]) : 0.f);
        if (p.gu) {
          p.gu[r * p.ldgu + c] = from_f32<T>(g);
          p.gu[r * p.ldgu + p.n + c] = from_f32<T>(u);
        }
        p.c[r * p.ldc + c] = from_f32<T>(activate<fast>(p.act, g).a * u);
      } else {
        const float g = to_f32(p.gu[r * p.ldgu + c]), u = to_f32(p.gu[r * p.ldgu + p.n + c]);
        const ActValue v = activate<fast>(p.act, g);
        p.dgu[r * p.ldgu + c] = from_f32<T>(acc[0][i][j] * u * v.da);
        p.dgu[r * p.ldgu + p.n + c] = from_f32<T>(acc[0][i][j] * v.a);
      }
    }
}

// Column sums of a [rows][cols] matrix, one block for 32 columns.
template <typename T>
__global__ void __launch_bounds__(1024) column_sums(int64_t rows, int64_t cols, const T *__restrict__ a, int64_t lda,
                                                    T *__restrict__ out) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * 32ll + lane;
  float s = 0.f;
  if (c < cols)
    for (int64_t r = wy; r < rows; r += 32) s += to_f32(a[r * lda + c]);
  sm[wy][lane] = s;
  __syncthreads();
  if (wy == 0 && c < cols) {
    float t = 0.f;
    for (int i = 0; i < 32; ++i) t += sm[i][lane];
    out[c] = from_f32<T>(t);
  }
}

template <typename T, int EPI>
void launch(const Product<T> &p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.n + kTile - 1) / kTile), (unsigned)((p.m + kTile - 1) / kTile));
  product_tile<T, EPI><<<grid, 256, 0, st>>>(p);
}

int64_t pitch(int64_t n) { return (n + 7) / 8 * 8; }

struct FfnLayout {
  size_t h, total;
};

FfnLayout saved_layout(const sla_ffn *f) {
  FfnLayout L;
  const size_t e = net_size(f->dtype);
  L.h = align256(e * (size_t)f->tokens * (size_t)pitch(2 * f->hidden));
  L.total = L.h + align256(e * (size_t)f->tokens * (size_t)pitch(f->hidden));
  return L;
}

sla_status check_ffn(const sla_ffn *f) {
  if (!f) return SLA_INVALID_ARG;
  const int64_t most = (int64_t)1 << 24;
  if (f->tokens < 0 || f->tokens > ((int64_t)1 << 31) - 1) return SLA_INVALID_ARG;
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

template <typename T>
sla_status forward(const sla_ffn *f, const T *x, int64_t ldx, const T *w_in, const T *b_in, const T *w_out,
                   const T *b_out, T *y, char *saved, char *ws, cudaStream_t st) {
  const FfnLayout L = saved_layout(f);
  T *h = (T *)(saved ? saved + L.h : ws);
  Product<T> p{};
  p.m = f->tokens, p.n = f->hidden, p.k = f->width;
  p.a = x, p.a_row = ldx, p.a_col = 1;
  p.b = w_in, p.b_row = f->width, p.b_col = 1, p.b_up = f->hidden * f->width;
  p.bias = b_in, p.c = h, p.ldc = pitch(f->hidden), p.gu = (T *)saved, p.ldgu = pitch(2 * f->hidden);
  p.act = f->activation;
  launch<T, kGate>(p, st);
  Product<T> q{};
  q.m = f->tokens, q.n = f->out, q.k = f->hidden;
  q.a = h, q.a_row = pitch(f->hidden), q.a_col = 1;
  q.b = w_out, q.b_row = f->hidden, q.b_col = 1;
  q.bias = b_out, q.c = y, q.ldc = f->out;
  launch<T, kStore>(q, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(e);
  count_launches(2);
  return SLA_OK;
}

template <typename T>
sla_status backward(const sla_ffn *f, const T *dy, int64_t lddy, const T *x, int64_t ldx, const T *w_in,
                    const T *w_out, const char *saved, T *dx, T *dw_in, T *dw_out, T *db_in, T *db_out, char *ws,
                    cudaStream_t st) {
  const FfnLayout L = saved_layout(f);
  const T *h = (const T *)(saved + L.h);
  T *dgu = (T *)ws;
  const int64_t ldgu = pitch(2 * f->hidden);
  uint64_t launches = 0;
  if (dx || dw_in || db_in) {
    Product<T> p{};
    p.m = f->tokens, p.n = f->hidden, p.k = f->out;
    p.a = dy, p.a_row = lddy, p.a_col = 1;
    p.b = w_out, p.b_row = 1, p.b_col = f->hidden;
    p.gu = (T *)saved, p.ldgu = ldgu, p.dgu = dgu, p.act = f->activation;
    launch<T, kGateBack>(p, st);
    ++launches;
  }
  auto product = [&](int64_t m, int64_t n, int64_t k, const T *a, int64_t ar, int64_t ac, const T *b, int64_t br,
                     int64_t bc, T *c) {
    Product<T> p{};
    p.m = m, p.n = n, p.k = k, p.a = a, p.a_row = ar, p.a_col = ac, p.b = b, p.b_row = br, p.b_col = bc;
    p.c = c, p.ldc = n;
    launch<T, kStore>(p, st);
    ++launches;
  };
  if (dx) product(f->tokens, f->width, 2 * f->hidden, dgu, ldgu, 1, w_in, 1, f->width, dx);
  if (dw_in) product(2 * f->hidden, f->width, f->tokens, dgu, 1, ldgu, x, 1, ldx, dw_in);
  if (dw_out) product(f->out, f->hidden, f->tokens, dy, 1, lddy, h, 1, pitch(f->hidden), dw_out);
  if (db_in) {
    column_sums<T><<<(unsigned)((2 * f->hidden + 31) / 32), 1024, 0, st>>>(f->tokens, 2 * f->hidden, dgu, ldgu, db_in);
    ++launches;
  }
  if (db_out) {
    column_sums<T><<<(unsigned)((f->out + 31) / 32), 1024, 0, st>>>(f->tokens, f->out, dy, lddy, db_out);
    ++launches;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(e);
  count_launches(launches);
  return SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

SLA_API size_t sla_gated_ffn_saved_bytes(const sla_ffn *f) {
  return check_ffn(f) == SLA_OK ? saved_layout(f).total : 0;
}

SLA_API size_t sla_gated_ffn_workspace_bytes(const sla_ffn *f) {
  if (check_ffn(f) != SLA_OK) return 0;
  return saved_layout(f).total - saved_layout(f).h;
}

SLA_API size_t sla_gated_ffn_backward_workspace_bytes(const sla_ffn *f) {
  if (check_ffn(f) != SLA_OK) return 0;
  return saved_layout(f).h;
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
  if (saved) SLA_CHECK(check_scratch(saved, saved_bytes, sla_gated_ffn_saved_bytes(f)));
  SLA_CHECK(check_scratch(workspace, ws_bytes, sla_gated_ffn_workspace_bytes(f)));
  if (f->tokens == 0) return SLA_OK;
#define SLA_FFN_FWD(T)                                                                                             \
  forward<T>(f, (const T *)x, ldx, (const T *)w_in, (const T *)b_in, (const T *)w_out, (const T *)b_out, (T *)y, \
             (char *)saved, (char *)workspace, (cudaStream_t)stream)
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
  SLA_CHECK(check_scratch(saved, saved_bytes, sla_gated_ffn_saved_bytes(f)));
  SLA_CHECK(check_scratch(workspace, ws_bytes, sla_gated_ffn_backward_workspace_bytes(f)));
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
              (T *)dx, (T *)dw_in, (T *)dw_out, (T *)db_in, (T *)db_out, (char *)workspace, st)
  return f->dtype == SLA_F32 ? SLA_FFN_BWD(float) : f->dtype == SLA_F16 ? SLA_FFN_BWD(f16) : SLA_FFN_BWD(bf16);
#undef SLA_FFN_BWD
}

}  // extern "C"
