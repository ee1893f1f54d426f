// The gated feed-forward block, forward and backward.
//
//   [g u] = x w_in^T + b_in,  h = act(g) u,  y = h w_out^T + b_out
//   dh = dy w_out,  dg = dh u act'(g),  du = dh act(g)
//   dx = [dg du] w_in,  dw_in = [dg du]^T x,  dw_out = dy^T h,  db_in = sum [dg du],  db_out = sum dy
//
// Six tensor-core products (sla_product.cuh); the activation, the product with u and their
// derivatives are the epilogues of the two that make g, u and dh.  How operands are laid out and products
// planned is in sla_dense.cuh.
#include <cuda_runtime.h>

#include <algorithm>

#include "sla_dense.cuh"
#include "sla_few.cuh"
#include "sla_narrow.cuh"

namespace sla {
namespace {

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
  w.runs = (float *)a.take(run_bytes(f->dtype));
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
  w.runs = (float *)a.take(run_bytes(f->dtype));
  w.total = a.used;
  return w;
}

// ------------------------------------------------------------------ narrow blocks

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

}  // extern "C"
