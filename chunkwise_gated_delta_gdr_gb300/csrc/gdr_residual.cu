// gdr_residual.cu -- what lies between two layers: a layer's output goes into the residual, and
// the sum is normed for the next layer; forward and backward. p = y or its norm uy wp, a = act(z)
// or 1, s a number or a channel's weight:
//   r' = r + s a p,  out = u w,  u = r' rho,  rho = 1 / sqrt(mean(r'^2) + eps)
//   g = dr' + rho (c - u mean(c u)),  c = dout w,  dw = sum dout u,  dr = g,  ds = sum g a p
//   dz = g s p a',  dp = g s a,  dy = dp, or behind a norm: dwp = sum dp uy,
//   dy = ry (dp wp - uy mean(dp wp uy))
//
// Every tensor is read once and written once: bound by HBM where there is enough of it, by the
// chain load - sums over the row - store of one row below. Measured on one GB300, bf16, a pass
// among others (a plain copy: 6.70 TB/s):
//   training step, 2 x 8192 x 4096: 196 us, 6.2 TB/s (forward 77, backward 104)
//   training step, 4096 x 1536, residual in 32 bits, y normed, gated and scaled per channel: 71 us
//   (22, 41, 8: 2.7 and 5.4 rows a block with one stage of copies, no row ahead: two would take 210
//   KB of an SM for its five blocks)
//   training step, 3 x 1021 x 777 in 32 bits, likewise without a row ahead: 50 us
//   training step, 2 x 8192 x 4096, residual in 32 bits 396 us, all in 32 bits 567: 4.7 and 4.3 TB/s
//   64 decode tokens x 2048 channels: 3.3 us
#include "gdr_norm.cuh"

namespace gdr {
namespace ops {
namespace {

struct ResArgs {
  View r, y, z, d, dr;           // r: the residual, backward: r'; d, dr: gradients of out and r'
  const float *w, *wp, *sv;      // [D] or null; sv: the scale per channel
  void *out, *r_out;             // forward; r_out null without y
  void *o_dr, *o_dy, *o_dz;      // backward, dense (o_dy, o_dz null without y, z)
  float* part;                   // [3][blocks][D]: of w, wp, sv; null: none
  int B, T, D, tokens, kind, post, want_p, want_s;
  int r_bf16, y_bf16, out_bf16;  // y_bf16: of y and z; out_bf16: of out and d
  int has_y, has_z, has_dr;
  int pieces, stages, groups;
  int flat;                      // the views' tokens are one stride apart, over batch rows too
  float eps, inv_d, s;
};

// The types of a call (residual; y and gate; out): the usual ones known when the kernel is
// compiled, the others from its arguments.
enum { kAnyTypes, kAllBf16, kF32Residual, kAllF32 };
template <int TY>
struct Types {
  __device__ static constexpr int r(const ResArgs& a) { return TY == kAnyTypes ? a.r_bf16 : TY == kAllBf16; }
  __device__ static constexpr int y(const ResArgs& a) { return TY == kAnyTypes ? a.y_bf16 : TY != kAllF32; }
  __device__ static constexpr int out(const ResArgs& a) { return TY == kAnyTypes ? a.out_bf16 : TY != kAllF32; }
};

// (With 16 elements a thread, 64 registers: an SM holds the kFwdPerSm threads that the plan counts on.)
template <class S, int TY>
__global__ void __launch_bounds__(kMaxThreads, S::N <= 16 && !S::kGroups ? 2 : 1) residual_fwd_kernel(ResArgs a) {
  constexpr int V = S::V, NV = S::NV, N = S::N;
  extern __shared__ __align__(16) char places[];
  __shared__ Red red;
  const Walk w = walk_of<S::LANES>(a.tokens, 1, a.groups);
  const int phase = S::SHIFT ? (int)(((long long)w.tok * a.D) & 7) : 0;
  const Ahead ahead(places, a.pieces, a.stages);
  Row<S, false> rr;                              // may be the result's own memory
  Row<S, true> ry, rz;
  const int r_bf16 = Types<TY>::r(a), y_bf16 = Types<TY>::y(a), out_bf16 = Types<TY>::out(a);
  auto has = [&](int it) { return (S::LANES == 0 || w.on) && w.tok + it * w.step < a.tokens; };
  auto locate = [&](int it) {
    const int tok = w.tok + it * w.step, rp = NV * (r_bf16 ? 1 : 2), yp = NV * (y_bf16 ? 1 : 2);
    rr.set(a.r.p, a.r.at(tok, a.T, a.flat, 0), r_bf16, 0);
    ry.set(a.y.p, a.y.at(tok, a.T, a.flat, 0), y_bf16, rp);
    rz.set(a.z.p, a.z.at(tok, a.T, a.flat, 0), y_bf16, rp + yp);
  };
  auto fetch = [&](int it, int stage) {
    if constexpr (S::kAhead || S::kRegs) {
      if (has(it)) {
        const uint32_t at = ahead.of(stage);
        locate(it);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int i = (c * w.threads + w.tid) * V - phase;
          if (i < a.D) {
            rr.fetch(ahead, at, c, i, a.D);
            if (a.has_y) ry.fetch(ahead, at, c, i, a.D);
            if (a.has_z) rz.fetch(ahead, at, c, i, a.D);
          }
        }
      }
      if constexpr (S::kAhead) ptx::cp_async_commit();
    }
  };
  begin_behind();
  for (int i = 0; i + 1 < a.stages; ++i) fetch(i, i);
  int turn = 0, stage = 0;
  for (int it = 0; it < w.iters; ++it, stage = stage + 1 == a.stages ? 0 : stage + 1) {
    rr.advance(), ry.advance(), rz.advance();
    fetch(it + a.stages - 1, stage == 0 ? a.stages - 1 : stage - 1);
    if constexpr (S::kAhead) ahead.wait();
    const bool on = S::LANES == 0 || has(it);
    if (S::LANES == 0 && !has(it)) break;        // the whole block
    if (!(S::kAhead || S::kRegs)) locate(it);
    const uint32_t at = ahead.of(stage);
    const size_t dense = (size_t)(w.tok + it * w.step) * a.D;
    float py = 1.f, s[1];
    if (a.post) {
      s[0] = 0.f;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        group_at<S>(w, c, a.D, ry);
        const int i = (c * w.threads + w.tid) * V - phase;
        if (!on || i >= a.D) continue;
        float y[V];
        ry.get(ahead, at, c, i, a.D, y);
        s[0] += dot_run<V>(y, y);
      }
      row_sum<S::LANES, 1>(s, red, turn);
      py = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
    }
    float r[N];
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      group_at<S>(w, c, a.D, rr);
      if (a.has_y) group_at<S>(w, c, a.D, ry);
      if (a.has_z) group_at<S>(w, c, a.D, rz);
      const int i = (c * w.threads + w.tid) * V - phase;
      if (!on || i >= a.D) continue;
      float* x = r + c * V;
      rr.get(ahead, at, c, i, a.D, x);
      if (a.has_y) {
        float y[V], k[V];
        ry.get(ahead, at, c, i, a.D, y);
        if (a.post) scale_run<V>(y, y, py);
        if (a.wp) {
          load_shared<S>(a.wp, i, a.D, k);
          mul_run<V>(y, y, k);
        }
        if (a.has_z) {
          rz.get(ahead, at, c, i, a.D, k);
          float g[V];
          gate_sigma<V>(g, k, a.kind);
          gate_open<V>(k, g, k, a.kind);
          mul_run<V>(y, y, k);
        }
        if (a.sv) {
          load_shared<S>(a.sv, i, a.D, k);
          fma_run<V>(x, k, y, x);
        } else {
          fma_run<V>(x, y, a.s, x);
        }
        store_row<S>(a.r_out, dense, i, a.D, r_bf16, x);
      }
      s[0] += dot_run<V>(x, x);
    }
    row_sum<S::LANES, 1>(s, red, turn);
    const float rho = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int i = (c * w.threads + w.tid) * V - phase;
      if (!on || i >= a.D) continue;
      float o[V], k[V];
      scale_run<V>(o, r + c * V, rho);
      if (a.w) {
        load_shared<S>(a.w, i, a.D, k);
        mul_run<V>(o, o, k);
      }
      store_row<S>(a.out, dense, i, a.D, out_bf16, o);
    }
  }
}

// FULL: y goes through a norm, a gate or a scale per channel; without, dy = s g.
template <class S, int TY, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, S::N <= 16 && !S::kGroups && !FULL ? 2 : 1) residual_bwd_kernel(ResArgs a) {
  constexpr int V = S::V, NV = S::NV, N = S::N;
  extern __shared__ __align__(16) char places[];
  __shared__ Red red;
  const Walk w = walk_of<S::LANES>(a.tokens, 1, a.groups);
  const int phase = S::SHIFT ? (int)(((long long)w.tok * a.D) & 7) : 0;
  const Ahead ahead(places, a.pieces, a.stages);
  float acc[FULL ? 3 : 1][N];
#pragma unroll
  for (int k = 0; k < (FULL ? 3 : 1); ++k)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[k][j] = 0.f;
  Row<S, true> rr, rd, rg, ry, rz;
  const int r_bf16 = Types<TY>::r(a), y_bf16 = Types<TY>::y(a), out_bf16 = Types<TY>::out(a);
  auto has = [&](int it) { return (S::LANES == 0 || w.on) && w.tok + it * w.step < a.tokens; };
  auto locate = [&](int it) {
    const int tok = w.tok + it * w.step;
    const int rp = NV * (r_bf16 ? 1 : 2), op = NV * (out_bf16 ? 1 : 2);
    const int yp = NV * (y_bf16 ? 1 : 2), at = rp + op + (a.has_dr ? rp : 0);
    rr.set(a.r.p, a.r.at(tok, a.T, a.flat, 0), r_bf16, 0);
    rd.set(a.d.p, a.d.at(tok, a.T, 1, 0), out_bf16, rp);
    rg.set(a.dr.p, a.dr.at(tok, a.T, 1, 0), r_bf16, rp + op);
    ry.set(a.y.p, a.y.at(tok, a.T, a.flat, 0), y_bf16, at);
    rz.set(a.z.p, a.z.at(tok, a.T, a.flat, 0), y_bf16, at + yp);
  };
  auto fetch = [&](int it, int stage) {
    if constexpr (S::kAhead || S::kRegs) {
      if (has(it)) {
        const uint32_t at = ahead.of(stage);
        locate(it);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int i = (c * w.threads + w.tid) * V - phase;
          if (i < a.D) {
            rr.fetch(ahead, at, c, i, a.D);
            rd.fetch(ahead, at, c, i, a.D);
            if (a.has_dr) rg.fetch(ahead, at, c, i, a.D);
            if (FULL) {
              ry.fetch(ahead, at, c, i, a.D);
              if (a.has_z) rz.fetch(ahead, at, c, i, a.D);
            }
          }
        }
      }
      if constexpr (S::kAhead) ptx::cp_async_commit();
    }
  };
  begin_behind();
  for (int i = 0; i + 1 < a.stages; ++i) fetch(i, i);
  int turn = 0, stage = 0;
  for (int it = 0; it < w.iters; ++it, stage = stage + 1 == a.stages ? 0 : stage + 1) {
    rr.advance(), rd.advance(), rg.advance(), ry.advance(), rz.advance();
    fetch(it + a.stages - 1, stage == 0 ? a.stages - 1 : stage - 1);
    if constexpr (S::kAhead) ahead.wait();
    const bool on = S::LANES == 0 || has(it);
    if (S::LANES == 0 && !has(it)) break;        // the whole block
    if (!(S::kAhead || S::kRegs)) locate(it);
    const uint32_t at = ahead.of(stage);
    const size_t dense = (size_t)(w.tok + it * w.step) * a.D;
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      group_at<S>(w, c, a.D, rr, rd);
      if (FULL && a.post) group_at<S>(w, c, a.D, ry);
      const int i = (c * w.threads + w.tid) * V - phase;
      if (!on || i >= a.D) continue;
      float x[V], d[V], k[V];
      rr.get(ahead, at, c, i, a.D, x);
      rd.get(ahead, at, c, i, a.D, d);
      if (a.w) {
        load_shared<S>(a.w, i, a.D, k);
        mul_run<V>(d, d, k);
      }
      s[0] += dot_run<V>(x, x);
      s[1] += dot_run<V>(d, x);
      if (FULL && a.post) {
        ry.get(ahead, at, c, i, a.D, x);
        s[2] += dot_run<V>(x, x);
      }
    }
    row_sum<S::LANES, FULL ? 3 : 2>(s, red, turn);
    const float rho = rsqrtf(fmaf(s[0], a.inv_d, a.eps)), m = s[1] * a.inv_d * rho;
    const float py = FULL && a.post ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 1.f;
    float dp[FULL ? N : 1], se[1] = {0.f};       // dp: dp wp behind a norm
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      group_at<S>(w, c, a.D, rr, rd);
      if (a.has_dr) group_at<S>(w, c, a.D, rg);
      if (FULL) group_at<S>(w, c, a.D, ry);
      if (FULL && a.has_z) group_at<S>(w, c, a.D, rz);
      const int i = (c * w.threads + w.tid) * V - phase;
      if (!on || i >= a.D) continue;
      float g[V], x[V], d[V], k[V];
      rr.get(ahead, at, c, i, a.D, x);
      rd.get(ahead, at, c, i, a.D, d);
      if (a.has_dr) {
        rg.get(ahead, at, c, i, a.D, g);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = 0.f;
      }
      scale_run<V>(x, x, rho);                   // u
      fma_run<V>(acc[0] + c * V, d, x, acc[0] + c * V);
      if (a.w) {
        load_shared<S>(a.w, i, a.D, k);
        mul_run<V>(d, d, k);
      }
      fma_run<V>(d, x, -m, d);
      fma_run<V>(g, d, rho, g);
      store_row<S>(a.o_dr, dense, i, a.D, r_bf16, g);
      if (!FULL) {
        if (a.o_dy) {
          scale_run<V>(g, g, a.s);
          store_row<S>(a.o_dy, dense, i, a.D, y_bf16, g);
        }
        continue;
      }
      if constexpr (FULL) {
        float y[V], z[V], p[V], q[V];
        ry.get(ahead, at, c, i, a.D, y);
        if (a.post) scale_run<V>(y, y, py);      // uy
        if (a.wp) {
          load_shared<S>(a.wp, i, a.D, k);
          mul_run<V>(p, y, k);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) p[e] = y[e];
        }
        if (a.has_z) {
          rz.get(ahead, at, c, i, a.D, z);
          float sg[V];
          gate_sigma<V>(sg, z, a.kind);
          gate_open<V>(q, sg, z, a.kind);        // a
          gate_slope<V>(z, sg, z, a.kind);       // a'
          mul_run<V>(z, z, g);
          mul_run<V>(z, z, p);
          mul_run<V>(q, q, g);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) q[e] = g[e];
        }
        if (a.sv) {                              // q: g a, then g a s
          fma_run<V>(acc[2] + c * V, q, p, acc[2] + c * V);
          load_shared<S>(a.sv, i, a.D, p);
          mul_run<V>(q, q, p);
          if (a.has_z) mul_run<V>(z, z, p);
        } else {
          scale_run<V>(q, q, a.s);
          if (a.has_z) scale_run<V>(z, z, a.s);
        }
        if (a.has_z) store_row<S>(a.o_dz, dense, i, a.D, y_bf16, z);
        float* dq = dp + c * V;
        if (a.post) {
          fma_run<V>(acc[1] + c * V, q, y, acc[1] + c * V);
          if (a.wp) {
            mul_run<V>(dq, q, k);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) dq[e] = q[e];
          }
          se[0] += dot_run<V>(dq, y);
        } else {
          store_row<S>(a.o_dy, dense, i, a.D, y_bf16, q);
        }
      }
    }
    if constexpr (FULL) {
      if (a.post) {
        row_sum<S::LANES, 1>(se, red, turn);
        const float my = se[0] * a.inv_d;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          group_at<S>(w, c, a.D, ry);
          const int i = (c * w.threads + w.tid) * V - phase;
          if (!on || i >= a.D) continue;
          float y[V];
          ry.get(ahead, at, c, i, a.D, y);
          fma_run<V>(y, y, -py * my, dp + c * V);
          scale_run<V>(y, y, py);
          store_row<S>(a.o_dy, dense, i, a.D, y_bf16, y);
        }
      }
    }
  }
  if (!a.part) return;
  __shared__ float sums[S::kSums];
#pragma unroll
  for (int k = 0; k < (FULL ? 3 : 1); ++k) {
    if ((k == 1 && !a.want_p) || (k == 2 && !a.want_s)) continue;
    block_part<S>(acc[k], sums, a.part + ((size_t)k * gridDim.x + blockIdx.x) * a.D, w, phase, a.D);
  }
}

// ------------------------------------------------------------------ host
gdr_status check(const gdr_residual_dims* d) {
  if (!d) return GDR_ERR_INVALID_ARG;
  if (d->B < 0 || d->T < 0 || d->D <= 0 || !is_dtype(d->residual_dtype) || !is_dtype(d->y_dtype) ||
      !is_dtype(d->out_dtype) || bad_act(d->activation) || bad_eps(d->eps) || !isfinite(d->scale))
    return GDR_ERR_INVALID_ARG;
  for (int64_t s : {d->residual_stride_b, d->residual_stride_t, d->y_stride_b, d->y_stride_t,
                    d->gate_stride_b, d->gate_stride_t})
    if (s < 0) return GDR_ERR_INVALID_ARG;
  if (d->D > kWidest || (long long)d->B * d->T > (1LL << 30)) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

// pieces: of all tensors of a row (see make_plan).
Plan residual_plan(const gdr_residual_dims* d, Fit fit, int pieces, int per_sm) {
  return make_plan(d->B * d->T, 1, d->D, pieces, fit, 256, false, per_sm);
}

gdr_status residual_args(ResArgs& a, const gdr_residual_dims* d, const void* r, const void* y,
                         const void* z, const float* w, const float* wp, const float* sv,
                         Fit* fit) {
  if (!is_aligned(r, dtype_size(d->residual_dtype)) || !is_aligned(y, dtype_size(d->y_dtype)) ||
      !is_aligned(z, dtype_size(d->y_dtype)) || !is_aligned(w, 16) || !is_aligned(wp, 16) ||
      !is_aligned(sv, 16))
    return GDR_ERR_ALIGNMENT;
  a.B = d->B; a.T = d->T; a.D = d->D; a.tokens = d->B * d->T;
  const int64_t b = d->B > 1, t = d->T > 1;
  a.r = {r, b * d->residual_stride_b, t * d->residual_stride_t, 0};
  a.y = {y, b * d->y_stride_b, t * d->y_stride_t, 0};
  a.z = {z, b * d->gate_stride_b, t * d->gate_stride_t, 0};
  a.w = w; a.wp = wp; a.sv = sv;
  a.has_y = y != nullptr;
  a.has_z = z != nullptr;
  a.post = d->post_norm != 0;
  a.kind = d->activation;
  a.r_bf16 = d->residual_dtype == GDR_BF16;
  a.y_bf16 = d->y_dtype == GDR_BF16;
  a.out_bf16 = d->out_dtype == GDR_BF16;
  a.eps = d->eps;
  a.inv_d = 1.f / d->D;
  a.s = d->scale;
  if (a.T == 1) a.r.t = a.r.b, a.y.t = a.y.b, a.z.t = a.z.b;   // tokens are batch rows
  a.flat = 1;
  for (const View* v : {&a.r, &a.y, &a.z})
    if (v->p && a.B > 1 && v->b != a.T * v->t) a.flat = 0;
  *fit = kVec;
  for (const View* v : {&a.r, &a.y, &a.z})
    if (v->p) *fit = worse(*fit, fit_of(v->p, a.B, a.T, 1, a.D, v->b, v->t, 0));
  return GDR_OK;
}
// f(the call's types) for the rows that go through shared memory; the others look at run time.
template <class S, typename F>
auto with_types(const ResArgs& a, F f) {
  if constexpr (S::kAhead && S::LANES == 0) {
    const int y = a.has_y || a.o_dy ? a.y_bf16 : a.out_bf16; // neither: any type of it
    if (y == a.out_bf16 && a.r_bf16 && y) return f(std::integral_constant<int, kAllBf16>());
    if (y == a.out_bf16 && !a.r_bf16)
      return y ? f(std::integral_constant<int, kF32Residual>())
               : f(std::integral_constant<int, kAllF32>());
  }
  return f(std::integral_constant<int, kAnyTypes>());
}
// A gate, a post norm or a scale per channel act on y.
bool needs_y(const gdr_residual_dims* d, const void* z, const float* wp, const float* sv) {
  return d->post_norm || z || wp || sv;
}
// wp belongs to the post norm.
bool bad_branch(const gdr_residual_dims* d, const void* y, const void* z, const float* wp,
                const float* sv) {
  return (!y && needs_y(d, z, wp, sv)) || (wp && !d->post_norm);
}

}  // namespace
}  // namespace ops
}  // namespace gdr

using namespace gdr;
using namespace gdr::ops;

extern "C" {

gdr_status gdr_residual_norm(const void* residual, const void* y, const void* gate,
                             const float* weight, const float* post_weight, const float* scale,
                             void* residual_out, void* out, const gdr_residual_dims* dims,
                             gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  ResArgs a = {};
  Fit fit = kSingle;
  const gdr_status ok =
      residual_args(a, dims, residual, y, gate, weight, post_weight, scale, &fit);
  if (ok != GDR_OK) return ok;
  if (!is_aligned(residual_out, 16) || !is_aligned(out, 16)) return GDR_ERR_ALIGNMENT;
  if (a.tokens == 0) return GDR_OK;
  if (!residual || !out || bad_branch(dims, y, gate, post_weight, scale) || !y != !residual_out)
    return GDR_ERR_INVALID_ARG;
  a.out = out;
  a.r_out = residual_out;
  const int re = a.r_bf16 ? 1 : 2, ye = a.y_bf16 ? 1 : 2;
  const Plan p = residual_plan(dims, fit, re + a.has_y * ye + a.has_z * ye, kFwdPerSm);
  a.pieces = p.pieces;
  a.stages = p.stages;
  a.groups = p.groups;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_shape<false>(p, [&](auto shape) {
    using S = decltype(shape);
    return with_types<S>(a, [&](auto types) {
      constexpr int TY = decltype(types)::value;
      struct Tag;
      if (p.smem > kPlainSmem && !allow_smem<Tag>(residual_fwd_kernel<S, TY>, kSmemPerSm))
        return GDR_ERR_CUDA;
      return launch_behind_smem(residual_fwd_kernel<S, TY>, dim3(p.blocks), p.threads, p.smem, s,
                                a);
    });
  });
}

size_t gdr_residual_norm_bwd_workspace_size(const gdr_residual_dims* dims) {
  if (check(dims) != GDR_OK) return 0;
  size_t most = kAlign;
  for (Fit fit : {dims->D % 8 ? kShift : kVec, kSingle}) {
    const size_t rows = residual_plan(dims, fit, 1, kBwdPerSm).rows;
    const size_t n = align_up(3 * rows * dims->D * sizeof(float));
    if (n > most) most = n;
  }
  return most;
}

gdr_status gdr_residual_norm_bwd(const void* d_out, const void* d_residual_out,
                                 const void* residual_out, const void* y, const void* gate,
                                 const float* weight, const float* post_weight, const float* scale,
                                 void* d_residual, void* d_y, void* d_gate, float* d_weight,
                                 float* d_post_weight, float* d_scale,
                                 const gdr_residual_dims* dims, void* workspace,
                                 size_t workspace_bytes, gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  ResArgs a = {};
  Fit fit = kSingle;
  const gdr_status ok =
      residual_args(a, dims, residual_out, y, gate, weight, post_weight, scale, &fit);
  if (ok != GDR_OK) return ok;
  for (const void* p : {d_out, d_residual_out, static_cast<const void*>(d_residual),
                        static_cast<const void*>(d_y), static_cast<const void*>(d_gate),
                        static_cast<const void*>(d_weight), static_cast<const void*>(d_post_weight),
                        static_cast<const void*>(d_scale)})
    if (!is_aligned(p, 16)) return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.tokens == 0) {
    for (float* p : {d_weight, d_post_weight, d_scale}) {
      const gdr_status z = zero(p, dims->D, s);
      if (z != GDR_OK) return z;
    }
    return GDR_OK;
  }
  const bool full = needs_y(dims, gate, post_weight, scale);
  if (!d_out || !residual_out || !d_residual || (full && !y) || (post_weight && !dims->post_norm) ||
      (full && !d_y) || !gate != !d_gate || (d_post_weight && !dims->post_norm) ||
      (d_scale && !scale))
    return GDR_ERR_INVALID_ARG;
  a.has_dr = d_residual_out != nullptr;
  const int re = a.r_bf16 ? 1 : 2, ye = a.y_bf16 ? 1 : 2, oe = a.out_bf16 ? 1 : 2;
  const int pieces = re * (1 + a.has_dr) + oe + (full ? ye * (1 + a.has_z) : 0);
  const Plan p = residual_plan(dims, fit, pieces, full ? kFullPerSm : kBwdPerSm);
  if (d_weight || d_post_weight || d_scale) {
    if (!workspace || workspace_bytes < gdr_residual_norm_bwd_workspace_size(dims))
      return GDR_ERR_WORKSPACE;
    if (!is_aligned(workspace, kAlign)) return GDR_ERR_ALIGNMENT;
    a.part = static_cast<float*>(workspace);
  }
  a.want_p = d_post_weight != nullptr;
  a.want_s = d_scale != nullptr;
  const int64_t t = dims->D;
  a.d = {d_out, t * dims->T, t, 0};
  a.dr = {d_residual_out, t * dims->T, t, 0};
  a.o_dr = d_residual;
  a.o_dy = d_y;
  a.o_dz = d_gate;
  a.pieces = p.pieces;
  a.stages = p.stages;
  a.groups = p.groups;
  const gdr_status run = with_shape<false>(p, [&](auto shape) {
    using S = decltype(shape);
    auto go = [&](auto* fn, auto* tag) {
      if (p.smem > kPlainSmem && !allow_smem<std::remove_pointer_t<decltype(tag)>>(fn, kSmemPerSm))
        return GDR_ERR_CUDA;
      // Blocks of a call that fills the device do not come early: their shared memory would be
      // taken from the kernel before. Training steps, early and not: with norm, gate and scale 1000 x
      // 1536 27.7 and 28.8 us, 4096 x 1536 71.8 and 70.1, 16384 x 1536 229 and 218, 8192 x 4096 326 and
      // 312; without, 600 x 4096 in bf16 17.0 and 18.8, 16384 x 4096 195 and 197, in 32 bits 3063 x 777
      // 36.7 and 33.0, 4096 x 2048 63.6 and 59.5.
      return p.blocks < kSms * 2 ? launch_behind_smem(fn, dim3(p.blocks), p.threads, p.smem, s, a)
                                 : launch_kernel(fn, dim3(p.blocks), p.threads, p.smem, s, a);
    };
    return with_types<S>(a, [&](auto types) {
      constexpr int TY = decltype(types)::value;
      struct Full;
      struct Plain;
      return full ? go(residual_bwd_kernel<S, TY, true>, static_cast<Full*>(nullptr))
                  : go(residual_bwd_kernel<S, TY, false>, static_cast<Plain*>(nullptr));
    });
  });
  if (run != GDR_OK || !a.part) return run;
  return sum_parts(a.part, d_weight, d_post_weight, d_scale, p.rows, dims->D, s);
}

}  // extern "C"
