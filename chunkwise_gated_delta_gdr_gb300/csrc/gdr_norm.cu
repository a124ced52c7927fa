// gdr_norm.cu -- the norms around a layer of a decoder, forward and backward.
//
// gated_norm, the norm of a layer's output heads with its output gate, a = act(z):
//   y = u w a,  u = x r,  r = 1 / sqrt(mean(x^2) + eps)        (gate behind the norm)
//   y = u w,    u = v r,  v = x a, r of v                      (gate before the norm)
// and with d the gradient of y
//   behind: dw = sum d a u,  c = d a w,  dx = r (c - u mean(c u)),  dz = d u w a'
//   before: dw = sum d u,    c = d w,    dv = r (c - u mean(c u)),  dx = dv a,  dz = dv x a'
//
// residual_norm, between two layers: p = y or its norm uy wp, a = act(z) or 1, s a number or a
// channel's weight:
//   r' = r + s a p,  out = u w,  u = r' rho
//   g = dr' + rho (c - u mean(c u)),  c = dout w,  dw = sum dout u,  dr = g,  ds = sum g a p
//   dz = g s p a',  dp = g s a,  dy = dp, or behind a norm: dwp = sum dp uy,
//   dy = ry (dp wp - uy mean(dp wp uy))
//
// Every tensor is read once and written once: bound by HBM where there is enough of it, by the
// chain load - sum over the row - store of one row below. Measured on one GB300, bf16, a pass
// among others (a plain copy: 6.70 TB/s):
//   gated_norm, 2 x 8192 x 32 heads of 128: 62.7 us, 6.4 TB/s; 64 decode tokens x 16 heads 2.5 us
//     training step, 4096 x 12 heads of 128: 24.9 us (forward 9, backward 15, weights' sums 5
//     with cold caches); 2 x 4096 x 4 groups of 512, gate first, weights per group 54.9 us
//   residual_norm, training step, 2 x 8192 x 4096: 196 us, 6.2 TB/s (forward 77, backward 104);
//     4096 x 1536, residual in 32 bits, y normed, gated and scaled per channel 71 us (22, 41,
//     8 us: 2.7 and 5.4 rows a block, whose loads, sums and stores fall together); 3 x 1021 x
//     777 in 32 bits 49 us; 64 decode tokens x 2048 channels 3.3 us
#include "gdr_norm.cuh"

namespace gdr {
namespace ops {
namespace {

constexpr int kMaxThreads = 512;

struct GatedArgs {
  View x, z, d;                  // d: the gradient of y (backward)
  const float* w;                // [D] or [H][D], or null
  void *y, *dx, *dz;             // dense
  float* part;                   // weight gradient's parts, or null
  int B, T, H, D, tokens, groups, per_head, kind, first;
  int in_bf16, out_bf16;         // out: of y and d
  int pieces, stages;
  int flat;                      // the views' tokens are one stride apart, over batch rows too
  float eps, inv_d;
};

// Sum over the block's groups of each element's acc (LANES > 0), in the first group's registers.
template <class S>
__device__ __forceinline__ void sum_groups(float* acc, float* s, int tid) {
  if constexpr (S::LANES > 0) {
    if constexpr (S::LANES < 32)
#pragma unroll
      for (int o = S::LANES; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < S::N; ++j) acc[j] += __shfl_xor_sync(~0u, acc[j], o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane < S::LANES)
#pragma unroll
      for (int j = 0; j < S::N; ++j) s[(warp * S::N + j) * S::LANES + tid] = acc[j];
    __syncthreads();
    if (threadIdx.x < S::LANES)
      for (int k = 1; k < warps; ++k)
#pragma unroll
        for (int j = 0; j < S::N; ++j) acc[j] += s[(k * S::N + j) * S::LANES + tid];
    __syncthreads();
  }
}

// A block's part of a weight gradient: its group's sums, or those of its groups added in order,
// element by element (groups of SHIFT have phases of their own).
constexpr int kBlockSum = 2048;                  // groups x elements of a block at most
template <class S>
__device__ __forceinline__ void block_part(const float* acc, float* s, float* to, const Walk& w,
                                           int phase, int D) {
  if constexpr (S::LANES == 0) {
#pragma unroll
    for (int c = 0; c < S::NV; ++c) {
      const int i = (c * w.threads + w.tid) * S::V - phase;
      if (i < D) store_part<S>(to, i, D, acc + c * S::V);
    }
  } else {
    const int groups = blockDim.x / S::LANES;
    __syncthreads();                             // the last sum's readers are done
#pragma unroll
    for (int c = 0; c < S::NV; ++c)
#pragma unroll
      for (int e = 0; e < S::V; ++e) {
        const int i = (c * w.threads + w.tid) * S::V - phase + e;
        if (i >= 0 && i < D) s[threadIdx.x / S::LANES * D + i] = acc[c * S::V + e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      float v = 0.f;
      for (int g = 0; g < groups; ++g) v += s[g * D + i];
      to[i] = v;
    }
  }
}

// Rows of at most 512 channels: a group of LANES lanes per row, NV runs of 8 channels a lane, UN
// rows at a time (the group's head in UN tokens), the next ones' loads under way meanwhile. What
// bounds the larger calls beside HBM is the number of instructions per row, so addresses step
// from row to row and sums and products go in pairs; the copies through shared memory that wider
// rows take cost twice the time here (2 x 8192 x 32 heads of 128 forward: 115 us so, 57 now).
template <typename T, int LANES, int NV, bool BWD, bool FIRST>
__global__ void __launch_bounds__(256, BWD ? 2 : 3) gated_rows_kernel(GatedArgs a) {
  typedef Shape<LANES, 8, NV> S;
  constexpr int TENSORS = BWD ? 3 : 2, UN = sizeof(T) == 2 && NV == 1 ? 2 : 1, N = 4 * NV;
  constexpr int Q = 8 * sizeof(T) / 16;          // 16-byte pieces of 8 channels
  constexpr bool AHEAD = NV == 1 || !BWD;        // else there are no registers for the next rows
  __shared__ float sums[BWD ? 8 * 32 * 8 * NV : 1];
  const Walk w = walk_of<LANES>(a.tokens, a.H, a.groups);
  bool mine[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) mine[c] = w.on && (c * LANES + w.tid) * 8 < a.D;
  const int ch = w.tid * 8;
  const T* base[TENSORS];
  int64_t pitch[TENSORS];
  base[0] = static_cast<const T*>(a.x.p) + w.head * a.x.h + ch;
  base[1] = static_cast<const T*>(a.z.p) + w.head * a.z.h + ch;
  pitch[0] = a.x.t;
  pitch[1] = a.z.t;
  if (BWD) {
    base[TENSORS - 1] = static_cast<const T*>(a.d.p) + w.head * a.d.h + ch;
    pitch[TENSORS - 1] = a.d.t;
  }
  struct Raw {
    uint4 q[NV * Q];
  };
  auto load = [&](int tok, Raw* r) {             // zeros where there is nothing
#pragma unroll
    for (int k = 0; k < TENSORS; ++k) {
      int64_t at = tok * pitch[k];
      if (!a.flat && k < 2) {
        const int b = tok / a.T;
        at = b * (k == 0 ? a.x.b : a.z.b) + (tok - b * a.T) * pitch[k];
      }
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const uint4* p = reinterpret_cast<const uint4*>(base[k] + at + c * LANES * 8);
#pragma unroll
        for (int i = 0; i < Q; ++i)
          r[k].q[c * Q + i] = mine[c] && tok < a.tokens ? __ldcs(p + i) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto pairs = [](const Raw& r, float2* f) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r.q);
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = sizeof(T) == 2 ? unpack2(u[i])
                            : make_float2(__uint_as_float(u[(2 * i) % (4 * NV * Q)]),
                                          __uint_as_float(u[(2 * i + 1) % (4 * NV * Q)]));
  };
  begin_behind();
  float2 wt[N], acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) wt[i] = make_float2(1.f, 1.f), acc[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < NV; ++c)
    if (a.w && mine[c]) {
      float f[8];
      load_run<float, 8, true>(a.w + (a.per_head ? (size_t)w.head * a.D : 0) + ch + c * LANES * 8, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) wt[4 * c + i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  Raw next[UN][TENSORS];
  if (AHEAD)
#pragma unroll
    for (int u = 0; u < UN; ++u) load(w.tok + u * w.step, next[u]);
  for (int it = 0; it < w.iters; it += UN) {
    const int tok0 = w.tok + it * w.step;
    Raw raw[UN][TENSORS];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (!AHEAD) load(tok0 + u * w.step, next[u]);
#pragma unroll
      for (int k = 0; k < TENSORS; ++k) raw[u][k] = next[u][k];
    }
    if (AHEAD && it + UN < w.iters)
#pragma unroll
      for (int u = 0; u < UN; ++u) load(tok0 + (UN + u) * w.step, next[u]);
    // p, q: forward a, or x a with the gate before the norm. Backward d a and d w a' (behind);
    // a and x a' (before).
    float2 p[UN][N], q[BWD ? UN : 1][N];
    float s[UN][2];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      float2 x[N], z[N], d[N], ss = make_float2(0.f, 0.f), se = make_float2(0.f, 0.f);
      pairs(raw[u][0], x);
      pairs(raw[u][1], z);
      if (BWD) pairs(raw[u][TENSORS - 1], d);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float2 g, slope;
        g.x = act(z[i].x, a.kind, slope.x);
        g.y = act(z[i].y, a.kind, slope.y);
        const float2 v = FIRST ? mul2(x[i], g) : x[i];
        ss = fma2(v, v, ss);
        if (!BWD) {
          p[u][i] = FIRST ? v : g;
        } else if (FIRST) {
          p[u][i] = g;
          q[u][i] = mul2(x[i], slope);
          se = fma2(mul2(d[i], wt[i]), v, se);
        } else {
          p[u][i] = mul2(d[i], g);
          q[u][i] = mul2(mul2(d[i], wt[i]), slope);
          se = fma2(mul2(p[u][i], wt[i]), v, se);
        }
      }
      s[u][0] = ss.x + ss.y;
      s[u][1] = se.x + se.y;
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        s[u][0] += __shfl_xor_sync(~0u, s[u][0], o);
        if (BWD) s[u][1] += __shfl_xor_sync(~0u, s[u][1], o);
      }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int tok = tok0 + u * w.step;
      const float r = rsqrtf(fmaf(s[u][0], a.inv_d, a.eps)), m = -s[u][1] * a.inv_d * r;
      const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
      const size_t dense = ((size_t)tok * a.H + w.head) * a.D + ch;
      float2 x[N], d[N];
      pairs(raw[u][0], x);
      if (BWD) pairs(raw[u][TENSORS - 1], d);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        float o[8], oz[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * c + j;
          float2 y, yz;
          if (!BWD) {
            y = FIRST ? mul2(mul2(p[u][i], r2), wt[i])
                      : mul2(mul2(mul2(x[i], r2), wt[i]), p[u][i]);
          } else if (FIRST) {
            const float2 un = mul2(mul2(x[i], p[u][i]), r2);
            const float2 dv = mul2(r2, fma2(un, m2, mul2(d[i], wt[i])));
            acc[i] = fma2(d[i], un, acc[i]);
            y = mul2(dv, p[u][i]);
            yz = mul2(dv, q[u][i]);
          } else {
            const float2 un = mul2(x[i], r2);
            acc[i] = fma2(p[u][i], un, acc[i]);
            y = mul2(r2, fma2(un, m2, mul2(p[u][i], wt[i])));
            yz = mul2(un, q[u][i]);
          }
          o[2 * j] = y.x;
          o[2 * j + 1] = y.y;
          if (BWD) {
            oz[2 * j] = yz.x;
            oz[2 * j + 1] = yz.y;
          }
        }
        if (mine[c] && tok < a.tokens) {
          store_run<T, 8>(static_cast<T*>(BWD ? a.dx : a.y) + dense + c * LANES * 8, o);
          if (BWD) store_run<T, 8>(static_cast<T*>(a.dz) + dense + c * LANES * 8, oz);
        }
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    float sum[8 * NV];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[2 * i] = acc[i].x, sum[2 * i + 1] = acc[i].y;
    if (!a.per_head) sum_groups<S>(sum, sums, w.tid);
    if (a.per_head ? !w.on : threadIdx.x >= LANES) return;
    float* to =
        a.part + (a.per_head ? ((size_t)w.tok * a.H + w.head) * a.D : (size_t)blockIdx.x * a.D);
#pragma unroll
    for (int c = 0; c < NV; ++c)
      if (ch + c * LANES * 8 < a.D) store_run<float, 8>(to + ch + c * LANES * 8, sum + 8 * c);
  }
}

// Any other row: wider ones, a block each, and those that do not allow 16-byte accesses.
template <class S, bool BWD>
__global__ void __launch_bounds__(kMaxThreads) gated_kernel(GatedArgs a) {
  constexpr int V = S::V, NV = S::NV, N = S::N, TENSORS = BWD ? 3 : 2;
  extern __shared__ __align__(16) char places[];
  __shared__ Red red;
  __shared__ float sums[BWD && S::LANES ? kBlockSum : 1];
  const Walk w = walk_of<S::LANES>(a.tokens, a.H, a.groups);
  const int phase = S::SHIFT ? (int)((((long long)w.tok * a.H + w.head) * a.D) & 7) : 0;
  const Ahead ahead(places, a.pieces, a.stages);
  const float* weight = a.w && a.per_head ? a.w + (size_t)w.head * a.D : a.w;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;

  Row<S, S::NV <= 4> row[TENSORS];
  auto has = [&](int it) { return w.on && w.tok + it * w.step < a.tokens; };
  auto locate = [&](int it) {
    const int tok = w.tok + it * w.step, per = NV * (a.in_bf16 ? 1 : 2);
    row[0].set(a.x.p, a.x.at(tok, a.T, a.flat, w.head), a.in_bf16, 0);
    row[1].set(a.z.p, a.z.at(tok, a.T, a.flat, w.head), a.in_bf16, per);
    if (BWD) row[TENSORS - 1].set(a.d.p, a.d.at(tok, a.T, 1, w.head), a.out_bf16, 2 * per);
  };
  auto fetch = [&](int it, int stage) {
    if constexpr (S::kAhead || S::kRegs) {
      if (has(it)) {
        const uint32_t at = ahead.of(stage);
        locate(it);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int i = (c * w.threads + w.tid) * V - phase;
          if (i < a.D)
#pragma unroll
            for (int k = 0; k < TENSORS; ++k) row[k].fetch(ahead, at, c, i, a.D);
        }
      }
      if constexpr (S::kAhead) ptx::cp_async_commit();
    }
  };
  begin_behind();
  for (int i = 0; i + 1 < a.stages; ++i) fetch(i, i);
  int turn = 0, stage = 0;
  for (int it = 0; it < w.iters; ++it, stage = stage + 1 == a.stages ? 0 : stage + 1) {
#pragma unroll
    for (int k = 0; k < TENSORS; ++k) row[k].advance();
    fetch(it + a.stages - 1, stage == 0 ? a.stages - 1 : stage - 1);
    if constexpr (S::kAhead) ahead.wait();
    const bool on = has(it);
    if (!(S::kAhead || S::kRegs) && on) locate(it);
    const uint32_t at = ahead.of(stage);
    const size_t dense = ((size_t)(w.tok + it * w.step) * a.H + w.head) * a.D;
    float s[2] = {0.f, 0.f};
    if (on)
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int i = (c * w.threads + w.tid) * V - phase;
        if (i >= a.D) continue;
        float x[V], z[V], d[V], wt[V];
        row[0].get(ahead, at, c, i, a.D, x);
        if (a.first || BWD) row[1].get(ahead, at, c, i, a.D, z);
        if (BWD) {
          row[TENSORS - 1].get(ahead, at, c, i, a.D, d);
          if (weight) load_shared<S>(weight, i, a.D, wt);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float g = a.first || BWD ? act(z[e], a.kind) : 1.f;
          const float v = a.first ? x[e] * g : x[e];
          s[0] = fmaf(v, v, s[0]);
          if (BWD) {
            const float dc = a.first ? d[e] : d[e] * g;
            s[1] = fmaf(weight ? dc * wt[e] : dc, v, s[1]);
          }
        }
      }
    row_sum<S::LANES, BWD ? 2 : 1>(s, red, turn);
    if (!on) continue;
    const float r = rsqrtf(fmaf(s[0], a.inv_d, a.eps)), m = s[1] * a.inv_d * r;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int i = (c * w.threads + w.tid) * V - phase;
      if (i >= a.D) continue;
      float x[V], z[V], d[V], wt[V], o[V], oz[V];
      row[0].get(ahead, at, c, i, a.D, x);
      row[1].get(ahead, at, c, i, a.D, z);
      if (BWD) row[TENSORS - 1].get(ahead, at, c, i, a.D, d);
      if (weight) {
        load_shared<S>(weight, i, a.D, wt);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) wt[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float slope;
        const float g = act(z[e], a.kind, slope);
        const float u = (a.first ? x[e] * g : x[e]) * r;
        if (!BWD) {
          o[e] = a.first ? u * wt[e] : u * wt[e] * g;
        } else if (a.first) {
          const float dv = r * fmaf(-u, m, d[e] * wt[e]);
          acc[c * V + e] = fmaf(d[e], u, acc[c * V + e]);
          o[e] = dv * g;
          oz[e] = dv * x[e] * slope;
        } else {
          const float dg = d[e] * g;
          acc[c * V + e] = fmaf(dg, u, acc[c * V + e]);
          o[e] = r * fmaf(-u, m, dg * wt[e]);
          oz[e] = d[e] * u * wt[e] * slope;
        }
      }
      if (BWD) {
        store_row<S>(a.dx, dense, i, a.D, a.in_bf16, o);
        store_row<S>(a.dz, dense, i, a.D, a.in_bf16, oz);
      } else {
        store_row<S>(a.y, dense, i, a.D, a.out_bf16, o);
      }
    }
  }
  if constexpr (BWD) {
    if (!a.part) return;
    // A row of parts per block; per group where its head has weights of its own.
    if (!a.per_head) {
      block_part<S>(acc, sums, a.part + (size_t)blockIdx.x * a.D, w, phase, a.D);
    } else if (w.on) {
      float* to = a.part + ((size_t)w.tok * a.H + w.head) * a.D;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int i = (c * w.threads + w.tid) * V - phase;
        if (i < a.D) store_part<S>(to, i, a.D, acc + c * V);
      }
    }
  }
}

// ------------------------------------------------------------------ residual
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
__global__ void __launch_bounds__(kMaxThreads, S::N <= 16 ? 2 : 1) residual_fwd_kernel(ResArgs a) {
  constexpr int V = S::V, NV = S::NV, N = S::N;
  extern __shared__ __align__(16) char places[];
  __shared__ Red red;
  const Walk w = walk_of<S::LANES>(a.tokens, 1, a.groups);
  const int phase = S::SHIFT ? (int)(((long long)w.tok * a.D) & 7) : 0;
  const Ahead ahead(places, a.pieces, a.stages);
  Row<S, false> rr;                              // may be the result's own memory
  Row<S, S::NV <= 4> ry, rz;
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
#pragma unroll
          for (int e = 0; e < V; ++e) k[e] = act(k[e], a.kind);
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
__global__ void __launch_bounds__(kMaxThreads, S::N <= 16 && !FULL ? 2 : 1) residual_bwd_kernel(ResArgs a) {
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
  Row<S, S::NV <= 4> rr, rd, rg, ry, rz;
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
#pragma unroll
          for (int e = 0; e < V; ++e) q[e] = act(z[e], a.kind, z[e]);    // a, and a' in z
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
  __shared__ float sums[S::LANES ? kBlockSum : 1];
#pragma unroll
  for (int k = 0; k < (FULL ? 3 : 1); ++k) {
    if ((k == 1 && !a.want_p) || (k == 2 && !a.want_s)) continue;
    block_part<S>(acc[k], sums, a.part + ((size_t)k * gridDim.x + blockIdx.x) * a.D, w, phase, a.D);
  }
}

// ------------------------------------------------------------------ host
constexpr int kSms = 152;
constexpr int kWidest = 16384;                   // elements of a row at most
constexpr int kSmemPerSm = 200 * 1024;         // of copies ahead, an SM and a block at most

constexpr int kPlainSmem = 36 * 1024;            // fits beside the static part without being asked for

// What a call's kernel looks like: threads of a block, groups and blocks, copies ahead.
struct Plan {
  int lanes, v, nv, threads, groups, blocks, rows;   // rows: of the parts, per weight
  bool shift;
  int pieces, stages, smem;
};

// f(Shape) for a plan.
template <typename F>
auto with_block(const Plan& p, F f) {
  if (p.shift) return f(Shape<0, 8, 2, true>());
  if (p.v == 8) return p.nv == 2 ? f(Shape<0, 8, 2>()) : f(Shape<0, 8, 4>());
  return p.nv == 4 ? f(Shape<0, 1, 4>()) : p.nv == 16 ? f(Shape<0, 1, 16>()) : f(Shape<0, 1, 32>());
}
// TWO: whether rows of more than 256 elements share a warp.
template <bool TWO, typename F>
auto with_shape(const Plan& p, F f) {
  if (p.lanes == 0) return with_block(p, f);
  if (p.shift)
    return p.lanes == 8    ? f(Shape<8, 8, 1, true>())
           : p.lanes == 16 ? f(Shape<16, 8, 1, true>())
                           : f(Shape<32, 8, 1, true>());
  if (p.v == 1) return f(Shape<32, 1, 8>());
  if constexpr (TWO)
    if (p.nv == 2) return f(Shape<32, 8, 2>());
  return p.lanes == 8    ? f(Shape<8, 8, 1>())
         : p.lanes == 16 ? f(Shape<16, 8, 1>())
                         : f(Shape<32, 8, 1>());
}

// How a call's rows lie: 16-byte accesses fit; fit but for a phase (Shape's SHIFT); or neither.
enum Fit { kVec, kShift, kSingle };

// pieces: 16-byte pieces per run of 8, over all tensors of a row. widest: elements of a row
// that shares a warp, at most (256 where rows have a phase or no alignment). per_sm: threads an SM is to hold.
Plan make_plan(int tokens, int H, int D, int pieces, Fit fit, int widest, bool per_head,
               int per_sm) {
  Plan p = {};
  p.shift = fit == kShift && D + 7 <= kMaxThreads * 16;
  const bool vec = fit == kVec || p.shift;
  p.v = vec ? 8 : 1;
  const int span = D + (p.shift ? 7 : 0);        // elements that a row's threads cover
  p.lanes = span > (fit == kVec ? widest : 256) ? 0
            : !vec || span > 128                          ? 32
            : span > 64                                   ? 16
                                                          : 8;
  int per_block = 1;                             // groups of a block
  if (p.lanes) {
    p.nv = !vec ? 8 : span > 256 ? 2 : 1;
    p.threads = 256;
    per_block = p.threads / p.lanes;
  } else {
    // Elements of a thread: 16, 32 in the widest rows, 4 in short ones element by element (more
    // threads then have more loads under way).
    p.nv = vec ? (D <= kMaxThreads * 16 ? 2 : 4)
               : D <= kMaxThreads * 4 ? 4 : D <= kMaxThreads * 16 ? 16 : 32;
    const int n = p.nv * p.v;
    p.threads = ((span + n - 1) / n + 31) / 32 * 32;
  }
  const long long rows = (long long)tokens * H;
  long long blocks = (rows + per_block - 1) / per_block;
  const long long most = (long long)kSms * (per_sm / p.threads > 1 ? per_sm / p.threads : 1);
  if (blocks > most) blocks = most;
  const long long least = (H + per_block - 1) / per_block;     // a group per head
  if (blocks < least) blocks = least;
  long long groups = blocks * per_block / H * H;
  if (p.shift && groups < rows) {                // steps of 8 tokens, for one phase per group
    const long long unit = 8LL * H;
    groups = groups < unit ? unit : groups / unit * unit;
    blocks = (groups + per_block - 1) / per_block;
  }
  p.blocks = (int)blocks;
  p.groups = (int)groups;
  p.rows = per_head ? p.groups / H : p.blocks;
  p.pieces = pieces * p.nv;
  p.stages = !vec && p.nv <= 8 ? 2 : 1;          // 2: the next row in registers
  if (p.v == 8 && p.nv <= 2) {
    const int stage = p.pieces * p.threads * 16;
    const int resident = per_sm / p.threads > 1 ? per_sm / p.threads : 1;
    p.stages = 3;
    while (p.stages > 1 && (long long)p.stages * stage * resident > kSmemPerSm) --p.stages;
    p.smem = p.stages * stage;
  }
  return p;
}

// The fit of a view [B, T, H, D] (strides of dimensions of one element: 0).
Fit fit_of(const void* p, int B, int T, int H, int D, int64_t b, int64_t t, int64_t h) {
  if (!is_aligned(p, 16)) return kSingle;
  const int64_t row = D, tok = row * H, batch = tok * T;
  if ((B > 1 && (b - batch) % 8) || (T > 1 && (t - tok) % 8) || (H > 1 && (h - row) % 8))
    return kSingle;
  return D % 8 ? kShift : kVec;
}
Fit worse(Fit a, Fit b) { return a > b ? a : b; }

// Column sums of the parts, behind the kernel that writes them.
gdr_status sum_parts(const float* part, float* o0, float* o1, float* o2, int rows, int cols,
                     cudaStream_t s) {
  return launch_behind(column_sum_kernel, dim3((cols + kSumCols - 1) / kSumCols, o1 || o2 ? 3 : 1),
                       kSumCols * kSumRows, s, part, o0, o1, o2, rows, cols);
}
gdr_status zero(float* p, size_t n, cudaStream_t s) {
  return !p || n == 0 ? GDR_OK : status_of(cudaMemsetAsync(p, 0, n * sizeof(float), s));
}

bool bad_eps(float e) { return !(isfinite(e) && e > 0.f); }
bool bad_act(int k) { return k != GDR_ACT_NONE && k != GDR_ACT_SIGMOID && k != GDR_ACT_SILU; }

gdr_status check(const gdr_gated_dims* d) {
  if (!d) return GDR_ERR_INVALID_ARG;
  if (d->B < 0 || d->T < 0 || d->H <= 0 || d->D <= 0 || !is_dtype(d->in_dtype) ||
      !is_dtype(d->out_dtype) || bad_act(d->activation) || bad_eps(d->eps))
    return GDR_ERR_INVALID_ARG;
  for (int64_t s : {d->x_stride_b, d->x_stride_t, d->x_stride_h, d->gate_stride_b,
                    d->gate_stride_t, d->gate_stride_h})
    if (s < 0) return GDR_ERR_INVALID_ARG;
  if (d->D > kWidest || (long long)d->B * d->T > (1LL << 30) || d->H > (1 << 20) ||
      (long long)d->H * d->D > (1LL << 30))
    return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

// Threads that an SM is to hold: of the kernels above (kFullPerSm: the residual's backward with a
// norm, gate or scale per channel, at most kBwdPerSm), and of gated_rows_kernel.
constexpr int kFwdPerSm = 1024, kBwdPerSm = 1024, kFullPerSm = 512;
constexpr int kFwdRowsPerSm = 768, kBwdRowsPerSm = 512;

Plan gated_plan(const gdr_gated_dims* d, Fit fit, bool bwd) {
  const int in = d->in_dtype == GDR_BF16 ? 1 : 2, out = d->out_dtype == GDR_BF16 ? 1 : 2;
  return make_plan(d->B * d->T, d->H, d->D, 2 * in + (bwd ? out : 0), fit, 512,
                   d->weight_per_head != 0,
                   fit == kVec && d->D <= 512 ? (bwd ? kBwdRowsPerSm : kFwdRowsPerSm)
                                      : (bwd ? kBwdPerSm : kFwdPerSm));
}
size_t gated_bytes(const gdr_gated_dims* d, const Plan& p) {
  const size_t cols = (size_t)d->D * (d->weight_per_head ? d->H : 1);
  return align_up((size_t)p.rows * cols * sizeof(float));
}

// Arguments that both directions share.
gdr_status gated_args(GatedArgs& a, const gdr_gated_dims* d, const void* x, const void* gate,
                      const float* w, Fit* fit) {
  if (!is_aligned(x, dtype_size(d->in_dtype)) || !is_aligned(gate, dtype_size(d->in_dtype)) ||
      !is_aligned(w, 16))
    return GDR_ERR_ALIGNMENT;
  a.B = d->B; a.T = d->T; a.H = d->H; a.D = d->D; a.tokens = d->B * d->T;
  // A dimension of one element is never stepped along.
  const int64_t b = d->B > 1, t = d->T > 1, h = d->H > 1;
  a.x = {x, b * d->x_stride_b, t * d->x_stride_t, h * d->x_stride_h};
  a.z = {gate, b * d->gate_stride_b, t * d->gate_stride_t, h * d->gate_stride_h};
  if (a.T == 1) a.x.t = a.x.b, a.z.t = a.z.b;      // tokens are batch rows
  a.flat = (a.B == 1 || (a.x.b == a.T * a.x.t && a.z.b == a.T * a.z.t)) ? 1 : 0;
  a.w = w;
  a.per_head = d->weight_per_head != 0;
  a.kind = d->activation;
  a.first = d->gate_first != 0;
  a.in_bf16 = d->in_dtype == GDR_BF16;
  a.out_bf16 = d->out_dtype == GDR_BF16;
  a.eps = d->eps;
  a.inv_d = 1.f / d->D;
  *fit = worse(fit_of(x, a.B, a.T, a.H, a.D, a.x.b, a.x.t, a.x.h),
               fit_of(gate, a.B, a.T, a.H, a.D, a.z.b, a.z.t, a.z.h));
  return GDR_OK;
}

template <bool BWD>
gdr_status launch_gated(GatedArgs& a, const Plan& p, cudaStream_t s) {
  a.groups = p.groups;
  a.pieces = p.pieces;
  a.stages = p.stages;
  if (p.lanes && p.v == 8 && !p.shift && a.in_bf16 == a.out_bf16)
    return with_dtype(a.in_bf16 ? GDR_BF16 : GDR_F32, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      auto go = [&](auto shape) {
        using S = decltype(shape);
        return launch_behind(a.first ? gated_rows_kernel<T, S::LANES, S::NV, BWD, true>
                                     : gated_rows_kernel<T, S::LANES, S::NV, BWD, false>,
                             dim3(p.blocks), p.threads, s, a);
      };
      return p.lanes == 8    ? go(Shape<8, 8, 1>())
             : p.lanes == 16 ? go(Shape<16, 8, 1>())
             : p.nv == 1     ? go(Shape<32, 8, 1>())
                             : go(Shape<32, 8, 2>());
    });
  return with_shape<true>(p, [&](auto shape) {
    using S = decltype(shape);
    struct Tag;
    if (p.smem > kPlainSmem && !allow_smem<Tag>(gated_kernel<S, BWD>, kSmemPerSm))
      return GDR_ERR_CUDA;
    return launch_behind_smem(gated_kernel<S, BWD>, dim3(p.blocks), p.threads, p.smem, s, a);
  });
}

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

gdr_status gdr_gated_norm(const void* x, const void* gate, const float* weight, void* y,
                          const gdr_gated_dims* dims, gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  GatedArgs a = {};
  Fit fit = kSingle;
  const gdr_status ok = gated_args(a, dims, x, gate, weight, &fit);
  if (ok != GDR_OK) return ok;
  if (!is_aligned(y, 16)) return GDR_ERR_ALIGNMENT;
  if (a.tokens == 0) return GDR_OK;
  if (!x || !gate || !y) return GDR_ERR_INVALID_ARG;
  a.y = y;
  return launch_gated<false>(a, gated_plan(dims, fit, false), reinterpret_cast<cudaStream_t>(stream));
}

size_t gdr_gated_norm_bwd_workspace_size(const gdr_gated_dims* dims) {
  if (check(dims) != GDR_OK) return 0;
  // The bases' alignment is not known here: room for every kernel.
  size_t most = kAlign;
  for (Fit fit : {dims->D % 8 ? kShift : kVec, kSingle}) {
    const size_t n = gated_bytes(dims, gated_plan(dims, fit, true));
    if (n > most) most = n;
  }
  return most;
}

gdr_status gdr_gated_norm_bwd(const void* d_y, const void* x, const void* gate, const float* weight,
                              void* dx, void* d_gate, float* d_weight, const gdr_gated_dims* dims,
                              void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  GatedArgs a = {};
  Fit fit = kSingle;
  const gdr_status ok = gated_args(a, dims, x, gate, weight, &fit);
  if (ok != GDR_OK) return ok;
  if (!is_aligned(d_y, 16) || !is_aligned(dx, 16) || !is_aligned(d_gate, 16) ||
      !is_aligned(d_weight, 16))
    return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int cols = dims->D * (a.per_head ? dims->H : 1);
  if (a.tokens == 0) return zero(d_weight, cols, s);
  if (!d_y || !x || !gate || !dx || !d_gate) return GDR_ERR_INVALID_ARG;
  const Plan p = gated_plan(dims, fit, true);
  if (d_weight) {
    if (!workspace || workspace_bytes < gdr_gated_norm_bwd_workspace_size(dims))
      return GDR_ERR_WORKSPACE;
    if (!is_aligned(workspace, kAlign)) return GDR_ERR_ALIGNMENT;
    a.part = static_cast<float*>(workspace);
  }
  const int64_t h = dims->D, t = h * dims->H;
  a.d = {d_y, t * dims->T, t, h};
  a.dx = dx;
  a.dz = d_gate;
  const gdr_status run = launch_gated<true>(a, p, s);
  if (run != GDR_OK || !d_weight) return run;
  return sum_parts(a.part, d_weight, nullptr, nullptr, p.rows, cols, s);
}

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
      // taken from the kernel before (training step of 4096 x 1536 with norm, gate and scale: 74.9 us
      // so, 70.7 not).
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
