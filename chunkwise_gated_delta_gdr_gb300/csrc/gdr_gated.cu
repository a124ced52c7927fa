// gdr_gated.cu -- the RMS norm of a layer's output heads with its output gate, forward and
// backward. With a = act(z):
//   y = u w a,  u = x r,  r = 1 / sqrt(mean(x^2) + eps)        (gate behind the norm)
//   y = u w,    u = v r,  v = x a, r of v                      (gate before the norm)
// and with d the gradient of y
//   behind: dw = sum d a u,  c = d a w,  dx = r (c - u mean(c u)),  dz = d u w a'
//   before: dw = sum d u,    c = d w,    dv = r (c - u mean(c u)),  dx = dv a,  dz = dv x a'
//
// Every tensor is read once and written once: bound by HBM where there is enough of it, by the
// chain load - sum over the row - store of one row below. Measured on one GB300, bf16, a pass
// among others (a plain copy: 6.70 TB/s):
//   2 x 8192 x 32 heads of 128: 62.7 us, 6.4 TB/s; 64 decode tokens x 16 heads 2.5 us
//   training step, 4096 x 12 heads of 128: 24.3 us (forward 9, backward 14, weights' sums 5 with
//   cold caches); 2 x 4096 x 4 groups of 512, gate first, weights per group 51.4 us; whole rows,
//   8192 x 1536 55 us, 4096 x 4096 69 us, 36288 rows of 173 58 us
#include "gdr_norm.cuh"

namespace gdr {
namespace ops {
namespace {

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

// Rows of at most 512 channels: a group of LANES lanes per row, NV runs of 8 channels a lane, UN
// rows at a time (the group's head in UN tokens), the next ones' loads under way meanwhile. What
// bounds the larger calls beside HBM is the number of instructions per row, so addresses step
// from row to row and sums and products go in pairs; the copies through shared memory that wider
// rows take cost twice the time here (2 x 8192 x 32 heads of 128 forward: 115 us so, 57 now).
// (Three blocks an SM forward, 80 registers, are for bf16; in 32 bits 257 to 512 channels spill some
// 90 bytes: 2 x 4096 x 4 groups of 512 34.4 us, 5.85 TB/s.)
template <typename T, int LANES, int NV, bool BWD, bool FIRST>
__global__ void __launch_bounds__(256, BWD ? 2 : 3) gated_rows_kernel(GatedArgs a) {
  typedef Shape<LANES, 8, NV> S;
  constexpr int TENSORS = BWD ? 3 : 2, UN = sizeof(T) == 2 && NV == 1 ? 2 : 1, N = 4 * NV;
  constexpr int Q = 8 * sizeof(T) / 16;          // 16-byte pieces of 8 channels
  constexpr bool AHEAD = NV == 1 || !BWD;        // else there are no registers for the next rows
  __shared__ float sums[BWD ? S::kSums : 1];
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
      float zs[2 * N], gs[2 * N], as[2 * N], sl[2 * N];
#pragma unroll
      for (int i = 0; i < N; ++i) put_pair(zs, 2 * i, z[i]);
#pragma unroll
      for (int c = 0; c < 2 * N; c += 8) {
        gate_sigma<8>(gs + c, zs + c, a.kind);
        gate_open<8>(as + c, gs + c, zs + c, a.kind);
        if (BWD) gate_slope<8>(sl + c, gs + c, zs + c, a.kind);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 g = pair_at(as, 2 * i);
        const float2 slope = BWD ? pair_at(sl, 2 * i) : g;
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
// TY: the types of a call, where they are the usual ones.
enum { kAnyTypes, kAllBf16, kAllF32 };
template <class S, int TY, bool BWD>
__global__ void __launch_bounds__(kMaxThreads, !BWD && S::N <= 16 && !S::SHIFT && !S::kGroups ? 2 : 1)
    gated_kernel(GatedArgs a) {
  constexpr int V = S::V, NV = S::NV, N = S::N, TENSORS = BWD ? 3 : 2;
  extern __shared__ __align__(16) char places[];
  __shared__ Red red;
  __shared__ float sums[BWD ? S::kSums : 1];
  const Walk w = walk_of<S::LANES>(a.tokens, a.H, a.groups);
  const int phase = S::SHIFT ? (int)((((long long)w.tok * a.H + w.head) * a.D) & 7) : 0;
  const int in_bf16 = TY == kAnyTypes ? a.in_bf16 : TY == kAllBf16;
  const int out_bf16 = TY == kAnyTypes ? a.out_bf16 : TY == kAllBf16;
  const Ahead ahead(places, a.pieces, a.stages);
  const float* weight = a.w && a.per_head ? a.w + (size_t)w.head * a.D : a.w;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;

  Row<S, true> row[TENSORS];
  auto has = [&](int it) { return w.on && w.tok + it * w.step < a.tokens; };
  auto locate = [&](int it) {
    const int tok = w.tok + it * w.step, per = NV * (in_bf16 ? 1 : 2);
    row[0].set(a.x.p, a.x.at(tok, a.T, a.flat, w.head), in_bf16, 0);
    row[1].set(a.z.p, a.z.at(tok, a.T, a.flat, w.head), in_bf16, per);
    if (BWD) row[TENSORS - 1].set(a.d.p, a.d.at(tok, a.T, 1, w.head), out_bf16, 2 * per);
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
    float s[2] = {0.f, 0.f}, g[N];               // g: the gates' sigmoids
    if (on)
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        group_at<S>(w, c, a.D, row[0]);
        if (a.first || BWD) group_at<S>(w, c, a.D, row[1]);
        if (BWD) group_at<S>(w, c, a.D, row[TENSORS - 1]);
        const int i = (c * w.threads + w.tid) * V - phase;
        if (i >= a.D) continue;
        float x[V], z[V], t[V];
        row[0].get(ahead, at, c, i, a.D, x);
        if (a.first || BWD) {
          row[1].get(ahead, at, c, i, a.D, z);
          gate_sigma<V>(g + c * V, z, a.kind);
          gate_open<V>(t, g + c * V, z, a.kind);
        }
        if (a.first) mul_run<V>(x, x, t);
        s[0] += dot_run<V>(x, x);
        if (BWD) {
          float d[V];
          row[TENSORS - 1].get(ahead, at, c, i, a.D, d);
          if (!a.first) mul_run<V>(d, d, t);
          if (weight) {
            load_shared<S>(weight, i, a.D, t);
            mul_run<V>(d, d, t);
          }
          s[1] += dot_run<V>(d, x);
        }
      }
    row_sum<S::LANES, BWD ? 2 : 1>(s, red, turn);
    if (!on) continue;
    const float r = rsqrtf(fmaf(s[0], a.inv_d, a.eps)), m = s[1] * a.inv_d * r;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      group_at<S>(w, c, a.D, row[0], row[1]);
      if (BWD) group_at<S>(w, c, a.D, row[TENSORS - 1]);
      const int i = (c * w.threads + w.tid) * V - phase;
      if (i >= a.D) continue;
      float *gc = g + c * V, x[V], z[V], t[V], u[V], wt[V];
      row[0].get(ahead, at, c, i, a.D, x);
      row[1].get(ahead, at, c, i, a.D, z);
      if (!BWD && !a.first) gate_sigma<V>(gc, z, a.kind);
      gate_open<V>(t, gc, z, a.kind);            // a
      if (weight) load_shared<S>(weight, i, a.D, wt);
      if (a.first) {
        mul_run<V>(u, x, t);
        scale_run<V>(u, u, r);
      } else {
        scale_run<V>(u, x, r);
      }
      if constexpr (!BWD) {
        if (weight) mul_run<V>(u, u, wt);
        if (!a.first) mul_run<V>(u, u, t);
        store_row<S>(a.y, dense, i, a.D, out_bf16, u);
      } else {
        float d[V], q[V];
        row[TENSORS - 1].get(ahead, at, c, i, a.D, d);
        gate_slope<V>(z, gc, z, a.kind);         // a'
        if (a.first) {
          fma_run<V>(acc + c * V, d, u, acc + c * V);
          if (weight) mul_run<V>(d, d, wt);
          fma_run<V>(q, u, -m, d);
          scale_run<V>(q, q, r);                 // dv
          mul_run<V>(t, t, q);                   // dx
          mul_run<V>(z, z, x);
          mul_run<V>(z, z, q);                   // dz
          store_row<S>(a.dx, dense, i, a.D, in_bf16, t);
        } else {
          mul_run<V>(q, d, t);
          fma_run<V>(acc + c * V, q, u, acc + c * V);
          if (weight) {
            mul_run<V>(q, q, wt);
            mul_run<V>(d, d, wt);
          }
          fma_run<V>(q, u, -m, q);
          scale_run<V>(q, q, r);                 // dx
          mul_run<V>(z, z, u);
          mul_run<V>(z, z, d);                   // dz
          store_row<S>(a.dx, dense, i, a.D, in_bf16, q);
        }
        store_row<S>(a.dz, dense, i, a.D, in_bf16, z);
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

// ------------------------------------------------------------------ host
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

Plan gated_plan(const gdr_gated_dims* d, Fit fit, bool bwd) {
  const int in = d->in_dtype == GDR_BF16 ? 1 : 2, out = d->out_dtype == GDR_BF16 ? 1 : 2;
  const int per_sm = fit == kVec && d->D <= 512 ? (bwd ? kBwdRowsPerSm : kFwdRowsPerSm)
                     : bwd                      ? kGatedBwdPerSm
                     : fit == kShift            ? kGatedShiftPerSm
                                                : kFwdPerSm;
  return make_plan(d->B * d->T, d->H, d->D, 2 * in + (bwd ? out : 0), fit, 512,
                   d->weight_per_head != 0, per_sm);
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
    auto go = [&](auto types) {
      constexpr int TY = decltype(types)::value;
      struct Tag;
      if (p.smem > kPlainSmem && !allow_smem<Tag>(gated_kernel<S, TY, BWD>, kSmemPerSm))
        return GDR_ERR_CUDA;
      return launch_behind_smem(gated_kernel<S, TY, BWD>, dim3(p.blocks), p.threads, p.smem, s, a);
    };
    if constexpr (S::kAhead && (S::LANES == 0 || S::SHIFT))
      if (a.in_bf16 == a.out_bf16)
        return a.in_bf16 ? go(std::integral_constant<int, kAllBf16>())
                         : go(std::integral_constant<int, kAllF32>());
    return go(std::integral_constant<int, kAnyTypes>());
  });
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

}  // extern "C"
