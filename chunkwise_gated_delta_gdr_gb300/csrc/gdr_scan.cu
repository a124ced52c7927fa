// gdr_scan.cu -- gated linear recurrence with one state per channel.
//
//   h_t = a_t h_{t-1} + u_t,  a = exp(g),  u = x or (1 - a) x
//   l_t = dh_t + a_{t+1} l_{t+1};  dx = l (1 - a, gated),  dg = l a (h_{t-1} - x, gated)
#include <type_traits>

#include "gdr_ops.cuh"

namespace gdr {
namespace ops {
namespace {

constexpr int CK = GDR_SCAN_CHECKPOINT;

struct ScanArgs {
  const void *x, *g, *dh;
  const float* s0;     // initial state (forward), gradient of the final state (backward); may be null
  void *h, *dx, *dg;
  float* sT;           // final state (forward), gradient of the initial state (backward); may be null
  float* ck;           // checkpoints; may be null in the forward
  int B, T, D, N;      // N = ceil(T / CK)
  int gated;
  int64_t xb, xt, gb, gt, db, dt;   // strides in elements
};

// One thread per V channels, tokens in order.
template <typename X, typename G, typename H, int V>
__global__ void __launch_bounds__(128) scan_serial_kernel(ScanArgs a) {
  const int d = (blockIdx.x * 128 + threadIdx.x) * V, b = blockIdx.y;
  if (d >= a.D) return;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  H* h = static_cast<H*>(a.h) + (size_t)b * a.T * a.D + d;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;
#pragma unroll 4
  for (int t = 0; t < a.T; ++t) {
    float xv[V], gv[V];
    load_f<X, V>(x + t * a.xt, xv);
    load_f<G, V>(g + t * a.gt, gv);
    if (a.ck && t % CK == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) a.ck[((size_t)b * a.N + t / CK) * a.D + d + i] = s[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = expf(gv[i]);
      s[i] = fmaf(e, s[i], a.gated ? (1.f - e) * xv[i] : xv[i]);
    }
    store_f<H, V>(h + (size_t)t * a.D, s);
  }
  if (a.sT) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[(size_t)b * a.D + d + i] = s[i];
  }
}

// One thread per V channels, blocks of CK tokens from the last: each block's states are
// rebuilt from its checkpoint in stretches of 8 tokens, whose starts stay in registers.
template <typename X, typename G, typename H, int V>
__global__ void __launch_bounds__(128) scan_serial_bwd_kernel(ScanArgs a) {
  constexpr int S = 8;
  const int d = (blockIdx.x * 128 + threadIdx.x) * V, b = blockIdx.y;
  if (d >= a.D) return;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  const H* dh = static_cast<const H*>(a.dh) + b * a.db + d;
  X* dx = static_cast<X*>(a.dx) + (size_t)b * a.T * a.D + d;
  G* dg = static_cast<G*>(a.dg) + (size_t)b * a.T * a.D + d;
  float mu[V];                                   // exp(g_{t+1}) l_{t+1}
#pragma unroll
  for (int i = 0; i < V; ++i) mu[i] = a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;
  for (int n = a.N - 1; n >= 0; --n) {
    const int t0 = n * CK, t1 = min(a.T, t0 + CK);
    float s[V], start[CK / S][V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = a.ck[((size_t)b * a.N + n) * a.D + d + i];
#pragma unroll
    for (int j = 0; j < CK / S; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) start[j][i] = s[i];
      for (int t = t0 + j * S; t < min(t1, t0 + (j + 1) * S); ++t) {
        float xv[V], gv[V];
        load_f<X, V>(x + t * a.xt, xv);
        load_f<G, V>(g + t * a.gt, gv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = expf(gv[i]);
          s[i] = fmaf(e, s[i], a.gated ? (1.f - e) * xv[i] : xv[i]);
        }
      }
    }
#pragma unroll
    for (int j = CK / S - 1; j >= 0; --j) {
      float past[S][V];
      const int j0 = t0 + j * S;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = start[j][i];
#pragma unroll
      for (int r = 0; r < S; ++r) {
        if (j0 + r < t1) {
          float xv[V], gv[V];
          load_f<X, V>(x + (j0 + r) * a.xt, xv);
          load_f<G, V>(g + (j0 + r) * a.gt, gv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            past[r][i] = a.gated ? s[i] - xv[i] : s[i];
            const float e = expf(gv[i]);
            s[i] = fmaf(e, s[i], a.gated ? (1.f - e) * xv[i] : xv[i]);
          }
        }
      }
#pragma unroll
      for (int r = S - 1; r >= 0; --r) {
        const int t = j0 + r;
        if (t < t1) {
          float gv[V], dv[V], ox[V], og[V];
          load_f<G, V>(g + t * a.gt, gv);
          load_f<H, V>(dh + t * a.dt, dv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float e = expf(gv[i]), l = dv[i] + mu[i];
            ox[i] = a.gated ? l * (1.f - e) : l;
            mu[i] = e * l;
            og[i] = mu[i] * past[r][i];
          }
          store_f<X, V>(dx + (size_t)t * a.D, ox);
          store_f<G, V>(dg + (size_t)t * a.D, og);
        }
      }
    }
  }
  if (a.sT) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[(size_t)b * a.D + d + i] = mu[i];
  }
}

gdr_status check(const gdr_scan_dims* d) {
  if (!d) return GDR_ERR_INVALID_ARG;
  if (d->B < 0 || d->T < 0 || d->D <= 0) return GDR_ERR_INVALID_ARG;
  if (!is_dtype(d->x_dtype) || !is_dtype(d->g_dtype) || !is_dtype(d->h_dtype))
    return GDR_ERR_INVALID_ARG;
  const int64_t st[] = {d->x_stride_b, d->x_stride_t, d->g_stride_b,
                        d->g_stride_t, d->dh_stride_b, d->dh_stride_t};
  for (int64_t s : st)
    if (s < 0) return GDR_ERR_INVALID_ARG;
  if (d->B > 65535 || d->T > (1 << 30) || d->D > (1 << 28)) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

ScanArgs make_args(const gdr_scan_dims* d) {
  ScanArgs a = {};
  a.B = d->B; a.T = d->T; a.D = d->D;
  a.N = (int)(((int64_t)d->T + CK - 1) / CK);
  a.gated = d->gated_input != 0;
  a.xb = d->x_stride_b; a.xt = d->x_stride_t;
  a.gb = d->g_stride_b; a.gt = d->g_stride_t;
  a.db = d->dh_stride_b; a.dt = d->dh_stride_t;
  if (a.B == 1) a.xb = a.gb = a.db = 0;          // never stepped along
  if (a.T == 1) a.xt = a.gt = a.dt = 0;
  return a;
}

// Whether V elements at a time stay aligned: the strides of the views and their bases
// (the dense tensors' rows follow D, their bases are 16-byte aligned).
bool vec_ok(const void* p, int dtype, int64_t sb, int64_t st, int V) {
  return sb % V == 0 && st % V == 0 && is_aligned(p, dtype_size(dtype) * V);
}

// T == 0: out = in (or zeros).
gdr_status copy_state(float* out, const float* in, size_t n, cudaStream_t s) {
  if (!out || out == in || n == 0) return GDR_OK;
  const cudaError_t e = in ? cudaMemcpyAsync(out, in, n * 4, cudaMemcpyDeviceToDevice, s)
                           : cudaMemsetAsync(out, 0, n * 4, s);
  return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

template <bool kBwd, int V>
gdr_status launch(const gdr_scan_dims* d, const ScanArgs& a, cudaStream_t s) {
  const dim3 grid((a.D + 128 * V - 1) / (128 * V), a.B);
  return with_dtype(d->x_dtype, [&](auto* x) {
    return with_dtype(d->g_dtype, [&](auto* g) {
      return with_dtype(d->h_dtype, [&](auto* h) {
        using X = std::remove_pointer_t<decltype(x)>;
        using G = std::remove_pointer_t<decltype(g)>;
        using H = std::remove_pointer_t<decltype(h)>;
        if constexpr (kBwd)
          scan_serial_bwd_kernel<X, G, H, V><<<grid, 128, 0, s>>>(a);
        else
          scan_serial_kernel<X, G, H, V><<<grid, 128, 0, s>>>(a);
        return launched();
      });
    });
  });
}

}  // namespace
}  // namespace ops
}  // namespace gdr

using namespace gdr;
using namespace gdr::ops;

extern "C" {

size_t gdr_linear_scan_checkpoints_size(const gdr_scan_dims* dims) {
  if (check(dims) != GDR_OK) return 0;
  return (size_t)dims->B * (((size_t)dims->T + CK - 1) / CK) * dims->D * sizeof(float);
}

gdr_status gdr_linear_scan_fwd(const void* x, const void* g, const float* initial_state, void* h,
                               float* final_state, float* checkpoints, const gdr_scan_dims* dims,
                               gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  const bool work = dims->B > 0 && dims->T > 0;
  if (work && (!x || !g || !h)) return GDR_ERR_INVALID_ARG;
  if (!is_aligned(x, dtype_size(dims->x_dtype)) || !is_aligned(g, dtype_size(dims->g_dtype)) ||
      !is_aligned(h, 16) || !is_aligned(initial_state, 16) || !is_aligned(final_state, 16) ||
      !is_aligned(checkpoints, 16))
    return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!work) return copy_state(final_state, initial_state, (size_t)dims->B * dims->D, s);
  ScanArgs a = make_args(dims);
  a.x = x; a.g = g; a.s0 = initial_state; a.h = h; a.sT = final_state; a.ck = checkpoints;
  const bool vec = dims->D % 2 == 0 && vec_ok(x, dims->x_dtype, a.xb, a.xt, 2) &&
                   vec_ok(g, dims->g_dtype, a.gb, a.gt, 2);
  return vec ? launch<false, 2>(dims, a, s) : launch<false, 1>(dims, a, s);
}

gdr_status gdr_linear_scan_bwd(const void* dh, const void* x, const void* g,
                               const float* checkpoints, const float* d_final_state, void* dx,
                               void* dg, float* d_initial_state, const gdr_scan_dims* dims,
                               gdr_stream_t stream) {
  const gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  const bool work = dims->B > 0 && dims->T > 0;
  if (work && (!dh || !x || !g || !checkpoints || !dx || !dg)) return GDR_ERR_INVALID_ARG;
  if (!is_aligned(x, dtype_size(dims->x_dtype)) || !is_aligned(g, dtype_size(dims->g_dtype)) ||
      !is_aligned(dh, dtype_size(dims->h_dtype)) || !is_aligned(checkpoints, 16) ||
      !is_aligned(d_final_state, 16) || !is_aligned(dx, 16) || !is_aligned(dg, 16) ||
      !is_aligned(d_initial_state, 16))
    return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!work) return copy_state(d_initial_state, d_final_state, (size_t)dims->B * dims->D, s);
  ScanArgs a = make_args(dims);
  a.x = x; a.g = g; a.dh = dh; a.s0 = d_final_state; a.sT = d_initial_state;
  a.dx = dx; a.dg = dg; a.ck = const_cast<float*>(checkpoints);
  const bool vec = dims->D % 2 == 0 && vec_ok(x, dims->x_dtype, a.xb, a.xt, 2) &&
                   vec_ok(g, dims->g_dtype, a.gb, a.gt, 2) &&
                   vec_ok(dh, dims->h_dtype, a.db, a.dt, 2);
  return vec ? launch<true, 2>(dims, a, s) : launch<true, 1>(dims, a, s);
}

}  // extern "C"
