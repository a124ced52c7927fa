// gdr_scan.cu -- gated linear recurrence with one state per channel.
//
//   h_t = a_t h_{t-1} + u_t,  a = exp(g),  u = x or (1 - a) x
//   l_t = dh_t + a_{t+1} l_{t+1};  dx = l (1 - a, gated),  dg = l a (h_{t-1} - x, gated)
#include <type_traits>

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"

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

// ------------------------------------------------------------ split along the sequence
// A cluster of S blocks walks the tokens of one column block (32 V channels) in steps of S
// tiles of TILE tokens, a tile per block, R tokens of it per warp. A stretch of tokens acts
// on the state as h -> A h + H (A the product of its a), and two stretches compose as
// (A2 A1, A2 H1 + H2). Per step each warp forms the pair of its tokens from registers, the
// warps' pairs meet in shared memory, the blocks' pairs in every block's shared memory
// (written remotely), and one cluster barrier later each warp knows the state before its
// first token and runs its tokens again, now with it, from the same registers. The next
// step's tokens load meanwhile. All orders are fixed.
constexpr int W = 8, R = 8, TILE = W * R, MAXS = 16;
static_assert(TILE == CK, "a tile starts at a checkpoint");

// Pairs (or triples) of the warps, double-buffered by step: one barrier per step suffices,
// as a buffer is written again only after the barrier of the step between.
template <int V>
struct alignas(16) ScanShared {
  float warp[2][W][3][32 * V];
  float block[2][MAXS][2][32 * V];
};

template <int V>
__device__ __forceinline__ void put_v(float* p, const float* v) {
  store_f<float, V>(p, v);
}
template <int V>
__device__ __forceinline__ void get_v(const float* p, float* v) {
  load_f<float, V>(p, v);
}
template <int V>
__device__ __forceinline__ void copy_v(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = v[i];
}

// Writes v to the same shared location in block `rank` of the cluster.
template <int V>
__device__ __forceinline__ void put_remote(float* p, uint32_t rank, const float* v) {
  const uint32_t at = ptx::mapa(ptx::smem_u32(p), rank);
#pragma unroll
  for (int i = 0; i < V; ++i)
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4 * i), "f"(v[i]) : "memory");
}

// The cluster's pairs applied to `carry`: in, the state before this step; returns the state
// before this block's tile, and leaves the state after the step in carry. tA, tH: this
// block's pair. Includes the step's barrier.
template <int V>
__device__ __forceinline__ void cluster_carry(ScanShared<V>& sm, int par, int S, int rank,
                                              int warp, int lane, const float* tA,
                                              const float* tH, float* carry, float* mine) {
  if (S == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine[i] = carry[i];
      carry[i] = fmaf(tA[i], carry[i], tH[i]);
    }
    return;
  }
  for (int q = warp; q < S; q += W) {
    put_remote<V>(&sm.block[par][rank][0][lane * V], q, tA);
    put_remote<V>(&sm.block[par][rank][1][lane * V], q, tH);
  }
  ptx::cluster_sync();
#pragma unroll 4
  for (int q = 0; q < S; ++q) {
    float qA[V], qH[V];
    get_v<V>(&sm.block[par][q][0][lane * V], qA);
    get_v<V>(&sm.block[par][q][1][lane * V], qH);
    if (q == rank) copy_v<V>(mine, carry);
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = fmaf(qA[i], carry[i], qH[i]);
  }
}

template <typename X, typename G, typename H, int V>
__global__ void __launch_bounds__(W * 32, 3) scan_kernel(ScanArgs a, int S) {
  __shared__ ScanShared<V> sm;
  const int rank = blockIdx.x % S, col = blockIdx.x / S, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = (col * 32 + lane) * V;
  const bool on = d < a.D;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  H* h = static_cast<H*>(a.h) + (size_t)b * a.T * a.D + d;
  float carry[V];
#pragma unroll
  for (int i = 0; i < V; ++i) carry[i] = on && a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;

  Raw<X, V> xr[R];
  Raw<G, V> gr[R];
  auto load = [&](int t0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (on && t0 + r < a.T) {
        xr[r] = load_once<X, V>(x + (t0 + r) * a.xt);
        gr[r] = load_once<G, V>(g + (t0 + r) * a.gt);
      }
    }
  };
  const int steps = (a.N + S - 1) / S;
  int t0 = rank * TILE + warp * R;
  load(t0);
  for (int step = 0; step < steps; ++step, t0 += S * TILE) {
    const int par = step & 1;
    float e[R][V], u[R][V], A[V], P[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, P[i] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (on && t0 + r < a.T) {
        to_float<X, V>(xr[r], u[r]);
        to_float<G, V>(gr[r], e[r]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[r][i] = expf(e[r][i]);
          if (a.gated) u[r][i] *= 1.f - e[r][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) e[r][i] = 1.f, u[r][i] = 0.f;
      }
    }
    load(t0 + S * TILE);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        P[i] = fmaf(e[r][i], P[i], u[r][i]);
        A[i] *= e[r][i];
      }
    put_v<V>(&sm.warp[par][warp][0][lane * V], A);
    put_v<V>(&sm.warp[par][warp][1][lane * V], P);
    __syncthreads();
    float pA[V], pH[V], tA[V], tH[V], s[V];      // before this warp; of the whole tile
#pragma unroll
    for (int i = 0; i < V; ++i) tA[i] = 1.f, tH[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w == warp) {
        copy_v<V>(pA, tA);
        copy_v<V>(pH, tH);
      }
      float wA[V], wH[V];
      get_v<V>(&sm.warp[par][w][0][lane * V], wA);
      get_v<V>(&sm.warp[par][w][1][lane * V], wH);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        tH[i] = fmaf(wA[i], tH[i], wH[i]);
        tA[i] *= wA[i];
      }
    }
    cluster_carry<V>(sm, par, S, rank, warp, lane, tA, tH, carry, s);
    if (a.ck && warp == 0 && on && t0 < a.T) {
#pragma unroll
      for (int i = 0; i < V; ++i) a.ck[((size_t)b * a.N + t0 / CK) * a.D + d + i] = s[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = fmaf(pA[i], s[i], pH[i]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = fmaf(e[r][i], s[i], u[r][i]);
      if (on && t0 + r < a.T) store_f<H, V>(h + (size_t)(t0 + r) * a.D, s);
    }
  }
  if (a.sT && rank == 0 && warp == 0 && on) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[(size_t)b * a.D + d + i] = carry[i];
  }
}

// The same walk from the last tile back. What travels is mu_t = a_t l_t, the gradient that
// reaches h_{t-1}: a stretch maps the mu after it to A mu + M, with the same A. The states
// inside a tile come from its checkpoint and the warps' forward pairs.
template <typename X, typename G, typename H, int V>
__global__ void __launch_bounds__(W * 32, 2) scan_bwd_kernel(ScanArgs a, int S) {
  __shared__ ScanShared<V> sm;
  const int rank = blockIdx.x % S, col = blockIdx.x / S, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = (col * 32 + lane) * V;
  const bool on = d < a.D;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  const H* dh = static_cast<const H*>(a.dh) + b * a.db + d;
  const float* ck = a.ck + (size_t)b * a.N * a.D + d;
  X* dx = static_cast<X*>(a.dx) + (size_t)b * a.T * a.D + d;
  G* dg = static_cast<G*>(a.dg) + (size_t)b * a.T * a.D + d;
  float carry[V];
#pragma unroll
  for (int i = 0; i < V; ++i) carry[i] = on && a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;

  Raw<X, V> xr[R];
  Raw<G, V> gr[R];
  Raw<H, V> dr[R];
  float cr[V];
  auto load = [&](int n) {
    if (!on || n < 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i) cr[i] = ck[(size_t)n * a.D + i];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = n * TILE + warp * R + r;
      if (t < a.T) {
        xr[r] = load_once<X, V>(x + t * a.xt);
        gr[r] = load_once<G, V>(g + t * a.gt);
        dr[r] = load_once<H, V>(dh + t * a.dt);
      }
    }
  };
  const int steps = (a.N + S - 1) / S;
  int n = a.N - 1 - rank;
  load(n);
  for (int step = 0; step < steps; ++step, n -= S) {
    const int par = step & 1, t0 = n * TILE + warp * R;
    float e[R][V], u[R][V], l[R][V], hs[V], A[V], P[V], M[V];
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, P[i] = M[i] = 0.f, hs[i] = cr[i];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (on && n >= 0 && t0 + r < a.T) {
        to_float<X, V>(xr[r], u[r]);
        to_float<G, V>(gr[r], e[r]);
        to_float<H, V>(dr[r], l[r]);
#pragma unroll
        for (int i = 0; i < V; ++i) e[r][i] = expf(e[r][i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) e[r][i] = 1.f, u[r][i] = l[r][i] = 0.f;
      }
    }
    load(n - S);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        P[i] = fmaf(e[r][i], P[i], a.gated ? (1.f - e[r][i]) * u[r][i] : u[r][i]);
        A[i] *= e[r][i];
      }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int i = 0; i < V; ++i) M[i] = e[r][i] * (l[r][i] + M[i]);
    put_v<V>(&sm.warp[par][warp][0][lane * V], A);
    put_v<V>(&sm.warp[par][warp][1][lane * V], P);
    put_v<V>(&sm.warp[par][warp][2][lane * V], M);
    __syncthreads();
    float pA[V], pM[V], tA[V], tM[V], mu[V];     // after this warp; of the whole tile
#pragma unroll
    for (int i = 0; i < V; ++i) tA[i] = 1.f, tM[i] = 0.f;
#pragma unroll
    for (int w = W - 1; w >= 0; --w) {
      if (w == warp) {
        copy_v<V>(pA, tA);
        copy_v<V>(pM, tM);
      }
      float wA[V], wM[V];
      get_v<V>(&sm.warp[par][w][0][lane * V], wA);
      get_v<V>(&sm.warp[par][w][2][lane * V], wM);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        tM[i] = fmaf(wA[i], tM[i], wM[i]);
        tA[i] *= wA[i];
      }
    }
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
      if (w < warp) {
        float wA[V], wH[V];
        get_v<V>(&sm.warp[par][w][0][lane * V], wA);
        get_v<V>(&sm.warp[par][w][1][lane * V], wH);
#pragma unroll
        for (int i = 0; i < V; ++i) hs[i] = fmaf(wA[i], hs[i], wH[i]);
      }
    cluster_carry<V>(sm, par, S, rank, warp, lane, tA, tM, carry, mu);
#pragma unroll
    for (int i = 0; i < V; ++i) mu[i] = fmaf(pA[i], mu[i], pM[i]);
    // u becomes what dg multiplies: h_{t-1}, minus x_t when gated.
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float past = a.gated ? hs[i] - u[r][i] : hs[i];
        hs[i] = fmaf(e[r][i], hs[i], a.gated ? (1.f - e[r][i]) * u[r][i] : u[r][i]);
        u[r][i] = past;
      }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float ox[V], og[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float lr = l[r][i] + mu[i];
        ox[i] = a.gated ? lr * (1.f - e[r][i]) : lr;
        mu[i] = e[r][i] * lr;
        og[i] = mu[i] * u[r][i];
      }
      if (on && n >= 0 && t0 + r < a.T) {
        store_f<X, V>(dx + (size_t)(t0 + r) * a.D, ox);
        store_f<G, V>(dg + (size_t)(t0 + r) * a.D, og);
      }
    }
  }
  if (a.sT && rank == 0 && warp == 0 && on) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.sT[(size_t)b * a.D + d + i] = carry[i];
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

// Tokens up to which one thread runs a channel's tokens by itself.
constexpr int kSerial = 8;

// Blocks along the sequence for a kernel: as many as keep every cluster resident at once.
int cluster_size(const void* fn, int resident, const ScanArgs& a, int V) {
  const long long cols = (a.D + 32 * V - 1) / (32 * V) * (long long)a.B;
  long long s = 152LL * resident / (cols > 0 ? cols : 1);
  if (s > MAXS) s = MAXS;
  if (s > a.N) s = a.N;
  (void)fn;
  return s < 1 ? 1 : (int)s;
}

template <bool kBwd, int V>
gdr_status launch(const gdr_scan_dims* d, const ScanArgs& a, cudaStream_t s) {
  return with_dtype(d->x_dtype, [&](auto* x) {
    return with_dtype(d->g_dtype, [&](auto* g) {
      return with_dtype(d->h_dtype, [&](auto* h) {
        using X = std::remove_pointer_t<decltype(x)>;
        using G = std::remove_pointer_t<decltype(g)>;
        using H = std::remove_pointer_t<decltype(h)>;
        if constexpr (!kBwd) {
          if (a.T <= kSerial) {
            const dim3 grid((a.D + 128 * V - 1) / (128 * V), a.B);
            scan_serial_kernel<X, G, H, V><<<grid, 128, 0, s>>>(a);
            return launched();
          }
        }
        auto fn = kBwd ? scan_bwd_kernel<X, G, H, V> : scan_kernel<X, G, H, V>;
        const int S = cluster_size((const void*)fn, kBwd ? 2 : 3, a, V);
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = S;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((a.D + 32 * V - 1) / (32 * V) * S, a.B);
        cfg.blockDim = dim3(W * 32);
        cfg.stream = s;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (S > 8 && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                         cudaSuccess) {
          (void)cudaGetLastError();
          return GDR_ERR_CUDA;
        }
        const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a, S);
        if (e != cudaSuccess) {
          (void)cudaGetLastError();
          return GDR_ERR_CUDA;
        }
        return GDR_OK;
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
