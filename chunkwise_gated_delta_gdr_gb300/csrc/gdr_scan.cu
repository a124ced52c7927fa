// gdr_scan.cu -- gated linear recurrence with one state per channel.
//
//   h_t = a_t h_{t-1} + u_t,  a = exp(g),  u = x or (1 - a) x
//   l_t = dh_t + a_{t+1} l_{t+1};  dx = l (1 - a, gated),  dg = l a (h_{t-1} - x, gated)
//
// About 4 operations per element forward and 14 with the backward, against 8 and 14 bytes
// (bf16 x, fp32 g): bound by HBM where there are channels or sequences enough, by the
// latency of a step (see below) where there are not. Every element is read once and written
// once: the sequence is split without a second pass.
//
// Measured on one GB300, fp32 g, us (TB/s; a plain copy: 6.78), forward and backward:
//   bf16 x         1 x 65000 x 4096       2 x 8192 x 4096      1 x 4096 x 1536
//     u = x        318 (6.7) 584 (6.4)    84 (6.4) 149 (6.3)   16.8 (3.0) 24.7 (3.6)
//     (1 - a) x    324 (6.6) 629 (5.9)    86 (6.2) 161 (5.8)   18.5 (2.7) 26.7 (3.3)
//   fp32 x, (1 - a) x                    139 (5.8) 201 (6.7)   19.4 (3.9) 28.8 (4.4)
//   fp32, 3 x 1021 x 777 (rows that no tensor copy can read): 10.4 (2.7) 16.6 (2.9); gated 11.5, 18.6
#include <type_traits>

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"
#include "gdr_tmap.cuh"

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
  long polls;          // bound of a wait
  int64_t xb, xt, gb, gt, db, dt;   // strides in elements
};

// g becomes a = exp(g), m the weights 1 - a of gated inputs. Near g = 0 the difference d = 1 - a
// loses what it is made of (13 % of it at g = -1e-6). There the weight is -g times the mean of
// exp over [0, g], taken by the trapezoidal rule with the first Euler-Maclaurin correction,
// 1 - d / 2 + g d / 12, whose next term is below 4e-7; beyond |g| = 0.13 the difference keeps
// a's error, under 1e-6 of it. (Pairs go two operations an instruction. Against the difference
// alone: 86 us instead of 83 forward, 161 instead of 153 backward, at 2 x 8192 x 4096.)
template <int V>
__device__ __forceinline__ void gate(float* g, float* m) {
  constexpr float kNear = 0.13f;
  if constexpr (V == 2) {
    auto both = [](float c) { return make_float2(c, c); };
    const float2 x = make_float2(g[0], g[1]), e = make_float2(expf(x.x), expf(x.y));
    const float2 d = fma2(e, both(-1.f), both(1.f));
    const float2 c = fma2(x, both(1.f / 12), both(-0.5f));
    const float2 w = mul2(x, fma2(d, c, both(1.f)));
    m[0] = fabsf(x.x) < kNear ? -w.x : d.x;
    m[1] = fabsf(x.y) < kNear ? -w.y : d.y;
    g[0] = e.x, g[1] = e.y;
  } else {
    const float x = g[0], e = expf(x), d = 1.f - e;
    const float w = x * fmaf(d, fmaf(x, 1.f / 12, -0.5f), 1.f);
    m[0] = fabsf(x) < kNear ? -w : d;
    g[0] = e;
  }
}

// One thread per V channels, tokens in order: decode steps and short prompts, bound by the
// launch (64 x 1 x 2048: 4.1 us a call, 3 us of it the kernel).
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
#pragma unroll 8
  for (int t = 0; t < a.T; ++t) {
    float xv[V], gv[V];
    load_f<X, V>(x + t * a.xt, xv);
    load_f<G, V>(g + t * a.gt, gv);
    if (a.ck && t % CK == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) a.ck[((size_t)b * a.N + t / CK) * a.D + d + i] = s[i];
    }
    if (a.gated) {
      float m[V];
      gate<V>(gv, m);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = fmaf(gv[i], s[i], m[i] * xv[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = fmaf(expf(gv[i]), s[i], xv[i]);
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
// tiles, a tile of W R tokens per block, R of them per warp. A stretch of tokens acts on the
// state as h -> A h + P (A the product of its a), and two stretches compose as
// (A2 A1, A2 P1 + P2). Per step each warp forms the pair of its tokens from registers, the
// warps' pairs meet in shared memory, the blocks' pairs in every block's shared memory, sent
// there with their bytes counted on a barrier of the receiver (one way, where a cluster
// barrier takes a round trip). Then each warp knows the state before its first token and
// runs its tokens again from the same registers, now with it. All orders are fixed.
// A step of a block alone on its SM takes about 1.6 us, 0.5 of them the exchange; with more
// warps and fewer rows each it took longer (16 warps of 8 rows: 1.54 instead of 1.15 us
// without the exchange).
constexpr int W = 8, MAXS = 8;

// Tokens per warp: as many as leave two blocks on an SM, registers and shared memory both.
template <typename X, typename G, int V>
constexpr int kRows = V == 1 || sizeof(X) + sizeof(G) <= 6 ? 16 : 8;

// Pairs (or triples) of the warps and pairs of the blocks, double-buffered by step: a buffer
// is written again only after the block barrier of the step between, and after every block
// has sent that step's pair, which it does once it has read this one.
template <int V, bool kBwd>
struct alignas(16) ScanShared {
  float warp[2][W][32][2 * V];
  float back[kBwd ? 2 : 1][kBwd ? W : 1][32][V];
  float block[2][MAXS][32][2 * V];
  uint64_t full[4];                  // ring stages (tensor copies)
  uint64_t met[2];                   // the blocks' pairs
};

template <int N>
__device__ __forceinline__ void put_v(float* p, const float* v) {
  store_f<float, N>(p, v);
}
template <int N>
__device__ __forceinline__ void get_v(const float* p, float* v) {
  load_f<float, N>(p, v);
}
template <int V>
__device__ __forceinline__ void copy_v(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = v[i];
}

// Waits are bounded. Each thread holds `lost`, 0 until one of its waits gives up (then one more
// than the number of tiles it has seen arrive). It then waits for nothing more, its channels'
// rows are NaN from that tile on, and so are the pairs formed with its own: no wrong state goes
// on as a finite number. It sends nothing more either, since pairs of two steps would be
// counted as one, so that blocks that wait for it give up as well. Thread 0 starts no copies
// then; see leave() for those under way.

// Bounded wait for the pairs of a step, acquiring what other blocks of the cluster sent.
__device__ __forceinline__ bool met_wait(uint64_t* bar, uint32_t parity, long polls) {
  const uint32_t at = ptx::smem_u32(bar);
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(at), "r"(parity)
      : "memory");
  for (long i = 0; !ok && i < polls; ++i)
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
  return ok != 0;
}

// The blocks' pairs of a step applied to `carry` (the state before the step): `mine` becomes
// the state before this block's tile, carry the state after the step.
template <int V, bool kBwd>
__device__ __forceinline__ void cluster_carry(ScanShared<V, kBwd>& sm, int step, int S, int rank,
                                              int warp, int lane, long polls, const float* tA,
                                              const float* tP, float* carry, float* mine,
                                              int& lost) {
  if (S == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine[i] = carry[i];
      carry[i] = fmaf(tA[i], carry[i], tP[i]);
    }
    return;
  }
  const int par = step & 1;
  if (threadIdx.x == 0 && !lost) ptx::mbar_expect_tx(&sm.met[par], S * 32 * 2 * V * 4);
  if (warp < S && !lost) {
    const uint32_t dst = ptx::mapa(ptx::smem_u32(sm.block[par][rank][lane]), warp);
    const uint32_t bar = ptx::mapa(ptx::smem_u32(&sm.met[par]), warp);
    if constexpr (V == 2)
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
          "[%5];" ::"r"(dst), "f"(tA[0]), "f"(tA[1]), "f"(tP[0]), "f"(tP[1]), "r"(bar)
          : "memory");
    else
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
              dst), "f"(tA[0]), "f"(tP[0]), "r"(bar)
          : "memory");
  }
  if (!lost && !met_wait(&sm.met[par], (step >> 1) & 1, polls)) lost = step + 2;
  if (lost) {
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = NAN;
  }
#pragma unroll 2
  for (int q = 0; q < S; ++q) {
    if (q == rank) copy_v<V>(mine, carry);
    float m[2 * V];
    get_v<2 * V>(sm.block[par][q][lane], m);
#pragma unroll
    for (int i = 0; i < V; ++i) carry[i] = fmaf(m[i], carry[i], m[V + i]);
  }
}

// A block's last act. Copies that thread 0 started and did not see arrive (where there(step)) are
// waited for, again with a bound. No block leaves while another may send to it; pairs sent
// before that barrier that a block has not seen arrive need a microsecond more: it stays a
// thousand.
constexpr long kDrainPolls = 1L << 20;           // about a second
template <int ST, typename F>
__device__ __forceinline__ void leave(uint64_t* full, int lost, int S, F there) {
  if constexpr (ST > 0) {
    if (lost && threadIdx.x == 0)
      for (int j = lost - 1; j < lost - 1 + ST; ++j)
        if (there(j)) (void)ptx::mbar_wait(&full[j % ST], (j / ST) & 1, kDrainPolls);
  }
  if (S == 1) return;
  __syncwarp();
  ptx::cluster_sync();
  if (lost)
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// One tensor's tiles on their way into a ring in shared memory, token-major. kTensor: a
// thread copies whole tiles, out-of-range tokens and channels arriving as zeros (so that
// a = exp(0) = 1 and u = 0 there: tokens that change nothing). Otherwise each thread copies
// its own channels' tokens, 4 or 8 bytes asynchronously, a single bf16 (too small for such a
// copy) through registers; it reads only those, so it waits for itself alone.
template <typename T, int V, int R, bool kTensor>
struct Feed {
  static constexpr bool kRing = kTensor || sizeof(T) * V >= 4;
  static constexpr int kBytes = kRing ? W * R * 32 * V * (int)sizeof(T) : 0;    // of a stage
  Raw<T, V> reg[kRing ? 1 : R];
  char* base;
  __device__ __forceinline__ Feed(char* ring, int warp, int lane)
      : base(ring + (warp * R * 32 + lane) * V * (int)sizeof(T)) {}
  __device__ __forceinline__ void fetch(int offset, int r, const T* p) {
    if constexpr (kRing)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                       ptx::smem_u32(base + offset + r * (32 * V * (int)sizeof(T)))),
                   "l"(p), "n"(V * (int)sizeof(T))
                   : "memory");
    else
      reg[r] = load_once<T, V>(p);
  }
  __device__ __forceinline__ void take(int offset, int r, float* f) const {
    if constexpr (kRing)
      load_f<T, V>(
          reinterpret_cast<const T*>(base + offset + r * (32 * V * (int)sizeof(T))), f);
    else
      to_float<T, V>(reg[r], f);
  }
};

// Tiles under way. Without a ring for every tensor: the one the registers hold.
template <typename X, typename G, typename H, int V, bool kTensor>
constexpr int kStages =
    kTensor || (sizeof(X) * V >= 4 && sizeof(G) * V >= 4 && sizeof(H) * V >= 4) ? 2 : 1;

struct ScanMaps {
  CUtensorMap x, g, dh;
};

template <typename X, typename G, typename H, int V, bool kTensor, bool kGated>
struct Fwd {
  static constexpr int R = kRows<X, G, V>, TILE = W * R, ST = kStages<X, G, float, V, kTensor>;
  static constexpr int XB = Feed<X, V, R, kTensor>::kBytes, GB = Feed<G, V, R, kTensor>::kBytes;
  static constexpr int SB = XB + GB, SMEM = ST * SB;
};

template <typename X, typename G, typename H, int V, bool kTensor, bool kGated>
__global__ void __launch_bounds__(W * 32, 2)
    scan_kernel(const __grid_constant__ ScanMaps maps, ScanArgs a, int S) {
  using F = Fwd<X, G, H, V, kTensor, kGated>;
  constexpr int R = F::R, TILE = F::TILE, ST = F::ST, SB = F::SB;
  extern __shared__ __align__(128) char ring[];
  __shared__ ScanShared<V, false> sm;
  const int rank = blockIdx.x % S, col = blockIdx.x / S, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = (col * 32 + lane) * V;
  const bool on = d < a.D;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  float carry[V];
#pragma unroll
  for (int i = 0; i < V; ++i) carry[i] = on && a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;

  int lost = 0;
  Feed<X, V, R, kTensor> xf(ring, warp, lane);
  Feed<G, V, R, kTensor> gf(ring + F::XB, warp, lane);
  // Tile `n` into `stage`: all threads (their own tokens), or thread 0 (the whole tile).
  auto load = [&](int stage, int n) {
    if constexpr (kTensor) {
      if (threadIdx.x == 0 && !lost && n * TILE < a.T) {
        ptx::mbar_expect_tx(&sm.full[stage], SB);
        const uint32_t dst = ptx::smem_u32(ring + stage * SB);
        ptx::tma_load3(dst, &maps.x, col * 32 * V, n * TILE, b, &sm.full[stage]);
        ptx::tma_load3(dst + F::XB, &maps.g, col * 32 * V, n * TILE, b, &sm.full[stage]);
      }
    } else {
      const int t0 = n * TILE + warp * R;
      if (on) {
        const X* xp = x + t0 * a.xt;
        const G* gp = g + t0 * a.gt;
#pragma unroll
        for (int r = 0; r < R; ++r, xp += a.xt, gp += a.gt)
          if (t0 + r < a.T) {
            xf.fetch(stage * SB, r, xp);
            gf.fetch(stage * SB, r, gp);
          }
      }
      ptx::cp_async_commit();
    }
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) ptx::mbar_init(&sm.full[i], 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&sm.met[i], 1);
    ptx::mbar_fence_init();
  }
  if (S > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  int n = rank;
#pragma unroll
  for (int i = 0; i < ST; ++i) load(i, n + i * S);
  H* h = static_cast<H*>(a.h) + ((size_t)b * a.T + n * TILE + warp * R) * a.D + d;
  const size_t hop = (size_t)S * TILE * a.D;
  const int tiles = (a.T + TILE - 1) / TILE, steps = (tiles + S - 1) / S;
  for (int step = 0; step < steps; ++step, n += S, h += hop) {
    const int par = step & 1, stage = step % ST, t0 = n * TILE + warp * R;
    const int rows = min(R, a.T - t0);           // of this warp; may be negative
    float e[R][V], u[R][V], A[V], P[V];
    if constexpr (kTensor) {
      if (n * TILE < a.T && !lost && !ptx::mbar_wait(&sm.full[stage], (step / ST) & 1, a.polls))
        lost = step + 1;
    } else {
      ptx::cp_async_wait<ST - 1>();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, P[i] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < V; ++i) e[r][i] = u[r][i] = 0.f;
      if (kTensor ? n * TILE < a.T : on && r < rows) {
        xf.take(stage * SB, r, u[r]);
        gf.take(stage * SB, r, e[r]);
      }
    }
    if constexpr (kGated) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float m[V];
        gate<V>(e[r], m);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          u[r][i] *= m[i];
          P[i] = fmaf(e[r][i], P[i], u[r][i]);
          A[i] *= e[r][i];
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[r][i] = expf(e[r][i]);
          P[i] = fmaf(e[r][i], P[i], u[r][i]);
          A[i] *= e[r][i];
        }
      }
    }
    if (lost) {
#pragma unroll
      for (int i = 0; i < V; ++i) P[i] = u[0][i] = NAN;
    }
    if constexpr (!kTensor) load(stage, n + ST * S);
    float w[2 * V];
    copy_v<V>(w, A);
    copy_v<V>(w + V, P);
    put_v<2 * V>(sm.warp[par][warp][lane], w);
    __syncthreads();
    if constexpr (kTensor) load(stage, n + ST * S);
    float pA[V], pP[V], tA[V], tP[V], s[V];      // before this warp; of the whole tile
#pragma unroll
    for (int i = 0; i < V; ++i) tA[i] = 1.f, tP[i] = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      if (v == warp) {
        copy_v<V>(pA, tA);
        copy_v<V>(pP, tP);
      }
      get_v<2 * V>(sm.warp[par][v][lane], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        tP[i] = fmaf(w[i], tP[i], w[V + i]);
        tA[i] *= w[i];
      }
    }
    cluster_carry<V, false>(sm, step, S, rank, warp, lane, a.polls, tA, tP, carry, s, lost);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = fmaf(pA[i], s[i], pP[i]);
    if (a.ck && warp * R % CK == 0 && on && rows > 0)
      put_v<V>(a.ck + ((size_t)b * a.N + t0 / CK) * a.D + d, s);
    if (on) {
      H* row = h;
#pragma unroll
      for (int r = 0; r < R; ++r, row += a.D) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = fmaf(e[r][i], s[i], u[r][i]);
        if (r < rows) store_f<H, V>(row, s);
      }
    }
  }
  if (a.sT && rank == 0 && warp == 0 && on) put_v<V>(a.sT + (size_t)b * a.D + d, carry);
  leave<kTensor ? ST : 0>(sm.full, lost, S,
                          [&](int j) { return (long long)(rank + j * S) * TILE < a.T; });
}

// The same walk from the last tile back. What travels is mu_t = a_t l_t, the gradient that
// reaches h_{t-1}: a stretch maps the mu after it to A mu + M, with the same A. The states
// inside a tile come from its checkpoint and the warps' forward pairs.
template <typename X, typename G, typename H, int V, bool kTensor, bool kGated>
struct Bwd {
  static constexpr int R = CK / W, TILE = CK, ST = kStages<X, G, H, V, kTensor>;
  static constexpr int XB = Feed<X, V, R, kTensor>::kBytes, GB = Feed<G, V, R, kTensor>::kBytes;
  static constexpr int DB = Feed<H, V, R, kTensor>::kBytes;
  static constexpr int SB = XB + GB + DB;
  // The weights of a gated input wait in shared memory between their two uses, where that
  // leaves the blocks per SM as they are, else in registers.
  static constexpr int PARK = W * 32 * R * V * 4, SM = 228 * 1024;
  static constexpr int USED = ST * SB + (int)sizeof(ScanShared<V, true>) + 1024;
  static constexpr bool kPark = kGated && (2 * USED > SM || 2 * (USED + PARK) <= SM);
  static constexpr int SMEM = ST * SB + (kPark ? PARK : 0);
};

template <typename X, typename G, typename H, int V, bool kTensor, bool kGated>
__global__ void __launch_bounds__(W * 32, 2)
    scan_bwd_kernel(const __grid_constant__ ScanMaps maps, ScanArgs a, int S) {
  using F = Bwd<X, G, H, V, kTensor, kGated>;
  constexpr int R = F::R, TILE = F::TILE, ST = F::ST, SB = F::SB;
  extern __shared__ __align__(128) char ring[];
  __shared__ ScanShared<V, true> sm;
  const int rank = blockIdx.x % S, col = blockIdx.x / S, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = (col * 32 + lane) * V;
  const bool on = d < a.D;
  const X* x = static_cast<const X*>(a.x) + b * a.xb + d;
  const G* g = static_cast<const G*>(a.g) + b * a.gb + d;
  const H* dh = static_cast<const H*>(a.dh) + b * a.db + d;
  const float* ck = a.ck + (size_t)b * a.N * a.D + d;
  float carry[V], cr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) carry[i] = on && a.s0 ? a.s0[(size_t)b * a.D + d + i] : 0.f;

  int lost = 0;
  Feed<X, V, R, kTensor> xf(ring, warp, lane);
  Feed<G, V, R, kTensor> gf(ring + F::XB, warp, lane);
  Feed<H, V, R, kTensor> df(ring + F::XB + F::GB, warp, lane);
  auto load = [&](int stage, int n, bool go) {
    if constexpr (kTensor) {
      if (threadIdx.x == 0 && go && n >= 0) {
        ptx::mbar_expect_tx(&sm.full[stage], SB);
        const uint32_t dst = ptx::smem_u32(ring + stage * SB);
        ptx::tma_load3(dst, &maps.x, col * 32 * V, n * TILE, b, &sm.full[stage]);
        ptx::tma_load3(dst + F::XB, &maps.g, col * 32 * V, n * TILE, b, &sm.full[stage]);
        ptx::tma_load3(dst + F::XB + F::GB, &maps.dh, col * 32 * V, n * TILE, b, &sm.full[stage]);
      }
    } else {
      const int t0 = n * TILE + warp * R;
      if (on && n >= 0) {
        const X* xp = x + t0 * a.xt;
        const G* gp = g + t0 * a.gt;
        const H* dp = dh + t0 * a.dt;
#pragma unroll
        for (int r = 0; r < R; ++r, xp += a.xt, gp += a.gt, dp += a.dt)
          if (t0 + r < a.T) {
            xf.fetch(stage * SB, r, xp);
            gf.fetch(stage * SB, r, gp);
            df.fetch(stage * SB, r, dp);
          }
      }
      ptx::cp_async_commit();
    }
  };
  float* park = reinterpret_cast<float*>(ring + ST * SB) + threadIdx.x * V;
  auto load_ck = [&](int n) {
#pragma unroll
    for (int i = 0; i < V; ++i) cr[i] = 0.f;
    if (on && n >= 0) load_f<float, V>(ck + (size_t)n * a.D, cr);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) ptx::mbar_init(&sm.full[i], 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&sm.met[i], 1);
    ptx::mbar_fence_init();
  }
  if (S > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  int n = a.N - 1 - rank;
#pragma unroll
  for (int i = 0; i < ST; ++i) load(i, n - i * S, true);
  load_ck(n);
  const int steps = (a.N + S - 1) / S;
  for (int step = 0; step < steps; ++step, n -= S) {
    const int par = step & 1, stage = step % ST, t0 = n * TILE + warp * R;
    const int rows = n < 0 ? 0 : min(R, a.T - t0);
    float e[R][V], m[kGated && !F::kPark ? R : 1][V], u[R][V], l[R][V], hs[V], A[V], P[V], M[V];
    if constexpr (kTensor) {
      if (n >= 0 && !lost && !ptx::mbar_wait(&sm.full[stage], (step / ST) & 1, a.polls))
        lost = step + 1;
    } else {
      ptx::cp_async_wait<ST - 1>();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) A[i] = 1.f, P[i] = M[i] = 0.f;
    copy_v<V>(hs, cr);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < V; ++i) e[r][i] = u[r][i] = l[r][i] = 0.f;
      if (kTensor ? n >= 0 : on && r < rows) {
        xf.take(stage * SB, r, u[r]);
        gf.take(stage * SB, r, e[r]);
        df.take(stage * SB, r, l[r]);
      }
    }
    // u becomes what dg multiplies (h_{t-1}, minus x_t when gated), but for what the state before
    // the warp adds to it.
    if constexpr (kGated) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float weight[V];
        gate<V>(e[r], weight);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = u[r][i];
          u[r][i] = P[i] - x;
          P[i] = fmaf(e[r][i], P[i], x * weight[i]);
          A[i] *= e[r][i];
        }
        if constexpr (F::kPark)
          put_v<V>(park + r * (W * 32 * V), weight);
        else
          copy_v<V>(m[r], weight);
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = u[r][i];
          e[r][i] = expf(e[r][i]);
          u[r][i] = P[i];
          P[i] = fmaf(e[r][i], P[i], x);
          A[i] *= e[r][i];
        }
    }
    if constexpr (!kTensor) load(stage, n - ST * S, true);
    load_ck(n - S);
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int i = 0; i < V; ++i) M[i] = e[r][i] * (l[r][i] + M[i]);
    if (lost) {
#pragma unroll
      for (int i = 0; i < V; ++i) P[i] = M[i] = l[R - 1][i] = NAN;
    }
    float w[2 * V];
    copy_v<V>(w, A);
    copy_v<V>(w + V, P);
    put_v<2 * V>(sm.warp[par][warp][lane], w);
    put_v<V>(sm.back[par][warp][lane], M);
    __syncthreads();
    // The stage is free. Its next tile is asked for here, or without gates, whose steps are
    // shorter, behind the exchange (2 x 8192 x 4096: 148 us there, 165 here; gated 164 and 162).
    if constexpr (kTensor && kGated) load(stage, n - ST * S, !lost);
    float pA[V], pM[V], tA[V], tM[V], mu[V];     // after this warp; of the whole tile
#pragma unroll
    for (int i = 0; i < V; ++i) tA[i] = 1.f, tM[i] = 0.f;
#pragma unroll
    for (int v = W - 1; v >= 0; --v) {
      if (v == warp) {
        copy_v<V>(pA, tA);
        copy_v<V>(pM, tM);
      }
      float wA[V], wM[V];
      get_v<V>(sm.warp[par][v][lane], wA);
      get_v<V>(sm.back[par][v][lane], wM);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        tM[i] = fmaf(wA[i], tM[i], wM[i]);
        tA[i] *= wA[i];
      }
    }
#pragma unroll
    for (int v = 0; v < W - 1; ++v)
      if (v < warp) {
        get_v<2 * V>(sm.warp[par][v][lane], w);
#pragma unroll
        for (int i = 0; i < V; ++i) hs[i] = fmaf(w[i], hs[i], w[V + i]);
      }
    cluster_carry<V, true>(sm, step, S, rank, warp, lane, a.polls, tA, tM, carry, mu, lost);
#pragma unroll
    for (int i = 0; i < V; ++i) mu[i] = fmaf(pA[i], mu[i], pM[i]);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[r][i] += hs[i];
        hs[i] *= e[r][i];
      }
    // (Also if the exchange of this very step gave up: leave() counts on it.)
    if constexpr (kTensor && !kGated) load(stage, n - ST * S, !lost || lost == step + 2);
    const size_t row0 = ((size_t)b * a.T + max(t0, 0)) * a.D + d;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      float ox[V], og[V], weight[V];
      if constexpr (kGated) {
        if constexpr (F::kPark)
          get_v<V>(park + r * (W * 32 * V), weight);
        else
          copy_v<V>(weight, m[r]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) weight[i] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float lr = l[r][i] + mu[i];
        ox[i] = lr * weight[i];
        mu[i] = e[r][i] * lr;
        og[i] = mu[i] * u[r][i];
      }
      if (on && r < rows) {
        store_f<X, V>(static_cast<X*>(a.dx) + row0 + (size_t)r * a.D, ox);
        store_f<G, V>(static_cast<G*>(a.dg) + row0 + (size_t)r * a.D, og);
      }
    }
  }
  if (a.sT && rank == 0 && warp == 0 && on) put_v<V>(a.sT + (size_t)b * a.D + d, carry);
  leave<kTensor ? ST : 0>(sm.full, lost, S, [&](int j) { return a.N - 1 - rank - j * S >= 0; });
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
  // A poll here may be suspended for about 1 us (measured), as long as sixteen of a flag take.
  a.polls = (long)(set_wait_limit(-1) / 16);
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
  return status_of(in ? cudaMemcpyAsync(out, in, n * 4, cudaMemcpyDeviceToDevice, s)
                      : cudaMemsetAsync(out, 0, n * 4, s));
}

constexpr int kSms = 152;
// Tokens up to which one thread runs its channels' tokens by itself: a few always; more where
// there are channels for more blocks than the walk keeps resident, whose tile of 128 tokens
// would be mostly empty (64 x 16 x 2048: 25 us by the walk, 6.4 so; 64 x 64 x 2048: 31, 41).
constexpr int kSerial = 8, kSerialWide = 32;
bool serial(const ScanArgs& a) {
  return a.T <= kSerial || (a.T <= kSerialWide && (long long)a.B * a.D >= 64LL * 2 * kSms);
}

// A view [B, T, D] as a tensor map with boxes of `rows` tokens x `cols` channels.
bool tmap_view(CUtensorMap* m, const void* p, int dtype, const ScanArgs& a, int64_t sb, int64_t st,
               int cols, int rows) {
  const int es = (int)dtype_size(dtype);
  const cuuint64_t row = (cuuint64_t)a.D * es;   // of a dimension that is never stepped along
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.T, (cuuint64_t)a.B};
  const cuuint64_t strides[2] = {a.T == 1 ? row : (cuuint64_t)st * es,
                                 a.B == 1 ? row : (cuuint64_t)sb * es};
  const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)rows, 1};
  return fast::tmap_encode(
      m, dtype == GDR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
      p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Whether a view can be copied by tensor maps: 16-byte aligned rows that differ.
bool tensor_ok(const void* p, int dtype, const ScanArgs& a, int64_t sb, int64_t st) {
  const int64_t es = (int64_t)dtype_size(dtype);
  return a.D * es % 16 == 0 && is_aligned(p, 16) &&
         (a.T == 1 || (st * es % 16 == 0 && st > 0)) && (a.B == 1 || (sb * es % 16 == 0 && sb > 0));
}

// Clusters of s blocks, s = 1 .. MAXS, that the device holds at once: with one block per SM
// (alone) and with as many as fit (packed). Asked of the runtime once per kernel (F names it)
// and device; false on a CUDA error.
struct Residency {
  int alone[MAXS + 1], packed[MAXS + 1];
};
template <typename F, typename Fn>
bool residency(Fn fn, Residency* r) {
  constexpr int kDevices = 16, kAlone = 120 * 1024;    // more than half an SM's shared memory
  static std::atomic<int> table[kDevices][2][MAXS + 1];   // [0][0]: filled
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return false;
  auto& row = table[dev];
  if (!row[0][0].load(std::memory_order_acquire)) {
    if (!allow_smem<F>(fn, F::SMEM > kAlone ? F::SMEM : kAlone)) return false;
    for (int k = 0; k < 2; ++k)
      for (int s = 1; s <= MAXS; ++s) {
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = s;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(s);
        cfg.blockDim = dim3(W * 32);
        cfg.dynamicSmemBytes = k == 0 && F::SMEM < kAlone ? kAlone : F::SMEM;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
          (void)cudaGetLastError();
          n = 0;
        }
        row[k][s].store(n, std::memory_order_relaxed);
      }
    row[0][0].store(1, std::memory_order_release);
  }
  for (int s = 1; s <= MAXS; ++s) {
    r->alone[s] = row[0][s].load(std::memory_order_relaxed);
    r->packed[s] = row[1][s].load(std::memory_order_relaxed);
  }
  return r->packed[1] > 0;
}

// Blocks per cluster (*best) with the least time for `clusters` of them over `tiles` tiles;
// returns that time in tenths of a step of a block that has its SM for itself. Two blocks
// that share an SM take 1.7 times as long for a step (measured: 1.6 and 2.7 us for forward
// steps at 1 x 16384 x 1024, S = 6 and 8; 1.7 and 2.6 us backward), three 2.5 times.
long long cluster_size(const Residency& r, long long clusters, int tiles, int* best) {
  long long least = -1;
  *best = 1;
  for (int s = 1; s <= MAXS && s <= tiles; ++s) {
    if (r.packed[s] <= 0) continue;
    const long long waves = (clusters + r.packed[s] - 1) / r.packed[s];
    const int share = clusters <= r.alone[s] ? 10 : clusters * s <= 2 * kSms ? 17 : 25;
    const long long cost = waves * ((tiles + s - 1) / s) * share;
    if (least < 0 || cost < least) least = cost, *best = s;
  }
  return least;
}

template <typename X, typename G, typename H, int V, bool kTensor, bool kBwd, bool kGated>
struct Walk {
  using F = std::conditional_t<kBwd, Bwd<X, G, H, V, kTensor, kGated>,
                               Fwd<X, G, H, V, kTensor, kGated>>;
  static auto kernel() {
    if constexpr (kBwd)
      return scan_bwd_kernel<X, G, H, V, kTensor, kGated>;
    else
      return scan_kernel<X, G, H, V, kTensor, kGated>;
  }
  // The time of this walk by the rule above, and its blocks per cluster; -1: a CUDA error.
  static long long plan(const ScanArgs& a, int* S) {
    Residency r;
    if (!residency<F>(kernel(), &r)) return -1;
    const long long cols = (a.D + 32LL * V - 1) / (32 * V);
    return cluster_size(r, cols * a.B, (a.T + F::TILE - 1) / F::TILE, S);
  }
  static gdr_status launch(const gdr_scan_dims* d, const ScanArgs& a, int S, cudaStream_t s) {
    ScanMaps m;
    if constexpr (kTensor) {
      if (!tmap_view(&m.x, a.x, d->x_dtype, a, a.xb, a.xt, 32 * V, F::TILE) ||
          !tmap_view(&m.g, a.g, d->g_dtype, a, a.gb, a.gt, 32 * V, F::TILE) ||
          (kBwd && !tmap_view(&m.dh, a.dh, d->h_dtype, a, a.db, a.dt, 32 * V, F::TILE)))
        return GDR_ERR_CUDA;
    }
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.D + 32LL * V - 1) / (32 * V) * S), a.B);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = F::SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return status_of(cudaLaunchKernelEx(&cfg, kernel(), m, a, S));
  }
};

// Two channels a lane or one. One halves a block's work for the same number of steps: a
// step takes 0.7 of the time (319 and 221 us at 1 x 16384 x 1024, S = 1, backward), and
// narrow problems get twice the blocks.
template <typename X, typename G, typename H, bool kBwd, bool kGated>
gdr_status launch_tensor(const gdr_scan_dims* d, const ScanArgs& a, cudaStream_t s) {
  using One = Walk<X, G, H, 1, true, kBwd, kGated>;
  using Two = Walk<X, G, H, 2, true, kBwd, kGated>;
  int S2 = 1, S1 = 1;
  const long long two = Two::plan(a, &S2), one = One::plan(a, &S1);
  if (two < 0 || one < 0) return GDR_ERR_CUDA;
  return one * 7 < two * 10 ? One::launch(d, a, S1, s) : Two::launch(d, a, S2, s);
}

template <typename X, typename G, typename H, int V, bool kBwd, bool kGated>
gdr_status launch_plain(const gdr_scan_dims* d, const ScanArgs& a, cudaStream_t s) {
  using Plain = Walk<X, G, H, V, false, kBwd, kGated>;
  int S = 1;
  return Plain::plan(a, &S) < 0 ? GDR_ERR_CUDA : Plain::launch(d, a, S, s);
}

enum Path { kPlain, kPairs, kTensorMaps };       // one channel; two; tiles by tensor maps

template <bool kBwd>
gdr_status launch(const gdr_scan_dims* d, const ScanArgs& a, Path path, cudaStream_t s) {
  return with_dtype(d->x_dtype, [&](auto* x) {
    return with_dtype(d->g_dtype, [&](auto* g) {
      return with_dtype(d->h_dtype, [&](auto* h) {
        using X = std::remove_pointer_t<decltype(x)>;
        using G = std::remove_pointer_t<decltype(g)>;
        using H = std::remove_pointer_t<decltype(h)>;
        if constexpr (!kBwd) {
          if (serial(a)) {
            const int V = path == kPlain ? 1 : 2;
            const dim3 grid((a.D + 128 * V - 1) / (128 * V), a.B);
            return launch_kernel(V == 1 ? scan_serial_kernel<X, G, H, 1>
                                        : scan_serial_kernel<X, G, H, 2>,
                                 grid, 128, 0, s, a);
          }
        }
        auto walk = [&](auto gated) {
          constexpr bool kGated = decltype(gated)::value;
          return path == kTensorMaps ? launch_tensor<X, G, H, kBwd, kGated>(d, a, s)
                 : path == kPairs    ? launch_plain<X, G, H, 2, kBwd, kGated>(d, a, s)
                                     : launch_plain<X, G, H, 1, kBwd, kGated>(d, a, s);
        };
        return a.gated ? walk(std::true_type()) : walk(std::false_type());
      });
    });
  });
}

Path choose(const gdr_scan_dims* d, const ScanArgs& a) {
  if (tensor_ok(a.x, d->x_dtype, a, a.xb, a.xt) && tensor_ok(a.g, d->g_dtype, a, a.gb, a.gt) &&
      (!a.dh || tensor_ok(a.dh, d->h_dtype, a, a.db, a.dt)))
    return kTensorMaps;
  return a.D % 2 == 0 && vec_ok(a.x, d->x_dtype, a.xb, a.xt, 2) &&
                 vec_ok(a.g, d->g_dtype, a.gb, a.gt, 2) &&
                 (!a.dh || vec_ok(a.dh, d->h_dtype, a.db, a.dt, 2))
             ? kPairs
             : kPlain;
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
  return launch<false>(dims, a, choose(dims, a), s);
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
  return launch<true>(dims, a, choose(dims, a), s);
}

}  // extern "C"
