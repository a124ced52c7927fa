// gdr_qk.cu -- RMS norm of query and key heads with the position rotation, its
// gradients, and the form that writes keys and values into a paged cache.
//
//   r = 1 / sqrt(mean(x^2) + eps),  u = r x,  y = turn(u w)
//   d = turn^-1(dy),  dw = sum d u,  dx = r (d w - u mean(d w u))
//
// Each head row is read once and written once (two reads in the backward): bound by HBM, and
// close behind it by the instructions per row. Measured on one GB300, bf16, heads of 128:
//   2 x 8192 x (32 + 4) heads, half of each turned: forward 53 us, 5.7 TB/s (a plain copy:
//   6.78 TB/s); backward 84 us, 5.4 TB/s
//   1 x 4096 x (12 + 12) heads: forward 15 us, backward 20 and the weights' sums 3 us
//   into pages: 66 us (5.1 TB/s) and 18.5 us
//   fp32: forward 107 us, backward 181, into pages 121 (5.6, 5.0 and 5.5 TB/s); 23, 33 and 28 us
//   64 decode tokens x (16 + 4 + 4) heads into their pages: 6.1 us a call, bound by the chain
//   position - page and angles - row of one token
#include <type_traits>

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"

namespace gdr {
namespace ops {
namespace {

enum Mode { kFwd = 0, kBwd = 1, kAppend = 2 };

struct QkArgs {
  const void *q, *k, *v;
  const float *wq, *wk, *cos, *sin;
  const void* pos;
  void *qo, *ko;              // forward outputs; backward: the gradients of q and k
  const void *dqo, *dko;      // backward: upstream gradients
  float* part;                // backward: [gridDim.x][2][D] sums for the weights, or null
  void *kc, *vc;              // append: the caches
  const int32_t* table;
  int B, T, HQ, HK, D, R, interleaved, pos64, rows;
  int num_pages, page, max_pages, cache_bf16;
  float eps;
  int64_t qb, qt, qh, kb, kt, kh, vb, vt, vh, pp, pt, ph;
  long long tokens;
};

__device__ __forceinline__ long long position(const QkArgs& a, long long tok) {
  if (!a.pos) return 0;
  return a.pos64 ? static_cast<const long long*>(a.pos)[tok] : static_cast<const int*>(a.pos)[tok];
}

// Offset of a token's row 0 in the caches, or -1 where it has no page.
__device__ __forceinline__ int64_t cache_row(const QkArgs& a, long long b, long long p) {
  if (p < 0 || p >= (long long)a.max_pages * a.page) return -1;
  const int j = (int)(p / a.page);
  const int32_t pg = a.table[b * a.max_pages + j];
  if (pg < 0 || pg >= a.num_pages) return -1;
  return pg * a.pp + (p - (long long)j * a.page) * a.pt;
}

__device__ __forceinline__ void store_cache(void* c, int64_t i, float v, int is_bf16) {
  if (is_bf16)
    static_cast<bf16*>(c)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(c)[i] = v;
}

// ------------------------------------------------------------ any size and stride
// One warp per head row, channel i at lane i % 32; the pairs of the rotation meet in
// shared memory. Covers what the vector kernel's alignment rules leave out.
constexpr int GW = 8;                            // warps per block
template <typename I, typename O, int MODE>
__global__ void __launch_bounds__(GW * 32) qk_any_kernel(QkArgs a) {
  constexpr int J = 8;                           // channels per lane: D <= 256
  if (MODE == kBwd) let_next_begin();
  __shared__ float row[GW][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = a.R >> 1;
  const int per = a.HQ + a.HK + (MODE == kAppend ? a.HK : 0);
  float* y = row[warp];
  float acc[2][J];
#pragma unroll
  for (int j = 0; j < J; ++j) acc[0][j] = acc[1][j] = 0.f;
  const long long total = a.tokens * per;
  for (long long r = (long long)blockIdx.x * GW + warp; r < total; r += (long long)gridDim.x * GW) {
    const long long tok = r / per, b = tok / a.T, t = tok - b * a.T;
    const int head = (int)(r - tok * per);
    const int kind = head < a.HQ ? 0 : head < a.HQ + a.HK ? 1 : 2;
    const int h = kind == 0 ? head : kind == 1 ? head - a.HQ : head - a.HQ - a.HK;
    const long long p = position(a, tok);
    bool bad = a.R > 0 && (p < 0 || p >= a.rows);
    int64_t at = 0;
    if (MODE == kAppend) {
      at = cache_row(a, b, p);
      bad = bad || at < 0;
      at += h * a.ph;
    }
    const I* src = kind == 0   ? static_cast<const I*>(a.q) + b * a.qb + t * a.qt + h * a.qh
                   : kind == 1 ? static_cast<const I*>(a.k) + b * a.kb + t * a.kt + h * a.kh
                               : static_cast<const I*>(a.v) + b * a.vb + t * a.vt + h * a.vh;
    if (MODE == kAppend && kind == 2) {
      if (!bad)                                  // values as they are
        for (int i = lane; i < a.D; i += 32) {
          if (a.cache_bf16 == (sizeof(I) == 2))
            static_cast<I*>(a.vc)[at + i] = src[i];
          else
            store_cache(a.vc, at + i, static_cast<float>(src[i]), a.cache_bf16);
        }
      continue;
    }
    const float* w = kind == 0 ? a.wq : a.wk;
    float x[J], ss = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = lane + 32 * j;
      x[j] = i < a.D ? static_cast<float>(src[i]) : 0.f;
      ss = fmaf(x[j], x[j], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    const float rs = rsqrtf(ss / a.D + a.eps);
    const int64_t dense = (tok * (kind == 0 ? a.HQ : a.HK) + h) * a.D;
    const O* dy = nullptr;
    if (MODE == kBwd) dy = static_cast<const O*>(kind == 0 ? a.dqo : a.dko) + dense;
    // Forward: the weighted unit row; backward: the upstream row.
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = lane + 32 * j;
      if (i < a.D) y[i] = MODE == kBwd ? static_cast<float>(dy[i]) : x[j] * rs * (w ? w[i] : 1.f);
    }
    __syncwarp();
    float z[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = lane + 32 * j;
      z[j] = 0.f;
      if (i >= a.D) continue;
      z[j] = y[i];
      if (i < a.R && !bad) {
        const int pr = a.interleaved ? i >> 1 : (i < half ? i : i - half);
        const bool first = a.interleaved ? (i & 1) == 0 : i < half;
        const int mate = a.interleaved ? i ^ 1 : (first ? i + half : i - half);
        const float c = a.cos[p * half + pr], s0 = a.sin[p * half + pr];
        const float s = (MODE == kBwd) == first ? s0 : -s0;
        z[j] = fmaf(y[mate], s, y[i] * c);
      }
      if (bad) z[j] = NAN;
    }
    __syncwarp();
    if (MODE == kBwd) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = lane + 32 * j;
        if (i >= a.D) continue;
        const float u = x[j] * rs;
        if (kind == 0)
          acc[0][j] = fmaf(z[j], u, acc[0][j]);
        else
          acc[1][j] = fmaf(z[j], u, acc[1][j]);
        z[j] *= w ? w[i] : 1.f;
        m = fmaf(z[j], u, m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(~0u, m, o);
      m /= a.D;
      I* dst = static_cast<I*>(kind == 0 ? a.qo : a.ko) + dense;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = lane + 32 * j;
        if (i < a.D) dst[i] = static_cast<I>(rs * (z[j] - x[j] * rs * m));
      }
    } else if (MODE == kAppend && kind == 1) {
      if (!bad)
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (lane + 32 * j < a.D) store_cache(a.kc, at + lane + 32 * j, z[j], a.cache_bf16);
    } else {
      O* dst = static_cast<O*>(kind == 0 ? a.qo : a.ko) + dense;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (lane + 32 * j < a.D) dst[lane + 32 * j] = static_cast<O>(z[j]);
    }
  }
  if (MODE == kBwd && a.part) {
    for (int n = 0; n < 2; ++n) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < J; ++j) row[warp][lane + 32 * j] = acc[n][j];
      __syncthreads();
      for (int i = threadIdx.x; i < a.D; i += GW * 32) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < GW; ++v) s += row[v][i];
        a.part[((size_t)blockIdx.x * 2 + n) * a.D + i] = s;
      }
    }
  }
}

// ------------------------------------------------------------ rows of 8 channels a lane
// A group of GL lanes (D / 8, rounded up to a power of two, at least 8) takes a head row; a
// lane holds two runs of four channels, chosen so that the members of its four rotation
// pairs are its own: the runs at 4 j and 4 j + R / 2 (2 x 4 neighbouring channels when pairs
// are neighbours, and beyond R). So the rotation needs no exchange, the norm one tree of
// shuffles. What bounds this kernel beside the bytes is the number of instructions per row:
// a group stays with one token for up to 32 of its rows, so that addresses, angles and
// weights are set up once for them, the weight is folded into the angles
//   y[j] = rs (M[j] x[j] + N[j] z[j]),   z[j] the other members of the pairs x[j],
// and fp32 goes two operations an instruction. A lane copies its own runs of the next rows
// asynchronously into its own places in shared memory (prefetching into registers held two
// rows and spilled), so it waits for itself alone.
constexpr int VT = 128;                          // threads per block

// A unit: `rows` head rows of one token, all of q, of k, or (append) of v. Units are numbered
// section by section.
struct VecPlan {
  int GL;                                        // lanes per row
  int rows[3], chunks[3];                        // per section: rows per unit, units per token
  unsigned units[3];
};

// The pairs that turn with x[0..3]: the other run's, or each pair swapped.
template <bool kNeighbours>
__device__ __forceinline__ float2 mate(const float2* x, int j) {
  return kNeighbours ? make_float2(x[j].y, x[j].x) : x[j ^ 2];
}

// Four elements, asynchronously into this thread's own place.
template <typename T>
__device__ __forceinline__ void copy_run(T* dst, const T* src) {
  if constexpr (sizeof(T) == 2)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(dst)), "l"(src)
                 : "memory");
  else
    ptx::cp_async16(ptx::smem_u32(dst), src, 16);
}

// Blocks an SM holds. Seven forward, with spills, changed no time by more than 4 % (1 x 4096
// tokens: 12 + 12 heads 14.4 us against 14.9, 32 + 8 heads 20.5 against 18.7).
constexpr int resident(int mode) { return mode == kBwd ? 4 : 6; }

template <typename I, typename O, int MODE, bool kNeighbours, int GL>
__global__ void __launch_bounds__(VT, resident(MODE)) qk_vec_kernel(QkArgs a, VecPlan v) {
  constexpr bool bwd = MODE == kBwd;
  if (bwd) let_next_begin();
  constexpr int K = bwd ? 1 : 2, DEPTH = 4;      // rows at work; steps of as many under way
  constexpr int XROW = 2 * VT * 4, DROW = bwd ? 2 * VT * 4 : 0;   // elements of a row of the block
  __shared__ __align__(16) I stage_x[DEPTH * K * XROW];
  __shared__ __align__(16) O stage_d[bwd ? DEPTH * K * DROW : 1];
  I* xs = stage_x + threadIdx.x * 4;
  O* ds = stage_d + (bwd ? threadIdx.x * 4 : 0);
  const int lane = threadIdx.x & (GL - 1), half = a.R >> 1, rot = a.R >> 3;
  const bool on = lane * 8 < a.D, turned = lane < rot;
  const bool split = !kNeighbours && turned;
  const int o0 = split ? 4 * lane : 8 * lane, o1 = split ? 4 * lane + half : 8 * lane + 4;
  const int run = o1 - o0;                       // from one run to the other
  const float inv = 1.f / a.D;
  // Groups of one warp may stand at different units: each exchanges among its own lanes.
  const unsigned mask = GL == 32 ? ~0u : ((1u << GL) - 1) << (threadIdx.x & 31 & ~(GL - 1));
  if (!on) {                                     // channels that are not there: zeros
    for (int s = 0; s < DEPTH * K * 2; ++s) {
      const float z[4] = {0.f, 0.f, 0.f, 0.f};
      store_f<I, 4>(xs + s * (XROW / 2), z);
      if constexpr (bwd) store_f<O, 4>(ds + s * (DROW / 2), z);
    }
  }
  const unsigned groups = gridDim.x * (VT / GL);
  unsigned unit = blockIdx.x * (VT / GL) + threadIdx.x / GL;
#pragma unroll 1
  for (int n = 0; n < (MODE == kAppend ? 3 : 2); ++n) {     // q, k, v
    const bool value = MODE == kAppend && n == 2;
    const int H = n == 0 ? a.HQ : a.HK;
    const float* wp = n == 0 ? a.wq : n == 1 ? a.wk : nullptr;
    float2 w[4], acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = make_float2(1.f, 1.f), acc[j] = make_float2(0.f, 0.f);
    if (wp && on && unit < v.units[n]) {
      load_pairs(wp + o0, w);
      load_pairs(wp + o1, w + 2);
    }
    const I* src = static_cast<const I*>(n == 0 ? a.q : n == 1 ? a.k : a.v);
    const int64_t sb = n == 0 ? a.qb : n == 1 ? a.kb : a.vb;
    const int64_t st = n == 0 ? a.qt : n == 1 ? a.kt : a.vt;
    const int64_t sh = n == 0 ? a.qh : n == 1 ? a.kh : a.vh;
#pragma unroll 1
    for (; unit < v.units[n]; unit += groups) {
      const unsigned tok = unit / v.chunks[n], b = tok / a.T, t = tok - b * a.T;
      const int r0 = (int)(unit - tok * v.chunks[n]) * v.rows[n], rows = min(H - r0, v.rows[n]);
      const int64_t dense = ((int64_t)tok * H + r0) * a.D + o0;
      const I* xp = src + b * sb + t * st + r0 * sh + o0;
      const O* dp = static_cast<const O*>(n == 0 ? a.dqo : a.dko) + dense;
      const long long pos = position(a, tok);
      // Step i: the K rows from i K, on their way into slot i % DEPTH of this lane.
      auto fetch = [&](int i) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (on && i * K + k < rows) {
            const int slot = (i % DEPTH) * K + k;
            copy_run<I>(xs + slot * XROW, xp);
            copy_run<I>(xs + slot * XROW + XROW / 2, xp + run);
            if constexpr (bwd) {
              copy_run<O>(ds + slot * DROW, dp);
              copy_run<O>(ds + slot * DROW + DROW / 2, dp + run);
            }
          }
          xp += sh;
          dp += a.D;
        }
        ptx::cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) fetch(i);
      bool bad = a.R > 0 && (pos < 0 || pos >= a.rows);
      char* to;                                  // this lane's place in the first result row
      int64_t step;
      bool to_bf16;
      if (MODE == kAppend && n > 0) {
        const int64_t at = cache_row(a, b, pos);
        bad = bad || at < 0;
        to_bf16 = a.cache_bf16;
        const int es = to_bf16 ? 2 : 4;
        to = static_cast<char*>(value ? a.vc : a.kc) + (at + r0 * a.ph + o0) * es;
        step = a.ph * es;
      } else {
        if (MODE == kAppend) bad = bad || cache_row(a, b, pos) < 0;
        to_bf16 = sizeof(O) == 2;
        if constexpr (bwd) to_bf16 = sizeof(I) == 2;
        const int es = to_bf16 ? 2 : 4;
        to = static_cast<char*>(n == 0 ? a.qo : a.ko) + dense * es;
        step = (int64_t)a.D * es;
      }
      const bool keep = on && !(MODE == kAppend && n > 0 && bad);
      // c and s of the lane's pairs, laid out like them; sg turns forward.
      float2 c[4], sg[4];
      if (turned && !bad) {
        const float4 cv = *reinterpret_cast<const float4*>(a.cos + pos * half + 4 * lane);
        const float4 sv = *reinterpret_cast<const float4*>(a.sin + pos * half + 4 * lane);
        if (kNeighbours) {
          c[0] = make_float2(cv.x, cv.x), c[1] = make_float2(cv.y, cv.y);
          c[2] = make_float2(cv.z, cv.z), c[3] = make_float2(cv.w, cv.w);
          sg[0] = make_float2(-sv.x, sv.x), sg[1] = make_float2(-sv.y, sv.y);
          sg[2] = make_float2(-sv.z, sv.z), sg[3] = make_float2(-sv.w, sv.w);
        } else {
          c[0] = c[2] = make_float2(cv.x, cv.y), c[1] = c[3] = make_float2(cv.z, cv.w);
          sg[2] = make_float2(sv.x, sv.y), sg[3] = make_float2(sv.z, sv.w);
          sg[0] = make_float2(-sv.x, -sv.y), sg[1] = make_float2(-sv.z, -sv.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = make_float2(1.f, 1.f), sg[j] = make_float2(0.f, 0.f);
      }
      if constexpr (bwd) {                       // back by the angle
#pragma unroll
        for (int j = 0; j < 4; ++j) sg[j] = make_float2(-sg[j].x, -sg[j].y);
      } else {
        float2 m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = mate<kNeighbours>(w, j);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j] = mul2(c[j], w[j]);               // M
          sg[j] = mul2(sg[j], m[j]);             // N
        }
      }
#pragma unroll 1
      for (int r = 0, i = 0; r < rows; r += K, ++i) {
        ptx::cp_async_wait<DEPTH - 1>();
        if (value) {                             // as they are, their type's rounding apart
          Raw<I, 4> x[K][2];
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int slot = (i % DEPTH) * K + k;
            x[k][0] = load_raw<I, 4>(xs + slot * XROW);
            x[k][1] = load_raw<I, 4>(xs + slot * XROW + XROW / 2);
          }
          fetch(i + DEPTH);
#pragma unroll
          for (int k = 0; k < K; ++k, to += step) {
            if (!keep || r + k >= rows) continue;
            if (to_bf16 == (sizeof(I) == 2)) {
              store_raw(reinterpret_cast<I*>(to), x[k][0]);
              store_raw(reinterpret_cast<I*>(to) + run, x[k][1]);
            } else {
              float2 y[4];
              to_pairs(x[k][0], y);
              to_pairs(x[k][1], y + 2);
              if (to_bf16) {
                store_pairs(reinterpret_cast<bf16*>(to), y);
                store_pairs(reinterpret_cast<bf16*>(to) + run, y + 2);
              } else {
                store_pairs(reinterpret_cast<float*>(to), y);
                store_pairs(reinterpret_cast<float*>(to) + run, y + 2);
              }
            }
          }
        } else {
          float2 x[K][4], d[K][4];
          float ss[K], dot[K];
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int slot = (i % DEPTH) * K + k;
            to_pairs(load_raw<I, 4>(xs + slot * XROW), x[k]);
            to_pairs(load_raw<I, 4>(xs + slot * XROW + XROW / 2), x[k] + 2);
            float2 q = mul2(x[k][0], x[k][0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) q = fma2(x[k][j], x[k][j], q);
            ss[k] = q.x + q.y;
            if constexpr (bwd) {
              float2 z[4];
              to_pairs(load_raw<O, 4>(ds + slot * DROW), z);
              to_pairs(load_raw<O, 4>(ds + slot * DROW + DROW / 2), z + 2);
              if (turned) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  d[k][j] = fma2(sg[j], mate<kNeighbours>(z, j), mul2(c[j], z[j]));
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[k][j] = z[j];
              }
              q = make_float2(0.f, 0.f);
#pragma unroll
              for (int j = 0; j < 4; ++j) q = fma2(mul2(d[k][j], w[j]), x[k][j], q);
              dot[k] = q.x + q.y;
            }
          }
          fetch(i + DEPTH);
#pragma unroll
          for (int o = GL / 2; o > 0; o >>= 1) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
              ss[k] += __shfl_xor_sync(mask, ss[k], o);
              if constexpr (bwd) dot[k] += __shfl_xor_sync(mask, dot[k], o);
            }
          }
#pragma unroll
          for (int k = 0; k < K; ++k) {
            // A bad position makes the whole row NaN (and stores nothing into the caches).
            const float rs = bad ? NAN : rsqrtf(fmaf(ss[k], inv, a.eps));
            const float2 rs2 = make_float2(rs, rs);
            float2 y[4];
            if constexpr (bwd) {
              // dx = rs (d w - u mean(d w u)), u = rs x
              const float m = -dot[k] * inv * rs;
              const float2 m2 = make_float2(m, m);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 u = mul2(x[k][j], rs2);
                acc[j] = fma2(d[k][j], u, acc[j]);
                y[j] = mul2(rs2, fma2(u, m2, mul2(d[k][j], w[j])));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = mul2(c[j], x[k][j]);
              if (turned) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fma2(sg[j], mate<kNeighbours>(x[k], j), y[j]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], rs2);
            }
            if (keep && r + k < rows) {
              if (to_bf16) {
                store_pairs(reinterpret_cast<bf16*>(to), y);
                store_pairs(reinterpret_cast<bf16*>(to) + run, y + 2);
              } else {
                store_pairs(reinterpret_cast<float*>(to), y);
                store_pairs(reinterpret_cast<float*>(to) + run, y + 2);
              }
            }
            to += step;
          }
        }
      }
    }
    unit -= v.units[n];
    if (bwd && a.part) {                         // the block's groups, in order
      __shared__ float red[VT / 8][8 * 8 + 4];   // groups x channels of eight lanes
      for (int l0 = 0; l0 < a.D / 8; l0 += 8) {
        __syncthreads();
        if (lane >= l0 && lane < l0 + 8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            red[threadIdx.x / GL][(lane - l0) * 8 + 2 * j] = acc[j].x;
            red[threadIdx.x / GL][(lane - l0) * 8 + 2 * j + 1] = acc[j].y;
          }
        }
        __syncthreads();
        const int of = l0 + (threadIdx.x >> 3), i = threadIdx.x & 7;
        if (threadIdx.x < 64 && of * 8 < a.D) {
          float sum = 0.f;
          for (int k = 0; k < VT / GL; ++k) sum += red[k][threadIdx.x];
          const bool sp = !kNeighbours && of < rot;
          const int ch = i < 4 ? (sp ? 4 * of : 8 * of) + i
                               : (sp ? 4 * of + half : 8 * of + 4) + i - 4;
          a.part[((size_t)blockIdx.x * 2 + n) * a.D + ch] = sum;
        }
      }
    }
  }
}

// ------------------------------------------------------------ the weights' gradients
// Eight columns (channels of dq_weight, then dk_weight) a block, so that the loads are a few
// per thread and spread over many SMs: row y of its threads adds every SR-th block's sums,
// then the rows are added in order.
constexpr int SX = 8, SR = 64;
__global__ void __launch_bounds__(SX * SR) qk_weight_kernel(const float* part, int blocks, int D,
                                                            float* dwq, float* dwk) {
  __shared__ float red[SR][SX];
  const int x = threadIdx.x % SX, y = threadIdx.x / SX, col = blockIdx.x * SX + x;
  wait_for_before();                             // the sums are written
  float s = 0.f;
  if (col < 2 * D) {
#pragma unroll 10
    for (int i = y; i < blocks; i += SR) s += part[(size_t)i * 2 * D + col];
  }
  red[y][x] = s;
  __syncthreads();
  if (y || col >= 2 * D) return;
  s = 0.f;
#pragma unroll 16
  for (int i = 0; i < SR; ++i) s += red[i][x];
  float* out = col < D ? dwq : dwk;
  if (out) out[col < D ? col : col - D] = s;
}

// ------------------------------------------------------------ host
constexpr int kMaxBlocks = 152 * 4;              // of the backward: rows of the partial sums

gdr_status check(const gdr_qk_dims* d) {
  if (!d) return GDR_ERR_INVALID_ARG;
  if (d->B < 0 || d->T < 0 || d->HQ <= 0 || d->HK <= 0 || d->D <= 0) return GDR_ERR_INVALID_ARG;
  if (d->R < 0 || d->R > d->D || d->R % 2 != 0 || d->table_rows < 0) return GDR_ERR_INVALID_ARG;
  if (!is_dtype(d->in_dtype) || !is_dtype(d->out_dtype)) return GDR_ERR_INVALID_ARG;
  if (d->position_bits != 32 && d->position_bits != 64) return GDR_ERR_INVALID_ARG;
  if (!(isfinite(d->eps) && d->eps > 0.f)) return GDR_ERR_INVALID_ARG;
  const int64_t st[] = {d->q_stride_b, d->q_stride_t, d->q_stride_h, d->k_stride_b, d->k_stride_t,
                        d->k_stride_h, d->v_stride_b, d->v_stride_t, d->v_stride_h};
  for (int64_t s : st)
    if (s < 0) return GDR_ERR_INVALID_ARG;
  if (d->D > 256 || d->HQ > (1 << 20) || d->HK > (1 << 20)) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

QkArgs make_args(const gdr_qk_dims* d, const float* wq, const float* wk, const float* cos,
                 const float* sin, const void* pos) {
  QkArgs a = {};
  a.wq = wq; a.wk = wk; a.cos = cos; a.sin = sin; a.pos = pos;
  a.B = d->B; a.T = d->T; a.HQ = d->HQ; a.HK = d->HK; a.D = d->D; a.R = d->R;
  a.interleaved = d->interleaved != 0;
  a.pos64 = d->position_bits == 64;
  a.rows = d->table_rows;
  a.eps = d->eps;
  a.qb = d->q_stride_b; a.qt = d->q_stride_t; a.qh = d->q_stride_h;
  a.kb = d->k_stride_b; a.kt = d->k_stride_t; a.kh = d->k_stride_h;
  a.vb = d->v_stride_b; a.vt = d->v_stride_t; a.vh = d->v_stride_h;
  a.tokens = (long long)d->B * d->T;
  if (a.B == 1) a.qb = a.kb = a.vb = 0;          // never stepped along
  if (a.T == 1) a.qt = a.kt = a.vt = 0;
  if (a.HQ == 1) a.qh = 0;
  if (a.HK == 1) a.kh = a.vh = 0;
  return a;
}

// The arguments every form shares: null pointers and alignment of the dense ones.
gdr_status check_shared(const gdr_qk_dims* d, const void* q, const void* k, const float* wq,
                        const float* wk, const float* cos, const float* sin, const void* pos,
                        bool need_pos) {
  if (d->B > 0 && d->T > 0) {
    if (!q || !k) return GDR_ERR_INVALID_ARG;
    if (d->R > 0 && (!cos || !sin)) return GDR_ERR_INVALID_ARG;
    if ((d->R > 0 || need_pos) && !pos) return GDR_ERR_INVALID_ARG;
  }
  const size_t e = dtype_size(d->in_dtype);
  if (!is_aligned(q, e) || !is_aligned(k, e) || !is_aligned(wq, 16) || !is_aligned(wk, 16) ||
      !is_aligned(cos, 16) || !is_aligned(sin, 16) || !is_aligned(pos, d->position_bits / 8))
    return GDR_ERR_ALIGNMENT;
  return GDR_OK;
}

// Whether the vector kernel takes these sizes, strides and bases: whole runs of four
// channels, aligned.
bool vec_ok(const gdr_qk_dims* d, const QkArgs& a, int mode, const gdr_paged_cache* c) {
  if (d->D % 8 != 0 || d->R % 8 != 0) return false;
  const size_t run = 4 * dtype_size(d->in_dtype);
  const int64_t s[] = {a.qb, a.qt, a.qh, a.kb, a.kt, a.kh,
                       mode == kAppend ? a.vb : 0, mode == kAppend ? a.vt : 0,
                       mode == kAppend ? a.vh : 0};
  for (int64_t x : s)
    if (x % 4 != 0) return false;
  if (!is_aligned(a.q, run) || !is_aligned(a.k, run)) return false;
  if (mode == kAppend && (!is_aligned(a.v, run) || c->page_stride % 4 != 0 ||
                          c->token_stride % 4 != 0 || c->head_stride % 4 != 0))
    return false;
  return a.tokens * (a.HQ + 2LL * a.HK) < (1LL << 31);
}

// The split of a token's heads into rows of at most `most` per group; returns the blocks.
long long vec_split(const QkArgs& a, int mode, int most, VecPlan& v) {
  const int heads[3] = {a.HQ, a.HK, mode == kAppend ? a.HK : 0};
  long long units = 0;
  for (int n = 0; n < 3; ++n) {
    if (!heads[n]) continue;
    const int chunks = (heads[n] + most - 1) / most;
    v.rows[n] = (heads[n] + chunks - 1) / chunks;
    v.chunks[n] = (heads[n] + v.rows[n] - 1) / v.rows[n];
    v.units[n] = (unsigned)(a.tokens * v.chunks[n]);
    units += v.units[n];
  }
  return (units * v.GL + VT - 1) / VT;
}

// More rows per group spread a token's angles and addresses over more work, until some SMs
// have none: the fewest of 1, 2, 4 .. 16 rows whose blocks are resident at once, else 16
// (2 x 512 x (32 + 8) heads forward: 4 rows 10.2 us, 8 rows 8.3, 32 rows 10.3); forward 32
// where that leaves four rounds (2 x 8192 x (32 + 4) heads: 53.4 us against 55.4; with their
// values into pages 67.6 against 71.1; backward 84.0 against 82.4, so not there).
VecPlan vec_plan(const QkArgs& a, int mode) {
  VecPlan v = {};
  v.GL = 8;
  while (v.GL * 8 < a.D) v.GL *= 2;
  const long long round = 152LL * resident(mode);
  if (mode != kBwd && vec_split(a, mode, 32, v) >= 4 * round) return v;
  for (int most = 1; vec_split(a, mode, most, v) > round && most < 16;) most *= 2;
  return v;
}

template <typename I, typename O, int MODE, bool kNeighbours>
gdr_status launch_vec(const QkArgs& a, const VecPlan& v, int blocks, cudaStream_t s) {
  return launch_kernel(v.GL == 8    ? qk_vec_kernel<I, O, MODE, kNeighbours, 8>
                       : v.GL == 16 ? qk_vec_kernel<I, O, MODE, kNeighbours, 16>
                                    : qk_vec_kernel<I, O, MODE, kNeighbours, 32>,
                       dim3(blocks), VT, 0, s, a, v);
}

// Launches with at most `most` blocks; returns how many through *blocks.
template <int MODE>
gdr_status launch(const gdr_qk_dims* d, const QkArgs& a, const gdr_paged_cache* c, int most,
                  int* blocks, cudaStream_t s) {
  const int per = a.HQ + a.HK + (MODE == kAppend ? a.HK : 0);
  const bool vec = vec_ok(d, a, MODE, c);
  const VecPlan v = vec ? vec_plan(a, MODE) : VecPlan();
  const long long units = (long long)v.units[0] + v.units[1] + v.units[2];
  const long long want = vec ? (units * v.GL + VT - 1) / VT
                             : (a.tokens * per + GW - 1) / GW;
  *blocks = (int)(want < most ? want : most);
  return with_dtype(d->in_dtype, [&](auto* i) {
    return with_dtype(d->out_dtype, [&](auto* o) {
      using I = std::remove_pointer_t<decltype(i)>;
      using O = std::remove_pointer_t<decltype(o)>;
      return !vec ? launch_kernel(qk_any_kernel<I, O, MODE>, dim3(*blocks), GW * 32, 0, s, a)
             : a.interleaved ? launch_vec<I, O, MODE, true>(a, v, *blocks, s)
                             : launch_vec<I, O, MODE, false>(a, v, *blocks, s);
    });
  });
}

}  // namespace
}  // namespace ops
}  // namespace gdr

using namespace gdr;
using namespace gdr::ops;

extern "C" {

gdr_status gdr_qk_norm_rope(const void* q, const void* k, const float* q_weight,
                            const float* k_weight, const float* cos, const float* sin,
                            const void* positions, void* q_out, void* k_out,
                            const gdr_qk_dims* dims, gdr_stream_t stream) {
  gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  st = check_shared(dims, q, k, q_weight, k_weight, cos, sin, positions, false);
  if (st != GDR_OK) return st;
  if (!is_aligned(q_out, 16) || !is_aligned(k_out, 16)) return GDR_ERR_ALIGNMENT;
  if (dims->B == 0 || dims->T == 0) return GDR_OK;
  if (!q_out || !k_out) return GDR_ERR_INVALID_ARG;
  QkArgs a = make_args(dims, q_weight, k_weight, cos, sin, positions);
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  int blocks;
  return launch<kFwd>(dims, a, nullptr, 1 << 30, &blocks, reinterpret_cast<cudaStream_t>(stream));
}

size_t gdr_qk_norm_rope_bwd_workspace_size(const gdr_qk_dims* dims) {
  if (check(dims) != GDR_OK) return 0;
  return align_up((size_t)kMaxBlocks * 2 * dims->D * sizeof(float));
}

gdr_status gdr_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                                const void* k, const float* q_weight, const float* k_weight,
                                const float* cos, const float* sin, const void* positions,
                                void* dq, void* dk, float* dq_weight, float* dk_weight,
                                const gdr_qk_dims* dims, void* workspace, size_t workspace_bytes,
                                gdr_stream_t stream) {
  gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  st = check_shared(dims, q, k, q_weight, k_weight, cos, sin, positions, false);
  if (st != GDR_OK) return st;
  if (!is_aligned(dq_out, 16) || !is_aligned(dk_out, 16) || !is_aligned(dq, 16) ||
      !is_aligned(dk, 16) || !is_aligned(dq_weight, 16) || !is_aligned(dk_weight, 16))
    return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->B == 0 || dims->T == 0) {            // no tokens: the sums are zero
    for (float* w : {dq_weight, dk_weight})
      if (w && st == GDR_OK) st = status_of(cudaMemsetAsync(w, 0, dims->D * sizeof(float), s));
    return st;
  }
  if (!dq_out || !dk_out || !dq || !dk) return GDR_ERR_INVALID_ARG;
  QkArgs a = make_args(dims, q_weight, k_weight, cos, sin, positions);
  a.q = q; a.k = k; a.dqo = dq_out; a.dko = dk_out; a.qo = dq; a.ko = dk;
  if (dq_weight || dk_weight) {
    if (!workspace || workspace_bytes < gdr_qk_norm_rope_bwd_workspace_size(dims))
      return GDR_ERR_WORKSPACE;
    if (!is_aligned(workspace, kAlign)) return GDR_ERR_ALIGNMENT;
    a.part = static_cast<float*>(workspace);
  }
  int blocks;
  st = launch<kBwd>(dims, a, nullptr, kMaxBlocks, &blocks, s);
  if (st != GDR_OK || !a.part) return st;
  return launch_behind(qk_weight_kernel, dim3((2 * a.D + SX - 1) / SX), SX * SR, s,
                       (const float*)a.part, blocks, a.D, dq_weight, dk_weight);
}

gdr_status gdr_qk_norm_rope_append(const void* q, const void* k, const void* v,
                                   const float* q_weight, const float* k_weight, const float* cos,
                                   const float* sin, const void* positions, void* q_out,
                                   void* k_cache, void* v_cache, const int32_t* page_table,
                                   const gdr_qk_dims* dims, const gdr_paged_cache* cache,
                                   gdr_stream_t stream) {
  gdr_status st = check(dims);
  if (st != GDR_OK) return st;
  st = check_cache(cache);
  if (st != GDR_OK) return st;
  if (cache->HK != dims->HK || cache->D != dims->D) return GDR_ERR_INVALID_ARG;
  st = check_shared(dims, q, k, q_weight, k_weight, cos, sin, positions, true);
  if (st != GDR_OK) return st;
  if (!is_aligned(v, dtype_size(dims->in_dtype)) || !is_aligned(q_out, 16) ||
      !is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(page_table, 4))
    return GDR_ERR_ALIGNMENT;
  if (dims->B == 0 || dims->T == 0) return GDR_OK;
  if (!v || !q_out || !has_arrays(cache, k_cache, v_cache, page_table)) return GDR_ERR_INVALID_ARG;
  QkArgs a = make_args(dims, q_weight, k_weight, cos, sin, positions);
  a.q = q; a.k = k; a.v = v; a.qo = q_out; a.kc = k_cache; a.vc = v_cache; a.table = page_table;
  a.num_pages = cache->num_pages; a.page = cache->page_size; a.max_pages = cache->max_pages;
  a.cache_bf16 = cache->dtype == GDR_BF16;
  a.pp = cache->page_stride; a.pt = cache->token_stride; a.ph = cache->head_stride;
  int blocks;
  return launch<kAppend>(dims, a, cache, 1 << 30, &blocks,
                         reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
