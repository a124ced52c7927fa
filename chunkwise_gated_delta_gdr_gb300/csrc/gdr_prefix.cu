// gdr_prefix.cu -- attention of one new token per sequence, for a batch whose sequences share a
// prompt: one softmax over the shared keys [0, P) and each sequence's own paged keys.
//
// The queries of all sequences that read one key-value head are the rows of a matrix product
// with the shared keys, which are read once for all of them instead of once per sequence. Over a
// stretch of keys, with a running maximum m per row (base 2: scores carry a factor log2(e)),
//   s = scale q . k,  p = 2^(s - m),  l = sum p,  o = sum p v
// and stretches join as  m = max m_i,  l = sum l_i 2^(m_i - m),  o likewise. A sequence's own
// keys are one more stretch (paged_decode_attn's result and its lse).
//
// Partition. An item is one (key-value head, tile of rows); its keys are cut into tiles. All
// tiles of the call, item after item, form one line that the blocks share out equally; each
// block leaves one part per item of its stretch, and a last kernel joins the parts of a row.
//
// Measured on one GB300, bf16, D = 128, a call among others:
//   128 sequences behind 65000 keys, 32 / 16 heads, 0 .. 1024 own keys: 264-267 us (own keys 98,
//     their join 8, shared keys 145 with the tensor cores 70 % busy, join 10-15; the bytes alone 160)
//   64 behind 8192, 32 / 4 heads, 0 .. 512 own keys: 41 us (16, 22 and 7-13)
//   4 behind 200, 16 / 16 heads: 12.7 us
// fp32, 5 behind 2999, 6 / 3 heads, D = 64: 17.6 us.
//
// The kernels start behind one another and each waits for the one before. That the shared keys'
// kernel would find the call's inputs ready without a wait, since the own keys' one waited for them
// before it let the next one start, is true of the device and promised nowhere; it was worth 2 us on
// 64 behind 8192, 2.6 and 3.6 on the two short ones.
#include <type_traits>

#include "gdr_prefix.cuh"
#include "gdr_prefix_tc.cuh"
#include "gdr_tmap.cuh"

namespace gdr {
namespace ops {
namespace {

// ------------------------------------------------------------ fp32 arithmetic, any type
// Up to 64 rows x 64 keys a step: scores as NI x 4 per thread from shared memory, then the rows'
// softmax by four lanes each, then NI rows x (D / 16) channels per thread of the product with V,
// NI = 1, 2 or 4 as there are rows. fp32 caches with 16-byte rows are copied asynchronously: the
// next tile's K while this one's weights and P V are computed, its V while the next scores are.
// 5 sequences behind 2999 keys, HK = 3, D = 64: a block has one tile, and the call is the chain
// page - row - scores - sums - join (17.6 us; 4 more with a page looked up per row, one row after
// the other). Queries come four channels at a time, up to eight of a thread's loads under way at
// once: 139 sequences behind 2 keys, 4 heads of 256, 32 us (channel by channel 42, and 26 so, when the
// kernel did not wait for the one before). Long prompts are bound by the reads of q and k from shared
// memory: 16 sequences behind 32768 keys, 32 / 8 heads of 128, 244 us where the bytes take 43.
constexpr int RM = 64, KT = 64, NT = 256;
template <int NJ>                                // channels in runs of 64: D <= 64 NJ
struct AnySmem {
  static constexpr int DP = NJ * 64, LD = DP + 4, LS = KT + 4;
  float q[RM * LD], k[KT * LD], v[KT * LD], s[RM * LS];
  float factor[RM];
  int64_t row[2][KT];                            // where the keys of a tile start; -1: none
  int bad;
};

// A tile of K or V into shared memory: asynchronously (to be waited for) or at once.
template <typename T, int NJ>
__device__ __forceinline__ void any_tile(const PrefixArgs& a, float* to, const T* cache,
                                         const int64_t* row, int vec) {
  constexpr int DP = NJ * 64, LD = DP + 4, PER = DP / 4;
#pragma unroll 4
  for (int e = threadIdx.x; e < KT * PER; e += NT) {
    const int r = e / PER, d = 4 * (e - r * PER);
    const int64_t at = row[r];
    if (sizeof(T) == 4 && vec) {
      const bool there = at >= 0 && d < a.D;
      ptx::cp_async16(ptx::smem_u32(to + r * LD + d), cache + (there ? at + d : 0), there ? 16 : 0);
      continue;
    }
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= 0 && d < a.D) {
      if (vec) {
        load_f<T, 4>(cache + at + d, f);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (d + i < a.D) f[i] = static_cast<float>(cache[at + d + i]);
      }
    }
    *reinterpret_cast<float4*>(to + r * LD + d) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// The first n rows of an item's queries, likewise (zeros where there are none).
template <typename T, int NJ>
__device__ __forceinline__ void any_queries(const PrefixArgs& a, float* to, int hk, int r0, int n,
                                            int q_vec) {
  constexpr int DP = NJ * 64, LD = DP + 4, PER = DP / 4;
#pragma unroll 8
  for (int e = threadIdx.x; e < n * PER; e += NT) {
    const int r = e / PER, d = 4 * (e - r * PER), m = r0 + r;
    const bool there = m < a.M && d < a.D;
    const int64_t at = there ? q_row(a, hk, m) + d : 0;
    if (!a.q_bf16 && q_vec) {
      ptx::cp_async16(ptx::smem_u32(to + r * LD + d), static_cast<const float*>(a.q) + at,
                      there ? 16 : 0);
      continue;
    }
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (there) {
      if (q_vec) {
        load_f<bf16, 4>(static_cast<const bf16*>(a.q) + at, f);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (d + i < a.D)
            f[i] = a.q_bf16 ? __bfloat162float(static_cast<const bf16*>(a.q)[at + i])
                            : static_cast<const float*>(a.q)[at + i];
      }
    }
    *reinterpret_cast<float4*>(to + r * LD + d) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// Scores of rows ty + 16 i, keys tx + 16 j; keys from `live` on get -inf.
template <int NJ, int NI>
__device__ __forceinline__ void any_scores(AnySmem<NJ>& sm, int live, float scale2) {
  constexpr int LD = AnySmem<NJ>::LD, LS = AnySmem<NJ>::LS;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float2 acc[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < NJ * 64; d += 4) {
    float4 qv[NI], kv[4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
      qv[i] = *reinterpret_cast<const float4*>(&sm.q[(ty + 16 * i) * LD + d]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      kv[j] = *reinterpret_cast<const float4*>(&sm.k[(tx + 16 * j) * LD + d]);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(make_float2(qv[i].x, qv[i].y), make_float2(kv[j].x, kv[j].y), acc[i][j]);
        acc[i][j] = fma2(make_float2(qv[i].z, qv[i].w), make_float2(kv[j].z, kv[j].w), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sm.s[(ty + 16 * i) * LS + tx + 16 * j] =
          tx + 16 * j < live ? scale2 * (acc[i][j].x + acc[i][j].y) : -INFINITY;
}

// o = factor o + P V for rows ty + 16 i, channels 64 j + 4 tx ..
template <int NJ, int NI>
__device__ __forceinline__ void any_values(const AnySmem<NJ>& sm, float (*o)[NJ * 4]) {
  constexpr int LD = AnySmem<NJ>::LD, LS = AnySmem<NJ>::LS;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float f = sm.factor[ty + 16 * i];
#pragma unroll
    for (int j = 0; j < NJ * 4; ++j) o[i][j] *= f;
  }
#pragma unroll 2
  for (int k = 0; k < KT; k += 4) {
    float4 p[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
      p[i] = *reinterpret_cast<const float4*>(&sm.s[(ty + 16 * i) * LS + k]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.v[(k + e) * LD + 64 * j + 4 * tx]);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
          float2* oo = reinterpret_cast<float2*>(&o[i][4 * j]);
          oo[0] = fma2(make_float2(w, w), make_float2(v.x, v.y), oo[0]);
          oo[1] = fma2(make_float2(w, w), make_float2(v.z, v.w), oo[1]);
        }
      }
  }
}

template <typename T, int NJ>
__global__ void __launch_bounds__(NT) prefix_any_kernel(PrefixArgs a, int vec, int q_vec) {
  extern __shared__ __align__(16) char raw[];
  typedef AnySmem<NJ> Smem;
  constexpr int LS = Smem::LS;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  let_next_begin();
  Stretch st = stretch_of(a, blockIdx.x);
  if (tid == 0) sm.bad = 0;
  wait_for_before();
  // The keys of tile t, each looked up by one thread.
  auto find = [&](int t) {
    if (tid < KT) {
      const int j = t * KT + tid;
      const int64_t r = j < a.P ? prefix_row(a, j) : -1;
      if (j < a.P && r < 0) sm.bad = 1;
      sm.row[t & 1][tid] = r;
    }
  };
  while (st.left > 0) {
    const int hk = st.item / a.row_tiles, r0 = (st.item - hk * a.row_tiles) * RM;
    const int last = min(a.tiles, st.tile + st.left), rows = min(RM, a.M - r0);
    const T* kc = static_cast<const T*>(a.kc) + hk * a.ph;
    const T* vc = static_cast<const T*>(a.vc) + hk * a.ph;
    __syncthreads();                             // the last item's tiles are done with
    find(st.tile);
    any_queries<T, NJ>(a, sm.q, hk, r0, rows <= 16 ? 16 : rows <= 32 ? 32 : RM, q_vec);
    float o[4][NJ * 4], m = -INFINITY, l = 0.f;  // m, l: of row tid / 4
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ * 4; ++j) o[i][j] = 0.f;
    __syncthreads();
    any_tile<T, NJ>(a, sm.k, kc, sm.row[st.tile & 1], vec);
    ptx::cp_async_commit();
    any_tile<T, NJ>(a, sm.v, vc, sm.row[st.tile & 1], vec);
    ptx::cp_async_commit();
    for (int t = st.tile; t < last; ++t) {
      const bool more = t + 1 < last;
      if (more) find(t + 1);
      ptx::cp_async_wait<1>();                   // K of this tile
      __syncthreads();
      if (rows <= 16)
        any_scores<NJ, 1>(sm, a.P - t * KT, a.scale2);
      else if (rows <= 32)
        any_scores<NJ, 2>(sm, a.P - t * KT, a.scale2);
      else
        any_scores<NJ, 4>(sm, a.P - t * KT, a.scale2);
      __syncthreads();
      if (more) any_tile<T, NJ>(a, sm.k, kc, sm.row[(t + 1) & 1], vec);
      ptx::cp_async_commit();
      if (tid >> 2 < (rows + 15) / 16 * 16) {    // four lanes per row, every fourth key each
        float* row = sm.s + (tid >> 2) * LS + (tid & 3);
        float top = m;
#pragma unroll
        for (int j = 0; j < KT; j += 4) top = fmaxf(top, row[j]);
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float f = top > m ? exp2f(m - top) : 1.f;    // 0 from -inf
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KT; j += 4) {
          const float w = exp2f(row[j] - base);
          row[j] = w;
          sum += w;
        }
        m = top;
        l = fmaf(l, f, sum);                     // of this lane's keys; the four meet at the end
        if ((tid & 3) == 0) sm.factor[tid >> 2] = f;
      }
      ptx::cp_async_wait<1>();                   // V of this tile
      __syncthreads();
      if (rows <= 16)
        any_values<NJ, 1>(sm, o);
      else if (rows <= 32)
        any_values<NJ, 2>(sm, o);
      else
        any_values<NJ, 4>(sm, o);
      __syncthreads();
      if (more) any_tile<T, NJ>(a, sm.v, vc, sm.row[(t + 1) & 1], vec);
      ptx::cp_async_commit();
    }
    l += __shfl_xor_sync(~0u, l, 1);
    l += __shfl_xor_sync(~0u, l, 2);
    const size_t part = part_of(a, st.item, blockIdx.x) * RM;
    if ((tid & 3) == 0) {
      a.part_ml[(part + (tid >> 2)) * 2] = m;
      a.part_ml[(part + (tid >> 2)) * 2 + 1] = sm.bad ? NAN : l;   // a bad page poisons the row
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ty + 16 * i < rows)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int d = 64 * j + 4 * tx;
          float* to = a.part_o + (part + ty + 16 * i) * a.D + d;
          if (a.D % 4 == 0) {
            if (d < a.D)
              *reinterpret_cast<float4*>(to) =
                  make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (d + e < a.D) to[e] = o[i][4 * j + e];
          }
        }
    st.left -= last - st.tile;
    st.tile = 0;
    ++st.item;
  }
}

// ------------------------------------------------------------ joining the stretches
// A row (a query head of a sequence) of few parts takes a warp; one of more the JW warps of a
// block, every JW-th part each (SPLIT). A lane holds V channels in a row, N runs of them, and
// has UN parts' loads under way, the first of them before the maximum is known (140 sequences of
// 256 heads of 256 channels behind 9 keys: 146 -> 140 us a call).
constexpr int JW = 4;
template <int V, bool SPLIT>
__global__ void __launch_bounds__(JW * 32) prefix_join_kernel(PrefixArgs a) {
  constexpr int N = 256 / (32 * V), UN = 4, STEP = SPLIT ? JW : 1;
  __shared__ float sum[JW], so[SPLIT ? JW : 1][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = SPLIT ? warp : 0;
  const long long row = SPLIT ? blockIdx.x : (long long)blockIdx.x * JW + warp;
  if (!SPLIT && row >= (long long)a.B * a.HQ) return;
  const int b = (int)(row / a.HQ), hq = (int)(row - (long long)b * a.HQ);
  const int hk = hq / a.G, r = b * a.G + hq - hk * a.G;
  const int item = hk * a.row_tiles + r / a.rows, in = r % a.rows;
  const int parts = parts_of(a, item) * a.units;
  const size_t first = (size_t)item * a.max_parts * a.units * a.rows + in;
  wait_for_before();                             // the stretches are written
  float2 ml[UN];
  float v[UN][N][V], o[N][V];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int c = c0 + STEP * u;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[u][i][k] = 0.f;
      if (c < parts) {
        const size_t at = first + (size_t)c * a.rows;
        ml[u] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int ch = (lane + 32 * i) * V;
          if (ch < a.D) load_f<float, V>(a.part_o + at * a.D + ch, v[u][i]);
        }
      }
    }
  };
  // All of the first loads under way before the first is waited for.
  const float own = a.own_lse[row] * LOG2E;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int ch = (lane + 32 * i) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) o[i][k] = 0.f;
    if (ch < a.D && w0 == 0) load_f<float, V>(a.own_o + (size_t)row * a.D + ch, o[i]);
  }
  load(w0);
  float m = own;
  for (int c = lane; c < parts; c += 32)
    m = fmaxf(m, a.part_ml[(first + (size_t)c * a.rows) * 2]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
  const float base = m == -INFINITY ? 0.f : m;
  float l = w0 == 0 ? exp2f(own - base) : 0.f;   // 0 without keys, NaN where they are bad
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) o[i][k] *= l;
  for (int c0 = w0; c0 < parts;) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const float f = exp2f(ml[u].x - base);
      l = fmaf(f, ml[u].y, l);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] = fmaf(f, v[u][i][k], o[i][k]);
    }
    c0 += STEP * UN;
    if (c0 < parts) load(c0);
  }
  if (SPLIT) {                                   // the warps' sums, in order
    if (lane == 0) sum[warp] = l;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) so[warp][(lane + 32 * i) * V + k] = o[i][k];
    __syncthreads();
    if (warp != 0) return;
    l = sum[0];
#pragma unroll
    for (int w = 1; w < JW; ++w) {
      l += sum[w];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) o[i][k] += so[SPLIT ? w : 0][(lane + 32 * i) * V + k];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int ch = (lane + 32 * i) * V;
    if (ch < a.D) {
#pragma unroll
      for (int k = 0; k < V; ++k) o[i][k] = l == 0.f ? 0.f : o[i][k] * inv;
      if (a.out_bf16)
        store_f<bf16, V>(static_cast<bf16*>(a.out) + (size_t)row * a.D + ch, o[i]);
      else
        store_f<float, V>(static_cast<float*>(a.out) + (size_t)row * a.D + ch, o[i]);
    }
  }
  if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

// ------------------------------------------------------------ host
constexpr int kSms = 152;
// Parts of a row from which the warps of a block share them. The whole call, shared and not: 8
// sequences behind 4096 keys, 16 query heads (16 parts) 15.7 and 17.9 us, 64 (4 parts) 30.5 and 32.2;
// 64 behind 8192, 32 heads (16 parts) 32.4 and 31.6, 128 heads (5 parts) 87 and 75, 192 (4 parts) 115
// and 95. It pays where rows are few, which this border does not ask.
constexpr int kSplitParts = 5;

// How the shared keys of a call are cut up.
struct Plan {
  bool tc, pair;                                 // on the tensor cores; 256 rows a tile
  int rows, keys, units;                         // of a tile; parts of a block per item
  int row_tiles, tiles, blocks, per, max_parts;
  size_t o_bytes, ml_bytes, own_bytes, lse_bytes, decode_bytes;
  size_t bytes() const { return o_bytes + ml_bytes + own_bytes + lse_bytes + decode_bytes; }
};

// f(Config of the head dimension) on the tensor cores.
template <typename F>
auto with_config(int D, F f) {
  return D == 64    ? f(tc::Config<64, true>())
         : D == 80  ? f(tc::Config<80, true>())
         : D == 96  ? f(tc::Config<96, true>())
         : D == 128 ? f(tc::Config<128, true>())
         : D == 192 ? f(tc::Config<192, true>())
                    : f(tc::Config<256, true>());
}

// Whether types, head dimension and strides allow the tensor cores: 16-byte pieces of every
// cache row (their bases are 16-byte aligned by contract).
bool tc_fits(const gdr_attn_dims* d, const gdr_paged_cache* c) {
  const int D = c->D;
  return d->q_dtype == GDR_BF16 && c->dtype == GDR_BF16 &&
         (D == 64 || D == 80 || D == 96 || D == 128 || D == 192 || D == 256) &&
         c->page_stride % 8 == 0 && c->token_stride % 8 == 0 && c->head_stride % 8 == 0;
}

Plan make_plan(const gdr_attn_dims* d, const gdr_paged_cache* c, int P) {
  Plan p = {};
  p.decode_bytes = gdr_paged_decode_attn_workspace_size(d, c);
  // No shared keys: paged_decode_attn's own work; no sequences: nothing to cut up.
  if (P == 0 || d->B == 0) return p;
  const int G = d->HQ / c->HK;
  const long long M = (long long)d->B * G;
  p.rows = RM;
  p.keys = KT;
  p.units = 1;
  int resident = c->D <= 64 ? 2 : 1;
  p.tc = tc_fits(d, c);
  if (p.tc)
    with_config(c->D, [&](auto config) {
      typedef decltype(config) F;
      p.pair = F::U == 2 && M > 128;
      p.rows = p.pair ? 256 : 128;
      p.keys = F::KT;
      p.units = F::U == 2 && !p.pair ? 2 : 1;
      resident = 1;
      return 0;
    });
  p.row_tiles = (int)((M + p.rows - 1) / p.rows);
  p.tiles = (P + p.keys - 1) / p.keys;
  const long long total = (long long)p.row_tiles * c->HK * p.tiles;
  const long long most = (long long)kSms * resident;
  p.blocks = (int)(total < most ? total : most);
  p.per = (int)((total + p.blocks - 1) / p.blocks);
  p.blocks = (int)((total + p.per - 1) / p.per);
  p.max_parts = (p.tiles - 1) / p.per + 2;
  const size_t rows = (size_t)p.row_tiles * c->HK * p.max_parts * p.units * p.rows;
  p.o_bytes = align_up(rows * c->D * sizeof(float));
  p.ml_bytes = align_up(rows * 2 * sizeof(float));
  p.own_bytes = align_up((size_t)d->B * d->HQ * c->D * sizeof(float));
  p.lse_bytes = align_up((size_t)d->B * d->HQ * sizeof(float));
  return p;
}

gdr_status check(const gdr_attn_dims* d, const gdr_paged_cache* c, int prefix_pages, int P) {
  if (!d) return GDR_ERR_INVALID_ARG;
  const gdr_status st = check_cache(c);
  if (st != GDR_OK) return st;
  if (d->B < 0 || d->HQ <= 0 || d->HQ % c->HK != 0 || !is_dtype(d->q_dtype) ||
      !is_dtype(d->out_dtype) || d->window != 0 || d->q_stride_b < 0 || d->q_stride_h < 0 ||
      !(isfinite(d->scale) && d->scale > 0.f) || prefix_pages < 0 || P < 0 ||
      P > (long long)prefix_pages * c->page_size)
    return GDR_ERR_INVALID_ARG;
  if (d->HQ > (1 << 20) || (long long)d->B * d->HQ > (1LL << 30) || P > (1 << 30))
    return GDR_ERR_UNSUPPORTED;
  // Tiles of the line, of 64 rows and keys: counts of them stay within an int.
  if (((double)d->B * d->HQ / 64 + c->HK) * ((double)P / 64 + 1) > (double)(1LL << 37))
    return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

// One of the caches as a tensor map: boxes of 64 channels of one head in `rows` tokens of a page.
bool cache_map(CUtensorMap* m, const void* p, const gdr_paged_cache* c, int rows) {
  const cuuint64_t dims[4] = {(cuuint64_t)c->D, (cuuint64_t)c->HK, (cuuint64_t)c->page_size,
                              (cuuint64_t)c->num_pages};
  const int64_t row = (c->D + 7) / 8 * 8;        // of a dimension that is never stepped along
  const cuuint64_t strides[3] = {
      (cuuint64_t)(c->HK == 1 ? row : c->head_stride) * 2,
      (cuuint64_t)(c->page_size == 1 ? row : c->token_stride) * 2,
      (cuuint64_t)(c->num_pages == 1 ? row : c->page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1};
  return fast::tmap_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool PAIR>
gdr_status launch_tc(const PrefixArgs& a, const gdr_paged_cache* c, cudaStream_t s) {
  const int q_vec = a.qb % 8 == 0 && a.qh % 8 == 0 && is_aligned(a.q, 16);
  CUtensorMap k = {}, v = {};
  auto go = [&](auto tma) {
    constexpr bool TMA = decltype(tma)::value;
    typedef tc::Config<D, TMA> F;
    struct Tag;
    if (!allow_smem<Tag>(tc::prefix_tc_kernel<D, PAIR, TMA>, F::SMEM)) return GDR_ERR_CUDA;
    return launch_behind_smem(tc::prefix_tc_kernel<D, PAIR, TMA>, dim3(a.blocks), F::THREADS,
                              F::SMEM, s, a, q_vec, k, v);
  };
  // Tensor copies where pages and tiles divide one another in runs of 8 rows (which the swizzle
  // repeats after), and the driver takes the strides (a stride of 0 is refused, for one). On 128
  // sequences and 65000 shared keys, HK = 16: 290 us so, 336 us row by row.
  constexpr int KT = tc::Config<D, true>::KT;
  const bool fits = c->page_size % 8 == 0 && (c->page_size % KT == 0 || KT % c->page_size == 0);
  const int rows = c->page_size < KT ? c->page_size : KT;
  if (fits && cache_map(&k, a.kc, c, rows) && cache_map(&v, a.vc, c, rows))
    return go(std::true_type());
  return go(std::false_type());
}

template <typename T, int NJ>
gdr_status launch_any(const PrefixArgs& a, int vec, int blocks, cudaStream_t s) {
  const int q_vec = a.D % 4 == 0 && a.qb % 4 == 0 && a.qh % 4 == 0 &&
                    is_aligned(a.q, a.q_bf16 ? 8 : 16);
  struct Tag;
  if (!allow_smem<Tag>(prefix_any_kernel<T, NJ>, sizeof(AnySmem<NJ>))) return GDR_ERR_CUDA;
  return launch_behind_smem(prefix_any_kernel<T, NJ>, dim3(blocks), NT, sizeof(AnySmem<NJ>), s, a,
                            vec, q_vec);
}

}  // namespace
}  // namespace ops
}  // namespace gdr

using namespace gdr;
using namespace gdr::ops;

extern "C" {

size_t gdr_paged_prefix_attn_workspace_size(const gdr_attn_dims* dims, const gdr_paged_cache* cache,
                                            int prefix_pages, int prefix_len) {
  if (check(dims, cache, prefix_pages, prefix_len) != GDR_OK) return 0;
  return make_plan(dims, cache, prefix_len).bytes();
}

gdr_status gdr_paged_prefix_attn(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* prefix_table, int prefix_pages, int prefix_len,
                                 const int32_t* page_table, const int32_t* lens, void* out,
                                 float* lse, const gdr_attn_dims* dims,
                                 const gdr_paged_cache* cache, void* workspace,
                                 size_t workspace_bytes, gdr_stream_t stream) {
  const gdr_status st = check(dims, cache, prefix_pages, prefix_len);
  if (st != GDR_OK) return st;
  if (!is_aligned(q, dtype_size(dims->q_dtype)) || !is_aligned(k_cache, 16) ||
      !is_aligned(v_cache, 16) || !is_aligned(page_table, 4) || !is_aligned(prefix_table, 4) ||
      !is_aligned(lens, 4) || !is_aligned(out, 16) || !is_aligned(lse, 16))
    return GDR_ERR_ALIGNMENT;
  if (dims->B == 0) return GDR_OK;
  if (!q || !lens || !out || !has_arrays(cache, k_cache, v_cache, page_table) ||
      (prefix_pages > 0 && !prefix_table))
    return GDR_ERR_INVALID_ARG;
  const Plan p = make_plan(dims, cache, prefix_len);
  if (!workspace || workspace_bytes < p.bytes()) return GDR_ERR_WORKSPACE;
  if (!is_aligned(workspace, kAlign)) return GDR_ERR_ALIGNMENT;
  if (prefix_len == 0)
    return gdr_paged_decode_attn(q, k_cache, v_cache, page_table, lens, out, lse, dims, cache,
                                 workspace, workspace_bytes, stream);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* at = static_cast<char*>(workspace);
  PrefixArgs a = {};
  a.part_o = reinterpret_cast<float*>(at);
  a.part_ml = reinterpret_cast<float*>(at += p.o_bytes);
  a.own_o = reinterpret_cast<float*>(at += p.ml_bytes);
  a.own_lse = reinterpret_cast<float*>(at += p.own_bytes);
  void* decode_ws = at += p.lse_bytes;
  a.q = q;
  a.kc = k_cache ? k_cache : workspace;          // never read without pages
  a.vc = v_cache ? v_cache : workspace;
  a.table = prefix_table;
  a.out = out;
  a.lse = lse;
  a.B = dims->B; a.HQ = dims->HQ; a.HK = cache->HK; a.D = cache->D;
  a.G = dims->HQ / cache->HK;
  a.M = dims->B * a.G;
  a.P = prefix_len;
  a.rows = p.rows; a.row_tiles = p.row_tiles; a.tiles = p.tiles; a.per = p.per;
  a.blocks = p.blocks; a.max_parts = p.max_parts;
  a.page = cache->page_size;
  a.num_pages = cache->num_pages;
  a.out_bf16 = dims->out_dtype == GDR_BF16;
  a.q_bf16 = dims->q_dtype == GDR_BF16;
  a.scale2 = dims->scale * LOG2E;
  a.qb = a.B > 1 ? dims->q_stride_b : 0;
  a.qh = a.HQ > 1 ? dims->q_stride_h : 0;
  a.pp = cache->page_stride; a.pt = cache->token_stride; a.ph = cache->head_stride;

  // The sequences' own keys first, bound by HBM; the shared ones' blocks, bound by the tensor
  // cores, come in where those leave an SM.
  gdr_attn_dims own = *dims;
  own.out_dtype = GDR_F32;
  gdr_status run = gdr_paged_decode_attn(q, k_cache, v_cache, page_table, lens, a.own_o, a.own_lse, &own,
                              cache, decode_ws, p.decode_bytes, stream);
  if (run != GDR_OK) return run;
  // A poll may be suspended for about 1 us, as long as sixteen of a flag take.
  a.polls = (long)(set_wait_limit(-1) / 16);
  a.units = p.units;
  if (p.tc) {
    run = with_config(a.D, [&](auto config) {
      constexpr int D = decltype(config)::D;
      if constexpr (decltype(config)::U == 2)
        if (p.pair) return launch_tc<D, true>(a, cache, s);
      return launch_tc<D, false>(a, cache, s);
    });
  } else {
    const int vec = a.D % 4 == 0 && a.pp % 4 == 0 && a.pt % 4 == 0 && a.ph % 4 == 0;
    run = with_dtype(cache->dtype, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      return a.D <= 64    ? launch_any<T, 1>(a, vec, p.blocks, s)
             : a.D <= 128 ? launch_any<T, 2>(a, vec, p.blocks, s)
             : a.D <= 192 ? launch_any<T, 3>(a, vec, p.blocks, s)
                          : launch_any<T, 4>(a, vec, p.blocks, s);
    });
  }
  if (run != GDR_OK) return run;
  // The join may start while the shared keys are being worked on; it waits for their kernel
  // itself, which ends behind the one for the sequences' own keys.
  const unsigned rows = (unsigned)(a.B * a.HQ);
  if ((p.max_parts - 1) * p.units >= kSplitParts)
    return launch_behind(a.D % 4 == 0 ? prefix_join_kernel<4, true> : prefix_join_kernel<1, true>,
                         dim3(rows), JW * 32, s, a);
  return launch_behind(a.D % 4 == 0 ? prefix_join_kernel<4, false> : prefix_join_kernel<1, false>,
                       dim3((rows + JW - 1) / JW), JW * 32, s, a);
}

}  // extern "C"
