// gdr_prefix_tc.cuh -- the shared keys' part of the attention behind a shared prompt, on the
// tensor cores (tcgen05): bf16 queries and caches.
//
// A step is a tile of 128 rows by KT keys: S = Q K^T into TMEM, the rows' softmax by 128 threads
// (one row each, so that no sum or maximum crosses a thread), the weights back into TMEM in the
// place of their scores, O += P V with P read from TMEM.
//
// Two units of 128 threads take steps in turn, so that one's softmax runs under the other's
// products. With more than 128 rows per key head (PAIR) a block takes 256 rows, one half per
// unit, and both read the same keys; with fewer the units take every other tile of keys and
// leave a part each. Heads of 256 channels leave TMEM for one unit, with two tiles of scores.
//
// Weights. As in paged_decode_attn, a weight goes into the product with V as two bf16: its upper
// bits as they are and what they leave over, rounded; 2^-15 of it is lost at most (one bf16 alone
// would put as much error into a bf16 result as rounding that does). That makes the products
// 3/2 of the plain count: (QK + 2 PV) = 6 rows keys D operations.
// Per 16 keys the weights' TMEM columns are 8 of upper parts and 8 of rests, in the columns of
// the scores they come from.
//
// What bounds it: the chain S - softmax - P V of two units. A step is 1536 cycles of products by
// count and takes 2200 (65000 keys, 256 rows per key head): Q K^T reads both operands from shared
// memory at its limit while the copies write there, and each of the two waits of a step between
// products costs some 200. The softmax is 1600 cycles of the other unit's time, some of it spills: the
// 168 registers that 9 or 10 warps share equally do not quite hold a row's 128 scores.
//
// Maximum. o and l are kept against a reference that is moved (and o rescaled in TMEM) only when
// a row's scores pass it by more than 2^8: weights stay below 2^8, far from any limit of fp32.
#pragma once

#include "gdr_prefix.cuh"

namespace gdr {
namespace ops {
namespace tc {

using namespace ptx;

// TMA: tiles come by tensor copies, a box per page and 64 channels; without, row by row (pages
// that do not fill whole runs of 8 rows of a tile).
template <int D_, bool TMA>
struct Config {
  static constexpr int D = D_, NB = (D + 63) / 64, C = D / 8;
  static constexpr int U = D <= 192 ? 2 : 1;               // units: TMEM columns U D + 2 KT <= 512
  static constexpr int KT = D <= 128 ? 128 : 64;           // keys of a tile
  static constexpr int QTILE = NB * 128 * 128, TILE = NB * KT * 128;   // bytes
  static constexpr int ST = D <= 64 ? 8 : 5;               // tiles of the ring, K and V in turn
  static constexpr int SOFT = 4 * U, LOAD = TMA ? 1 : 3, THREADS = 32 * (SOFT + LOAD + 1);
  static constexpr int SMEM = U * QTILE + ST * TILE + 1024 + 256;
  static constexpr uint32_t T_S = 0, T_O = 2 * KT;         // TMEM columns: S x 2, O x U
  static_assert(U * D + 2 * KT <= 512 && SMEM <= 232448, "");
};
constexpr int LAG = 3;                                     // tiles of copies in flight, less one
constexpr long kDrainPolls = 1L << 20;                     // of the last waits; about a second

__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                             int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc));
}
// 32 columns of this warp's lanes, without waiting for them; tmem_take() makes them usable.
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_take(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// 16 columns, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_put_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {            // 2^x, 2 ulp; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// One lane of a converged warp. What it guards runs with the warp's uniform registers, which a
// test of the lane's number would not allow (the products' descriptors: 386 -> 304 us on
// 128 sequences, 65000 shared keys, HK = 16).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// A row's scores from TMEM.
template <int KT>
__device__ __forceinline__ void tile_scores(uint32_t s_at, uint32_t* x) {
#pragma unroll
  for (int c = 0; c < KT / 32; ++c) tmem_get(s_at + 32 * c, x + 32 * c);
#pragma unroll
  for (int c = 0; c < KT / 32; ++c) tmem_take(x + 32 * c);
}
// The largest of them; those from `live` on become -inf.
template <int KT, bool MASK>
__device__ __forceinline__ float tile_max(uint32_t* x, int live) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (MASK) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
      if (k >= live) x[k] = 0xff800000u;
  }
#pragma unroll
  for (int k = 0; k < KT; k += 2)
    top[(k >> 1) & 3] = max3(top[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
  return fmaxf(max3(top[0], top[1], top[2]), top[3]);
}
// A row's weights 2^(scale s - ref), in TMEM in the place of its scores; returns their sum. What
// bounds this is the pipe of the 32-bit integer and conversion instructions (two cycles each):
// per pair of keys two extractions, two packings and, above, one maximum.
template <int KT>
__device__ __forceinline__ float tile_weights(uint32_t s_at, const uint32_t* x, float scale2,
                                              float ref) {
  const float2 scale = make_float2(scale2, scale2), off = make_float2(-ref, -ref);
  const float2 one = make_float2(1.f, 1.f), more = make_float2(1.f + 0x1p-20f, 1.f + 0x1p-20f);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < KT / 16; ++c) {
    uint32_t w[16];                                        // 8 upper parts, 8 rests
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const uint32_t* y = x + 16 * c + k;
      float2 p = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), scale, off);
      p.x = ex2(p.x);
      p.y = ex2(p.y);
      sum[(k >> 1) & 1] = fma2(p, one, sum[(k >> 1) & 1]);
      const uint32_t hi = __byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x7632);
      // 2^-20 of the weight on top: the rest is not 0 beside an upper part that is not (down to
      // weights of 2^-106), so that an infinite v gives what w v gives.
      const float2 hif = unpack2(hi), rest = fma2(p, more, make_float2(-hif.x, -hif.y));
      w[k >> 1] = hi;
      w[8 + (k >> 1)] = pack2(rest.x, rest.y);
    }
    tmem_put16(s_at + 16 * c, w);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}
// 8 consecutive words of one thread, 32-byte aligned.
__device__ __forceinline__ void store8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

struct Bars {
  uint64_t kv_full[8], kv_empty[8];   // a tile of K or V: LOAD arrivals; commit of its last product
  uint64_t s_full[2], p_full[2];      // scores: commit; weights in their place: 4 arrivals
  uint64_t pv_done[2];                // commit of the step's product with V
  uint64_t q_full, fin;               // an item's queries: SOFT arrivals; all products, at the end
  uint32_t tmem, dead, bad;           // dead: a wait gave up; bad: a page out of range
};

// A wait that gives up after `polls`, or when another role has: then every role runs to its end,
// the block's remaining parts get a sum of NaN, and copies and products under way are waited for,
// again with a limit.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, long polls,
                                         volatile uint32_t* dead) {
  if (mbar_test(bar, parity)) return true;
  for (long i = 0; i < polls; ++i) {
    if (mbar_wait(bar, parity, 1)) return true;
    if (*dead) return false;
  }
  *dead = 1;
  return false;
}

// PAIR: 256 rows a block, a half per unit, every tile of keys taken by both.
template <int D, bool PAIR, bool TMA>
__global__ void __launch_bounds__(Config<D, TMA>::THREADS, 1)
    prefix_tc_kernel(PrefixArgs a, int q_vec, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  typedef Config<D, TMA> F;
  constexpr int U = F::U, KT = F::KT, ST = F::ST, C = F::C, PER_TILE = PAIR ? 2 : 1;
  constexpr int ROWS = PAIR ? 256 : 128;
  static_assert(!PAIR || U == 2, "");
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                       ~static_cast<uintptr_t>(1023));
  __shared__ Bars bars;
  let_next_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_at = smem_u32(base), ring = q_at + U * F::QTILE;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.kv_full[i], F::LOAD);
      mbar_init(&bars.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.q_full, F::SOFT);
    mbar_init(&bars.fin, 1);
    bars.dead = bars.bad = 0;
    mbar_fence_init();
  }
  if (warp == F::SOFT + F::LOAD) tmem_alloc(&bars.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile uint32_t* dead = &bars.dead;
  Stretch st = stretch_of(a, blockIdx.x);
  wait_for_before();                                       // nothing above touches global memory
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, a.polls, dead); };

  if (warp < F::SOFT) {
    // ------------------------------------------------------------ softmax
    const int unit = warp >> 2, row = threadIdx.x & 127;   // row = TMEM lane
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_at = tmem + lanes + F::T_O + unit * D;
    bool ok = true;
    int g = 0, n0 = 0;                                     // steps and tiles of the block so far
    for (; st.left > 0; ++st.item, st.tile = 0) {
      const int hk = st.item / a.row_tiles, r0 = (st.item - hk * a.row_tiles) * ROWS;
      const int last = min(a.tiles, st.tile + st.left), steps = (last - st.tile) * PER_TILE;
      if (ok) {
        for (int e = threadIdx.x; e < ROWS * C; e += 128 * U) {
          const int r = e / C, ch = e - r * C, m = r0 + r;
          const uint32_t to = (r >> 7) * F::QTILE + (ch >> 3) * 16384 + (r & 127) * 128 +
                              (((ch ^ r) & 7) << 4);
          const bf16* src = static_cast<const bf16*>(a.q) + (m < a.M ? q_row(a, hk, m) + ch * 8 : 0);
          if (q_vec) {                                     // all of a thread's pieces under way at once
            cp_async16(q_at + to, src, m < a.M ? 16 : 0);
          } else {
            const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m < a.M)
              v = make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16,
                             s[4] | (uint32_t)s[5] << 16, s[6] | (uint32_t)s[7] << 16);
            *reinterpret_cast<uint4*>(base + to) = v;
          }
        }
        cp_async_wait_all();
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_full);
      }
      float m = -INFINITY, l = 0.f;
      int prev = -1;                                       // this unit's last step
      for (int i = 0; i < steps && ok; ++i, ++g) {
        const int buf = g & 1;
        // Unit of a step: its half of the rows, or whose turn it is.
        if (U == 2 && buf != unit) continue;
        const uint32_t s_at = tmem + lanes + F::T_S + buf * KT;
        const int key0 = (st.tile + (PAIR ? i >> 1 : i)) * KT, live = a.P - key0;
        ok = wait(&bars.s_full[buf], (g >> 1) & 1);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[KT];
        tile_scores<KT>(s_at, x);
        float top = live >= KT ? tile_max<KT, false>(x, live) : tile_max<KT, true>(x, live);
        top *= a.scale2;
        if (__any_sync(~0u, top > m + 8.f)) {              // and from -inf
          const float to = fmaxf(m, top), f = to > m ? ex2(m - to) : 1.f;    // 0 from -inf
          m = to;
          l *= f;
          if (prev >= 0) {
            ok = wait(&bars.pv_done[prev & 1], (prev >> 1) & 1);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(o_at + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_put16(o_at + 16 * c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        l += tile_weights<KT>(s_at, x, a.scale2, ref);
        if (TMA && live < KT && (!PAIR || unit == 0)) {
          // Rows of V behind the prompt's end, whatever they hold: their weights are 0.
          const int n = n0 + 2 * (PAIR ? i >> 1 : i) + 1;
          ok = __all_sync(~0u, wait(&bars.kv_full[n % ST], (n / ST) & 1));
          if (!ok) break;
          char* v = base + U * F::QTILE + (n % ST) * F::TILE;
          for (int e = row; e < (KT - live) * F::NB * 8; e += 128) {
            const int r = live + e / (F::NB * 8), c = e % (F::NB * 8);
            *reinterpret_cast<uint4*>(v + (c >> 3) * (KT * 128) + r * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        tmem_put_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[buf]);
        prev = g;
      }
      if (ok && prev >= 0) {
        ok = wait(&bars.pv_done[prev & 1], (prev >> 1) & 1);
        ok = __all_sync(~0u, ok);
        tc_fence_after();
      }
      // This unit's part: a row of its half of the tile, or of its share of the keys.
      const size_t part = PAIR || U == 1
                              ? part_of(a, st.item, blockIdx.x) * ROWS + (PAIR ? unit * 128 : 0) + row
                              : (part_of(a, st.item, blockIdx.x) * 2 + unit) * ROWS + row;
      const bool mine = r0 + (PAIR ? unit * 128 : 0) + row < a.M;
      if (mine) {
        a.part_ml[part * 2] = m;
        a.part_ml[part * 2 + 1] = !ok || *(volatile uint32_t*)&bars.bad ? NAN : l;
      }
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          if (prev >= 0) {
            tmem_ld16(o_at + 16 * c, o);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0u;
          }
          if (mine) {
            store8(a.part_o + part * D + 16 * c, o);
            store8(a.part_o + part * D + 16 * c + 8, o + 8);
          }
        }
        tc_fence_before();
      }
      st.left -= last - st.tile;
      n0 += 2 * (last - st.tile);
      // All scores of the item are in, so its queries are done with.
      if (U == 2 && st.left > 0) asm volatile("bar.sync 1, 256;" ::: "memory");
      if (U == 1 && st.left > 0) asm volatile("bar.sync 1, 128;" ::: "memory");
      ok = __all_sync(~0u, ok && !*dead);
    }
  } else if (TMA && warp == F::SOFT) {
    // ------------------------------------------------------------ copies, page by page
    const int R = min(a.page, KT), boxes = KT / R * F::NB; // rows of a box
    int n = 0;                                             // tiles issued
    bool ok = true;
    int tok = 0;                                           // of this lane's page: its first row
    auto find = [&](int tile) {                            // -1: no such keys, or a bad page
      const int j = tile * KT + lane * R;
      if (lane >= KT / R || j >= a.P) return -1;
      const int pj = j / a.page, pg = a.table[pj];
      tok = j - pj * a.page;
      if (pg >= 0 && pg < a.num_pages) return pg;
      bars.bad = 1;
      return -1;
    };
    for (; st.left > 0 && ok; ++st.item, st.tile = 0) {
      const int hk = st.item / a.row_tiles;
      const int last = min(a.tiles, st.tile + st.left);
      int next = find(st.tile);
      for (int t = st.tile; t < last && ok; ++t) {
        const int pg = next, at = tok;
        if (t + 1 < last) next = find(t + 1);              // looked up meanwhile
        const int pages = __popc(__ballot_sync(~0u, pg >= 0));
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int slot = n % ST;
          if (n >= ST) {
            ok = __all_sync(~0u, wait(&bars.kv_empty[slot], (n / ST - 1) & 1));
            if (!ok) break;
          }
          if (lane == 0) mbar_expect_tx(&bars.kv_full[slot], pages * F::NB * R * 128);
          __syncwarp();
          for (int e0 = 0; e0 < boxes; e0 += 32) {
            const int e = e0 + lane, i = e / F::NB, c = e - i * F::NB;
            const int p = __shfl_sync(~0u, pg, i & 31), row = __shfl_sync(~0u, at, i & 31);
            if (e < boxes && p >= 0)
              tma_load4(ring + slot * F::TILE + c * (KT * 128) + i * (R * 128), kv ? &v_map : &k_map,
                        c * 64, hk, row, p, &bars.kv_full[slot]);
          }
        }
      }
      st.left -= last - st.tile;
    }
    for (int k = max(0, n - ST); k < n; ++k)               // no copy outlives the block
      mbar_wait(&bars.kv_full[k % ST], (k / ST) & 1, kDrainPolls);
  } else if (!TMA && warp < F::SOFT + F::LOAD) {
    // ------------------------------------------------------------ copies, row by row
    // Warp w takes every third row from w on. (A fourth warp would leave the softmax 128 registers
    // instead of 168; with these, tiles of 128 keys spill 80 to 142 bytes, those of 64 keys nothing.)
    constexpr int RW = (KT + F::LOAD - 1) / F::LOAD, NO = (RW + 31) / 32;   // rows of a warp, a lane
    const int w = warp - F::SOFT;
    const bf16 *kc = static_cast<const bf16*>(a.kc), *vc = static_cast<const bf16*>(a.vc);
    int n = 0, sent = 0;                                   // tiles issued, tiles handed over
    bool ok = true;
    auto hand_over = [&]() {                               // this warp's copies of tile `sent` are in
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.kv_full[sent % ST]);
      ++sent;
    };
    // Where this lane's rows of a tile start; -1: no such key, or a bad page.
    auto find = [&](int tile, int64_t* off) {
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const int in = w + F::LOAD * (lane + 32 * i), j = tile * KT + in;
        off[i] = -1;
        if (in < KT && j < a.P) {
          off[i] = prefix_row(a, j);
          if (off[i] < 0) bars.bad = 1;
        }
      }
    };
    for (; st.left > 0 && ok; ++st.item, st.tile = 0) {
      const int hk = st.item / a.row_tiles;
      const int last = min(a.tiles, st.tile + st.left);
      int64_t next[NO];
      find(st.tile, next);
      for (int t = st.tile; t < last && ok; ++t) {
        int64_t off[NO];
#pragma unroll
        for (int i = 0; i < NO; ++i) off[i] = next[i];
        if (t + 1 < last) find(t + 1, next);               // looked up meanwhile
#pragma unroll 1
        for (int kv = 0; kv < 2 && ok; ++kv, ++n) {
          const int slot = n % ST;
          if (n >= ST) {
            const uint32_t parity = (n / ST - 1) & 1;
            if (!__all_sync(~0u, mbar_test(&bars.kv_empty[slot], parity))) {
              // Nothing is held back while this waits.
              cp_async_wait<0>();
              while (sent < n) hand_over();
              ok = __all_sync(~0u, wait(&bars.kv_empty[slot], parity));
              if (!ok) break;
            }
          }
          const bf16* src = (kv ? vc : kc) + hk * a.ph;
          const uint32_t to = ring + slot * F::TILE;
#pragma unroll 8
          for (int i = 0; i < (RW * C + 31) / 32; ++i) {
            const int e = lane + 32 * i, r = e / C, ch = e - r * C, in = w + F::LOAD * r;
            int64_t o = __shfl_sync(~0u, off[0], r & 31);
            if (NO > 1) {
              const int64_t o1 = __shfl_sync(~0u, off[NO - 1], r & 31);
              if (r >= 32) o = o1;
            }
            if (in < KT)
              cp_async16(to + (ch >> 3) * (KT * 128) + in * 128 + (((ch ^ in) & 7) << 4),
                         src + (o < 0 ? 0 : o + ch * 8), o < 0 ? 0 : 16);
          }
          cp_async_commit();
          if (n - sent >= LAG) {
            cp_async_wait<LAG>();
            hand_over();
          }
        }
      }
      st.left -= last - st.tile;
    }
    cp_async_wait<0>();
    while (sent < n) hand_over();
  } else if (warp == F::SOFT + F::LOAD && elect()) {
    // ------------------------------------------------------------ products
    // S of the next step but one goes right behind O += P V of this one, whose place in TMEM it
    // takes: that keeps the units out of step, one's softmax under the other's products. (A
    // thread each for S and for P V queued both units' P V first, and both softmaxes met: 316 us
    // instead of 290 on 128 sequences, 65000 shared keys, HK = 16.)
    constexpr uint32_t ID_QK = idesc_bf16_kk(128, KT), ID_PV = idesc_bf16(128, D, 0, 1);
    const uint64_t q_desc = sdesc_sw128(q_at), k_desc = sdesc_sw128(ring);
    const uint64_t v_desc = sdesc_sw128_lbo(ring, KT * 128);
    int g0 = 0, n0 = 0;                                    // steps and tiles before this item
    bool ok = true;
    for (int item = 0; st.left > 0 && ok; ++item, st.tile = 0) {
      const int tiles = min(a.tiles - st.tile, st.left), steps = tiles * PER_TILE;
      auto scores = [&](int i) {                           // S of step i
        const int n = n0 + 2 * (PAIR ? i >> 1 : i), slot = n % ST, g = g0 + i;
        if (!PAIR || (i & 1) == 0) ok = ok && wait(&bars.kv_full[slot], (n / ST) & 1);
        // The weights of two steps ago, in the same place, have been used.
        if (g >= 2) ok = ok && wait(&bars.pv_done[g & 1], ((g >> 1) - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        // Descriptors count 16 bytes.
        const uint64_t q = q_desc + (PAIR ? (i & 1) * (F::QTILE >> 4) : 0);
        const uint64_t k = k_desc + slot * (F::TILE >> 4);
        const uint32_t d = tmem + F::T_S + (g & 1) * KT;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          umma_bf16(d, q + (c >> 2) * 1024 + (c & 3) * 2, k + (c >> 2) * (KT * 8) + (c & 3) * 2,
                    ID_QK, c > 0);
        umma_commit(&bars.s_full[g & 1]);
        if (!PAIR || (i & 1)) umma_commit(&bars.kv_empty[slot]);
      };
      ok = wait(&bars.q_full, item & 1);
      if (ok) scores(0);
      if (ok && steps > 1) scores(1);
      for (int i = 0; i < steps && ok; ++i) {
        const int n = n0 + 2 * (PAIR ? i >> 1 : i) + 1, slot = n % ST, g = g0 + i;
        if (!PAIR || (i & 1) == 0) ok = ok && wait(&bars.kv_full[slot], (n / ST) & 1);
        ok = ok && wait(&bars.p_full[g & 1], (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t p = tmem + F::T_S + (g & 1) * KT, o = tmem + F::T_O + (U == 2 ? g & 1 : 0) * D;
        const uint64_t v = v_desc + slot * (F::TILE >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int c = 0; c < KT / 16; ++c)
            umma_bf16_ts(o, p + 16 * c + 8 * part, v + c * 128, ID_PV, i >= U || part || c);
        umma_commit(&bars.pv_done[g & 1]);
        if (!PAIR || (i & 1)) umma_commit(&bars.kv_empty[slot]);
        if (i + 2 < steps) scores(i + 2);
      }
      g0 += steps;
      n0 += 2 * tiles;
      st.left -= tiles;
    }
    umma_commit(&bars.fin);                                // and no product
    mbar_wait(&bars.fin, 0, kDrainPolls);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == F::SOFT + F::LOAD) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace tc
}  // namespace ops
}  // namespace gdr
