// gdr_paged.cu -- attention of one new token per sequence over a paged key-value cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - m),  lse = m + log sum_j p_j
//
// over the keys lo <= j < len, lo = max(0, len - window). The running maximum m and the
// sums are kept per stretch of keys; two stretches join as
//   m = max(m1, m2),  l = l1 e^{m1 - m} + l2 e^{m2 - m},  o likewise.
// All of it runs in base 2: scores carry a factor log2(e).
//
// Partition. An item is one (sequence, key-value head, group of query heads); its keys are
// cut into tiles of TILE keys. All tiles of the call, item after item, form one line that
// the blocks share out equally, whatever the lengths are: block c takes the tiles
// [c per, (c + 1) per), per = ceil(total / blocks). The lengths are read on the device, so
// the host needs none of them. A block that holds a whole item writes its result; an item
// cut by a block boundary leaves partial results, at most two per block (slot 0: the item
// began in an earlier block, slot 1: it began here), which paged_join_kernel joins in order.
//
// The cache is read once: 2 len HK D elements, against 4 len HQ D operations, a few % of the
// tensor rate at 8 queries a head. Bound by HBM from some 100 MB on, by the chain length -
// page - row - sums below. Measured on one GB300, bf16, D = 128, kv heads of the cache HK:
//   1 x 65000 keys, HK = 16, 2 queries a head: 90-92 us, 5.8-6.0 TB/s (a plain copy: 6.78 TB/s)
//   64 sequences of 0 .. 8192 keys, HK = 4, 8 queries a head: 104-106 us, 75-77 % of the copy rate
//   4 x 200 keys, HK = 16: 7.1 us a call (8.2 when it starts after the kernel before has ended)
// 16 x 8000 keys, HK = 8, D = 128: 4 queries a head 92 us, 5.7 TB/s; 16 97 us; 32 182 us, since the
// cache is read once per group of 16.
// fp32, 16 x 8000 keys, HK = 8: D = 256 309 us, 6.8 TB/s; D = 64 92 us, 5.7; D = 128 with 4
// queries a head 174 us, 6.0; with 8 241 us, 4.3, bound by the reads of q from shared memory
// (that pipe is 65 % busy, fp32 arithmetic 17 %).
// The general kernel, same keys: fp32 D = 72, 2 queries a head 277 us, 2.1 TB/s; bf16, 4 queries,
// D = 40 529 us and D = 136 858 us, 0.3 and 0.6 TB/s: its rows come through registers, a few keys
// at a time, once per 4 query heads (2 beyond D = 128).
#include <type_traits>

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"

namespace gdr {
namespace ops {
namespace {

constexpr int TILE = 64;          // keys per tile
constexpr int WARPS = 4;          // per block
constexpr int GMAX = 16;          // query heads of an item at most
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct AttnArgs {
  const void *q, *kc, *vc;
  const int32_t *table, *lens;
  void* out;
  float* lse;                     // may be null
  float *part_o, *part_ml;        // [blocks][2][GMAX][D], [blocks][2][GMAX][2]
  int by_item, hb;                // of the join: a block per item, or per boundary; heads per block
  int B, HQ, HK, D, G, GH, groups;  // G = HQ / HK; GH query heads per item, groups per kv head
  int page, shift;                // shift: log2(page) if page is a power of two, else -1
  int num_pages, max_pages, window, whole, blocks, out_bf16, q_bf16;
  float scale2;                   // scale log2(e)
  int64_t qb, qh, pp, pt, ph;
  long long cap;                  // max_pages * page
};

// Keys of sequence b: [lo, n), and whether its length is valid.
struct Span {
  int lo, n;
  bool ok;
  __device__ int tiles() const { return (n - lo + TILE - 1) / TILE; }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  const int n = a.lens[b];
  Span s;
  s.ok = n >= 0 && n <= a.cap;
  s.n = s.ok ? n : 0;
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  return s;
}

// A place on the line of tiles.
struct Place {
  int b, item, tile;   // sequence, (kv head, group), tile of it
  Span s;
};

// All lanes of a warp: tiles of the whole call.
__device__ __forceinline__ long long total_tiles(const AttnArgs& a, int lane) {
  long long t = 0;
  for (int b = lane; b < a.B; b += 32) t += span_of(a, b).tiles();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
  return t * a.HK * a.groups;
}

// All lanes of a warp: the place of tile w < total of the line.
__device__ __forceinline__ Place locate(const AttnArgs& a, long long w, int lane) {
  const int per_b = a.HK * a.groups;
  long long base = 0;
  for (int b0 = 0;; b0 += 32) {
    const long long t = b0 + lane < a.B ? (long long)span_of(a, b0 + lane).tiles() * per_b : 0;
    long long inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned hit = __ballot_sync(~0u, base + inc > w);
    if (hit || b0 + 32 >= a.B) {
      const int src = hit ? __ffs(hit) - 1 : 0;
      const long long first = __shfl_sync(~0u, base + inc - t, src);
      Place p;
      p.b = min(b0 + src, a.B - 1);
      p.s = span_of(a, p.b);
      const int tiles = max(1, p.s.tiles());
      p.item = (int)((w - first) / tiles);
      p.tile = (int)((w - first) - (long long)p.item * tiles);
      return p;
    }
    base += __shfl_sync(~0u, inc, 31);
  }
}

// The first item after p that has tiles (there has to be one).
__device__ __forceinline__ void next_item(const AttnArgs& a, Place& p) {
  p.tile = 0;
  if (++p.item < a.HK * a.groups) return;
  p.item = 0;
  do {
    p.s = span_of(a, ++p.b);
  } while (p.s.tiles() == 0 && p.b + 1 < a.B);
}

__device__ __forceinline__ void put(void* out, size_t i, float v, int is_bf16) {
  if (is_bf16)
    static_cast<bf16*>(out)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(out)[i] = v;
}

// Results of head `hq` of sequence b (channel d) from the sums, m in base 2.
__device__ __forceinline__ void finish_lse(const AttnArgs& a, int b, int hq, float m, float l) {
  if (a.lse) a.lse[(size_t)b * a.HQ + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}
__device__ __forceinline__ void finish(const AttnArgs& a, int b, int hq, int d, float m, float l,
                                       float o) {
  const size_t row = (size_t)b * a.HQ + hq;
  put(a.out, row * a.D + d, l == 0.f ? 0.f : o / l, a.out_bf16);
  if (d == 0) finish_lse(a, b, hq, m, l);
}

// Sequences without tiles: zeros and -inf (no keys), NaN (an invalid length).
__device__ __forceinline__ void empty_rows(const AttnArgs& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Span s = span_of(a, b);
    if (s.tiles()) continue;
    const float o = s.ok ? 0.f : NAN;
    for (int i = threadIdx.x; i < a.HQ * a.D; i += blockDim.x)
      put(a.out, (size_t)b * a.HQ * a.D + i, o, a.out_bf16);
    if (a.lse)
      for (int i = threadIdx.x; i < a.HQ; i += blockDim.x)
        a.lse[(size_t)b * a.HQ + i] = s.ok ? -INFINITY : NAN;
  }
}

// This block's stretch of the line: its first place and its number of tiles (0: none).
__device__ __forceinline__ long long stretch(const AttnArgs& a, int lane, Place* p) {
  if (a.whole) {                   // one block per item
    p->b = blockIdx.x / (a.HK * a.groups);
    p->item = blockIdx.x - p->b * (a.HK * a.groups);
    p->tile = 0;
    p->s = span_of(a, p->b);
    return p->s.tiles();
  }
  const long long total = total_tiles(a, lane), per = (total + a.blocks - 1) / a.blocks;
  const long long first = blockIdx.x * per, last = min(total, first + per);
  if (first >= last) return 0;
  *p = locate(a, first, lane);
  return last - first;
}

// Element offset of key j of sequence b (kv head 0), or -1 for a bad table entry.
__device__ __forceinline__ int64_t key_row(const AttnArgs& a, int b, int j) {
  const int pj = a.shift >= 0 ? j >> a.shift : j / a.page;
  const int32_t pg = a.table[(size_t)b * a.max_pages + pj];
  if (pg < 0 || pg >= a.num_pages) return -1;
  return pg * a.pp + (j - pj * a.page) * a.pt;
}

// ------------------------------------------------------------ fp32 arithmetic, any type
// Eight lanes per key: lane c of an octet holds the channels 4 (c + 8 i) .. + 3, i < NC,
// so a warp works on four keys at a time and a row is read in 16-byte pieces (8-byte for
// bf16). Each octet keeps its own maximum and sums for the item's GH heads.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int ch, int D, bool vec, float* f) {
  if (vec) {
    if (ch < D)
      load_f<T, 4>(row + ch, f);
    else
      f[0] = f[1] = f[2] = f[3] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = ch + e < D ? static_cast<float>(row[ch + e]) : 0.f;
  }
}

template <typename T, int NC, int GH>
__global__ void __launch_bounds__(WARPS * 32) paged_any_kernel(AttnArgs a, int vec) {
  constexpr int DP = NC * 32, KU = NC == 2 ? 4 : NC == 4 ? 2 : 1;   // keys in flight per octet
  __shared__ float so[WARPS][GH][DP], sml[WARPS][GH][2];
  begin_behind();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7, oct = lane >> 3;
  empty_rows(a);
  Place p;
  long long left = stretch(a, lane, &p);
  while (left > 0) {
    const int tiles = p.s.tiles();
    const int t1 = (int)min((long long)tiles, p.tile + left);
    const int hk = p.item / a.groups, g0 = (p.item - hk * a.groups) * GH;
    const int heads = min(GH, a.G - g0), hq0 = hk * a.G + g0;
    float q[GH][NC * 4], o[GH][NC * 4], m[GH], l[GH];
#pragma unroll
    for (int g = 0; g < GH; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int i = 0; i < NC * 4; ++i) {
        const int ch = 4 * (c + 8 * (i >> 2)) + (i & 3);
        o[g][i] = 0.f;
        q[g][i] = 0.f;
        if (g < heads && ch < a.D) {
          const int64_t at = p.b * a.qb + (hq0 + g) * a.qh + ch;
          q[g][i] = a.scale2 * (a.q_bf16 ? __bfloat162float(static_cast<const bf16*>(a.q)[at])
                                         : static_cast<const float*>(a.q)[at]);
        }
      }
    }
    const int end = min(p.s.n, p.s.lo + t1 * TILE);
    const T* kc = static_cast<const T*>(a.kc) + hk * a.ph;
    const T* vc = static_cast<const T*>(a.vc) + hk * a.ph;
    // KU keys per octet at a time; the next ones' pages are looked up meanwhile.
    int j0 = p.s.lo + p.tile * TILE + warp * 4 + oct;
    int64_t row[KU];
    auto find = [&](int j) {
#pragma unroll
      for (int u = 0; u < KU; ++u)               // -1: bad page, -2: no such key
        row[u] = j + 16 * u < end ? key_row(a, p.b, j + 16 * u) : -2;
    };
    find(j0);
    for (int jw = j0 - oct; jw < end; jw += 16 * KU, j0 += 16 * KU) {
      float s[KU][GH], vv[KU][NC * 4];
      int64_t at[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) at[u] = row[u];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        float kv[NC * 4];
#pragma unroll
        for (int i = 0; i < NC * 4; ++i) kv[i] = vv[u][i] = 0.f;
        if (at[u] >= 0) {
#pragma unroll
          for (int i = 0; i < NC; ++i) load4<T>(kc + at[u], 4 * (c + 8 * i), a.D, vec, kv + 4 * i);
#pragma unroll
          for (int i = 0; i < NC; ++i)
            load4<T>(vc + at[u], 4 * (c + 8 * i), a.D, vec, vv[u] + 4 * i);
        }
#pragma unroll
        for (int g = 0; g < GH; ++g) {
          s[u][g] = 0.f;
#pragma unroll
          for (int i = 0; i < NC * 4; ++i) s[u][g] = fmaf(q[g][i], kv[i], s[u][g]);
        }
      }
      find(j0 + 16 * KU);
#pragma unroll
      for (int x = 4; x > 0; x >>= 1)
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
          for (int g = 0; g < GH; ++g) s[u][g] += __shfl_xor_sync(~0u, s[u][g], x);
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        float top = m[g];
#pragma unroll
        for (int u = 0; u < KU; ++u) top = fmaxf(top, at[u] == -2 ? -INFINITY : s[u][g]);
        if (top > m[g]) {
          const float f = exp2f(m[g] - top);     // 0 from -inf
          m[g] = top;
          l[g] *= f;
#pragma unroll
          for (int i = 0; i < NC * 4; ++i) o[g][i] *= f;
        }
        const float base = m[g] == -INFINITY ? 0.f : m[g];
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          // A bad page poisons the item.
          const float w = at[u] == -2 ? 0.f : at[u] == -1 ? NAN : exp2f(s[u][g] - base);
          l[g] += w;
#pragma unroll
          for (int i = 0; i < NC * 4; ++i) o[g][i] = fmaf(w, vv[u][i], o[g][i]);
        }
      }
    }
    __syncwarp();
    // Octets, then warps.
#pragma unroll
    for (int g = 0; g < GH; ++g) {
      float mm = m[g];
#pragma unroll
      for (int x = 8; x < 32; x <<= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, x));
      const float f = m[g] == -INFINITY ? (l[g] == 0.f ? 0.f : 1.f) : exp2f(m[g] - mm);
      l[g] *= f;
#pragma unroll
      for (int x = 8; x < 32; x <<= 1) l[g] += __shfl_xor_sync(~0u, l[g], x);
#pragma unroll
      for (int i = 0; i < NC * 4; ++i) {
        o[g][i] *= f;
#pragma unroll
        for (int x = 8; x < 32; x <<= 1) o[g][i] += __shfl_xor_sync(~0u, o[g][i], x);
        if (oct == 0) so[warp][g][4 * (c + 8 * (i >> 2)) + (i & 3)] = o[g][i];
      }
      if (lane == 0) {
        sml[warp][g][0] = mm;
        sml[warp][g][1] = l[g];
      }
    }
    __syncthreads();
    const bool done = p.tile == 0 && t1 == tiles;
    const size_t slot = (size_t)blockIdx.x * 2 + (p.tile == 0 ? 1 : 0);
    for (int e = threadIdx.x; e < heads * a.D; e += WARPS * 32) {
      const int g = e / a.D, d = e - g * a.D;
      float mm = -INFINITY, ll = 0.f, oo = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, sml[w][g][0]);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = sml[w][g][0] == -INFINITY ? 1.f : exp2f(sml[w][g][0] - mm);
        ll += f * sml[w][g][1];
        oo += f * so[w][g][d];
      }
      if (done) {
        finish(a, p.b, hq0 + g, d, mm, ll, oo);
      } else {
        a.part_o[(slot * GMAX + g) * a.D + d] = oo;
        if (d == 0) {
          a.part_ml[(slot * GMAX + g) * 2] = mm;
          a.part_ml[(slot * GMAX + g) * 2 + 1] = ll;
        }
      }
    }
    __syncthreads();
    left -= t1 - p.tile;
    if (left > 0) next_item(a, p);
  }
}

// ------------------------------------------------------------ rings of gathered rows
// A warp takes KEYS keys of a tile at a time (SUB such steps, so that NW warps cover the
// tile) and needs nobody else for them: it copies its own K and V rows (16-byte pieces,
// gathered by page) into its own ring of ST slots, and keeps a running maximum and sums of
// its own; the warps meet once per item, each leaving its sums in the slot it has just used
// up. The pieces of a row are swizzled by the row's number in rows of a multiple of 128
// bytes, so that neither the reads conflict nor the copies split (rows padded to an odd
// number of pieces cost 1.5 times the L2 reads). A Core is the arithmetic on a slot.

// bf16 on the tensor cores. The 16 rows of an m16n8k16 product are the query heads that
// share a kv head: S = Q K^T, the softmax in registers, O += P V. The work is bound by the
// bytes of the cache, not by the products (a few % of the tensor rate at 8 heads), so what
// matters is that a row passes through shared memory once and that 100 KB or more of copies
// are under way per SM.
template <int D>
struct MmaCore {
  typedef bf16 T;
  static constexpr int DIM = D, NW = 4, KEYS = 16, SUB = 1, ST = 3, HEADS = GMAX, KS = D / 16;
  static constexpr int C = D / 8, RS = (C + 7) / 8 * 128, SLOT = 2 * KEYS * RS;
  static constexpr int OCC = D <= 64 ? 4 : D <= 128 ? 2 : 1;
  static constexpr int QS = 0;                   // floats of shared memory for q
  static constexpr int OS = RS / 2;              // floats per row of a warp's sums,
  static_assert(16 * OS * 4 == SLOT, "which fill its slot");
  __device__ static int piece(int r, int ch) { return (ch ^ (r & 7)) << 4; }
  // Where channel d of head g of the sums lies (swizzled likewise).
  __device__ static int sum_at(int g, int d) { return g * OS + (d ^ ((g & 7) << 3)); }

  uint32_t q[KS][4];
  float o[D / 8][4], m[2], l[2];

  __device__ __forceinline__ void begin(const AttnArgs& a, int b, int hq0, int heads, float*) {
    const int lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const bf16* qp = static_cast<const bf16*>(a.q) + b * a.qb + (hq0 + row) * a.qh + 2 * quad;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int h = 0; h < 4; ++h)                // rows row, row + 8; channels +0, +8
        q[k][h] = row + 8 * (h & 1) < heads
                      ? *reinterpret_cast<const uint32_t*>(qp + 8 * (h & 1) * a.qh + 16 * k +
                                                           8 * (h >> 1))
                      : 0u;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int h = 0; h < 4; ++h) o[i][h] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  __device__ __forceinline__ void step(const AttnArgs& a, char* slot, int live, bool bad,
                                       const float*, float*) {
    const int lane = threadIdx.x & 31, quad = lane & 3;
    const uint32_t kd = ptx::smem_u32(slot), vd = kd + KEYS * RS;
    // Row and first piece (swizzled, as a byte offset) of this lane's matrix rows in K and V.
    const int krow = ((lane & 7) + (lane >> 4) * 8) * RS;
    const int vrow = ((lane & 7) + ((lane >> 3) & 1) * 8) * RS;
    const int kpc = (((lane >> 3) & 1) ^ (lane & 7)) << 4, vpc = ((lane >> 4) ^ (lane & 7)) << 4;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 4; ++h) s[n][h] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t f[4];
      ptx::ldsm_x4(f, kd + krow + (kpc ^ (32 * k)));
      ptx::mma_bf16_16816(s[0], q[k], f[0], f[1]);
      ptx::mma_bf16_16816(s[1], q[k], f[2], f[3]);
    }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        s[n][h] *= a.scale2;
        if (n * 8 + 2 * quad + (h & 1) >= live) s[n][h] = -INFINITY;
        top[h >> 1] = fmaxf(top[h >> 1], s[n][h]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
    }
    if (__any_sync(~0u, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = top[r] > m[r] ? exp2f(m[r] - top[r]) : 1.f;    // 0 from -inf
        m[r] = top[r];
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * r] *= f;
          o[i][2 * r + 1] *= f;
        }
      }
    }
    const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        s[n][h] = exp2f(s[n][h] - base[h >> 1]);
        l[h >> 1] += s[n][h];                    // unrounded; the lanes' sums meet at the end
      }
    if (bad) l[0] = l[1] = NAN;
    // A weight goes into the product with V as two bf16: its upper bits as they are, then what
    // they leave over, rounded; 2^-15 of it is lost at most (one bf16 alone would put as much
    // error into a bf16 result as rounding that does). Neither part is negative, and the second
    // is never 0 beside a first that is not, so that an infinite v gives what w v gives. One pass
    // over V per part (16 x 8000 keys, HK = 8, G = 4: D = 192 146 us, D = 256 198; both parts in
    // one pass, where products of one sum follow each other, 174 and 209; one bf16 158 and 188).
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* w = &s[i >> 1][2 * (i & 1)];
      float rest[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        rest[e] = fmaxf(w[e] - __uint_as_float(__float_as_uint(w[e]) & 0xffff0000u),
                        fminf(w[e], 0x1p-126f));
      hi[i] = __byte_perm(__float_as_uint(w[0]), __float_as_uint(w[1]), 0x7632);
      lo[i] = pack2(rest[0], rest[1]);
    }
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t f[4];
        ptx::ldsm_x4_t(f, vd + vrow + (vpc ^ (32 * i)));
        ptx::mma_bf16_16816(o[2 * i], part ? lo : hi, f[0], f[1]);
        ptx::mma_bf16_16816(o[2 * i + 1], part ? lo : hi, f[2], f[3]);
      }
  }

  // The warp's sums into its slot, maxima and weights into sml[head][2].
  __device__ __forceinline__ void leave(float* so, float (*sml)[2]) {
    const int lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      if (quad == 0) {
        sml[row + 8 * r][0] = m[r];
        sml[row + 8 * r][1] = l[r];
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(so + sum_at(row + 8 * r, 8 * i + 2 * quad)) =
            make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
  }
};

// fp32 throughout, for GH query heads of a kv head. Eight keys a step: four lanes per key
// take a quarter of its channels for the scores of all heads (q from shared memory), then
// each of the four goes on with every fourth head's softmax; the weights pass through shared
// memory and a lane sums the channels 4 lane .. + 3 (and + 128) of V for all heads.
template <int D, int GH_>
struct F32Core {
  typedef float T;
  static constexpr int DIM = D, GH = GH_, HEADS = GH_, KEYS = 8, NW = D <= 128 ? 8 : 4;
  static constexpr int SUB = TILE / (NW * KEYS), ST = 3, OCC = D <= 64 ? 2 : 1;
  static constexpr int C = D / 4, RS = (C + 7) / 8 * 128, SLOT = 2 * KEYS * RS;
  static constexpr int QS = GH * D;              // q of the item
  static constexpr int NH = GH < 4 ? 1 : GH / 4; // heads of a lane's softmax
  static constexpr int NV = (D + 127) / 128;     // runs of four channels of a lane
  static_assert(GH * D * 4 <= SLOT, "a slot holds a warp's sums");
  __device__ static int piece(int r, int ch) { return (ch ^ ((r & 1) << 2)) << 4; }
  __device__ static int sum_at(int g, int d) { return g * D + d; }

  float4 o[GH][NV];
  float m[NH], l[NH];                            // of heads (lane & 3) + 4 i

  __device__ __forceinline__ void begin(const AttnArgs& a, int b, int hq0, int heads, float* sq) {
    for (int e = threadIdx.x; e < GH * D; e += NW * 32) {
      const int g = e / D;
      float v = 0.f;
      if (g < heads) {
        const int64_t at = b * a.qb + (hq0 + g) * a.qh + (e - g * D);
        v = a.scale2 * (a.q_bf16 ? __bfloat162float(static_cast<const bf16*>(a.q)[at])
                                 : static_cast<const float*>(a.q)[at]);
      }
      sq[e] = v;
    }
#pragma unroll
    for (int g = 0; g < GH; ++g)
#pragma unroll
      for (int i = 0; i < NV; ++i) o[g][i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NH; ++i) m[i] = -INFINITY, l[i] = 0.f;
  }

  // sw: [KEYS + 1][GH] floats of this warp: the weights of a step, and factors for o.
  __device__ __forceinline__ void step(const AttnArgs& a, char* slot, int live, bool bad,
                                       const float* sq, float* sw) {
    const int lane = threadIdx.x & 31, key = lane >> 2, part = lane & 3;
    float2 acc[GH];
#pragma unroll
    for (int g = 0; g < GH; ++g) acc[g] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < C / 4; ++i) {
      const int ch = 4 * i + part;
      const float4 k = *reinterpret_cast<const float4*>(slot + key * RS + piece(key, ch));
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const float4 q = *reinterpret_cast<const float4*>(sq + g * D + 4 * ch);
        acc[g] = fma2(make_float2(k.x, k.y), make_float2(q.x, q.y), acc[g]);
        acc[g] = fma2(make_float2(k.z, k.w), make_float2(q.z, q.w), acc[g]);
      }
    }
    float s[GH];
#pragma unroll
    for (int g = 0; g < GH; ++g) {
      s[g] = acc[g].x + acc[g].y;
      s[g] += __shfl_xor_sync(~0u, s[g], 1);
      s[g] += __shfl_xor_sync(~0u, s[g], 2);
    }
    bool moved = false;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      float v = s[4 * i];                        // this lane's head, part + 4 i
#pragma unroll
      for (int g = 1; g < 4; ++g)
        if (4 * i + g < GH && part == g) v = s[4 * i + g];
      if (key >= live) v = -INFINITY;
      float top = fmaxf(m[i], v);
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
      const float f = top > m[i] ? exp2f(m[i] - top) : 1.f;            // 0 from -inf
      moved = moved || top > m[i];
      m[i] = top;
      const float w = exp2f(v - (top == -INFINITY ? 0.f : top));
      l[i] = fmaf(l[i], f, w);                   // of this key's lanes; they meet at the end
      if (bad) l[i] = NAN;
      if (part + 4 * i < GH) {
        sw[key * GH + part + 4 * i] = w;
        if (key == 0) sw[KEYS * GH + part + 4 * i] = f;
      }
    }
    moved = __any_sync(~0u, moved);
    __syncwarp();
    if (moved) {
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const float f = sw[KEYS * GH + g];
#pragma unroll
        for (int i = 0; i < NV; ++i)
          o[g][i] = make_float4(o[g][i].x * f, o[g][i].y * f, o[g][i].z * f, o[g][i].w * f);
      }
    }
    const char* vs = slot + KEYS * RS;
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      float4 v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        v[i] = lane + 32 * i < C
                   ? *reinterpret_cast<const float4*>(vs + k * RS + piece(k, lane + 32 * i))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const float w = sw[k * GH + g];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float2* oo = reinterpret_cast<float2*>(&o[g][i]);
          oo[0] = fma2(make_float2(w, w), make_float2(v[i].x, v[i].y), oo[0]);
          oo[1] = fma2(make_float2(w, w), make_float2(v[i].z, v[i].w), oo[1]);
        }
      }
    }
    __syncwarp();                                // sw is written again by the next step
  }

  __device__ __forceinline__ void leave(float* so, float (*sml)[2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(~0u, l[i], x);
      if (lane < 4 && lane + 4 * i < GH) {
        sml[lane + 4 * i][0] = m[i];
        sml[lane + 4 * i][1] = l[i];
      }
    }
#pragma unroll
    for (int g = 0; g < GH; ++g)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane + 32 * i < C)
          *reinterpret_cast<float4*>(so + sum_at(g, 4 * lane + 128 * i)) = o[g][i];
  }
};

template <class Core>
__global__ void __launch_bounds__(Core::NW * 32, Core::OCC) paged_ring_kernel(AttnArgs a) {
  typedef typename Core::T T;
  constexpr int D = Core::DIM, NW = Core::NW, ST = Core::ST, C = Core::C, RS = Core::RS;
  constexpr int KEYS = Core::KEYS, SUB = Core::SUB, SLOT = Core::SLOT, PER = 16 / sizeof(T);
  static_assert(NW * KEYS * SUB == TILE && KEYS * C % 32 == 0, "");
  extern __shared__ __align__(128) char ring[];
  __shared__ float sml[NW][Core::HEADS][2];
  __shared__ int sbad[NW][ST];
  __shared__ __align__(16) float sq[Core::QS ? Core::QS : 1];
  __shared__ float sw[NW][Core::QS ? (KEYS + 1) * Core::HEADS : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  begin_behind();
  empty_rows(a);
  Place pc;                                      // the tile being computed
  long long left = stretch(a, lane, &pc);
  if (left <= 0) return;
  Place pi = pc;                                 // the tile being copied
  long long to_copy = left;
  int sub_copy = 0;
  char* slots = ring + warp * ST * SLOT;
  const T* kc = static_cast<const T*>(a.kc);
  const T* vc = static_cast<const T*>(a.vc);

  // Where this lane's key of the step at pi starts (-1: bad page, -2: no such key).
  auto find = [&]() -> int64_t {
    const int j = pi.s.lo + pi.tile * TILE + (sub_copy * NW + warp) * KEYS + (lane & (KEYS - 1));
    if (j >= pi.s.n) return -2;
    const int64_t r = key_row(a, pi.b, j);
    return r < 0 ? -1 : r + (pi.item / a.groups) * a.ph;
  };
  int64_t off = find();
  auto copy = [&](int slot) {
    if (to_copy > 0) {
      const unsigned bad = __ballot_sync(~0u, off == -1);
      if (lane == 0) sbad[warp][slot] = bad != 0;
      const uint32_t kd = ptx::smem_u32(slots + slot * SLOT), vd = kd + KEYS * RS;
#pragma unroll
      for (int i = 0; i < KEYS * C / 32; ++i) {
        const int e = lane + 32 * i, r = e / C, ch = e - r * C;
        const int64_t o = __shfl_sync(~0u, off, r);
        const int64_t at = o < 0 ? 0 : o + ch * PER;
        const uint32_t to = r * RS + Core::piece(r, ch);
        ptx::cp_async16(kd + to, kc + at, o < 0 ? 0 : 16);
        ptx::cp_async16(vd + to, vc + at, o < 0 ? 0 : 16);
      }
      if (++sub_copy == SUB) {
        sub_copy = 0;
        if (--to_copy > 0 && ++pi.tile == pi.s.tiles()) next_item(a, pi);
      }
      if (to_copy > 0) off = find();             // the next step's rows, looked up meanwhile
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) copy(i);

  Core core;
  int hq0 = 0, heads = 0, tile0 = 0, sub = 0;
  auto begin = [&]() {
    const int hk = pc.item / a.groups, g0 = (pc.item - hk * a.groups) * Core::HEADS;
    hq0 = hk * a.G + g0;
    heads = min(Core::HEADS, a.G - g0);
    tile0 = pc.tile;
    core.begin(a, pc.b, hq0, heads, sq);
  };
  begin();
  if (Core::QS) __syncthreads();

  for (int slot = 0;; slot = slot + 1 == ST ? 0 : slot + 1) {
    ptx::cp_async_wait<ST - 1>();
    __syncwarp();
    const int live = pc.s.n - (pc.s.lo + pc.tile * TILE + (sub * NW + warp) * KEYS);
    if (live > 0) core.step(a, slots + slot * SLOT, live, sbad[warp][slot] != 0, sq, sw[warp]);
    const int tiles = pc.s.tiles();
    if (++sub < SUB) {
      __syncwarp();
      copy(slot);
      continue;
    }
    sub = 0;
    --left;
    if (pc.tile + 1 == tiles || left == 0) {     // the item's end, or this block's
      __syncwarp();                              // the slot's last readers are done
      core.leave(reinterpret_cast<float*>(slots + slot * SLOT), sml[warp]);
      __syncthreads();
      const bool done = tile0 == 0 && pc.tile + 1 == tiles;
      const size_t part = (size_t)blockIdx.x * 2 + (tile0 == 0 ? 1 : 0);
      for (int e = threadIdx.x; e < heads * (D / 4); e += NW * 32) {   // four channels each
        const int g = e / (D / 4), d = 4 * (e - g * (D / 4));
        float mm = -INFINITY, ll = 0.f;
        float2 oo[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, sml[w][g][0]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = sml[w][g][0] == -INFINITY ? 1.f : exp2f(sml[w][g][0] - mm);
          const float4 v = *reinterpret_cast<const float4*>(
              ring + (w * ST + slot) * SLOT + 4 * Core::sum_at(g, d));
          ll = fmaf(f, sml[w][g][1], ll);
          oo[0] = fma2(make_float2(f, f), make_float2(v.x, v.y), oo[0]);
          oo[1] = fma2(make_float2(f, f), make_float2(v.z, v.w), oo[1]);
        }
        if (done) {
          const size_t at = ((size_t)pc.b * a.HQ + hq0 + g) * D + d;
          const float r = ll == 0.f ? 0.f : 1.f / ll;    // no weight: zeros
          oo[0] = ll == 0.f ? make_float2(0.f, 0.f) : mul2(oo[0], make_float2(r, r));
          oo[1] = ll == 0.f ? make_float2(0.f, 0.f) : mul2(oo[1], make_float2(r, r));
          if (a.out_bf16)
            store_pairs(static_cast<bf16*>(a.out) + at, oo);
          else
            store_pairs(static_cast<float*>(a.out) + at, oo);
          if (d == 0) finish_lse(a, pc.b, hq0 + g, mm, ll);
        } else {
          store_pairs(a.part_o + (part * GMAX + g) * D + d, oo);
          if (d == 0) {
            a.part_ml[(part * GMAX + g) * 2] = mm;
            a.part_ml[(part * GMAX + g) * 2 + 1] = ll;
          }
        }
      }
      if (left > 0) {
        next_item(a, pc);
        begin();
      }
      __syncthreads();
      if (left == 0) break;
    } else {
      ++pc.tile;
    }
    __syncwarp();
    copy(slot);
  }
}

// ------------------------------------------------------------ items cut by block boundaries
// Launched behind the kernel above and waits for it before it reads the lengths, too: they may come
// from the kernel before that one. (64 sequences of 0 .. 8192 keys: 104-106 us a call; 97-101 were
// measured with the items looked up ahead of the wait, on other draws of the lengths.) Block (x, y):
// heads y hb and on of item x, or, with more items than blocks, of the item that the boundary after
// stretch x is the first to cut. The JW warps share a head's parts (hb < JW) or take every JW-th
// head; a lane has V channels in a row at a time.
constexpr int JW = 4;
template <int V>
__global__ void __launch_bounds__(JW * 32) paged_join_kernel(AttnArgs a) {
  constexpr int N = 256 / (32 * V);              // runs of V channels of a lane
  __shared__ float red[JW][256], sum[JW];
  begin_behind();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_b = a.HK * a.groups;
  const long long total = total_tiles(a, lane), per = (total + a.blocks - 1) / a.blocks;
  Place p = {};
  long long first = 0;
  bool mine = total > 0;
  if (a.by_item) {
    p.b = blockIdx.x / per_b;
    p.item = blockIdx.x - p.b * per_b;
    p.s = span_of(a, p.b);
    long long before = 0;
    for (int b = lane; b < p.b; b += 32) before += span_of(a, b).tiles();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(~0u, before, o);
    first = before * per_b + (long long)p.item * p.s.tiles();
    mine = mine && p.s.tiles() > 0;
  } else {
    const long long at = (blockIdx.x + 1) * per;
    mine = mine && at < total;
    if (mine) {
      p = locate(a, at, lane);
      first = at - p.tile;
      mine = p.tile > 0 && first / per == blockIdx.x;
    }
  }
  const long long c0 = mine ? first / per : 0;
  const int parts = mine ? (int)((first + p.s.tiles() - 1) / per - c0) + 1 : 0;
  const int hk = p.item / a.groups, g0 = (p.item - hk * a.groups) * a.GH;
  const int heads = min(a.GH, a.G - g0), h0 = blockIdx.y * a.hb, h1 = min(heads, h0 + a.hb);
  if (parts < 2) return;
  const int share = a.hb < JW ? JW / a.hb : 1;             // warps per head
  const int w0 = warp % share;
  for (int g = h0 + warp / share; g < h1; g += JW / share) {
    auto slot = [&](int c) { return ((size_t)(c0 + c) * 2 + (c == 0)) * GMAX + g; };
    auto ml_of = [&](int c) { return *reinterpret_cast<const float2*>(a.part_ml + slot(c) * 2); };
    float m = -INFINITY, l = 0.f, o[N][V];
    for (int c = lane; c < parts; c += 32) m = fmaxf(m, ml_of(c).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) o[i][v] = 0.f;
#pragma unroll 8
    for (int c = w0; c < parts; c += share) {
      const size_t s = slot(c);
      const float2 ml = ml_of(c);
      const float f = ml.x == -INFINITY ? 1.f : exp2f(ml.x - m);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int ch = (lane + 32 * i) * V;
        if (ch < a.D) {
          float v[V];
          load_f<float, V>(a.part_o + s * a.D + ch, v);
#pragma unroll
          for (int k = 0; k < V; ++k) o[i][k] = fmaf(f, v[k], o[i][k]);
        }
      }
    }
    const int hq = hk * a.G + g0 + g;
    if (share == 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int ch = (lane + 32 * i) * V + v;
          if (ch < a.D) finish(a, p.b, hq, ch, m, l, o[i][v]);
        }
    } else {                                     // once: hb < JW heads a block
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) red[warp][(lane + 32 * i) * V + v] = o[i][v];
      if (lane == 0) sum[warp] = l;
      __threadfence_block();
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / share), "r"(share * 32) : "memory");
      l = 0.f;
      for (int w = warp - w0; w < warp - w0 + share; ++w) l += sum[w];
      for (int d = w0 * 32 + lane; d < a.D; d += share * 32) {
        float v = 0.f;
        for (int w = warp - w0; w < warp - w0 + share; ++w) v += red[w][d];
        finish(a, p.b, hq, d, m, l, v);
      }
    }
  }
}

// ------------------------------------------------------------ host
constexpr int kSms = 152;
constexpr long long kMaxKeys = (1LL << 31) - 1024;   // tile ends stay within an int
constexpr int kWholeTiles = 8;    // capacity up to which one block takes a whole item

enum Kind { kAny, kMma, kF32 };                  // which kernel

struct Plan {
  Kind kind;
  int GH, groups, whole, blocks, by_item, joins, hb;
  size_t o_bytes, ml_bytes;
};

// Whether sizes, types and strides allow a ring kernel (16-byte pieces of every cache row;
// their bases are 16-byte aligned by contract): on the tensor cores for bf16 q and caches,
// in fp32 for fp32 caches.
Kind kind_of(const gdr_attn_dims* d, const gdr_paged_cache* c) {
  const int D = c->D, run = c->dtype == GDR_BF16 ? 8 : 4;
  if (D != 64 && D != 80 && D != 96 && D != 128 && D != 192 && D != 256) return kAny;
  if (c->page_stride % run != 0 || c->token_stride % run != 0 || c->head_stride % run != 0)
    return kAny;
  if (c->dtype == GDR_F32) return kF32;
  return d->q_dtype == GDR_BF16 && (d->q_stride_b % 2 == 0 || d->B == 1) &&
                 (d->q_stride_h % 2 == 0 || d->HQ == 1)
             ? kMma
             : kAny;
}

// f(null pointer of the Core) for a ring kernel of head dimension D.
template <typename F>
auto with_core(Kind kind, int D, int G, F f) {
  auto pick = [&](auto dim) {
    constexpr int N = decltype(dim)::value;
    if (kind == kMma) return f(static_cast<MmaCore<N>*>(nullptr));
    return G <= 2   ? f(static_cast<F32Core<N, 2>*>(nullptr))
           : G <= 4 ? f(static_cast<F32Core<N, 4>*>(nullptr))
                    : f(static_cast<F32Core<N, 8>*>(nullptr));
  };
  return D == 64    ? pick(std::integral_constant<int, 64>())
         : D == 80  ? pick(std::integral_constant<int, 80>())
         : D == 96  ? pick(std::integral_constant<int, 96>())
         : D == 128 ? pick(std::integral_constant<int, 128>())
         : D == 192 ? pick(std::integral_constant<int, 192>())
                    : pick(std::integral_constant<int, 256>());
}

Plan make_plan(const gdr_attn_dims* d, const gdr_paged_cache* c, Kind kind) {
  Plan p;
  const int G = d->HQ / c->HK;
  p.kind = kind;
  int resident = 2;                              // blocks per SM
  p.GH = c->D <= 128 ? 4 : 2;
  if (kind != kAny)
    with_core(kind, c->D, G, [&](auto* core) {
      using Core = std::remove_pointer_t<decltype(core)>;
      p.GH = Core::HEADS;
      resident = Core::OCC;
      return 0;
    });
  p.groups = (G + p.GH - 1) / p.GH;
  long long keys = (long long)c->max_pages * c->page_size;
  if (d->window > 0 && keys > d->window) keys = d->window;
  const long long items = (long long)d->B * c->HK * p.groups;
  p.whole = keys <= kWholeTiles * TILE && items < (1LL << 31);
  p.blocks = p.whole ? (int)items : kSms * resident;
  p.o_bytes = p.whole ? 0 : align_up((size_t)p.blocks * 2 * GMAX * c->D * sizeof(float));
  p.ml_bytes = p.whole ? 0 : align_up((size_t)p.blocks * 2 * GMAX * 2 * sizeof(float));
  // The join's blocks: as few heads each as leave two of them per SM.
  p.by_item = !p.whole && items <= p.blocks;
  p.joins = p.by_item ? (int)items : p.blocks - 1;
  const int heads = G < p.GH ? G : p.GH;
  p.hb = 1;
  while (p.hb < heads && (long long)p.joins * ((heads + p.hb - 1) / p.hb) > 2 * kSms) p.hb *= 2;
  return p;
}

// Never 0, which stands for invalid arguments.
size_t plan_bytes(const Plan& p) { return p.whole ? kAlign : p.o_bytes + p.ml_bytes; }

template <class Core>
gdr_status launch_ring(const AttnArgs& a, cudaStream_t s) {
  constexpr int bytes = Core::NW * Core::ST * Core::SLOT;
  if (!allow_smem<Core>(paged_ring_kernel<Core>, bytes)) return GDR_ERR_CUDA;
  return launch_behind_smem(paged_ring_kernel<Core>, dim3(a.blocks), Core::NW * 32, bytes, s, a);
}

gdr_status check(const gdr_attn_dims* d, const gdr_paged_cache* c) {
  if (!d) return GDR_ERR_INVALID_ARG;
  const gdr_status st = check_cache(c);
  if (st != GDR_OK) return st;
  if (d->B < 0 || d->HQ <= 0 || d->HQ % c->HK != 0 || !is_dtype(d->q_dtype) ||
      !is_dtype(d->out_dtype) || d->window < 0 || d->q_stride_b < 0 || d->q_stride_h < 0 ||
      !(isfinite(d->scale) && d->scale > 0.f))
    return GDR_ERR_INVALID_ARG;
  if (d->HQ > (1 << 20)) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

}  // namespace
}  // namespace ops
}  // namespace gdr

using namespace gdr;
using namespace gdr::ops;

extern "C" {

size_t gdr_paged_decode_attn_workspace_size(const gdr_attn_dims* dims,
                                            const gdr_paged_cache* cache) {
  if (check(dims, cache) != GDR_OK) return 0;
  // q's alignment is not known here: room for either kernel.
  const size_t any = plan_bytes(make_plan(dims, cache, kAny));
  const size_t ring = plan_bytes(make_plan(dims, cache, kind_of(dims, cache)));
  return any > ring ? any : ring;
}

gdr_status gdr_paged_decode_attn(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* page_table, const int32_t* lens, void* out,
                                 float* lse, const gdr_attn_dims* dims,
                                 const gdr_paged_cache* cache, void* workspace,
                                 size_t workspace_bytes, gdr_stream_t stream) {
  const gdr_status st = check(dims, cache);
  if (st != GDR_OK) return st;
  if (!is_aligned(q, dtype_size(dims->q_dtype)) || !is_aligned(k_cache, 16) ||
      !is_aligned(v_cache, 16) || !is_aligned(page_table, 4) || !is_aligned(lens, 4) ||
      !is_aligned(out, 16) || !is_aligned(lse, 16))
    return GDR_ERR_ALIGNMENT;
  if (dims->B == 0) return GDR_OK;
  if (!q || !lens || !out || !has_arrays(cache, k_cache, v_cache, page_table))
    return GDR_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < gdr_paged_decode_attn_workspace_size(dims, cache))
    return GDR_ERR_WORKSPACE;
  if (!is_aligned(workspace, kAlign)) return GDR_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Kind kind = kind_of(dims, cache);
  if (kind == kMma && !is_aligned(q, 4)) kind = kAny;
  const Plan p = make_plan(dims, cache, kind);
  AttnArgs a = {};
  // Copies of rows that are not there read nothing, from the address of row 0 all the same.
  a.kc = k_cache ? k_cache : workspace;
  a.vc = v_cache ? v_cache : workspace;
  a.q = q; a.table = page_table; a.lens = lens;
  a.out = out; a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.o_bytes);
  a.B = dims->B; a.HQ = dims->HQ; a.HK = cache->HK; a.D = cache->D;
  a.G = dims->HQ / cache->HK; a.GH = p.GH; a.groups = p.groups;
  a.page = cache->page_size;
  a.shift = (a.page & (a.page - 1)) == 0 ? __builtin_ctz(a.page) : -1;
  a.num_pages = cache->num_pages; a.max_pages = cache->max_pages;
  a.window = dims->window; a.whole = p.whole; a.blocks = p.blocks;
  a.out_bf16 = dims->out_dtype == GDR_BF16; a.q_bf16 = dims->q_dtype == GDR_BF16;
  a.by_item = p.by_item; a.hb = p.hb;
  a.scale2 = dims->scale * LOG2E;
  a.qb = dims->q_stride_b; a.qh = dims->q_stride_h;
  a.pp = cache->page_stride; a.pt = cache->token_stride; a.ph = cache->head_stride;
  if (a.B == 1) a.qb = 0;                        // never stepped along
  if (a.HQ == 1) a.qh = 0;
  a.cap = (long long)cache->max_pages * cache->page_size;
  if (a.cap > kMaxKeys) a.cap = kMaxKeys;
  gdr_status run = GDR_OK;
  if (p.kind != kAny) {
    run = with_core(p.kind, a.D, a.G, [&](auto* core) {
      return launch_ring<std::remove_pointer_t<decltype(core)>>(a, s);
    });
  } else {
    const int vec = a.D % 4 == 0 && a.pp % 4 == 0 && a.pt % 4 == 0 && a.ph % 4 == 0;
    run = with_dtype(cache->dtype, [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      return launch_behind(a.D <= 64    ? paged_any_kernel<T, 2, 4>
                           : a.D <= 128 ? paged_any_kernel<T, 4, 4>
                                        : paged_any_kernel<T, 8, 2>,
                           dim3(p.blocks), WARPS * 32, s, a, vec);
    });
  }
  if (run != GDR_OK || p.whole) return run;
  // The join may start while the last parts are being written; it waits for them itself.
  const int heads = a.G < p.GH ? a.G : p.GH;
  return launch_behind(a.D % 4 == 0 ? paged_join_kernel<4> : paged_join_kernel<1>,
                       dim3(p.joins, (heads + p.hb - 1) / p.hb), JW * 32, s, a);
}

}  // extern "C"
