// gdr_prefix.cuh -- what the kernels of the attention behind a shared prompt have in common:
// arguments, the line of tiles that the blocks share out, and the rows of queries and keys.
#pragma once

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"

namespace gdr {
namespace ops {

struct PrefixArgs {
  const void *q, *kc, *vc;
  const int32_t* table;           // the shared pages
  float *part_o, *part_ml;        // [items][max_parts][units][rows][D], the same [2]
  float *own_o, *own_lse;         // [B][HQ][D], [B][HQ]: of the sequences' own keys
  void* out;
  float* lse;                     // may be null
  int B, HQ, HK, D, G, M, P;      // G = HQ / HK, M = B G rows per kv head, P shared keys
  int rows, row_tiles, tiles;     // rows of a tile, tiles of M and of P
  int blocks, per, max_parts;     // tiles of a block; blocks of an item at most
  int units;                      // parts that a block leaves per item
  int page, num_pages, out_bf16, q_bf16;
  float scale2;                   // scale log2(e)
  long polls;                     // bound of a wait
  int64_t qb, qh, pp, pt, ph;
};

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Element offset of row m of kv head hk: query head hk G + m % G of sequence m / G.
__device__ __forceinline__ int64_t q_row(const PrefixArgs& a, int hk, int m) {
  const int b = m / a.G;
  return b * a.qb + (int64_t)(hk * a.G + m - b * a.G) * a.qh;
}
// Element offset of shared key j < P (kv head 0), or -1 for a bad page.
__device__ __forceinline__ int64_t prefix_row(const PrefixArgs& a, int j) {
  const int pj = j / a.page;
  const int32_t pg = a.table[pj];
  if (pg < 0 || pg >= a.num_pages) return -1;
  return pg * a.pp + (int64_t)(j - pj * a.page) * a.pt;
}

// A block's stretch of the line: its first item and tile, and its number of tiles.
struct Stretch {
  int item, tile, left;
};
__device__ __forceinline__ Stretch stretch_of(const PrefixArgs& a, int block) {
  const long long total = (long long)a.row_tiles * a.HK * a.tiles, first = (long long)block * a.per;
  Stretch s;
  s.left = (int)max(0LL, min((long long)a.per, total - first));
  s.item = (int)(first / a.tiles);
  s.tile = (int)(first - (long long)s.item * a.tiles);
  return s;
}
// Place of a block's part of an item among all parts (units aside), and the blocks of an item.
__device__ __forceinline__ size_t part_of(const PrefixArgs& a, int item, int block) {
  return (size_t)item * a.max_parts + (block - (int)((long long)item * a.tiles / a.per));
}
__device__ __forceinline__ int parts_of(const PrefixArgs& a, int item) {
  const long long first = (long long)item * a.tiles;
  return (int)((first + a.tiles - 1) / a.per - first / a.per) + 1;
}

}  // namespace ops
}  // namespace gdr
