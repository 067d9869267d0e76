// weigh_tiles.cuh -- which keys and row tiles a block of weigh.cu's passes takes, in whole
// numbers. Plain C++ too, so that the rule can be tested on the host.
#pragma once

#ifdef __CUDACC__
#define ATTN_TILES_FN __host__ __device__ __forceinline__
#else
#define ATTN_TILES_FN inline
#endif

namespace attn {
namespace weigh_tiles {

constexpr int kRows = 32;   // rows of a row tile: 128 (row, head) pairs
constexpr int kKeys = 128;  // keys of a tile

ATTN_TILES_FN int lesser(int a, int b) { return a < b ? a : b; }

// A sequence's keys cut evenly into `splits` segments of whole tiles: segment s is [k0, k1).
ATTN_TILES_FN void segment(int keys, int splits, int s, int* k0, int* k1) {
  const int len = ((keys + splits - 1) / splits + kKeys - 1) / kKeys * kKeys;
  const long long from = (long long)s * len, to = from + len;
  *k0 = from < keys ? (int)from : keys;
  *k1 = to < keys ? (int)to : keys;
}

// The end of a segment's keys that some row of row tile rt sees, and the tiles that hold them.
ATTN_TILES_FN int visible(int ctx, int rows, int k1, int rt) { return lesser(k1, ctx + lesser(rows, (rt + 1) * kRows)); }
ATTN_TILES_FN int tiles(int ctx, int rows, int k0, int k1, int rt) {
  const int n = visible(ctx, rows, k1, rt) - k0;
  return n > 0 ? (n + kKeys - 1) / kKeys : 0;
}

// The first of the row tiles rt0 .. rt1 - 1 that sees a key of the segment, as all after it do;
// rt1 where none does.
ATTN_TILES_FN int first_seeing(int ctx, int k0, int k1, int rt0, int rt1) {
  if (k0 >= k1) return rt1;
  const int rt = k0 > ctx ? (k0 - ctx) / kRows : 0;
  return rt < rt0 ? rt0 : lesser(rt, rt1);
}

}  // namespace weigh_tiles
}  // namespace attn
