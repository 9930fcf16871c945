// kv_plan.cuh -- the layout of a cache plan (see ws_kv_plan): what
// k_kv_plan writes on the device and the append and attention kernels read.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ws {

constexpr int kPage = WS_KV_PAGE;
constexpr int kTileRows = 16;  // rows of a tile of the decode kernel
constexpr int kWarpsPerSm = 12;  // of the decode kernel, resident

// Rows are a sequence's (new token, query head of one kv head) pairs, token by
// token.  Everything is per kv head; all kv heads have the same plan.
struct KvHeader {
  int n_append;  // touched pages
  int n_tiles;   // 16-row tiles
  int pages;     // sum of the tiles' pages
  int units;     // equal shares of those pages, one warp each
  int n_split;   // tiles cut by a unit's end
  int pad[11];
};
// All int4 arrays.
//   seq     {tokens before the call, first row of q, new tokens, 0}
//   append  {first row, page (-1: none), first place in it, rows}
//   tile    {sequence, first row, pages of the tiles before it, index among the cut ones or -1},
//           one more at the end with the pages of all
//   split   {tile, first slot, pieces, 0}
// and int  unit   first tile of each unit.
struct KvLayout {
  size_t seq, pre, append, tile, split, unit, bytes;  // byte offsets; pre: prefix sums over sequences
  int64_t max_append, max_tiles, max_units;
};

struct KvShape {
  int64_t T;
  int n_seq, max_pages, max_new, nh, nkv, hd;
};

inline KvLayout kv_layout(const KvShape& s) {
  KvLayout L = {};
  const int64_t live = std::min<int64_t>(s.n_seq, s.T), G = s.nh / s.nkv;
  // n rows touch (n + 62) / 64 + 1 pages at most
  L.max_append = std::min<int64_t>(std::min<int64_t>(s.T, live * (((int64_t)s.max_new + 62) / kPage + 1)),
                                   s.T / kPage + 2 * live);
  L.max_tiles = std::min<int64_t>(s.T * G / kTileRows + live, live * (((int64_t)s.max_new * G + kTileRows - 1) / kTileRows));
  L.max_units = std::max<int64_t>(1, (int64_t)device_sm_count() * kWarpsPerSm / s.nkv);
  size_t o = sizeof(KvHeader);
  auto take = [&](size_t n) {
    const size_t at = o;
    o += (n + 15) / 16 * 16;
    return at;
  };
  L.seq = take((size_t)s.n_seq * 16);
  L.pre = take((size_t)(s.n_seq + 1) * 8);
  L.append = take((size_t)L.max_append * 16);
  L.tile = take((size_t)(L.max_tiles + 1) * 16);
  L.split = take((size_t)L.max_units * 16);
  L.unit = take((size_t)(L.max_units + 1) * 4);
  L.bytes = o;
  return L;
}

// Pages of unit u: [unit_start(u), unit_start(u + 1)) of the W pages of all
// tiles; unit_of is its inverse.
__host__ __device__ inline int unit_start(int u, int W, int U) { return (int)((int64_t)u * W / U); }
__host__ __device__ inline int unit_of(int page, int W, int U) {
  return (int)((((int64_t)page + 1) * U - 1) / W);
}

}  // namespace ws
