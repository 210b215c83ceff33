// The plan of masked attention: what the kernels know of a batch's documents.
//
// With contiguous documents the keys that a query sees, and the queries that see a key, are one
// interval of tokens each, whatever of the causal, document, prefix and padding masks is in force:
//   query i of document [a, a + len), prefix end pe:  [a, max(i + 1, pe)) causal, else [a, a + len)
//   key j:                                            queries [a or j, a + len): j where causal and j >= pe
// (empty for a token outside every document's valid part).  The plan holds both interval lists, and
// per 128-token tile the range of opposite tiles that any of its rows meets, the part of that range
// in which every row sees every column (no masking there), and the order in which the tiles are
// worked on: the longest first.
#pragma once

#include "common.cuh"

namespace xt {
namespace attn_plan {

constexpr int BT = 128;               // tokens per tile
constexpr int kMagic = 0x58544150;
constexpr int kHeader = 16;           // ints

// First element of each part, in ints from the plan's start (every part 16-byte aligned).
struct Layout {
  int64_t tiles, qrange, krange, pairs, qs, ks, q_iv, k_iv, total;
  __host__ __device__ explicit Layout(int64_t T) {
    tiles = (T + BT - 1) / BT;
    qrange = kHeader;
    krange = qrange + 4 * tiles;
    pairs = krange + 4 * tiles;
    qs = pairs + 12 * ((tiles + 1) / 2);
    ks = qs + 8 * tiles;
    q_iv = ks + 8 * tiles;
    k_iv = q_iv + 2 * BT * tiles;
    total = k_iv + 2 * BT * tiles;
  }
};

// A plan as a kernel reads it.  Ranges are (first, end, full first, full end) of opposite tiles.
struct View {
  const int32_t* base;
  int64_t T;
  int tiles;
  const int4* pairs;         // pairs of query tiles, most work first: (first tile, first key tile, end, 0), two ranges
  const int4 *qs, *ks;       // query tiles and key tiles, most work first: (tile, 0, 0, 0), range
  const int2 *q_iv, *k_iv;   // per token [first, end)
};

inline View view(const void* plan, int64_t T) {
  const Layout l(T);
  const int32_t* b = static_cast<const int32_t*>(plan);
  View v;
  v.base = b;
  v.T = T;
  v.tiles = int(l.tiles);
  v.pairs = reinterpret_cast<const int4*>(b + l.pairs);
  v.qs = reinterpret_cast<const int4*>(b + l.qs);
  v.ks = reinterpret_cast<const int4*>(b + l.ks);
  v.q_iv = reinterpret_cast<const int2*>(b + l.q_iv);
  v.k_iv = reinterpret_cast<const int2*>(b + l.k_iv);
  return v;
}

// The plan was made for these tokens (read after the wait for the preceding kernel).
__device__ __forceinline__ bool valid(const View& v) {
  return v.base[0] == kMagic && v.base[1] == int32_t(v.T);
}

}  // namespace attn_plan
}  // namespace xt
