// How the keys of a call are split over the device, and what the parts leave for the join.
//
// An item is a sequence, a key-value head and a chunk of up to `rows` query rows (tokens x query
// heads of the group); its keys are tiles of `tile` places.  All items' tiles in a row, sequence
// by sequence, are cut into equal shares, one per block: the lengths are on the device, so every
// block counts the tiles by itself and finds its share.  An item begins with `cost` places in the
// row that stand for its own beginning and end, so that blocks with many short items get fewer
// tiles.  A block walks the items of its share; an item that lies in it whole is written out, a part
// goes to the workspace as (maximum, sum, unnormalised output) per row: a block has at most two
// parts, the rest of an item that begins in an earlier block (slot 0) and the beginning of one that
// goes on in the next (slot 1).  The join kernel looks at each block that cut an item at its end,
// and adds that item's parts in the order of the blocks.
//
// Short tables: a block takes one whole item, no lengths are counted and there is no join; where the
// caller reads the status, a kernel of one block looks through the table for it.
#pragma once

#include "kda_attn.cuh"

namespace kda {
namespace attn {

constexpr int kMinPlaces = 256;  // of a block's share, where there are as many
// A table of up to 512 places (256 where places take long, with float32 queries or more than 16 rows,
// and items are fewer than half the SMs) is short.  Split and joined / a block per item, us on the GPU:
// 8 items of bf16 heads of 128, 4 rows, 64 places 7.3 / 4.9, 256 9.4 / 7.2, 512 10.7 / 9.8, 1024 10.7 / 14.5;
// float32, 256 14.4 / 11.5, 512 15.6 / 18.1, 128 items of 512 23.1 / 18.6; 32 rows over bf16, 8 items of
// 256 16.2 / 12.0, 512 15.8 / 16.6, 128 items of 512 23.1 / 17.1; 256 sequences of 1 to 512 bf16 places and
// 8 heads, cold, 68 / 61.  Many more items than blocks do better in equal shares: 512 sequences of 100 to 300
// places, 8 heads, 4 tokens over bf16 138 / 150, float32 275 / 301.  A table of more entries would take the
// kernel that looks through it too long.
constexpr int kShortPlaces = 512, kShortEntries = 4096;

struct Split {
  unsigned int* status;   // workspace header
  unsigned int* verdict;  // [blocks]: what each block found
  int64_t* cut;           // [blocks]: the item that begins in the block and goes on in the next, or -1
  int64_t* last;          // [blocks]: the block in which that item ends
  float* part;            // [blocks][2][rows (d + 2)]
  int64_t blocks, items;
  int rows, tile, cost, chunks, part_floats;
  int64_t least;  // tiles of a share
  bool one;       // a block per item
};
inline int64_t pad256(int64_t b) { return (b + 255) / 256 * 256; }

inline Split split_of(const AttnArgs& a, int rows, int tile, int cost, int per_sm) {
  Split s{};
  s.rows = rows;
  s.tile = tile;
  s.cost = cost;
  s.least = kMinPlaces / tile;
  s.chunks = (a.T * a.rep + rows - 1) / rows;
  s.items = (int64_t)a.B * a.hk * s.chunks;
  s.blocks = a.sms * per_sm;
  const int64_t cap = (int64_t)a.t.max_pages << a.t.shift;
  const bool quick = a.bf16 && rows <= 16;
  s.one = cap <= (quick || s.items >= a.sms / 2 ? kShortPlaces : kShortPlaces / 2) && s.items <= 5 * s.blocks &&
          (int64_t)a.B * a.t.max_pages <= kShortEntries;
  if (s.one) {
    s.blocks = s.items;
    return s;
  }
  // no more blocks than the table has tiles for
  const int64_t tiles = (cap + tile - 1) / tile + 1 + cost;
  const int64_t most = s.items * ((tiles + s.least - 1) / s.least);
  if (most < s.blocks) s.blocks = most;
  s.part_floats = rows * (a.d + 2);
  return s;
}
inline size_t split_bytes(const Split& s) {
  if (s.one) return kWsHeader;
  return kWsHeader + pad256(4 * s.blocks) + 2 * pad256(8 * s.blocks) +
         pad256(s.blocks * 2 * s.part_floats * (int64_t)sizeof(float));
}
inline void split_place(Split& s, void* ws) {
  char* p = static_cast<char*>(ws);
  s.status = reinterpret_cast<unsigned int*>(p);
  if (s.one) return;
  p += kWsHeader;
  s.verdict = reinterpret_cast<unsigned int*>(p);
  p += pad256(4 * s.blocks);
  s.cut = reinterpret_cast<int64_t*>(p);
  p += pad256(8 * s.blocks);
  s.last = reinterpret_cast<int64_t*>(p);
  p += pad256(8 * s.blocks);
  s.part = reinterpret_cast<float*>(p);
}

// The places of sequence n that any of its tokens sees: [first, hi); lo is first rounded down to a tile.
struct Keys {
  int64_t first, lo, hi;
  int64_t tiles;  // at least 1, so that an empty item has a block that writes its zeros
};
__device__ __forceinline__ Keys keys_of(const AttnArgs& a, int tile, int n) {
  const int64_t cap = (int64_t)a.t.max_pages << a.t.shift, len = a.t.lens[n];
  Keys k;
  k.hi = len < 0 ? 0 : len < cap ? len : cap;
  k.first = 0;
  if (a.window > 0) {
    k.first = len - a.T + 1 - a.window;
    k.first = k.first < 0 ? 0 : k.first > k.hi ? k.hi : k.first;
  }
  k.lo = k.first - k.first % tile;
  k.tiles = (k.hi - k.lo + tile - 1) / tile;
  if (k.tiles < 1) k.tiles = 1;
  return k;
}

// Where a block starts: item (n, j) with j = head and chunk, tile t of it; its tiles.
struct Start {
  int64_t at, end;  // positions [at, end)
  int64_t share;    // of a block
  int64_t before;   // places in the row of one (head, chunk) of the sequences before n
  int n;
};
// All threads of the block take part (NT of them); `scratch` holds 34 values.
template <int NT>
__device__ __forceinline__ bool find_start(const AttnArgs& a, const Split& s, int64_t* scratch, Start& out) {
  const int64_t each = (int64_t)a.hk * s.chunks;
  if (s.one) {
    out.n = blockIdx.x / (unsigned)each;
    out.share = keys_of(a, s.tile, out.n).tiles + s.cost;
    out.at = (blockIdx.x - out.n * each) * out.share;
    out.end = out.at + out.share;
    out.before = 0;
    __syncthreads();
    return true;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + NT - 1) / NT, n0 = min(tid * per, a.B), n1 = min(n0 + per, a.B);
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += keys_of(a, s.tile, n).tiles + s.cost;
  int64_t up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) scratch[warp] = up;
  __syncthreads();
  int64_t total = 0, before = up - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  int64_t share = (total * each + s.blocks - 1) / s.blocks;
  if (share < s.least) share = s.least;
  out.share = share;
  out.at = blockIdx.x * share;
  out.end = min(out.at + share, total * each);
  if (out.at >= out.end) return false;
  if (before * each <= out.at && out.at < (before + mine) * each) {
    int n = n0;
    for (;; ++n) {
      const int64_t t = keys_of(a, s.tile, n).tiles + s.cost;
      if (out.at < (before + t) * each) break;
      before += t;
    }
    scratch[32] = before;
    scratch[33] = n;
  }
  __syncthreads();
  out.before = scratch[32];
  out.n = (int)scratch[33];
  return true;
}

// one part of an item: where it begins in the workspace, [rows] maxima, [rows] sums, [rows][d]
__device__ __forceinline__ float* part_of(const Split& s, int64_t block, int slot) {
  return s.part + (block * 2 + slot) * s.part_floats;
}

cudaError_t launch_attn_join(const AttnArgs& a, const Split& s);
cudaError_t launch_attn_table(const AttnArgs& a, const Split& s);

}  // namespace attn
}  // namespace kda
