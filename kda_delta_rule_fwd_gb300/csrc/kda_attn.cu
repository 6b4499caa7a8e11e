// Attention of new tokens over the paged cache: products on the tensor cores.
//
// Bound by the bytes of keys and values: 1 to 64 query rows per key are few operations, so the
// products are warp-level ones (m16n8k16), with the keys as rows and 8 queries as columns, and
// everything else serves a steady stream of loads.  Each of a block's four key groups takes 16 or
// 32 of a tile's places: its warps copy them into a ring of stages of their own (cp.async, 16
// bytes a lane, swizzled by row) and wait for nobody else; a running maximum, sum and output per
// warp are joined when an item ends.  The next items' tiles are requested while the present one
// is worked on.
//
//     S^T = K Q^T:  A = keys as they lie (ldmatrix), B = queries, kept as fragments
//     O^T = V^T P^T: A = values (ldmatrix.trans), B = the weights: S^T's accumulators, packed to
//                    16 bits and transposed 8 x 8 in registers (movmatrix)
//
// Above 16 rows the outputs of all channels no longer leave a warp enough registers for others to
// run beside it (253 of them: two warps to a scheduler, five cycles to an instruction).  There the four
// groups share their weights through shared memory and each adds up a quarter of the channels for all
// places of the tile; the rows' bases are then the block's, three barriers to a tile.
//
// Types.  bf16 caches: products of bf16, exact in float32; a weight enters as two bf16 parts
// (16 bits), since one alone would cost as much as the output's own rounding.  Codes become f16,
// exactly; queries become f16 after a power of two per row has brought their largest to 2^13,
// which keeps every bit down to 2^-27 of it.  A value's power of two joins its weight, and a query
// row's base follows the largest product of the two that it meets, which f16 gets as 2^9 to 2^15:
// products down to 2^-23 of the largest keep all 11 bits, what is below is off by 2^-34 of it at most.  Up to
// 8 rows, where the bytes bind, a second f16 part makes them 22 bits (4 rows over e4m3 195 us with one part or
// two; 16 rows 201 and 215, 32 rows 298 and 365, 64 rows 507 and 668: one part from 9 rows on).
// A row of large power takes nothing from the others where its weight is small or it is not seen.
// (With 2^11 to 2^15 the bases move more often: 32 and 64 rows over int8 330 and 582 us, with 2^9 320 and
// 532, with 2^7 316 and 520.)  The sum of weights is float32 and counts from the same base: its terms fall
// with the largest power (2^-112 for 2^121, the largest that is written).  A base stays within 2^103
// of the largest weight, so that sums of weights of rows of zeros (power 2^-126) stay finite: where all
// that a row sees has powers below 2^-87, they keep fewer bits.
//
// float32 queries over codes are two f16 parts (22 bits), as are their weights; over a float32 cache
// keys, values, queries and weights are three bf16 parts each (all 24 bits), whose six largest products
// leave out 2^-24.
//
// Codes lie four to a 32-bit word, and the products' order of channels is free as long as both
// operands have the same: a word of a key's row is channels 4t .. 4t + 3, used as the two pairs
// of a k-step; ldmatrix.trans on pairs of bytes gives two channels of two places, which one
// byte permutation sorts by channel, so that a thread's outputs are pairs of adjacent channels.
//
// Places that a row does not see: the tiles at the ends of the seen range give them the weight 0,
// and values that are not finite become zeros there once the rows that do see them have got them
// (0 times infinity would reach the others).  Such a value, seen, leaves its channel's sum infinite or NaN,
// whatever the weight's parts; at the item's end those sums are replaced by the sum of the channel's values
// that are not finite (a weight is above 0, though its parts may be 0).
#include <type_traits>

#include "kda_attn_split.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kGroups = 4;    // key groups of a block
// Places that an item's beginning and end take the time of.  256 sequences of up to 8192 e4m3 places, 4
// rows (3.4 us an item, 2 us for 128 places, from the blocks' own times): 368 us with 0, 334 with 256
// and with 512.  16 sequences of up to 32768 int8 places, 32 rows: 153, 150, 148 and 152 us with 192,
// 256, 384 and 640.
constexpr int item_cost(int eights) { return eights == 4 ? 384 : 256; }
// The base of a row's weights follows where a weight, times the power of its value's codes, passes it by this much
template <bool kCoded> constexpr float lazy() { return kCoded ? 6.f : 8.f; }
constexpr float kFill = 9.f, kDeep = 96.f;  // codes: the largest product in f16 as the base is set; the smallest power that counts
constexpr float kNone = -3e38f;           // the base of a row that has seen nothing: every score passes it
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros when `have` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void matrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void matrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool kBf16>
__device__ __forceinline__ void product(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two numbers as N parts of 16 bits each, their sum the number: bf16 or f16 to the nearest, each part of
// what the ones before it left; three bf16 parts are cut off a float32's 24 bits, exactly.
template <bool kBf16, int N, bool kCut = N == 3>
__device__ __forceinline__ void split(float x, float y, uint32_t (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float xh, yh;
    if constexpr (kCut) {
      part[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
      xh = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      yh = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    } else if constexpr (kBf16) {
      part[i] = layer::pack_bf16(x, y);
      layer::unpack2(part[i], xh, yh);
    } else {
      part[i] = pack_half(x, y);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&part[i]));
      xh = f.x;
      yh = f.y;
    }
    if (i + 1 < N) {
      x -= xh;
      y -= yh;
    }
  }
}
// a value's byte as the exponent that a base allows for: its power, less what f16 holds of the product
__device__ __forceinline__ float ask(int byte) { return fmaxf((float)(byte - 127) - kFill, -kDeep); }
// two codes as f16
__device__ __forceinline__ uint32_t open2(uint16_t two) {
  uint32_t f;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(two));
  return f;
}
// four codes as two pairs of f16
template <int CACHE>
__device__ __forceinline__ void open4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CACHE == KDA_CACHE_E4M3) {
    lo = open2((uint16_t)w);
    hi = open2((uint16_t)(w >> 16));
  } else {  // 1024 + 128 + code in f16's mantissa, less 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}
// whether a 32-bit word of values (a float32, two bf16 or four e4m3 codes) holds one that is not finite
template <int CACHE>
__device__ __forceinline__ bool wild(uint32_t w) {
  if constexpr (CACHE == KDA_CACHE_BF16) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  else if constexpr (CACHE == KDA_CACHE_F32) return (w & 0x7f800000u) == 0x7f800000u;
  else if constexpr (CACHE == KDA_CACHE_E4M3) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
  else return false;
}
template <int CACHE>
__device__ __forceinline__ uint32_t tamed(uint32_t w) {  // such values as zeros
  if constexpr (CACHE == KDA_CACHE_BF16) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
  } else if constexpr (CACHE == KDA_CACHE_F32) {
    return wild<CACHE>(w) ? 0u : w;
  } else {
    return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
}
__device__ __forceinline__ uint32_t transposed(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

// A channel of a row whose sum came out infinite or NaN: the sum of the values [from, to) of sequence n that
// are not finite, 0 where all are.
template <typename TC, int D>
__device__ __noinline__ float sum_of_wild(const AttnArgs& a, int n, int head, int ch, int from, int to) {
  float sum = 0.f;
  for (int p = from; p < to && sum == sum; ++p) {
    const int id = page_of(a.t, n, p);
    if (id < 0) continue;
    const int64_t row = ((int64_t)head << a.t.shift) + (p & ((1 << a.t.shift) - 1));
    const float x = to_f32(static_cast<const TC*>(a.vc)[id * a.ldpage + row * D + ch]);
    if (!isfinite(x)) sum += x;
  }
  return sum;
}

// Places of tiles in the block's share, item by item.
struct Cursor {
  int64_t left;     // of the share from here on
  int n, head, chunk;
  int t, tiles;     // tile of the item, the item's number
  int first, hi;    // the sequence's places that a token sees
  __device__ __forceinline__ void enter(const AttnArgs& a, const Split& s) {
    const Keys k = keys_of(a, s.tile, n);
    first = (int)k.first;
    hi = (int)k.hi;
    tiles = (int)k.tiles;
  }
  // where its tiles begin
  template <int TILE> __device__ __forceinline__ int lo() const { return first & ~(TILE - 1); }
  // past `by` tiles of the item
  __device__ __forceinline__ void pass(const AttnArgs& a, const Split& s, int by) {
    left -= by;
    t += by;
    if (t < tiles) return;
    t = 0;
    left -= s.cost;
    if (++chunk < s.chunks) return;
    chunk = 0;
    if (++head < a.hk) return;
    head = 0;
    ++n;
    if (left > 0) enter(a, s);
  }
};

// FQ: float32 queries; NT: query rows of a warp in eights; WM: warps with rows of their own; KT: places
// of a key group in a tile; PER: blocks to an SM; SHARE: the groups share their weights
template <bool FQ, int CACHE, int D, int NT, int WM, int KT, int PER, bool SHARE = false>
struct Shape {
  static constexpr bool kCoded = CACHE == KDA_CACHE_E4M3 || CACHE == KDA_CACHE_INT8, kF32 = CACHE == KDA_CACHE_F32;
  // 16-bit parts of a key or value, of a query, of a weight
  static constexpr int kParts = kF32 ? 3 : 1, kQParts = kF32 ? 3 : FQ ? 2 : 1, kWParts = kF32 ? 3 : kCoded && !FQ && NT > 1 ? 1 : 2;
  static constexpr int kThreads = kGroups * WM * 32, kPerSm = PER;
  static constexpr int kRows = 8 * NT * WM, kTile = kGroups * KT, kCost = item_cost(NT) / kTile;
  static constexpr int kElem = kCoded ? 1 : kF32 ? 4 : 2;
  static constexpr int kChunks = D * kElem / 16;           // 16-byte pieces of a row
  static constexpr int kHalf = KT * D * kElem;             // a group's keys (or values) of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kSlice = NT == 1 ? 16 : 32, kPitch = kSlice + 2;  // channels of an item's end that meet at once
  static constexpr int kMerge = kGroups * kRows * kPitch * 4;
  // shared weights: fragments of all groups' weights; bases that the groups ask for
  static constexpr int kWBytes = kGroups * kWParts * NT * 32 * 8, kTops = kGroups * kRows * 4;
  static constexpr int kTail = SHARE ? kWBytes + kTops : 2 * kMerge;
  static constexpr int kQBytes = kRows * D * 2 * kQParts;
  static constexpr int bytes(int stages) {
    return kGroups * stages * (kStage + 2 * KT + 4) + kQBytes + 12 * kRows + kGroups * kRows * 8 + kTail;
  }
  // as many stages as the SM's 228 KB hold for its blocks (each takes 1.5 KB for itself), up to six
  static constexpr int fit() {
    int n = 2;
    while (n < 6 && PER * (bytes(n + 1) + 1536) <= 228 * 1024) ++n;
    return n;
  }
  static constexpr int kStages = fit();
  static_assert(PER * (bytes(kStages) + 1536) <= 228 * 1024, "shared memory");
  static constexpr int oQ = kGroups * kStages * kStage;
  static constexpr int oScale = oQ + kQBytes;
  static constexpr int oSeen = oScale + kGroups * kStages * 2 * KT;
  static constexpr int oRow = oSeen + kGroups * kStages * 4;
  static constexpr int oStats = oRow + 12 * kRows;
  static constexpr int oMerge = oStats + kGroups * kRows * 8;
  static constexpr int kBytes = bytes(kStages);
  static_assert(oMerge % 16 == 0 && oMerge + kTail == kBytes, "layout");
};
// a row's 16-byte piece c, moved so that 8 rows' pieces c lie in different banks
template <int CHUNKS>
__device__ __forceinline__ int piece(int row, int c) {
  if constexpr (CHUNKS >= 8) return row * CHUNKS + (c ^ (row & 7));
  else return row * CHUNKS + (c ^ ((row >> 1) & 3));
}

// float32 keys are read 16 bytes a lane, 4 pieces of 2 rows at once: adjacent rows in other halves
template <int CHUNKS, bool kF32>
__device__ __forceinline__ int key_piece(int row, int c) {
  if constexpr (kF32) return row * CHUNKS + (c ^ ((row & 1) << 2 | (row >> 1 & 3)));
  else return piece<CHUNKS>(row, c);
}

template <bool FQ, int CACHE, int D, int NT, int WM, int KT, int PER, bool SHARE>
__global__ void __launch_bounds__(Shape<FQ, CACHE, D, NT, WM, KT, PER, SHARE>::kThreads, PER)
attn_mma_kernel(AttnArgs a, Split s, bool words) {
  using S = Shape<FQ, CACHE, D, NT, WM, KT, PER, SHARE>;
  using TQ = std::conditional_t<FQ, float, __nv_bfloat16>;
  constexpr bool kCoded = S::kCoded, kF32 = S::kF32;
  constexpr int AP = S::kParts, QP = S::kQParts, PP = S::kWParts;
  // a thread's outputs are channels 16 i + 2 g + (0, 1), or 16 i + g and 8 behind it
  constexpr bool kNext = kCoded || kF32;
  constexpr int KS = D / 16, KM = KT / 16, CH = S::kChunks;
  constexpr bool kHoldQ = NT * KS * QP <= 8;  // queries stay in registers
  constexpr int OB = SHARE ? D / 16 / kGroups : D / 16;  // blocks of 16 channels that a warp adds up
  static_assert(!SHARE || (!FQ && WM == 1 && KT == 16), "shared weights");
  constexpr unsigned kAll = KT == 32 ? 0xffffffffu : 0xffffu;
  extern __shared__ __align__(128) char raw[];
  __shared__ int64_t scratch[34];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp % kGroups, wm = warp / kGroups;  // key group; which query rows
  const int g = lane >> 2, t4 = lane & 3;
  if (tid == 0) {
    bad = 0;
    if (!s.one) s.cut[blockIdx.x] = -1;
  }
  Start st;
  if (!find_start<S::kThreads>(a, s, scratch, st)) {
    if (tid == 0 && !s.one) s.verdict[blockIdx.x] = KDA_OK;
    return;
  }
  const int mask = (1 << a.t.shift) - 1;
  Cursor now;
  {
    now.n = st.n;
    now.left = st.end - st.at;
    now.enter(a, s);
    const int64_t off = st.at - st.before * (a.hk * s.chunks);
    const int all = now.tiles + s.cost, j = (int)(off / all);
    now.t = (int)(off % all) - s.cost;
    if (now.t < 0) {
      now.left += now.t;
      now.t = 0;
    }
    now.head = j / s.chunks;
    now.chunk = j % s.chunks;
  }
  Cursor ahead = now;
  char* const kv = raw + grp * S::kStages * S::kStage;
  uint8_t* const sc = reinterpret_cast<uint8_t*>(raw + S::oScale) + grp * S::kStages * 2 * KT;
  unsigned* const seen_of = reinterpret_cast<unsigned*>(raw + S::oSeen) + grp * S::kStages;
  float* const row_factor = reinterpret_cast<float*>(raw + S::oRow);
  int* const row_end = reinterpret_cast<int*>(raw + S::oRow) + S::kRows;
  int* const row_place = row_end + S::kRows;  // the row among a sequence's rows of the output
  uint2* const shared_w = reinterpret_cast<uint2*>(raw + S::oMerge);  // [parts][groups][rows / 8][lanes]
  float* const shared_top = reinterpret_cast<float*>(raw + S::oMerge + S::kWBytes);  // [groups][rows]
  uint2* const qs = reinterpret_cast<uint2*>(raw + S::oQ) + wm * NT * KS * 32;  // [parts][rows / 8][steps][lanes]

  // The table's entries of the next request are read one request early.
  int ids[KM];
  auto look = [&]() {
    if (a.t.shift < 4 || ahead.left <= 0) return;
#pragma unroll
    for (int u = 0; u < KM; ++u) {
      const unsigned pos = (unsigned)ahead.template lo<S::kTile>() + (unsigned)ahead.t * S::kTile + grp * KT + u * 16;
      const int64_t col = pos >> a.t.shift;
      ids[u] = pos < (unsigned)ahead.hi && col < a.t.max_pages ? a.t.pages[(int64_t)ahead.n * a.t.max_pages + col] : -1;
    }
  };
  // The group's places of the tile at `ahead` into a stage (its WM warps take a share each).
  auto request = [&](int stage) {
    if (ahead.left > 0) {
      const unsigned pos = (unsigned)ahead.template lo<S::kTile>() + (unsigned)ahead.t * S::kTile + grp * KT;
      const uint32_t dst = smem_at(kv + stage * S::kStage);
      unsigned seen = 0;  // the places that a token sees, on pages of the pool
      if (a.t.shift >= 4) {  // a page holds 16 places in a row
        const char *k[KM], *v[KM];
        int have[KM];
#pragma unroll
        for (int u = 0; u < KM; ++u) {
          const unsigned p = pos + u * 16;
          const bool some = p < (unsigned)ahead.hi;
          const bool ok = some && (unsigned)ids[u] < (unsigned)a.t.num_pages;
          have[u] = ok ? (int)min(16u, (unsigned)ahead.hi - p) : 0;
          if (some && !ok && p + 16 > (unsigned)ahead.first) bad = 1;
          seen |= ((1u << have[u]) - 1) << (u * 16);
          const int64_t row = ((int64_t)ahead.head << a.t.shift) + (p & mask);
          const int64_t from = ok ? (ids[u] * a.ldpage + row * D) * S::kElem : 0;
          k[u] = static_cast<const char*>(a.kc) + from;
          v[u] = static_cast<const char*>(a.vc) + from;
          if (kCoded && wm == 0 && ok && (lane >> 1) == u) {
            const int64_t b = (((int64_t)ids[u] * a.hk) << a.t.shift) + row;
            copy16(smem_at(sc + stage * 2 * KT + (lane & 1) * KT + u * 16), (lane & 1 ? a.vs : a.ks) + b);
          }
        }
        constexpr int kTurns = KT * CH / 32 / WM, kRowsOf = 32 / CH;
        const bool full = seen == kAll;
        if (pos < (unsigned)ahead.first) {  // no token sees these
          const unsigned before = min(ahead.first - pos, 31u);
          seen = seen >> before << before;
        }
        if (full) {
#pragma unroll
          for (int i = 0; i < kTurns; ++i) {
            const int x = (i * WM + wm) * 32 + lane, u = i * WM * kRowsOf / 16;
            const int r = x / CH, c = x % CH, from = (x % (16 * CH)) * 16;
            copy16(dst + key_piece<CH, kF32>(r, c) * 16, k[u] + from);
            copy16(dst + S::kHalf + piece<CH>(r, c) * 16, v[u] + from);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kTurns; ++i) {
            const int x = (i * WM + wm) * 32 + lane, r = x / CH, u = r / 16;
            const bool ok = (r & 15) < (KM == 2 && u ? have[KM - 1] : have[0]);
            const int c = x % CH, from = ok ? (x % (16 * CH)) * 16 : 0;
            copy16(dst + key_piece<CH, kF32>(r, c) * 16, (KM == 2 && u ? k[KM - 1] : k[0]) + from, ok);
            copy16(dst + S::kHalf + piece<CH>(r, c) * 16, (KM == 2 && u ? v[KM - 1] : v[0]) + from, ok);
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < KT * CH / 32 / WM; ++i) {
          const int x = (i * WM + wm) * 32 + lane, r = x / CH, c = x % CH;
          const int id = pos + r < (unsigned)ahead.hi ? page_of(a.t, ahead.n, pos + r) : -1;
          const int64_t row = ((int64_t)ahead.head << a.t.shift) + ((pos + r) & mask);
          const int64_t from = id >= 0 ? (id * a.ldpage + row * D) * S::kElem + c * 16 : 0;
          copy16(dst + key_piece<CH, kF32>(r, c) * 16, static_cast<const char*>(a.kc) + from, id >= 0);
          copy16(dst + S::kHalf + piece<CH>(r, c) * 16, static_cast<const char*>(a.vc) + from, id >= 0);
        }
        const bool some = lane < KT && pos + lane < (unsigned)ahead.hi && pos + lane >= (unsigned)ahead.first;
        const int id = some ? page_of(a.t, ahead.n, pos + lane) : -1;
        if (some && id < 0) bad = 1;
        seen = __ballot_sync(0xffffffffu, id >= 0);
        if (kCoded && wm == 0 && id >= 0) {
          const int64_t b = (((int64_t)id * a.hk + ahead.head) << a.t.shift) + ((pos + lane) & mask);
          sc[stage * 2 * KT + lane] = a.ks[b];
          sc[stage * 2 * KT + KT + lane] = a.vs[b];
        }
      }
      if (wm == 0 && lane == 0) seen_of[stage] = seen;
      ahead.pass(a, s, 1);
      look();
    }
    copy_commit();
  };
  // all that the group's warps wrote of a stage is there, and nobody reads the one before
  auto meet = [&]() {
    if constexpr (SHARE) __syncthreads();
    else if constexpr (WM == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WM) : "memory");
  };

  look();
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) request(i);
  int stage = 0;
  // ldmatrix: the lane's row of 16 places and piece of two, (places, pieces) = 0 0, 1 0, 0 1, 1 1
  // by eights of lanes; bf16 values take 0 0, 0 1, 1 0, 1 1
  const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mcol = lane >> 4;
  const int vrow = kCoded ? mrow : (lane & 7) + (lane >> 4) * 8, vcol = kCoded ? mcol : (lane >> 3) & 1;

  while (now.left > 0) {
    // ---- an item begins: its queries as fragments of B, one row per warp and turn
    const int n = now.n, head = now.head, row0 = now.chunk * S::kRows;
    const int rows = min(S::kRows, a.T * a.rep - row0);
    const int len = max(a.t.lens[n], -8);  // nothing is seen at 0 and below
    const int t0 = now.t, t1 = (int)min((int64_t)now.tiles, now.t + now.left);
    if (tid == 0) {
      if ((int64_t)len > (int64_t)a.t.max_pages << a.t.shift) bad = 1;
      if (t0 == 0 && t1 < now.tiles) {
        s.cut[blockIdx.x] = ((int64_t)n * a.hk + head) * s.chunks + now.chunk;
        s.last[blockIdx.x] = (st.end - now.left + now.tiles - 1) / st.share;
      }
    }
    __syncthreads();
    constexpr int kTurns = S::kRows / (S::kThreads / 32);  // rows of a warp, all loaded before the first is used
    using Pair = std::conditional_t<FQ, float2, __nv_bfloat162>;
    Pair held[kTurns][D / 64];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int r = warp + k * (S::kThreads / 32), row = row0 + r, tok = row / a.rep;
      const TQ* q = static_cast<const TQ*>(a.q) + ((int64_t)n * a.T + tok) * a.ldq +
                    (int64_t)(head * a.rep + row - tok * a.rep) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int p = lane + 32 * i;
        held[k][i].x = held[k][i].y = from_f32<TQ>(0.f);
        if (r < rows) {
          if (words) held[k][i] = reinterpret_cast<const Pair*>(q)[p];
          else { held[k][i].x = q[2 * p]; held[k][i].y = q[2 * p + 1]; }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int r = warp + k * (S::kThreads / 32), tok = (row0 + r) / a.rep;
      const Pair (&x)[D / 64] = held[k];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        most = max(most, max(__float_as_uint(to_f32(x[i].x)) & 0x7fffffffu, __float_as_uint(to_f32(x[i].y)) & 0x7fffffffu));
      // the sign of the scale goes into the query, so that factors are positive; no scale: no query
      float up = a.scale < 0.f ? -1.f : a.scale > 0.f ? 1.f : 0.f, f = fabsf(a.scale) * kLog2e;
      if constexpr (kCoded) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        // 2^13 over the largest's power of two, kept a normal number
        const int e = (int)(most >> 23);
        const int k = e == 0 || e == 255 ? 0 : min(max(127 + 13 - e, -120), 120);
        up *= __uint_as_float((uint32_t)(127 + k) << 23);
        f *= __uint_as_float((uint32_t)(127 - k) << 23);
      }
      if (lane == 0) {
        row_factor[r] = f > 1e-37f ? f : 1e-37f;
        row_end[r] = len - a.T + tok + 1;  // the row sees places below this
        row_place[r] = tok * a.hq + row0 + r - tok * a.rep;
      }
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int p = lane + 32 * i, ks = p / 8, w = p % 8;
        const int t = kNext ? w / 2 : w % 4, hi = kNext ? w & 1 : w / 4;
        uint32_t* to = reinterpret_cast<uint32_t*>(raw + S::oQ) + ((r / 8) * KS + ks) * 64 + ((r & 7) * 4 + t) * 2 + hi;
        uint32_t part[QP];
        split<!kCoded, QP>(to_f32(x[i].x) * up, to_f32(x[i].y) * up, part);
#pragma unroll
        for (int j = 0; j < QP; ++j) to[j * (S::kRows / 8) * KS * 64] = part[j];
      }
    }
    __syncthreads();
    float base[NT][2], l[NT][2], rf[NT][2];  // the weights' bases and sums, the scores' factors
    float o[OB][NT][4];
    uint2 qh[kHoldQ ? QP * NT * KS : 1];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        base[i][e] = kNone;
        l[i][e] = 0.f;
        rf[i][e] = row_factor[(wm * NT + i) * 8 + 2 * t4 + e];
      }
#pragma unroll
    for (int i = 0; i < OB; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    if (kHoldQ) {
#pragma unroll
      for (int i = 0; i < QP * NT * KS; ++i) qh[i] = qs[(i / (NT * KS) * (S::kRows / 8) * KS + i % (NT * KS)) * 32 + lane];
    }
    auto query = [&](int part, int nt, int ks) {
      return kHoldQ ? qh[(part * NT + nt) * KS + ks] : qs[(part * (S::kRows / 8) * KS + nt * KS + ks) * 32 + lane];
    };
    // c += A's parts times B's, down to the smallest that count.  The tensor cores cut what they add to a
    // sum off instead of rounding it, which over many steps is a drift: with float32 queries the
    // largest product of a step starts from 0 and is added in float32, the small ones add up in `rest`.
    auto scores = [&](float (&c)[NT][4], float (&rest)[NT][4], const uint4 (&w)[AP], int ks) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int b = 0; b < QP; ++b) {
          const uint2 q = query(b, j, ks);
#pragma unroll
          for (int i = 0; i < AP; ++i) {
            if (i + b >= (AP > QP ? AP : QP)) continue;
            if (FQ && i + b == 0) {
              float one[4] = {0.f, 0.f, 0.f, 0.f};
              product<!kCoded>(one, w[i], q.x, q.y);
#pragma unroll
              for (int e = 0; e < 4; ++e) c[j][e] += one[e];
            } else {
              product<!kCoded>(FQ ? rest[j] : c[j], w[i], q.x, q.y);
            }
          }
        }
    };
    const int hi_min = len - a.T + row0 / a.rep + 1;
    const int lo_max =
        a.window > 0 ? (int)max((int64_t)len - a.T + (row0 + rows - 1) / a.rep + 1 - a.window, (int64_t)INT_MIN) : INT_MIN;

    for (int t = t0; t < t1; ++t) {
      copy_wait<S::kStages - 2>();
      meet();
      request(stage == 0 ? S::kStages - 1 : stage - 1);
      char* const here = kv + stage * S::kStage;
      const uint8_t* const bytes = sc + stage * 2 * KT;
      const unsigned seen = seen_of[stage];
      // what the decisions go by that the sharing warps take alike: the group's places, or the tile's
      unsigned some = seen, all = seen;
      if constexpr (SHARE) {
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
          const unsigned x = seen_of[((grp + i) % kGroups - grp) * S::kStages + stage];
          some |= x;
          all &= x;
        }
      }
      const int here_at = stage * S::kStage;
      const int now_stage = stage;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
      if (some == 0) continue;
      const int first = (int)((unsigned)now.template lo<S::kTile>() + (unsigned)t * S::kTile), pos = (int)((unsigned)first + grp * KT);
      const bool edge = all != kAll || (SHARE ? first > hi_min - S::kTile || first < lo_max : pos > hi_min - KT || pos < lo_max);
      const uint32_t kbase = smem_at(here), vbase = kbase + S::kHalf;
      // ---- scores: c[places][queries]
      float c[KM][NT][4], rest[KM][NT][4];
#pragma unroll
      for (int u = 0; u < KM; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[u][j][e] = rest[u][j][e] = 0.f;
      if constexpr (kF32) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int u = 0; u < KM; ++u) {  // channels 4 t .. 4 t + 3 of the step, places g and g + 8
            const float4 x = *reinterpret_cast<const float4*>(here + key_piece<CH, true>(u * 16 + g, 4 * ks + t4) * 16);
            const float4 y = *reinterpret_cast<const float4*>(here + key_piece<CH, true>(u * 16 + 8 + g, 4 * ks + t4) * 16);
            uint32_t p[4][3];
            split<true, 3>(x.x, x.y, p[0]);
            split<true, 3>(y.x, y.y, p[1]);
            split<true, 3>(x.z, x.w, p[2]);
            split<true, 3>(y.z, y.w, p[3]);
            uint4 w[AP];
#pragma unroll
            for (int k = 0; k < AP; ++k) w[k] = make_uint4(p[0][k], p[1][k], p[2][k], p[3][k]);
            scores(c[u], rest[u], w, ks);
          }
      } else {
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
#pragma unroll
          for (int u = 0; u < KM; ++u) {
            uint32_t b[4];
            matrix4(b, kbase + piece<CH>(u * 16 + mrow, 2 * i + mcol) * 16);
            if constexpr (!kCoded) {
              const uint4 w[1] = {make_uint4(b[0], b[1], b[2], b[3])};
              scores(c[u], rest[u], w, i);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint4 w[1];
                open4<CACHE>(b[2 * k], w[0].x, w[0].z);
                open4<CACHE>(b[2 * k + 1], w[0].y, w[0].w);
                scores(c[u], rest[u], w, 2 * i + k);
              }
            }
          }
      }
      if (FQ) {
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[u][j][e] += rest[u][j][e];
      }
      // powers of two of places g and g + 8, each worked out by one lane.  The readers of a value's row that
      // is not finite become NaN through their sums.
      float kf[KM][2], vf[KM][2];
      unsigned nan_rows = 0;
      int vb = 0;
      float most = 0.f;  // the largest power, as an exponent that a base is asked to allow for
      if constexpr (kCoded) {
        const int kb = bytes[lane];
        vb = KT == 16 ? kb : bytes[KT + lane];
        const bool mine = KT == 16 ? lane >= 16 && (seen >> (lane & 15) & 1) : seen >> lane & 1;
        nan_rows = __ballot_sync(0xffffffffu, mine && vb == 255);
        if (KT == 16) nan_rows >>= 16;
        most = ask((int)__reduce_max_sync(0xffffffffu, mine && vb != 255 ? vb : 0));
        const float kfac = power(kb);
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) kf[u][e] = __shfl_sync(0xffffffffu, kfac, u * 16 + e * 8 + g);
      }
      if constexpr (kCoded) {
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[u][j][e] *= kf[u][e >> 1];
      }
      // ---- weights
      if (edge) {
        unsigned on[NT][2];  // the places that a query sees
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int64_t end = (int64_t)row_end[(wm * NT + j) * 8 + 2 * t4 + e] - pos;
            const int64_t from = a.window > 0 ? end - a.window : 0;
            unsigned m = end >= KT ? kAll : end <= 0 ? 0u : (1u << end) - 1;
            if (from > 0) m = from >= KT ? 0u : m & ~((1u << from) - 1);
            on[j][e] = m & seen;
            if (on[j][e] & nan_rows) l[j][e] = NAN;
#pragma unroll
            for (int u = 0; u < KM; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!(on[j][e] >> (u * 16 + h * 8 + g) & 1)) c[u][j][2 * h + e] = -INFINITY;
          }
        if (CACHE != KDA_CACHE_INT8) {
          bool found = false;
          for (int i = lane; i < S::kHalf / 16; i += 32) {
            const uint4 w = reinterpret_cast<const uint4*>(here + S::kHalf)[i];
            found |= wild<CACHE>(w.x) || wild<CACHE>(w.y) || wild<CACHE>(w.z) || wild<CACHE>(w.w);
          }
          if (SHARE ? __syncthreads_or(found) : __any_sync(0xffffffffu, found)) {
            // the rows that do see such a value take it (their output stays so), then it is 0
#pragma unroll 1
            for (int key = 0; key < (SHARE ? S::kTile : KT); ++key) {
              const int from = SHARE ? key / KT : grp, k = key % KT, place = first + from * KT + k;
              const bool there = seen_of[(from - grp) * S::kStages + now_stage] >> k & 1;
              const char* const row = raw + from * S::kStages * S::kStage + here_at + S::kHalf;
#pragma unroll
              for (int i = 0; i < OB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int ch = (SHARE ? grp * OB * 16 : 0) + (kNext ? i * 16 + 2 * g + h : i * 16 + h * 8 + g);
                  const int byte = ch * S::kElem;
                  const char* at = row + piece<CH>(k, byte / 16) * 16 + byte % 16;
                  float x;
                  if constexpr (kCoded) x = (*reinterpret_cast<const uint8_t*>(at) & 0x7f) == 0x7f ? NAN : 0.f;
                  else if constexpr (kF32) x = *reinterpret_cast<const float*>(at);
                  else x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
                  if (there && !isfinite(x)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        const int end = row_end[(wm * NT + j) * 8 + 2 * t4 + e];
                        if (place < end && (a.window == 0 || place >= end - a.window)) o[i][j][2 * h + e] += x;
                      }
                  }
                }
            }
            meet();
            if (wm == 0)
              for (int i = lane; i < S::kHalf / 4; i += 32) {
                uint32_t* w = reinterpret_cast<uint32_t*>(here + S::kHalf) + i;
                *w = tamed<CACHE>(*w);
              }
            meet();
          }
        }
      } else if (nan_rows) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) l[j][e] = NAN;
      }
      // The base of a row's weights follows its maximum (over codes the largest of weights times powers) only
      // where a score passes it by more than 2^lazy: the outputs are then rarely scaled again, the rows' maxima
      // rarely looked for across the warp, and a weight is 2^lazy at most.  Whether one does is told by the
      // largest power of all fetched places; by how much, below, from the places that the row sees.
      float high = -INFINITY;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int u = 0; u < KM; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) high = fmaxf(high, fmaf(c[u][j][2 * h + e], rf[j][e], -base[j][e]));
      const bool past = high > lazy<kCoded>() - most;
      if (SHARE ? __syncthreads_or(past) : __any_sync(0xffffffffu, past)) {
        float want[NT][2], add[KM][2];
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            add[u][h] = kCoded ? __shfl_sync(0xffffffffu, ask(vb == 255 ? 0 : vb), (KT == 16 ? 16 : u * 16) + h * 8 + g) : 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = -INFINITY;
#pragma unroll
            for (int u = 0; u < KM; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) x = fmaxf(x, fmaf(c[u][j][2 * h + e], rf[j][e], add[u][h]));
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, i));
            want[j][e] = x;
            if (SHARE && g == 0) shared_top[grp * S::kRows + j * 8 + 2 * t4 + e] = x;
          }
        if constexpr (SHARE) {  // the largest of the tile
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) want[j][e] = fmaxf(want[j][e], shared_top[i * S::kRows + j * 8 + 2 * t4 + e]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float al = 1.f;
            if (want[j][e] - base[j][e] > lazy<kCoded>()) {
              const float x = kCoded ? floorf(want[j][e]) : want[j][e];  // whole: an item's end moves it exactly
              al = exp2_of(base[j][e] - x);
              base[j][e] = x;
              l[j][e] *= al;
            }
#pragma unroll
            for (int i = 0; i < OB; ++i) {
              o[i][j][e] *= al;
              o[i][j][2 + e] *= al;
            }
          }
      }
      if constexpr (kCoded) {  // a value's power, 0 for a row that is not finite
        const float vfac = vb == 255 ? 0.f : power(vb);
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) vf[u][e] = __shfl_sync(0xffffffffu, vfac, (KT == 16 ? 16 : u * 16) + e * 8 + g);
      }
      uint32_t pw[PP][KM][NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int u = 0; u < KM; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = c[u][j][2 * h + e];
              x = exp2_of(fmaf(x, rf[j][e], -base[j][e]));
              l[j][e] += x;
              if (kCoded) x *= vf[u][h];
            }
        }
#pragma unroll
        for (int u = 0; u < KM; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t part[PP];
            split<!kCoded, PP, kF32>(c[u][j][2 * h], c[u][j][2 * h + 1], part);
#pragma unroll
            for (int k = 0; k < PP; ++k) pw[k][u][j][h] = transposed(part[k]);
          }
      }
      // ---- outputs
      auto outputs = [&](float (&o)[NT][4], const uint4 (&w)[AP], int u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float large[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < PP; ++b)
#pragma unroll
            for (int i = 0; i < AP; ++i)
              if (i + b < (AP > PP ? AP : PP))
                product<!kCoded>(!FQ ? o[j] : i + b ? small : large, w[i], pw[b][u][j][0], pw[b][u][j][1]);
          if (FQ) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] += large[e] + small[e];
          }
        }
      };
      if constexpr (SHARE) {
        // all groups' weights through shared memory; each warp adds up a quarter of the channels
#pragma unroll
        for (int b = 0; b < PP; ++b)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            shared_w[((b * kGroups + grp) * NT + j) * 32 + lane] = make_uint2(pw[b][0][j][0], pw[b][0][j][1]);
        __syncthreads();
        const uint32_t values = smem_at(raw + here_at + S::kHalf);  // of group 0
        constexpr uint32_t kApart = S::kStages * S::kStage;         // to the next group's
        auto add = [&](float (&o)[NT][4], const uint4& w, int u) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int b = 0; b < PP; ++b) {
              const uint2 p = shared_w[((b * kGroups + u) * NT + j) * 32 + lane];
              product<!kCoded>(o[j], w, p.x, p.y);
            }
        };
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          uint32_t b[4];
          if constexpr (!kCoded) {
#pragma unroll
            for (int i = 0; i < OB; ++i) {
              matrix4_trans(b, values + u * kApart + piece<CH>(vrow, (grp * OB + i) * 2 + vcol) * 16);
              add(o[i], make_uint4(b[0], b[1], b[2], b[3]), u);
            }
          } else {
            // two blocks of a group's values, or one block of two groups'
            if (OB == 1 && (u & 1)) continue;
            const uint32_t at = OB == 2 ? piece<CH>(mrow, grp * 2 + mcol) * 16 : mcol * kApart + piece<CH>(mrow, grp) * 16;
            matrix4_trans(b, values + u * kApart + at);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint4 w;
              open4<CACHE>(__byte_perm(b[2 * k], 0u, 0x3120), w.x, w.y);
              open4<CACHE>(__byte_perm(b[2 * k + 1], 0u, 0x3120), w.z, w.w);
              add(o[OB == 2 ? k : 0], w, OB == 2 ? u : u + k);
            }
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < KM; ++u) {
          if constexpr (kF32) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {  // channels 2 g and 2 g + 1, places 2 t, 2 t + 1 and 8 behind them
              float2 x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = u * 16 + 2 * t4 + (k & 1) + (k >> 1) * 8;
                x[k] = *reinterpret_cast<const float2*>(here + S::kHalf + piece<CH>(r, 4 * i + (g >> 1)) * 16 + (g & 1) * 8);
              }
              uint32_t p[4][3];
              split<true, 3>(x[0].x, x[1].x, p[0]);
              split<true, 3>(x[0].y, x[1].y, p[1]);
              split<true, 3>(x[2].x, x[3].x, p[2]);
              split<true, 3>(x[2].y, x[3].y, p[3]);
              uint4 w[AP];
#pragma unroll
              for (int k = 0; k < AP; ++k) w[k] = make_uint4(p[0][k], p[1][k], p[2][k], p[3][k]);
              outputs(o[i], w, u);
            }
          } else {
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              uint32_t b[4];
              matrix4_trans(b, vbase + piece<CH>(u * 16 + vrow, 2 * i + vcol) * 16);
              if constexpr (!kCoded) {
                const uint4 w[1] = {make_uint4(b[0], b[1], b[2], b[3])};
                outputs(o[i], w, u);
              } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint4 w[1];  // even channels of places 0-7, odd ones, the same of 8-15
                  open4<CACHE>(__byte_perm(b[2 * k], 0u, 0x3120), w[0].x, w[0].y);
                  open4<CACHE>(__byte_perm(b[2 * k + 1], 0u, 0x3120), w[0].z, w[0].w);
                  outputs(o[2 * i + k], w, u);
                }
              }
            }
          }
        }
      }
    }

    // ---- the item's end: the groups' outputs of the same rows, weighted by 2^(m - the largest m),
    // add up through shared memory, kSlice channels at a time in two buffers by turns.  Over codes a base counts
    // from the largest product of weight and power: the sum's own power goes into the maximum first.
    const bool whole = t0 == 0 && t1 == now.tiles;
    float2* const stats = reinterpret_cast<float2*>(raw + S::oStats);  // [groups][rows]: maximum, sum
    float scale_by[NT][2];
    float odd = 0.f;  // plus 0 times the sums: NaN where one is not finite
    if constexpr (!kCoded) {
#pragma unroll
      for (int i = 0; i < OB; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) odd = fmaf(o[i][j][e], 0.f, odd);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], i);
        if (base[j][e] == kNone) base[j][e] = -INFINITY;
        float m = base[j][e], sum = l[j][e];
        if (kCoded && sum > 0.f) {
          const int k = min((int)(__float_as_uint(sum) >> 23) - 127, 126);  // 126: an infinity
          sum *= __uint_as_float((uint32_t)(127 - k) << 23);
          m += (float)k;
        }
        if (g == 0) stats[grp * S::kRows + (wm * NT + j) * 8 + 2 * t4 + e] = make_float2(m, sum);
      }
    const bool wild_sums = __syncthreads_or(odd != odd);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (wm * NT + j) * 8 + 2 * t4 + e;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) m = fmaxf(m, stats[i * S::kRows + r].x);
        scale_by[j][e] = exp2_of(base[j][e] - (m == -INFINITY ? 0.f : m));
      }
    float* const part = part_of(s, blockIdx.x, t0 == 0 ? 1 : 0);
    // the sum of a row, and its maximum
    auto row_sum = [&](int r, float& m) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) m = fmaxf(m, stats[i * S::kRows + r].x);
      const float base = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) sum += stats[i * S::kRows + r].y * exp2_of(stats[i * S::kRows + r].x - base);
      return sum;
    };
    const int64_t out0 = (int64_t)n * a.T * a.hq + head * a.rep;  // with row_place the row's place in the output
    if (tid < rows) {
      float m;
      const float sum = row_sum(tid, m);
      if (!whole) {
        part[tid] = m;
        part[S::kRows + tid] = sum;
      } else if (a.lse) {
        a.lse[out0 + row_place[tid]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
      }
    }
    if constexpr (SHARE) {  // each warp has the sums of its channels
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = j * 8 + 2 * t4 + e;
          if (r >= rows) continue;
          float m, f = kCoded ? scale_by[j][e] : 1.f;  // the base is the same in all groups
          if (whole) {
            const float sum = row_sum(r, m);
            f = sum == 0.f ? 0.f : f / sum;
          }
          TQ* const to = static_cast<TQ*>(a.out) + (out0 + row_place[r]) * D;
#pragma unroll
          for (int i = 0; i < OB; ++i) {
            const float x = o[i][j][e] * f, z = o[i][j][2 + e] * f;
            const int ch = (grp * OB + i) * 16 + (kNext ? 2 * g : g), next = kNext ? 1 : 8;
            if (!whole) {
              part[2 * S::kRows + r * D + ch] = x;
              part[2 * S::kRows + r * D + ch + next] = z;
            } else if (kNext && words) {
              *reinterpret_cast<uint32_t*>(to + ch) = layer::pack_bf16(x, z);
            } else {
              to[ch] = from_f32<TQ>(x);
              to[ch + next] = from_f32<TQ>(z);
            }
          }
        }
    } else {
      constexpr int kSlice = S::kSlice, kPairs = kSlice / 2;
      // a thread's rows and channels of a slice are the same in every turn
      constexpr int kPer = (S::kRows * kPairs + S::kThreads - 1) / S::kThreads;
      float inverse[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = (i * S::kThreads + tid) / kPairs;
        float m, sum = 1.f;
        if (r < rows && whole) sum = row_sum(r, m);
        inverse[i] = sum == 0.f ? 0.f : 1.f / sum;
      }
#pragma unroll
      for (int q = 0; q < D / kSlice; ++q) {
        float* const buf = reinterpret_cast<float*>(raw + S::oMerge + (q & 1) * S::kMerge);  // [groups][rows][kPitch]
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* const to = buf + (grp * S::kRows + (wm * NT + j) * 8 + 2 * t4 + e) * S::kPitch;
#pragma unroll
            for (int i = 0; i < kSlice / 16; ++i) {
              const float x = o[q * (kSlice / 16) + i][j][e] * scale_by[j][e];
              const float z = o[q * (kSlice / 16) + i][j][2 + e] * scale_by[j][e];
              if constexpr (kNext) {
                *reinterpret_cast<float2*>(to + i * 16 + 2 * g) = make_float2(x, z);
              } else {
                to[i * 16 + g] = x;
                to[i * 16 + 8 + g] = z;
              }
            }
          }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int x = i * S::kThreads + tid, r = x / kPairs, ch = x % kPairs * 2;
          if (r >= rows) break;
          float2 v = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            const float2 w = *reinterpret_cast<const float2*>(buf + (k * S::kRows + r) * S::kPitch + ch);
            v.x += w.x;
            v.y += w.y;
          }
          if (whole) {
            TQ* to = static_cast<TQ*>(a.out) + (out0 + row_place[r]) * D + q * kSlice + ch;
            if (words && FQ) {
              *reinterpret_cast<float2*>(to) = make_float2(v.x * inverse[i], v.y * inverse[i]);
            } else if (words) {
              *reinterpret_cast<uint32_t*>(to) = layer::pack_bf16(v.x * inverse[i], v.y * inverse[i]);
            } else {
              to[0] = from_f32<TQ>(v.x * inverse[i]);
              to[1] = from_f32<TQ>(v.y * inverse[i]);
            }
          } else {
            *reinterpret_cast<float2*>(part + 2 * S::kRows + r * D + q * kSlice + ch) = v;
          }
        }
      }
    }
    if constexpr (!kCoded) {
      if (wild_sums) {
        __syncthreads();
        using TC = std::conditional_t<kF32, float, __nv_bfloat16>;
        const int from = now.template lo<S::kTile>() + t0 * S::kTile, to = (int)min((int64_t)now.template lo<S::kTile>() + (int64_t)t1 * S::kTile, (int64_t)now.hi);
#pragma unroll 1
        for (int i = tid; i < rows * D; i += S::kThreads) {
          const int r = i / D, end = row_end[r];
          TQ* const at = static_cast<TQ*>(a.out) + (out0 + row_place[r]) * D + i % D;
          const float x = whole ? to_f32(*at) : part[2 * S::kRows + i];
          float m;
          const float sum = row_sum(r, m);
          if (isfinite(x) || sum != sum) continue;  // scores that are NaN
          const int seen = a.window > 0 ? (int)max((int64_t)end - a.window, (int64_t)from) : from;
          const float wild = sum_of_wild<TC, D>(a, n, head, i % D, seen, min(to, end));
          if (wild == 0.f) continue;
          if (whole) *at = from_f32<TQ>(wild);
          else part[2 * S::kRows + i] = wild;
        }
      }
    }
    now.pass(a, s, t1 - t0);
  }
  copy_wait<0>();
  __syncthreads();
  if (tid == 0 && !s.one) s.verdict[blockIdx.x] = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
}

template <bool FQ, int CACHE, int D, int NT, int WM, int KT, int PER, bool SHARE>
cudaError_t launch(Shape<FQ, CACHE, D, NT, WM, KT, PER, SHARE>, const AttnArgs& a, const Split& s) {
  using S = Shape<FQ, CACHE, D, NT, WM, KT, PER, SHARE>;
  auto* kernel = attn_mma_kernel<FQ, CACHE, D, NT, WM, KT, PER, SHARE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  constexpr uintptr_t two = FQ ? 8 : 4;  // whole pairs of q and out
  const bool words = (uintptr_t)a.q % two == 0 && (uintptr_t)a.out % two == 0 && a.ldq % 2 == 0;
  kernel<<<(unsigned)s.blocks, S::kThreads, S::kBytes, a.stream>>>(a, s, words);
  return cudaGetLastError();
}

// f(Shape) for the rows of a call: 8, 16, 32 or 64 to a block.  One GB300, us: 256 sequences of up
// to 8192 e4m3 places, 4 rows: 32 places a group and 3 blocks to an SM 334, 16 and 4 blocks 389, 32
// and 2 blocks 488 (before the ends were weighed in); 131071 bf16 places: 3 blocks 92, 2 blocks 94;
// 16 sequences of up to 32768 int8 places, 32 rows: shared weights with 3 blocks to an SM 148, with 4
// or 2 blocks 160, all channels in each warp 172; 32 sequences of 8192 bf16 places, 32 and 64 rows:
// shared 226 and 353, not shared 273 and 385 (shared today 210 and 352; the int8 case 154).
template <int CACHE, int D, class F>
auto by_rows(const AttnArgs& a, F f) {
  constexpr bool kCoded = CACHE == KDA_CACHE_E4M3 || CACHE == KDA_CACHE_INT8;
  constexpr int kPlaces = kCoded ? 32 : 16;
  const int rows = a.T * a.rep;
  if (rows <= 8) return f(Shape<false, CACHE, D, 1, 1, kPlaces, 3>());
  if (rows <= 16) return f(Shape<false, CACHE, D, 2, 1, kPlaces, 2>());
  if (rows <= 32) return f(Shape<false, CACHE, D, 4, 1, 16, kCoded ? 3 : 2, true>());
  return f(Shape<false, CACHE, D, 8, 1, 16, 2, true>());
}
// float32 queries: their parts take room, so 32 rows at most
template <int CACHE, int D, class F>
auto by_rows_f32(const AttnArgs& a, F f) {
  constexpr int kPer = CACHE == KDA_CACHE_F32 && D == 128 ? 1 : 2;
  const int rows = a.T * a.rep;
  if (rows <= 8) return f(Shape<true, CACHE, D, 1, 1, 16, kPer>());
  if (rows <= 16) return f(Shape<true, CACHE, D, 2, 1, 16, kPer>());
  return f(Shape<true, CACHE, D, 2, 2, 16, 1>());
}
template <int D, class F>
auto by_cache(const AttnArgs& a, F f) {
  if (a.cache == KDA_CACHE_E4M3) return a.bf16 ? by_rows<KDA_CACHE_E4M3, D>(a, f) : by_rows_f32<KDA_CACHE_E4M3, D>(a, f);
  if (a.cache == KDA_CACHE_INT8) return a.bf16 ? by_rows<KDA_CACHE_INT8, D>(a, f) : by_rows_f32<KDA_CACHE_INT8, D>(a, f);
  return a.bf16 ? by_rows<KDA_CACHE_BF16, D>(a, f) : by_rows_f32<KDA_CACHE_F32, D>(a, f);  // of q's type
}
template <class F>
auto by_type(const AttnArgs& a, F f) {
  return a.d == 128 ? by_cache<128>(a, f) : by_cache<64>(a, f);
}

Split split_for(const AttnArgs& a) {
  return by_type(a, [&](auto shape) { return split_of(a, shape.kRows, shape.kTile, shape.kCost, shape.kPerSm); });
}

}  // namespace

size_t attn_workspace(const AttnArgs& a) { return split_bytes(split_for(a)); }

cudaError_t launch_attn(const AttnArgs& a) {
  if (a.B == 0) return a.ws ? cudaMemsetAsync(a.ws, 0, 4, a.stream) : cudaSuccess;
  Split s = split_for(a);
  split_place(s, a.ws);
  cudaError_t e = by_type(a, [&](auto shape) { return launch(shape, a, s); });
  if (e != cudaSuccess) return e;
  if (s.one) return a.ws ? launch_attn_table(a, s) : e;
  return launch_attn_join(a, s);
}

}  // namespace attn
}  // namespace kda
