// Attention of new tokens over the paged cache, bf16 queries: products on the tensor cores.
//
// Bound by the bytes of keys and values: 8 to 64 query rows per key are few operations, so the
// products are warp-level ones (m16n8k16, 16 query rows), and everything else serves a steady
// stream of loads.  Each of a block's four key groups takes 16 of a tile's 64 places: its warps
// copy them into a ring of stages of their own (cp.async, 16 bytes a lane, swizzled by row) and
// wait for nobody else; a running maximum, sum and output per warp are joined when an item ends.
// The next items' tiles are requested while the present one is worked on.
//
//     S = Q K^T: A = queries, B = keys (their rows are B's columns: ldmatrix as they lie)
//     O = P V:   A = the weights, whose accumulator layout is A's; B = values (ldmatrix.trans)
//
// Types.  bf16 caches: products of bf16, exact in float32; a weight enters as two bf16 parts
// (16 bits), since one alone would cost as much as the output's own rounding.  Codes become f16,
// exactly; queries become f16 after a power of two per row has brought their largest to 2^13,
// which keeps every bit down to 2^-27 of it.  A value's power of two joins the weight in the
// exponent, 2^(s + e - M) with M the row's own running maximum of s + e, so that f16 holds the
// largest contributions with 11 bits and smaller ones to 2^-25 of them; the sum of weights
// stays 2^(s - m) in float32.
//
// Codes lie four to a 32-bit word, and the products' order of channels is free as long as both
// operands have the same: a word of a key's row is channels 4t .. 4t + 3, used as the two pairs
// of a k-step; ldmatrix.trans on pairs of bytes gives two channels of two places, which one
// byte permutation sorts by channel, so that a thread's outputs are four adjacent channels.
//
// Places that a row does not see: the tiles at the ends of the seen range replace their scores
// by -inf, and values that are not finite by zeros, whose rows get them added afterwards if they
// do see them (0 times infinity would reach the others).
#include "kda_attn_split.cuh"

namespace kda {
namespace attn {
namespace {

constexpr int kGroups = 4;  // key groups of a block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
// whether a half of the pair is an infinity or NaN; such halves are cleared
template <bool kBf16>
__device__ __forceinline__ bool clear_wild(uint32_t& w) {
  constexpr uint32_t m = kBf16 ? 0x7f80u : 0x7c00u;
  bool wild = false;
  if ((w & m) == m) { w &= 0xffff0000u; wild = true; }
  if (((w >> 16) & m) == m) { w &= 0xffffu; wild = true; }
  return wild;
}

// Places of tiles in the block's share, item by item.
struct Cursor {
  int64_t left;  // tiles of the share from here on
  int n, j;      // sequence; head and chunk
  int t, tiles;  // tile of the item, the item's number
  int lo, hi;    // the sequence's places
  __device__ __forceinline__ void enter(const AttnArgs& a) {
    const Keys k = keys_of(a, n);
    lo = (int)k.lo;
    hi = (int)k.hi;
    tiles = (int)k.tiles;
  }
  __device__ __forceinline__ void next(const AttnArgs& a, int each) {
    --left;
    if (++t < tiles) return;
    t = 0;
    if (++j < each) return;
    j = 0;
    ++n;
    if (left > 0) enter(a);
  }
};

template <int CACHE, int D, int MT, int WM>
struct Shape {
  static constexpr bool kCoded = CACHE == KDA_CACHE_E4M3 || CACHE == KDA_CACHE_INT8;
  static constexpr int kThreads = kGroups * WM * 32;
  static constexpr int kRows = 16 * MT * WM;
  static constexpr int kRowBytes = D * (kCoded ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;           // 16-byte pieces of a row
  static constexpr int kHalf = 16 * kRowBytes;             // a group's keys (or values) of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kMergeWarp = 16 * MT * (D + 2) * 4;  // a warp's output, maxima and sums
  static constexpr int kQBytes = WM * MT * (D / 16) * 32 * 16;
  static constexpr int bytes(int stages) {
    return kGroups * stages * (kStage + 32 + 4) + kQBytes + (kRows * 4 + 15) / 16 * 16 + WM * kMergeWarp;
  }
  // two blocks to an SM where three stages of each fit (228 KB, of which a block takes 1.5 KB
  // for itself), with up to five stages; otherwise one block with up to six
  static constexpr int kRoom = 228 * 1024;
  static constexpr bool kTwo = WM == 1 && 2 * (bytes(3) + 1536) <= kRoom;
  static constexpr int fit() {
    int n = 2;
    while (n < (kTwo ? 5 : 6) && (kTwo ? 2 : 1) * (bytes(n + 1) + 1536) <= kRoom) ++n;
    return n;
  }
  static constexpr int kStages = fit();
  static constexpr int kPerSm = kTwo ? 2 : 1;
  // shared memory
  static constexpr int oQ = kGroups * kStages * kStage;
  static constexpr int oScale = oQ + kQBytes;
  static constexpr int oSeen = oScale + kGroups * kStages * 32;
  static constexpr int oRow = oSeen + kGroups * kStages * 4;
  static constexpr int oMerge = oRow + (kRows * 4 + 15) / 16 * 16;
  static constexpr int kBytes = bytes(kStages);
  static_assert(oMerge % 16 == 0 && kMergeWarp % 16 == 0 && oMerge + WM * kMergeWarp == kBytes, "layout");
};
// a row's 16-byte piece c, moved so that 8 rows' pieces c lie in different banks
template <int CHUNKS>
__device__ __forceinline__ int piece(int row, int c) {
  if constexpr (CHUNKS >= 8) return row * CHUNKS + (c ^ (row & 7));
  else return row * CHUNKS + (c ^ ((row >> 1) & 3));
}

template <int CACHE, int D, int MT, int WM>
__global__ void __launch_bounds__(Shape<CACHE, D, MT, WM>::kThreads, Shape<CACHE, D, MT, WM>::kPerSm)
attn_mma_kernel(AttnArgs a, Split s, bool words) {
  using S = Shape<CACHE, D, MT, WM>;
  constexpr int KS = D / 16;
  extern __shared__ __align__(128) char raw[];
  __shared__ int64_t scratch[34];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp % kGroups, wm = warp / kGroups;  // key group; which query rows
  const int g = lane >> 2, t4 = lane & 3;
  if (tid == 0) bad = 0;
  Start st;
  const bool work = find_start<S::kThreads>(a, s, scratch, st);
  if (!work) {
    if (tid == 0) s.verdict[blockIdx.x] = KDA_OK;
    return;
  }
  const int each = a.hk * s.chunks;
  const int mask = (1 << a.t.shift) - 1;
  Cursor now;
  {
    now.n = st.n;
    now.left = st.end - st.at;
    now.enter(a);
    const int64_t off = st.at - st.before * each;
    now.j = (int)(off / now.tiles);
    now.t = (int)(off % now.tiles);
  }
  Cursor ahead = now;
  char* const kv = raw + grp * S::kStages * S::kStage;
  uint8_t* const sc = reinterpret_cast<uint8_t*>(raw + S::oScale) + grp * S::kStages * 32;
  int* const seen_of = reinterpret_cast<int*>(raw + S::oSeen) + grp * S::kStages;
  float* const row_factor = reinterpret_cast<float*>(raw + S::oRow);
  uint4* const qs = reinterpret_cast<uint4*>(raw + S::oQ);

  // The group's 16 places of the tile at `ahead` into a stage (its WM warps take a share each).
  auto request = [&](int stage) {
    if (ahead.left > 0) {
      const int head = ahead.j / s.chunks;
      const int64_t pos = (int64_t)ahead.lo + (int64_t)ahead.t * kTile + grp * 16;
      const uint32_t dst = smem_at(kv + stage * S::kStage);
      unsigned seen = 0;
      if (a.t.shift >= 4) {  // a page holds all 16
        const int id = pos < ahead.hi ? page_of(a.t, ahead.n, pos) : -1;
        const int have = pos < ahead.hi ? (int)min((int64_t)16, ahead.hi - pos) : 0;
        if (id >= 0) seen = (1u << have) - 1;
        else if (have > 0) bad = 1;
        const int64_t row = ((int64_t)head << a.t.shift) + (pos & mask);
        const int64_t from = id >= 0 ? (id * a.ldpage + row * D) * (S::kCoded ? 1 : 2) : 0;
        const char* k = static_cast<const char*>(a.kc) + from;
        const char* v = static_cast<const char*>(a.vc) + from;
#pragma unroll
        for (int i = 0; i < 16 * S::kChunks / 32 / WM; ++i) {
          const int x = (i * WM + wm) * 32 + lane, r = x / S::kChunks, c = x % S::kChunks;
          const bool ok = id >= 0 && r < have;
          const int to = piece<S::kChunks>(r, c) * 16;
          copy16(dst + to, ok ? k + x * 16 : k, ok);
          copy16(dst + S::kHalf + to, ok ? v + x * 16 : v, ok);
        }
        if (S::kCoded && wm == 0 && lane < 2 && id >= 0) {
          const int64_t b = (((int64_t)id * a.hk) << a.t.shift) + row;
          copy16(smem_at(sc + stage * 32 + lane * 16), (lane ? a.vs : a.ks) + b, true);
        }
      } else {
        for (int i = 0; i < 16 * S::kChunks / 32 / WM; ++i) {
          const int x = (i * WM + wm) * 32 + lane, r = x / S::kChunks, c = x % S::kChunks;
          const int id = pos + r < ahead.hi ? page_of(a.t, ahead.n, pos + r) : -1;
          const int64_t row = ((int64_t)head << a.t.shift) + ((pos + r) & mask);
          const int64_t from = id >= 0 ? (id * a.ldpage + row * D) * (S::kCoded ? 1 : 2) + c * 16 : 0;
          const int to = piece<S::kChunks>(r, c) * 16;
          copy16(dst + to, static_cast<const char*>(a.kc) + from, id >= 0);
          copy16(dst + S::kHalf + to, static_cast<const char*>(a.vc) + from, id >= 0);
        }
        const int r = lane & 15;
        const int id = pos + r < ahead.hi ? page_of(a.t, ahead.n, pos + r) : -1;
        if (id < 0 && pos + r < ahead.hi) bad = 1;
        seen = __ballot_sync(0xffffffffu, id >= 0) & 0xffffu;
        if (S::kCoded && wm == 0 && id >= 0) {
          const int64_t row = ((int64_t)head << a.t.shift) + ((pos + r) & mask);
          const int64_t b = (((int64_t)id * a.hk) << a.t.shift) + row;
          sc[stage * 32 + lane] = (lane < 16 ? a.ks : a.vs)[b];
        }
      }
      if (wm == 0 && lane == 0) seen_of[stage] = (int)seen;
      ahead.next(a, each);
    }
    copy_commit();
  };
  // all that the group's warps wrote of a stage is there, and nobody reads the one before
  auto meet = [&]() {
    if constexpr (WM == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WM) : "memory");
  };

#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) request(i);
  int stage = 0;

  while (now.left > 0) {
    // ---- an item begins: its queries as fragments of A, one row per warp and turn
    const int n = now.n, head = now.j / s.chunks, row0 = now.j % s.chunks * S::kRows;
    const int rows = min(S::kRows, a.T * a.rep - row0);
    const int len = max(a.t.lens[n], -8);  // nothing is seen at 0 and below
    const int t0 = now.t, t1 = (int)min((int64_t)now.tiles, now.t + now.left);
    if (tid == 0) {
      if ((int64_t)len > (int64_t)a.t.max_pages << a.t.shift) bad = 1;
      if (t0 == 0) s.first[(int64_t)n * each + now.j] = st.end - now.left;
    }
    __syncthreads();
    for (int r = warp; r < S::kRows; r += S::kThreads / 32) {
      const int row = row0 + r;
      __nv_bfloat162 x[D / 64];
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
          ((int64_t)n * a.T + row / a.rep) * a.ldq + (int64_t)(head * a.rep + row % a.rep) * D;
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int p = lane + 32 * i;
        x[i] = __floats2bfloat162_rn(0.f, 0.f);
        if (r < rows) {
          if (words) x[i] = reinterpret_cast<const __nv_bfloat162*>(q)[p];
          else { x[i].x = q[2 * p]; x[i].y = q[2 * p + 1]; }
        }
        most = max(most, max(__float_as_uint(__bfloat162float(x[i].x)) & 0x7fffffffu,
                             __float_as_uint(__bfloat162float(x[i].y)) & 0x7fffffffu));
      }
      float up = 1.f;
      if constexpr (S::kCoded) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        // 2^13 over the largest's power of two, kept a normal number
        const int e = (int)(most >> 23);
        const int k = e == 0 || e == 255 ? 0 : min(max(127 + 13 - e, -120), 120);
        up = __uint_as_float((uint32_t)(127 + k) << 23);
        if (lane == 0) row_factor[r] = a.scale * kLog2e * __uint_as_float((uint32_t)(127 - k) << 23);
      }
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int p = lane + 32 * i, ks = p / 8, w = p % 8;
        const int t = S::kCoded ? w / 2 : w % 4, hi = S::kCoded ? w & 1 : w / 4;
        uint32_t v;
        if constexpr (S::kCoded) v = pack_half(__bfloat162float(x[i].x) * up, __bfloat162float(x[i].y) * up);
        else v = *reinterpret_cast<const uint32_t*>(&x[i]);
        uint32_t* to = reinterpret_cast<uint32_t*>(&qs[((r / 16) * KS + ks) * 32 + (r & 7) * 4 + t]);
        to[hi * 2 + ((r >> 3) & 1)] = v;
      }
    }
    __syncthreads();
    float m[MT][2], M[MT][2], l[MT][2], rf[MT][2];
    float o[MT][D / 8][4];
    int hi_of[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (wm * MT + mt) * 16 + h * 8 + g;
        m[mt][h] = M[mt][h] = -INFINITY;
        l[mt][h] = 0.f;
        rf[mt][h] = S::kCoded ? row_factor[r] : a.scale * kLog2e;
        hi_of[mt][h] = len - a.T + (row0 + r) / a.rep + 1;  // the row sees places below this
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
    const int hi_min = len - a.T + row0 / a.rep + 1;
    const int lo_max = a.window > 0 ? len - a.T + (row0 + rows - 1) / a.rep + 1 - a.window : INT_MIN;

    for (int t = t0; t < t1; ++t) {
      copy_wait<S::kStages - 2>();
      meet();
      request(stage == 0 ? S::kStages - 1 : stage - 1);
      const int pos = now.lo + t * kTile + grp * 16;
      const unsigned seen = (unsigned)seen_of[stage];
      const bool edge = seen != 0xffffu || pos > hi_min - 16 || pos < lo_max;
      const uint32_t kbase = smem_at(kv + stage * S::kStage), vbase = kbase + S::kHalf;
      // ---- scores of 16 places: c[mt][places 0-7, 8-15]
      float c[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[mt][i][e] = 0.f;
      if constexpr (!S::kCoded) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          // matrices: places 0-7 and 8-15 by channels 0-7 and 8-15 of the step
          uint32_t b[4];
          const int r = (lane & 7) + (lane >> 4) * 8;
          matrix4(b, kbase + piece<S::kChunks>(r, 2 * ks + ((lane >> 3) & 1)) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 q = qs[((wm * MT + mt) * KS + ks) * 32 + lane];
            product<true>(c[mt][0], q, b[0], b[1]);
            product<true>(c[mt][1], q, b[2], b[3]);
          }
        }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          // matrices: places 0-7 and 8-15 by steps 2 k2 and 2 k2 + 1 (16 bytes each)
          uint32_t b[4];
          const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
          matrix4(b, kbase + piece<S::kChunks>(r, 2 * k2 + (lane >> 4)) * 16);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t x0, x1, y0, y1;
            open4<CACHE>(b[2 * k], x0, x1);
            open4<CACHE>(b[2 * k + 1], y0, y1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint4 q = qs[((wm * MT + mt) * KS + 2 * k2 + k) * 32 + lane];
              product<false>(c[mt][0], q, x0, x1);
              product<false>(c[mt][1], q, y0, y1);
            }
          }
        }
      }
      float kf[2][2], ev[2][2];  // a key's power of two; a value's exponent
      if constexpr (S::kCoded) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = stage * 32 + i * 8 + 2 * t4 + e;
            const int b = sc[at + 16];
            kf[i][e] = power(sc[at]);
            ev[i][e] = b == 255 ? INFINITY : (float)(b - 127);
          }
      }
      // ---- weights
      bool moved = false;
      float al[MT][2];  // the output's factor
      uint4 ph[MT], pl[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float p[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY, Mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = c[mt][i][2 * h + e];
              x *= rf[mt][h];
              if (S::kCoded) x *= kf[i][e];
              if (edge) {
                const int key = i * 8 + 2 * t4 + e;
                const bool ok = ((seen >> key) & 1) && pos + key < hi_of[mt][h] &&
                                (a.window == 0 || pos + key >= hi_of[mt][h] - a.window);
                if (!ok) x = -INFINITY;
              }
              mx = fmaxf(mx, x);
              if (S::kCoded) Mx = fmaxf(Mx, edge && x == -INFINITY ? x : x + ev[i][e]);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[mt][h], mx);
          const float mb = mn == -INFINITY ? 0.f : mn;
          const float am = exp2_of(m[mt][h] - mb);
          l[mt][h] *= am;
          al[mt][h] = am;
          moved |= mn != m[mt][h];
          m[mt][h] = mn;
          float Mb = 0.f;
          if (S::kCoded) {
            Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, 1));
            Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, 2));
            const float Mn = fmaxf(M[mt][h], Mx);
            Mb = Mn == -INFINITY ? 0.f : Mn;
            al[mt][h] = exp2_of(M[mt][h] - Mb);
            moved |= Mn != M[mt][h];
            M[mt][h] = Mn;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = c[mt][i][2 * h + e];
              const float w = exp2_of(x - mb);
              l[mt][h] += w;
              p[i][2 * h + e] = w;
              if (S::kCoded) p[i][2 * h + e] = edge && x == -INFINITY ? 0.f : exp2_of(x + ev[i][e] - Mb);
            }
        }
        uint32_t w[4], v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // A's words: rows g, g + 8 of places 0-7, then of 8-15
          const float x = p[k >> 1][(k & 1) * 2], y = p[k >> 1][(k & 1) * 2 + 1];
          if constexpr (S::kCoded) {
            w[k] = pack_half(x, y);
          } else {
            w[k] = layer::pack_bf16(x, y);
            float xh, yh;
            layer::unpack2(w[k], xh, yh);
            v[k] = layer::pack_bf16(x - xh, y - yh);
          }
        }
        ph[mt] = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (!S::kCoded) pl[mt] = make_uint4(v[0], v[1], v[2], v[3]);
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][0] *= al[mt][0];
            o[mt][i][1] *= al[mt][0];
            o[mt][i][2] *= al[mt][1];
            o[mt][i][3] *= al[mt][1];
          }
      }
      // ---- outputs; each ldmatrix gives 16 bytes of channels twice
      bool wild = false;
#pragma unroll
      for (int i = 0; i < S::kChunks / 2; ++i) {
        uint32_t b[4];
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
        matrix4_trans(b, vbase + piece<S::kChunks>(r, 2 * i + (lane >> 4)) * 16);
        if constexpr (!S::kCoded) {
          if (edge) {
#pragma unroll
            for (int k = 0; k < 4; ++k) wild |= clear_wild<true>(b[k]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              product<true>(o[mt][2 * i + k], ph[mt], b[2 * k], b[2 * k + 1]);
              product<true>(o[mt][2 * i + k], pl[mt], b[2 * k], b[2 * k + 1]);
            }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t x0, x1, y0, y1;  // even channels of places 0-7 (8-15), odd channels
            open4<CACHE>(__byte_perm(b[2 * k], 0u, 0x3120), x0, x1);
            open4<CACHE>(__byte_perm(b[2 * k + 1], 0u, 0x3120), y0, y1);
            if (CACHE == KDA_CACHE_E4M3 && edge) {
              wild |= clear_wild<false>(x0);
              wild |= clear_wild<false>(x1);
              wild |= clear_wild<false>(y0);
              wild |= clear_wild<false>(y1);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              product<false>(o[mt][2 * (2 * i + k)], ph[mt], x0, y0);
              product<false>(o[mt][2 * (2 * i + k) + 1], ph[mt], x1, y1);
            }
          }
        }
      }
      if (edge && CACHE != KDA_CACHE_INT8 && __any_sync(0xffffffffu, wild)) {
        // the rows that do see such a value take it
        const char* v = kv + stage * S::kStage + S::kHalf;
        for (int key = 0; key < 16; ++key)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int h = e >> 1, lim = hi_of[mt][h];
                const int ch = S::kCoded ? (i / 2) * 16 + 4 * t4 + 2 * (e & 1) + (i & 1) : i * 8 + 2 * t4 + (e & 1);
                const int byte = ch * (S::kCoded ? 1 : 2);
                const char* at = v + piece<S::kChunks>(key, byte / 16) * 16 + byte % 16;
                float x;
                if constexpr (S::kCoded) x = (*reinterpret_cast<const uint8_t*>(at) & 0x7f) == 0x7f ? NAN : 0.f;
                else x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
                const bool ok = ((seen >> key) & 1) && pos + key < lim && (a.window == 0 || pos + key >= lim - a.window);
                if (ok && !isfinite(x)) o[mt][i][e] += x;
              }
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }

    // ---- the item's end: the groups' outputs of the same rows join, one after the other
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 1);
        l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 2);
        if (S::kCoded) {  // from the outputs' own base to the weights'
          const float f = m[mt][h] == -INFINITY ? 1.f : exp2_of(M[mt][h] - m[mt][h]);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][2 * h] *= f;
            o[mt][i][2 * h + 1] *= f;
          }
        }
      }
#pragma unroll
    for (int up = kGroups - 1; up > 0; --up) {
      float* buf = reinterpret_cast<float*>(raw + S::oMerge + wm * S::kMergeWarp);
      __syncthreads();
      if (grp == up) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float4*>(buf + ((mt * (D / 8) + i) * 32 + lane) * 4) =
                make_float4(o[mt][i][0], o[mt][i][1], o[mt][i][2], o[mt][i][3]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (t4 == 0) {
              buf[16 * MT * D + mt * 16 + h * 8 + g] = m[mt][h];
              buf[16 * MT * (D + 1) + mt * 16 + h * 8 + g] = l[mt][h];
            }
        }
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float fa[2], fb[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mo = buf[16 * MT * D + mt * 16 + h * 8 + g], lo = buf[16 * MT * (D + 1) + mt * 16 + h * 8 + g];
            const float mn = fmaxf(m[mt][h], mo), base = mn == -INFINITY ? 0.f : mn;
            fa[h] = exp2_of(m[mt][h] - base);
            fb[h] = exp2_of(mo - base);
            l[mt][h] = l[mt][h] * fa[h] + lo * fb[h];
            m[mt][h] = mn;
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(buf + ((mt * (D / 8) + i) * 32 + lane) * 4);
            o[mt][i][0] = o[mt][i][0] * fa[0] + x.x * fb[0];
            o[mt][i][1] = o[mt][i][1] * fa[0] + x.y * fb[0];
            o[mt][i][2] = o[mt][i][2] * fa[1] + x.z * fb[1];
            o[mt][i][3] = o[mt][i][3] * fa[1] + x.w * fb[1];
          }
        }
      }
    }
    if (grp == 0) {
      const bool whole = t0 == 0 && t1 == now.tiles;
      float* part = whole ? nullptr : part_of(s, blockIdx.x, t0 == 0 ? 1 : 0);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (wm * MT + mt) * 16 + h * 8 + g, row = row0 + r;
          if (r >= rows) continue;
          const float lr = l[mt][h];
          if (!whole) {
            if (t4 == 0) {
              part[r] = m[mt][h];
              part[S::kRows + r] = lr;
            }
            float* to = part + 2 * S::kRows + r * D;
            if constexpr (S::kCoded) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float4*>(to + i * 16 + 4 * t4) =
                    make_float4(o[mt][2 * i][2 * h], o[mt][2 * i + 1][2 * h], o[mt][2 * i][2 * h + 1], o[mt][2 * i + 1][2 * h + 1]);
            } else {
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(to + i * 8 + 2 * t4) = make_float2(o[mt][i][2 * h], o[mt][i][2 * h + 1]);
            }
            continue;
          }
          const int64_t at = ((int64_t)n * a.T + row / a.rep) * a.hq + head * a.rep + row % a.rep;
          const float f = lr == 0.f ? 0.f : 1.f / lr;
          if (t4 == 0 && a.lse) a.lse[at] = lr == 0.f ? -INFINITY : (m[mt][h] + log2f(lr)) * kLn2;
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at * D;
          auto put = [&](int ch, float x, float y) {
            if (words) {
              *reinterpret_cast<uint32_t*>(to + ch) = layer::pack_bf16(x, y);
            } else {
              to[ch] = __float2bfloat16_rn(x);
              to[ch + 1] = __float2bfloat16_rn(y);
            }
          };
          if constexpr (S::kCoded) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              put(i * 16 + 4 * t4, o[mt][2 * i][2 * h] * f, o[mt][2 * i + 1][2 * h] * f);
              put(i * 16 + 4 * t4 + 2, o[mt][2 * i][2 * h + 1] * f, o[mt][2 * i + 1][2 * h + 1] * f);
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) put(i * 8 + 2 * t4, o[mt][i][2 * h] * f, o[mt][i][2 * h + 1] * f);
          }
        }
    }
    // on to the next item
    now.left -= t1 - t0;
    if (t1 == now.tiles) {
      now.t = 0;
      if (++now.j == each) {
        now.j = 0;
        ++now.n;
        if (now.left > 0) now.enter(a);
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
  if (tid == 0) s.verdict[blockIdx.x] = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
}

template <int CACHE, int D, int MT, int WM>
cudaError_t launch(const AttnArgs& a, const Split& s) {
  using S = Shape<CACHE, D, MT, WM>;
  cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<CACHE, D, MT, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const bool words = (uintptr_t)a.q % 4 == 0 && (uintptr_t)a.out % 4 == 0 && a.ldq % 2 == 0;
  attn_mma_kernel<CACHE, D, MT, WM><<<(unsigned)s.blocks, S::kThreads, S::kBytes, a.stream>>>(a, s, words);
  return cudaGetLastError();
}

// f(Shape) for the rows of a call: 16, 32 or 64 to a block
template <int CACHE, int D, class F>
auto by_rows(const AttnArgs& a, F f) {
  const int rows = a.T * a.rep;
  if (rows <= 16) return f(Shape<CACHE, D, 1, 1>());
  if (rows <= 32) return f(Shape<CACHE, D, 2, 1>());
  return f(Shape<CACHE, D, 2, 2>());
}
template <class F>
auto by_type(const AttnArgs& a, F f) {
  if (a.d == 128) {
    if (a.cache == KDA_CACHE_E4M3) return by_rows<KDA_CACHE_E4M3, 128>(a, f);
    if (a.cache == KDA_CACHE_INT8) return by_rows<KDA_CACHE_INT8, 128>(a, f);
    return by_rows<KDA_CACHE_BF16, 128>(a, f);
  }
  if (a.cache == KDA_CACHE_E4M3) return by_rows<KDA_CACHE_E4M3, 64>(a, f);
  if (a.cache == KDA_CACHE_INT8) return by_rows<KDA_CACHE_INT8, 64>(a, f);
  return by_rows<KDA_CACHE_BF16, 64>(a, f);
}
template <int CACHE, int D, int MT, int WM>
cudaError_t launch_of(Shape<CACHE, D, MT, WM>, const AttnArgs& a, const Split& s) {
  return launch<CACHE, D, MT, WM>(a, s);
}

}  // namespace

Split attn_mma_split(const AttnArgs& a) {
  return by_type(a, [&](auto shape) { return split_of(a, shape.kRows, shape.kPerSm); });
}

cudaError_t launch_attn_mma(const AttnArgs& a) {
  Split s = attn_mma_split(a);
  split_place(s, a.ws);
  cudaError_t e = by_type(a, [&](auto shape) { return launch_of(shape, a, s); });
  return e != cudaSuccess ? e : launch_attn_join(a, s);
}

}  // namespace attn
}  // namespace kda
