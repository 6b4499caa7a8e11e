// The paged key-value cache: rows written as given or as 8-bit codes with a power of two per
// row, and read back.
//
// Codes.  The row's power 2^e is the smallest with max |x| <= top 2^e (top = 448 or 127), read
// off the exponent and mantissa of the largest magnitude; x 2^-e is exact, so that one rounding
// (to nearest, ties to even) gives the code.  Magnitudes are compared as integers, which puts
// NaN above infinity above every number: a row with either is told by its maximum.
//
// Both directions move each value once and are bound by memory traffic.  A block takes the rows
// (heads, keys and values) of a few consecutive tokens: their places are looked up once, then
// d / 16 lanes move a row, twice 8 channels each.
#include <type_traits>

#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

using namespace layer;

constexpr int kThreads = 256, kMaxTile = 16;  // kMaxTile: tokens of a block

// Places of the tile's tokens: the page and the row in it, page -1 for a token without a place
// and -2 for one of no sequence (behind the last).
// (One warp: each step of the search for the first token's sequence looks at 32 offsets at once.)
__device__ __forceinline__ int find_seq(const Seqs& q, int64_t t) {
  if (!q.cu) return (int)(t / q.T);
  const int lane = threadIdx.x & 31;
  int lo = 0, n = q.N;  // the last of [lo, lo + n) that begins at t or before (or lo)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && (int64_t)q.cu[at] <= t);
    const int i = le ? 31 - __clz(le) : 0;
    n = min(step, n - i * step);
    lo += i * step;
  }
  return lo;
}
__device__ __forceinline__ void find_places(const CacheArgs& a, int64_t t0, int tile, int2* place) {
  const int i = threadIdx.x;
  if (i < 32) {
    int n = find_seq(a.q, t0);
    int2 r = make_int2(-2, 0);
    const int64_t t = t0 + i;
    if (i < tile && t < a.q.total) {
      if (!a.q.cu) n = (int)(t / a.q.T);
      else while (n + 1 < a.q.N && (int64_t)a.q.cu[n + 1] <= t) ++n;
      int64_t start, end;
      a.q.range(n, start, end);
      if (t >= start && t < end) {
        const int64_t pos = (int64_t)a.t.lens[n] - (end - t);
        r.x = -1;
        if (pos >= 0) {
          r.x = page_of(a.t, n, pos);
          r.y = (int)(pos & ((1 << a.t.shift) - 1));
          if (r.x < 0) latch_status(a.status, KDA_ERR_INVALID_ARG);
        }
      }
    }
    if (i < tile) place[i] = r;
  }
  // one block looks over the offsets
  if (blockIdx.x == 0 && a.status && a.q.cu)
    for (int n = threadIdx.x; n <= a.q.N; n += blockDim.x) {
      const int64_t v = a.q.cu[n];
      if ((n == 0 && v != 0) || (n == a.q.N && v != a.q.total) || (n > 0 && v < a.q.cu[n - 1]))
        latch_status(a.status, KDA_ERR_BAD_SEQLENS);
    }
  __syncthreads();
}

// 8 values as a cache row's codes, rounded to nearest, ties to even
template <int CACHE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t b[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = x[2 * i] * inv, hi = x[2 * i + 1] * inv;
    uint32_t two;
    if constexpr (CACHE == KDA_CACHE_E4M3) {
      uint16_t h;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
      two = h;
    } else {
      two = (uint32_t)(__float2int_rn(lo) & 0xff) | (uint32_t)(__float2int_rn(hi) & 0xff) << 8;
    }
    b[i / 2] |= two << (16 * (i & 1));
  }
  return make_uint2(b[0], b[1]);
}
template <int CACHE>
__device__ __forceinline__ void decode8(uint2 v, float scale, float (&x)[8]) {
  const uint32_t b[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t h = (uint16_t)(b[i / 2] >> (16 * (i & 1)));
    if constexpr (CACHE == KDA_CACHE_E4M3) {
      uint32_t f;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f));
      x[2 * i] = g.x * scale;
      x[2 * i + 1] = g.y * scale;
    } else {
      x[2 * i] = (float)(int8_t)(h & 0xff) * scale;
      x[2 * i + 1] = (float)(int8_t)(h >> 8) * scale;
    }
  }
}

template <typename T, bool kWide>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (kWide) {
    store<8>(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = from_f32<T>(x[e]);
  }
}

// A lane's two runs of 8 values of a row (of 8 L channels each) as they lie in memory, held while in
// flight
template <typename T, bool kWide> struct Held { layer::Raw<T, 8> v[2]; };
template <typename T> struct Held<T, false> { T v[2][8]; };
template <typename T, bool kWide>
__device__ __forceinline__ void fetch16(const T* p, int apart, Held<T, kWide>& h) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (kWide) {
      h.v[k] = fetch<T, 8>(p + k * apart);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h.v[k][e] = p[k * apart + e];
    }
  }
}
template <typename T, bool kWide>
__device__ __forceinline__ void open8(const Held<T, kWide>& h, int k, float (&x)[8]) {
  if constexpr (kWide) {
    open<T, 8>(h.v[k], x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f32(h.v[k][e]);
  }
}
// the largest magnitude of a row's L lanes as float32 bits; of bf16 pairs two to an instruction
template <int L, typename T, bool kWide>
__device__ __forceinline__ uint32_t peak(const Held<T, kWide>& h, unsigned mask) {
  uint32_t m = 0;
  if constexpr (kWide && sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 w = h.v[k].v;
      m = __vmaxu2(m, w.x & 0x7fff7fffu);
      m = __vmaxu2(m, w.y & 0x7fff7fffu);
      m = __vmaxu2(m, w.z & 0x7fff7fffu);
      m = __vmaxu2(m, w.w & 0x7fff7fffu);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(mask, m, o));
    return max(m << 16, m & 0xffff0000u);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x[8];
      open8<T, kWide>(h, k, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
    return m;
  }
}

// A group of L = D / 16 lanes takes one head (of keys or of values) of the tile's tokens, some of
// them in flight; groups that outnumber the heads share a head's tokens.
template <int D, class F>
__device__ __forceinline__ void each_head(const CacheArgs& a, F f) {
  constexpr int kGroups = kThreads / (D / 16);
  const int group = threadIdx.x / (D / 16), heads = 2 * a.heads;
  if (heads >= kGroups) {
    for (int r = group; r < heads; r += kGroups) f(r >= a.heads, r >= a.heads ? r - a.heads : r, 0, 1);
  } else {
    const int ways = kGroups / heads, r = group % heads, way = group / heads;
    if (way < ways) f(r >= a.heads, r >= a.heads ? r - a.heads : r, way, ways);
  }
}
// Rows in flight of values of `size` bytes, and blocks to an SM.  58511 tokens of 8 heads of 128 in
// e4m3, written and read back, take 122 us with 4 rows and 3 blocks, 131 with 2 and 4, 122 with 2 and 6.
constexpr int ahead(int size) { return size == 4 ? 2 : 4; }
constexpr int kPerSm = 3;

template <typename T, int CACHE, int D, bool kWide>
__global__ void __launch_bounds__(kThreads, kPerSm) cache_write_kernel(CacheArgs a, int tile) {
  constexpr int L = D / 16, kAhead = ahead(sizeof(T));  // L: lanes of a row
  __shared__ int2 place[kMaxTile];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  find_places(a, t0, tile, place);
  const int lane = threadIdx.x % L;
  // the lanes of a row leave and stay together
  const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1) << (threadIdx.x & 31 & ~(L - 1));
  each_head<D>(a, [&](bool kv, int h, int first, int step) {
    const int64_t ld = kv ? a.ldv : a.ldk;
    const T* src = static_cast<const T*>(kv ? a.v : a.k) + t0 * ld + (int64_t)h * D + lane * 8;
    void* const pool = kv ? a.vc : a.kc;
    for (int base = first; base < tile; base += step * kAhead) {
      Held<T, kWide> held[kAhead];
      int2 at[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = base + k * step;
        at[k] = i < tile ? place[i] : make_int2(-2, 0);
        if (at[k].x >= 0) fetch16<T, kWide>(src + i * ld, 8 * L, held[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (at[k].x < 0) continue;  // the same for all lanes of the row
        const int64_t row = ((int64_t)h << a.t.shift) + at[k].y;
        const int64_t to = at[k].x * a.ldpage + row * D + lane * 8;
        if constexpr (CACHE == KDA_CACHE_F32 || CACHE == KDA_CACHE_BF16) {
          using TC = std::conditional_t<CACHE == KDA_CACHE_F32, float, __nv_bfloat16>;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x[8];
            open8<T, kWide>(held[k], r, x);
            store<8>(static_cast<TC*>(pool) + to + r * 8 * L, x);
          }
        } else {
          const uint32_t m = peak<L, T, kWide>(held[k], mask);
          // 448 = 1.75 2^8, 127 = 1.984375 2^6
          constexpr uint32_t top = CACHE == KDA_CACHE_E4M3 ? 0x600000u : 0x7e0000u;
          int e = (int)(m >> 23) - 127 - (CACHE == KDA_CACHE_E4M3 ? 8 : 6) + ((m & 0x7fffffu) > top);
          e = max(e, -126);
          const bool finite = m < 0x7f800000u;
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x[8];
            open8<T, kWide>(held[k], r, x);
            uint2 code = encode8<CACHE>(x, inv);
            if (!finite) code = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + to + r * 8 * L) = code;
          }
          if (lane == 0)
            (kv ? a.vs : a.ks)[(((int64_t)at[k].x * a.heads) << a.t.shift) + row] = finite ? (uint8_t)(e + 127) : 255;
        }
      }
    }
  });
}

// 8 codes or values of a cache row
template <int CACHE> struct Row8 { uint2 v; };
template <> struct Row8<KDA_CACHE_F32> { layer::Raw<float, 8> v; };
template <> struct Row8<KDA_CACHE_BF16> { layer::Raw<__nv_bfloat16, 8> v; };

template <typename T, int CACHE, int D, bool kWide>
__global__ void __launch_bounds__(kThreads, kPerSm) cache_read_kernel(CacheArgs a, int tile) {
  constexpr int L = D / 16;
  constexpr bool kCoded = CACHE == KDA_CACHE_E4M3 || CACHE == KDA_CACHE_INT8;
  constexpr int kElem = CACHE == KDA_CACHE_F32 ? 4 : CACHE == KDA_CACHE_BF16 ? 2 : 1, kAhead = ahead(kElem);
  __shared__ int2 place[kMaxTile];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  find_places(a, t0, tile, place);
  const int lane = threadIdx.x % L;
  each_head<D>(a, [&](bool kv, int h, int first, int step) {
    T* const out = static_cast<T*>(kv ? a.vo : a.ko);
    if (!out) return;
    const char* const pool = static_cast<const char*>(kv ? a.vc : a.kc);
    for (int base = first; base < tile; base += step * kAhead) {
      Row8<CACHE> held[kAhead][2];
      uint8_t byte[kAhead];
      int2 at[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = base + k * step;
        at[k] = i < tile ? place[i] : make_int2(-2, 0);
        if (at[k].x >= 0) {
          const int64_t row = ((int64_t)h << a.t.shift) + at[k].y;
          const char* from = pool + (at[k].x * a.ldpage + row * D + lane * 8) * kElem;
          held[k][0] = *reinterpret_cast<const Row8<CACHE>*>(from);
          held[k][1] = *reinterpret_cast<const Row8<CACHE>*>(from + 8 * L * kElem);
          if (kCoded) byte[k] = (kv ? a.vs : a.ks)[(((int64_t)at[k].x * a.heads) << a.t.shift) + row];
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (at[k].x == -2) continue;
        const float p = kCoded && at[k].x >= 0 ? power(byte[k]) : 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
          if (at[k].x >= 0) {
            if constexpr (CACHE == KDA_CACHE_F32) open<float, 8>(held[k][r].v, x);
            else if constexpr (CACHE == KDA_CACHE_BF16) open<__nv_bfloat16, 8>(held[k][r].v, x);
            else decode8<CACHE>(held[k][r].v, p, x);
          }
          store8<T, kWide>(out + ((t0 + base + k * step) * a.heads + h) * D + lane * 8 + r * 8 * L, x);
        }
      }
    }
  });
}

template <typename T, int CACHE, int D, bool kWide>
void launch(const CacheArgs& a, bool write) {
  // few tokens: fewer of them per block, so that the device is filled
  int tile = kMaxTile;
  while (tile > 1 && a.q.total < 2 * tile * a.sms) tile /= 2;
  const unsigned grid = (unsigned)((a.q.total + tile - 1) / tile);
  if (write) cache_write_kernel<T, CACHE, D, kWide><<<grid, kThreads, 0, a.stream>>>(a, tile);
  else cache_read_kernel<T, CACHE, D, kWide><<<grid, kThreads, 0, a.stream>>>(a, tile);
}
template <typename T, int CACHE>
void by_size(const CacheArgs& a, bool write, bool wide) {
  if (a.d == 128) wide ? launch<T, CACHE, 128, true>(a, write) : launch<T, CACHE, 128, false>(a, write);
  else wide ? launch<T, CACHE, 64, true>(a, write) : launch<T, CACHE, 64, false>(a, write);
}
template <typename T>
void by_cache(const CacheArgs& a, bool write, bool wide) {
  switch (a.cache) {
    case KDA_CACHE_F32: return by_size<T, KDA_CACHE_F32>(a, write, wide);
    case KDA_CACHE_BF16: return by_size<T, KDA_CACHE_BF16>(a, write, wide);
    case KDA_CACHE_E4M3: return by_size<T, KDA_CACHE_E4M3>(a, write, wide);
    default: return by_size<T, KDA_CACHE_INT8>(a, write, wide);
  }
}
cudaError_t run(const CacheArgs& a, bool write, bool wide) {
  if (a.q.total == 0) return cudaSuccess;
  if (a.bf16) by_cache<__nv_bfloat16>(a, write, wide);
  else by_cache<float>(a, write, wide);
  return cudaGetLastError();
}
bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace

cudaError_t launch_cache_write(const CacheArgs& a) {
  const int64_t v = a.bf16 ? 8 : 4;
  return run(a, true, al16(a.k) && al16(a.v) && a.ldk % v == 0 && a.ldv % v == 0);
}
cudaError_t launch_cache_read(const CacheArgs& a) { return run(a, false, al16(a.ko) && al16(a.vo)); }

}  // namespace attn
}  // namespace kda
