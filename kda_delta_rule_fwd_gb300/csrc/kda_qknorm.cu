// Norms of queries and keys per head with the position's rotation, and their gradient.
//
//     n = x k w,  k = 1 / sqrt(mean(x^2) + eps);   (a, b) -> (a cos f - b sin f, a sin f + b cos f)
//     backward:  g = the rotation by -f of dy,  dw = sum of g x k,  p = g w,
//                dx = k (p - n0 mean(p n0)),  n0 = x k      (dx = g without a weight)
//
// Angles.  f / 2 pi per position is a fraction of a turn in 64-bit fixed point, and position
// times it modulo 2^64 is the place on the circle: whole turns fall off the top, exactly, for
// positions of either sign, and half a unit of the fraction times 2^31 is 2^-34 of a turn.  The top 32
// bits then go to sincospi.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

using layer::Raw;
using layer::dot_v;
using layer::fma_v;
using layer::mul_v;
using layer::open;
using layer::store;

using u64 = unsigned long long;

// freq / 2 pi in 64-bit fixed point, modulo 1, to the nearest: the mantissa times 2^130 / 2 pi (128 bits) in 192
// bits, moved by the exponent (whole numbers: 64 float64 operations of every thread would take 10 us).
// With only the upper 64 bits of 2^130 / 2 pi a frequency of 2^20 was 2^-48 of a turn off.
__device__ __forceinline__ u64 turn_of(double freq) {
  const u64 bits = (u64)__double_as_longlong(freq), m = (bits & 0xfffffffffffffull) | 1ull << 52;
  constexpr u64 hi = 0xa2f9836e4e441529ull, lo = 0xfc2757d1f534ddc1ull;
  const u64 p1 = __umul64hi(m, lo) + m * hi;                     // the product's second word
  const u64 p2 = __umul64hi(m, hi) + (p1 < m * hi ? 1 : 0);      // and its third
  const int r = max(1077 - (int)(bits >> 52 & 0x7ff), 34);       // whole turns lie above bit 64 + r; 34: 2^20
  u64 t = 0, half = 0;
  if (r < 64) {
    t = p2 << (64 - r) | p1 >> r;
    half = p1 >> (r - 1) & 1;
  } else if (r < 128) {
    t = p2 >> (r - 64);
    half = (r == 64 ? p1 >> 63 : p2 >> (r - 65)) & 1;
  }
  t += half;
  return bits >> 63 ? 0 - t : t;
}
__device__ __forceinline__ float2 angle(u64 turn, int pos) {  // (cos, sin)
  const u64 f = turn * (u64)(long long)pos;
  float2 r;
  sincospif((float)(int)(f >> 32) * 4.656612873077392578125e-10f, &r.y, &r.x);  // half turns
  return r;
}

// The two channels of pair j; behind the rotated ones adjacent channels make pairs that stay.
__device__ __forceinline__ int2 pair_at(const QKArgs& a, int j) {
  const int half = a.rot / 2;
  if (j < half && !a.interleaved) return make_int2(j, j + half);
  return make_int2(2 * j, 2 * j + 1);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kNarrowWarps = 4, kPairs = 4;  // up to 256 channels: 4 pairs per lane

// Any alignment, stride and size: a warp per row, a pair of single channels per lane and load.
template <typename T, bool kBwd>
__global__ void __launch_bounds__(32 * kNarrowWarps) qknorm_narrow_kernel(QKArgs a) {
  const QKPart& p = a.p[blockIdx.y];
  if ((int)blockIdx.x >= p.ctas) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = a.tokens * p.heads, step = (int64_t)p.ctas * kNarrowWarps;
  const int pairs = a.d / 2, half = a.rot / 2;
  int2 at[kPairs];
  u64 turn[kPairs];
  float2 w[kPairs], dw[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int j = lane + 32 * i;
    at[i] = pair_at(a, j);
    turn[i] = j < half ? turn_of(a.freqs[j]) : 0;
    w[i] = p.w && j < pairs ? make_float2(p.w[at[i].x], p.w[at[i].y]) : make_float2(1.f, 1.f);
    dw[i] = make_float2(0.f, 0.f);
  }
  for (int64_t row = (int64_t)blockIdx.x * kNarrowWarps + warp; row < rows; row += step) {
    const int64_t tok = row / p.heads;
    const T* x = static_cast<const T*>(p.x) + tok * p.ld + (row - tok * p.heads) * a.d;
    const int pos = a.rot ? a.pos[tok] : 0;
    float2 v[kPairs], g[kPairs];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      v[i] = g[i] = make_float2(0.f, 0.f);
      if (lane + 32 * i < pairs) {
        v[i] = make_float2(to_f32(x[at[i].x]), to_f32(x[at[i].y]));
        if (kBwd) {
          const T* dy = static_cast<const T*>(p.dy) + row * a.d;
          g[i] = make_float2(to_f32(dy[at[i].x]), to_f32(dy[at[i].y]));
        }
      }
      ss = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, ss));
    }
    const float k = p.w ? rsqrtf(fmaf(warp_sum(ss), a.inv_d, a.eps)) : 1.f;
    float pn = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 cs = lane + 32 * i < half ? angle(turn[i], pos) : make_float2(1.f, 0.f);
      v[i].x *= k;
      v[i].y *= k;
      if (kBwd) {
        const float ga = g[i].x * cs.x + g[i].y * cs.y, gb = g[i].y * cs.x - g[i].x * cs.y;
        dw[i].x = fmaf(ga, v[i].x, dw[i].x);
        dw[i].y = fmaf(gb, v[i].y, dw[i].y);
        g[i] = make_float2(ga * w[i].x, gb * w[i].y);
        pn = fmaf(g[i].x, v[i].x, fmaf(g[i].y, v[i].y, pn));
      } else {
        const float na = v[i].x * w[i].x, nb = v[i].y * w[i].y;
        v[i] = make_float2(na * cs.x - nb * cs.y, na * cs.y + nb * cs.x);
      }
    }
    if (kBwd && p.w) {
      const float mean = warp_sum(pn) * a.inv_d;
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        g[i] = make_float2(k * (g[i].x - v[i].x * mean), k * (g[i].y - v[i].y * mean));
    }
    T* y = static_cast<T*>(kBwd ? p.dx : p.y) + row * a.d;
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (lane + 32 * i < pairs) {
        y[at[i].x] = from_f32<T>(kBwd ? g[i].x : v[i].x);
        y[at[i].y] = from_f32<T>(kBwd ? g[i].y : v[i].y);
      }
  }
  if (!kBwd || !p.dw) return;
  __shared__ float fold[kNarrowWarps][256];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    if (lane + 32 * i < pairs) {
      fold[warp][at[i].x] = dw[i].x;
      fold[warp][at[i].y] = dw[i].y;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kNarrowWarps; ++q) s += fold[q][c];
    p.part[(int64_t)blockIdx.x * a.d + c] = s;
  }
}

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(void* dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(have ? 16 : 0) : "memory");
}

// Aligned rows: TPR threads hold a row in two chunks of 16 bytes each, chosen so that both members
// of a pair are in one thread (chunk c and c + rot / 2 of halves, adjacent channels of one chunk),
// and nothing but the row's sum leaves a thread.  A group of TPR threads takes a token's heads (or
// `per` of them, where tokens are few): the angles are made once for them.  Blocks are persistent
// and request the next row before they work on the present one; a block serves q or k, in
// proportion to their heads, so that its weights and its sums for their gradient stay in registers.
constexpr int kWide = 256;  // threads of a block
// Blocks to an SM and rows in flight.  16384 tokens of 40 heads of 128 in bf16 took 66 us forwards (with
// four rows 70, with four blocks 99: too few registers), their gradient 97 (two or three rows 99), before
// the items were made equal; they take 64 and 91, bound by memory: a copy of as many bytes takes 60 and
// 85, and without the rotation, the angles or most of the sum the forward kernel takes 65.
template <bool kBwd> constexpr int wide_blocks() { return kBwd ? 2 : 3; }
template <bool kBwd> constexpr int wide_ahead() { return kBwd ? 4 : 3; }

template <typename T, int TPR, bool kInter, bool kBwd>
__global__ void __launch_bounds__(kWide, wide_blocks<kBwd>()) qknorm_wide_kernel(QKArgs a, int2 per_of) {
  constexpr int VEC = 16 / sizeof(T), kGroups = kWide / TPR;
  constexpr int kAhead = wide_ahead<kBwd>(), kWords = kBwd ? 4 : 2;  // 16-byte words of a thread's row
  extern __shared__ uint4 ring[];  // [kAhead][kWords][kWide]: each thread copies what it reads itself
  __shared__ u64 turns[128];
  const bool second = (int)blockIdx.x >= a.p[0].ctas;
  const QKPart& p = a.p[second];
  const int block = blockIdx.x - (second ? a.p[0].ctas : 0);
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int chunks = a.d / VEC, half = a.rot / 2, per = second ? per_of.y : per_of.x;
  for (int j = threadIdx.x; j < half; j += kWide) turns[j] = turn_of(a.freqs[j]);
  __syncthreads();
  // the thread's chunks: channels at[0] .. and at[1] .., -1 behind the row's end; its first pairs
  int at[2];
  bool turned = true;  // halves: whether the chunks are each other's partners
  if (kInter) {
    const int width = (chunks + 1) / 2;
    at[0] = lane < width ? lane * VEC : -1;
    at[1] = lane < width && lane + width < chunks ? (lane + width) * VEC : -1;
  } else {
    const int both = half / VEC, i = lane - both;
    turned = i < 0;
    const int c = turned ? lane : 2 * both + 2 * i;
    at[0] = c < chunks ? c * VEC : -1;
    at[1] = turned ? (lane + both) * VEC : c + 1 < chunks ? (c + 1) * VEC : -1;
  }
  const auto weight = [&](int i, int e) { return p.w && at[i] >= 0 ? p.w[at[i] + e] : 1.f; };
  float w[2][VEC], sum[2][VEC];  // the backward's
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = kBwd ? weight(i, e) : 1.f;
      sum[i][e] = 0.f;
    }
  // items (token, heads [c per, c per + per)) of this group; all groups of a warp run as often as
  // its first
  const int parts = (p.heads + per - 1) / per;
  const int64_t items = a.tokens * parts, step = (int64_t)p.ctas * kGroups;
  int64_t item = (int64_t)block * kGroups + group;
  int64_t first = (int64_t)block * kGroups + threadIdx.x / 32 * (32 / TPR);
  struct Place {
    const T *x, *dy;  // the item's first row
    int64_t row;      // its place among the dense rows
    int rows, tok_pos;
  };
  const auto locate = [&](int64_t it) {
    Place l{nullptr, nullptr, 0, 0, 0};
    if (it < items) {
      const int64_t tok = parts == 1 ? it : it / parts;
      const int head = (int)(it - tok * parts) * per;
      l.row = tok * p.heads + head;
      l.x = static_cast<const T*>(p.x) + tok * p.ld + head * a.d;
      if (kBwd) l.dy = static_cast<const T*>(p.dy) + l.row * a.d;
      l.rows = min(per, p.heads - head);
      l.tok_pos = half ? a.pos[tok] : 0;
    }
    return l;
  };
  // the next row to request: head `req_h` of the item at `req`
  Place req = locate(item);
  int64_t req_item = item;
  int req_h = 0;
  const auto request = [&](int slot) {
    const bool on = req_h < req.rows;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4* const to = ring + (slot * kWords + i) * kWide + threadIdx.x;
      const bool have = on && at[i] >= 0;
      copy16(to, have ? req.x + req_h * a.d + at[i] : static_cast<const T*>(p.x), have);
      if (kBwd) copy16(to + 2 * kWide, have ? req.dy + req_h * a.d + at[i] : static_cast<const T*>(p.dy), have);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++req_h == per) {
      req_h = 0;
      req_item += step;
      req = locate(req_item);
    }
  };
  Place now = req;
#pragma unroll
  for (int d = 0; d < kAhead; ++d) request(d);
  int h = 0, slot = 0;
  // A pair's rotation (a, b) -> (f0 a + f1 b, f2 a + f3 b), with the weights in it forwards and turned
  // back backwards; halves: pair e of the thread, adjacent: of the two chunks' pairs in a row.
  float f0[VEC], f1[VEC], f2[VEC], f3[VEC];
  while (first < items) {
    if (h == 0) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = e < VEC / 2 ? at[0] + 2 * e : at[1] + 2 * e - VEC;
        const int j = kInter ? c >> 1 : at[0] + e;
        const bool turn = kInter ? (e < VEC / 2 ? at[0] : at[1]) >= 0 && j < half : turned && j < half;
        const float2 r = turn ? angle(turns[j], now.tok_pos) : make_float2(1.f, 0.f);
        const int ia = kInter ? e / (VEC / 2) : 0, ea = kInter ? e % (VEC / 2) * 2 : e;
        const int ib = kInter ? ia : 1, eb = kInter ? ea + 1 : e;
        const float wa = kBwd ? 1.f : weight(ia, ea), wb = kBwd ? 1.f : weight(ib, eb);
        const float sine = kBwd ? -r.y : r.y;
        f0[e] = wa * r.x;
        f1[e] = -wb * sine;
        f2[e] = wa * sine;
        if (!kBwd) f3[e] = wb * r.x;  // backwards it is f0
      }
    }
    float v[2][VEC], g[2][VEC];
    const bool here = h < now.rows;
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4* const from = ring + (slot * kWords + i) * kWide + threadIdx.x;
      open<T, VEC>(*reinterpret_cast<const Raw<T, VEC>*>(from), v[i]);
      if (kBwd) open<T, VEC>(*reinterpret_cast<const Raw<T, VEC>*>(from + 2 * kWide), g[i]);
    }
    request(slot);
    slot = slot + 1 == kAhead ? 0 : slot + 1;
    float k = 1.f;
    if (p.w) {
      float2 ss = make_float2(0.f, 0.f);
      dot_v(v[0], v[0], ss);
      dot_v(v[1], v[1], ss);
      float s = ss.x + ss.y;
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      k = here ? rsqrtf(fmaf(s, a.inv_d, a.eps)) : 0.f;
    }
    const auto turn_pairs = [&](float (&y)[2][VEC]) {
      if constexpr (kInter) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float &u = y[e / (VEC / 2)][e % (VEC / 2) * 2], &t = y[e / (VEC / 2)][e % (VEC / 2) * 2 + 1];
          const float x0 = fmaf(t, f1[e], u * f0[e]), x1 = fmaf(t, kBwd ? f0[e] : f3[e], u * f2[e]);
          u = x0;
          t = x1;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 u = make_float2(y[0][e], y[0][e + 1]), t = make_float2(y[1][e], y[1][e + 1]);
          const float2 x0 = fma2(t, make_float2(f1[e], f1[e + 1]), mul2(u, make_float2(f0[e], f0[e + 1])));
          const float2 last = kBwd ? make_float2(f0[e], f0[e + 1]) : make_float2(f3[e], f3[e + 1]);
          const float2 x1 = fma2(t, last, mul2(u, make_float2(f2[e], f2[e + 1])));
          y[0][e] = x0.x;
          y[0][e + 1] = x0.y;
          y[1][e] = x1.x;
          y[1][e + 1] = x1.y;
        }
      }
    };
    if constexpr (!kBwd) {
      turn_pairs(v);
      mul_v(v[0], k);
      mul_v(v[1], k);
    } else {
      turn_pairs(g);
      if (p.w) {  // with g k for g: the weights' sums, then dx = g k w - x k^2 mean(g k w x)
        mul_v(g[0], k);
        mul_v(g[1], k);
        fma_v(g[0], v[0], sum[0]);
        fma_v(g[1], v[1], sum[1]);
        mul_v(g[0], w[0]);
        mul_v(g[1], w[1]);
        float2 pn = make_float2(0.f, 0.f);
        dot_v(g[0], v[0], pn);
        dot_v(g[1], v[1], pn);
        float s = pn.x + pn.y;
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        float back = -s * a.inv_d * k;
        if (k > 0x1p60f) {  // rows near float32's smallest, with eps as small: k^2 would not do
          mul_v(v[0], k);
          mul_v(v[1], k);
        } else {
          back *= k;
        }
        fma_v(v[0], back, g[0]);
        fma_v(v[1], back, g[1]);
      }
    }
    if (here) {
      T* y = static_cast<T*>(kBwd ? p.dx : p.y) + (now.row + h) * a.d;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (at[i] >= 0) store<VEC>(y + at[i], kBwd ? g[i] : v[i]);
    }
    if (++h == per) {
      h = 0;
      first += step;
      item += step;
      now = locate(item);
    }
  }
  if (!kBwd || !p.dw) return;
  static_assert(kAhead * kWords * 16 >= 2 * VEC * 4, "room for the sums");
  float* const fold = reinterpret_cast<float*>(ring);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at[i] >= 0) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) fold[group * a.d + at[i] + e] = sum[i][e];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kWide) {
    float s = 0.f;
    for (int q = 0; q < kGroups; ++q) s += fold[q * a.d + c];
    p.part[(int64_t)block * a.d + c] = s;
  }
}

// The weights' gradients: 32 columns per block, whose warps take every 32nd block's sums.
__global__ void __launch_bounds__(1024) qknorm_reduce_kernel(QKArgs a) {
  __shared__ float fold[32][33];
  const QKPart& p = a.p[blockIdx.y];
  if (!p.dw) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.d)
    for (int b = warp; b < p.ctas; b += 32) s += p.part[(int64_t)b * a.d + c];
  fold[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s += fold[q][lane];
    p.dw[c] = s;
  }
}

constexpr int kPerSm = 4;  // blocks of a part, at most

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }
// whole 16-byte chunks everywhere, and no chunk that is rotated in part
bool wide_ok(const QKArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  bool ok = a.d % v == 0 && (a.interleaved || a.rot / 2 % v == 0);
  for (const QKPart& p : a.p)
    ok = ok && (p.heads == 0 || (p.ld % v == 0 && al16(p.x) && al16(p.dy) && al16(p.y) && al16(p.dx)));
  return ok;
}

template <typename T, int TPR, bool kInter, bool kBwd>
void launch_wide(QKArgs& a) {
  constexpr int kGroups = kWide / TPR;
  const int64_t most = a.sms * wide_blocks<kBwd>();
  // a token's angles take about as long as two of its heads
  const int heads = a.p[0].heads + (a.p[1].heads ? a.p[1].heads + 4 : 2);
  int per[2] = {1, 1};
  for (int i = 0; i < 2; ++i) {
    QKPart& p = a.p[i];
    p.ctas = 0;
    if (p.heads == 0) continue;
    int64_t share = (most * (p.heads + 2) + heads / 2) / heads;
    if (share < 1) share = 1;
    // A token's heads in equal items: many even the groups' work out (a group takes whole ones),
    // each makes the angles again.
    const int64_t groups = share * kGroups;
    int64_t best = INT64_MAX, items = a.tokens * p.heads;  // a head each where the groups suffice
    const bool few = items <= groups;
    for (int parts = 1; !few && parts <= p.heads && parts <= 64; ++parts) {
      const int n = (p.heads + parts - 1) / parts;
      const int64_t all = a.tokens * ((p.heads + n - 1) / n), cost = (all + groups - 1) / groups * (n + 2);
      if (cost < best) {
        best = cost;
        per[i] = n;
        items = all;
      }
    }
    const int64_t need = (items + kGroups - 1) / kGroups;
    const int64_t limit = qknorm_bwd_ctas(a.tokens, p.heads, a.sms);
    p.ctas = (int)(need < share ? need : share);
    if (p.ctas > limit) p.ctas = (int)limit;
  }
  const int grid = a.p[0].ctas + a.p[1].ctas;
  if (grid == 0) return;
  constexpr int bytes = wide_ahead<kBwd>() * (kBwd ? 4 : 2) * kWide * 16;
  if (bytes > 40 * 1024)  // with the table more than a block gets unasked
    cudaFuncSetAttribute(qknorm_wide_kernel<T, TPR, kInter, kBwd>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  qknorm_wide_kernel<T, TPR, kInter, kBwd><<<grid, kWide, bytes, a.stream>>>(a, make_int2(per[0], per[1]));
}
template <typename T, int TPR>
void by_kind(QKArgs& a, bool bwd) {
  if (a.interleaved) bwd ? launch_wide<T, TPR, true, true>(a) : launch_wide<T, TPR, true, false>(a);
  else bwd ? launch_wide<T, TPR, false, true>(a) : launch_wide<T, TPR, false, false>(a);
}
template <typename T>
void by_size(QKArgs& a, bool bwd) {
  const int chunks = a.d * (int)sizeof(T) / 16;
  // threads of a row: pairs of chunks, those left over behind the rotated ones two by two
  const int lanes = (chunks + 1) / 2;
  if (lanes <= 4) return by_kind<T, 4>(a, bwd);
  if (lanes <= 8) return by_kind<T, 8>(a, bwd);
  if (lanes <= 16) return by_kind<T, 16>(a, bwd);
  by_kind<T, 32>(a, bwd);
}

cudaError_t run(QKArgs& a, bool bwd) {
  using bf = __nv_bfloat16;
  if (wide_ok(a)) {
    a.bf16 ? by_size<bf>(a, bwd) : by_size<float>(a, bwd);
    return cudaGetLastError();
  }
  int most = 0;
  for (QKPart& p : a.p) {
    p.ctas = (int)qknorm_bwd_ctas(a.tokens, p.heads, a.sms);
    most = p.ctas > most ? p.ctas : most;
  }
  if (most == 0) return cudaSuccess;
  const dim3 grid(most, a.p[1].heads > 0 ? 2 : 1), block(32 * kNarrowWarps);
  if (bwd)
    a.bf16 ? qknorm_narrow_kernel<bf, true><<<grid, block, 0, a.stream>>>(a)
           : qknorm_narrow_kernel<float, true><<<grid, block, 0, a.stream>>>(a);
  else
    a.bf16 ? qknorm_narrow_kernel<bf, false><<<grid, block, 0, a.stream>>>(a)
           : qknorm_narrow_kernel<float, false><<<grid, block, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

int64_t qknorm_bwd_ctas(int64_t tokens, int heads, int64_t sms) {
  const int64_t blocks = (tokens * heads + kNarrowWarps - 1) / kNarrowWarps, most = kPerSm * sms;
  return blocks < most ? blocks : most;
}

cudaError_t launch_qknorm_fwd(QKArgs a) { return run(a, false); }

cudaError_t launch_qknorm_bwd(QKArgs a) {
  cudaError_t e = run(a, true);
  if (e != cudaSuccess || (!a.p[0].dw && !a.p[1].dw)) return e;
  qknorm_reduce_kernel<<<dim3((a.d + 31) / 32, 2), 1024, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
