// Attention of new tokens over the paged cache, float32 queries: float32 arithmetic on the CUDA
// cores; and the join of the parts.
//
// One pass over the keys with the running maximum and sum: a tile of 64 places is brought to
// shared memory as float32, each thread forms the scores of one place with 8 query rows, a warp
// takes 4 rows' maxima and weights, then each thread adds up one channel of all rows.  Scores
// count in units of log 2.  The power of two of a key's codes multiplies its score, that of a
// value its weight.  A place that a row does not see has no part in its sums: its score is
// replaced (not added to), and where its weight is 0 its value is not multiplied.
#include "kda_attn_split.cuh"

namespace kda {
namespace attn {
namespace {

using namespace layer;

constexpr int kThreads = 128, kRows = 16, kTile = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename TC> __device__ __forceinline__ void load4(const TC* p, float (&x)[4]);
template <> __device__ __forceinline__ void load4(const float* p, float (&x)[4]) { load<4>(p, x); }
struct E4M3 { uint8_t v; };
struct Int8 { int8_t v; };
template <> __device__ __forceinline__ void load4(const E4M3* p, float (&x)[4]) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(u >> (16 * i))));
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f));
    x[2 * i] = g.x;
    x[2 * i + 1] = g.y;
  }
}
template <> __device__ __forceinline__ void load4(const Int8* p, float (&x)[4]) {
  const char4 u = *reinterpret_cast<const char4*>(p);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}

template <int D> struct Shared {
  float q[kRows][D];
  float k[kTile][D + 4];
  float v[kTile][D];
  float p[kRows][kTile];
  float ks[kTile], vs[kTile];
  float m[kRows], l[kRows], alpha[kRows];
  int64_t scratch[34];
  int seen[kTile];  // the place lies in the sequence and on a page of the pool
  int bad;
};

template <typename TC, int D>
__global__ void __launch_bounds__(kThreads) attn_kernel(AttnArgs a, Split s) {
  constexpr bool kCoded = sizeof(TC) == 1;
  constexpr int kGroups = kThreads / D;       // threads of a channel
  constexpr int kOwn = kRows / kGroups;       // rows of a thread in the second product
  extern __shared__ __align__(16) char raw[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sh.bad = 0;
    s.cut[blockIdx.x] = -1;
  }
  Start st;
  const bool work = find_start<kThreads>(a, s, sh.scratch, st);
  const int64_t each = (int64_t)a.hk * s.chunks;
  const int64_t cap = (int64_t)a.t.max_pages << a.t.shift;
  int n = work ? st.n : 0;
  int64_t before = work ? st.before : 0;
  for (int64_t at = work ? st.at : 0; work && at < st.end;) {
    const Keys keys = keys_of(a, s.tile, n);
    const int64_t j = (at - before * each) / (keys.tiles + s.cost);       // head and chunk
    const int64_t item_at = before * each + j * (keys.tiles + s.cost);
    const int64_t tile_at = item_at + s.cost;                             // the item's first tile
    if (tile_at >= st.end) break;
    const int64_t t0 = max(at - tile_at, (int64_t)0), t1 = min(keys.tiles, st.end - tile_at);
    const int head = (int)(j / s.chunks), row0 = (int)(j % s.chunks) * kRows;
    const int rows = min(kRows, a.T * a.rep - row0);
    const int64_t len = a.t.lens[n];
    __syncthreads();
    if (tid == 0 && len > cap) sh.bad = 1;
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = i / D, c = i % D, row = row0 + r;
      float x = 0.f;
      if (r < rows) {
        const float* q = static_cast<const float*>(a.q) + ((int64_t)n * a.T + row / a.rep) * a.ldq;
        x = q[(int64_t)(head * a.rep + row % a.rep) * D + c] * a.scale * kLog2e;
      }
      sh.q[r][c] = x;
    }
    if (tid < kRows) {
      sh.m[tid] = -INFINITY;
      sh.l[tid] = 0.f;
    }
    float acc[kOwn];
#pragma unroll
    for (int r = 0; r < kOwn; ++r) acc[r] = 0.f;
    for (int64_t t = t0; t < t1; ++t) {
      const int64_t k0 = keys.lo + t * kTile;
      __syncthreads();
      // the tile, two halves of the block for keys and values; places unseen are zeros
      for (int i = tid; i < kTile * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const int64_t pos = k0 + r;
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        int id = -1;
        if (pos < keys.hi) {
          id = page_of(a.t, n, pos);
          if (id < 0) sh.bad = 1;
        }
        float sk = 1.f, sv = 1.f;
        if (id >= 0) {
          const int64_t row = ((int64_t)head << a.t.shift) + (pos & ((1 << a.t.shift) - 1));
          load4<TC>(static_cast<const TC*>(a.kc) + id * a.ldpage + row * D + c, x);
          load4<TC>(static_cast<const TC*>(a.vc) + id * a.ldpage + row * D + c, y);
          if (kCoded && c == 0) {
            const int64_t b = (((int64_t)id * a.hk) << a.t.shift) + row;
            sk = power(a.ks[b]);
            sv = power(a.vs[b]);
          }
        }
        *reinterpret_cast<float4*>(&sh.k[r][c]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&sh.v[r][c]) = make_float4(y[0], y[1], y[2], y[3]);
        if (c == 0) {
          sh.seen[r] = id >= 0;
          sh.ks[r] = sk;
          sh.vs[r] = sv;
        }
      }
      __syncthreads();
      {
        const int key = tid % kTile, r0 = tid / kTile * (kRows / 2);
        float dot[kRows / 2];
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) dot[r] = 0.f;
        for (int c = 0; c < D; c += 4) {
          const float4 x = *reinterpret_cast<const float4*>(&sh.k[key][c]);
#pragma unroll
          for (int r = 0; r < kRows / 2; ++r) {
            const float4 y = *reinterpret_cast<const float4*>(&sh.q[r0 + r][c]);
            dot[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot[r]))));
          }
        }
        const int64_t pos = k0 + key;
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) {
          const int64_t hi = len - a.T + (row0 + r0 + r) / a.rep + 1;
          const bool seen = sh.seen[key] && r0 + r < rows && pos < hi && (a.window == 0 || pos >= hi - a.window);
          sh.p[r0 + r][key] = seen ? dot[r] * sh.ks[key] : -INFINITY;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const int r = warp * (kRows / 4) + i;
        const float x = sh.p[r][lane], y = sh.p[r][lane + 32];
        // a score that is NaN makes the row NaN through its sum
        float m = fmaxf(x, y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float old = sh.m[r];
        m = fmaxf(m, old);
        const float base = m == -INFINITY ? 0.f : m;
        const float px = exp2f(x - base), py = exp2f(y - base);
        float l = px + py;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        // a weight of 0 stays 0, whatever its value's power
        sh.p[r][lane] = px == 0.f ? 0.f : px * sh.vs[lane];
        sh.p[r][lane + 32] = py == 0.f ? 0.f : py * sh.vs[lane + 32];
        __syncwarp();
        if (lane == 0) {
          const float alpha = exp2f(old - base);
          sh.alpha[r] = alpha;
          sh.l[r] = fmaf(sh.l[r], alpha, l);
          sh.m[r] = m;
        }
      }
      __syncthreads();
      {
        const int c = tid % D, r0 = tid / D * kOwn;
#pragma unroll
        for (int r = 0; r < kOwn; ++r) acc[r] *= sh.alpha[r0 + r];
        for (int key = 0; key < kTile; ++key) {
          const float v = sh.v[key][c];
#pragma unroll
          for (int r = 0; r < kOwn; ++r) {
            const float p = sh.p[r0 + r][key];
            if (p != 0.f) acc[r] = fmaf(p, v, acc[r]);
          }
        }
      }
    }
    __syncthreads();
    const int c = tid % D, r0 = tid / D * kOwn;
    if (t0 == 0 && t1 == keys.tiles) {
#pragma unroll
      for (int r = 0; r < kOwn; ++r) {
        const int row = row0 + r0 + r;
        if (r0 + r >= rows) break;
        const int64_t o = ((int64_t)n * a.T + row / a.rep) * a.hq + head * a.rep + row % a.rep;
        const float l = sh.l[r0 + r];
        static_cast<float*>(a.out)[o * D + c] = l == 0.f ? 0.f : acc[r] / l;
        if (c == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (sh.m[r0 + r] + log2f(l)) * kLn2;
      }
    } else {
      float* part = part_of(s, blockIdx.x, t0 == 0 ? 1 : 0);
      if (t0 == 0 && tid == 0) {
        s.cut[blockIdx.x] = (int64_t)n * each + j;
        s.cut_at[blockIdx.x] = item_at;
      }
      if (tid < kRows) {
        part[tid] = sh.m[tid];
        part[kRows + tid] = sh.l[tid];
      }
#pragma unroll
      for (int r = 0; r < kOwn; ++r) part[2 * kRows + (r0 + r) * D + c] = acc[r];
    }
    at = tile_at + t1;
    if (t1 == keys.tiles && j == each - 1) {
      before += keys.tiles + s.cost;
      ++n;
    }
  }
  __syncthreads();
  if (tid == 0) s.verdict[blockIdx.x] = sh.bad ? KDA_ERR_INVALID_ARG : KDA_OK;
}

// One block per cut item and row: the parts' outputs weighted by 2^(m - the largest m), over the
// sum of their sums.  A lane has four channels, each warp every fourth part.
constexpr int kJoinWarps = 4;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(AttnArgs a, Split s) {
  __shared__ float4 fold[kJoinWarps][32];
  __shared__ float sums[kJoinWarps], tops[kJoinWarps];
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    unsigned int bad = 0;
    for (int64_t b = tid; b < s.blocks; b += blockDim.x) bad |= s.verdict[b];
    bad = __syncthreads_or(bad);
    if (tid == 0) *s.status = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
  }
  const int64_t item = s.cut[blockIdx.x];
  if (item < 0) return;
  const int64_t each = (int64_t)a.hk * s.chunks;
  const int n = (int)(item / each), head = (int)(item % each) / s.chunks;
  const int r = blockIdx.y, row = (int)(item % s.chunks) * s.rows + r;
  if (row >= a.T * a.rep) return;
  const int64_t b0 = blockIdx.x, b1 = (s.cut_at[b0] + s.cost + keys_of(a, s.tile, n).tiles - 1) / *s.share;
  float m = -INFINITY;
  for (int64_t b = b0 + tid; b <= b1; b += blockDim.x) m = fmaxf(m, part_of(s, b, b == b0)[r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) tops[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) m = fmaxf(m, tops[i]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int64_t b = b0 + warp; b <= b1; b += kJoinWarps) {
    const float* p = part_of(s, b, b == b0);
    const float w = exp2f(p[r] - base);
    l = fmaf(p[s.rows + r], w, l);
    if (lane * 4 < D) {
      const float4 x = *reinterpret_cast<const float4*>(p + 2 * s.rows + r * D + lane * 4);
      o.x = fmaf(x.x, w, o.x);
      o.y = fmaf(x.y, w, o.y);
      o.z = fmaf(x.z, w, o.z);
      o.w = fmaf(x.w, w, o.w);
    }
  }
  fold[warp][lane] = o;
  if (lane == 0) sums[warp] = l;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int i = 1; i < kJoinWarps; ++i) {
    const float4 x = fold[i][lane];
    o.x += x.x;
    o.y += x.y;
    o.z += x.z;
    o.w += x.w;
    l += sums[i];
  }
  const int64_t to = ((int64_t)n * a.T + row / a.rep) * a.hq + head * a.rep + row % a.rep;
  const float f = l == 0.f ? 0.f : 1.f / l;
  if (lane * 4 < D) {
    T* out = static_cast<T*>(a.out) + to * D + lane * 4;
    out[0] = from_f32<T>(o.x * f);
    out[1] = from_f32<T>(o.y * f);
    out[2] = from_f32<T>(o.z * f);
    out[3] = from_f32<T>(o.w * f);
  }
  if (lane == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename TC, int D>
cudaError_t launch(const AttnArgs& a, const Split& s) {
  constexpr int bytes = sizeof(Shared<D>);
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<TC, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  attn_kernel<TC, D><<<(unsigned)s.blocks, kThreads, bytes, a.stream>>>(a, s);
  return cudaGetLastError();
}
template <int D>
cudaError_t by_cache(const AttnArgs& a, const Split& s) {
  switch (a.cache) {
    case KDA_CACHE_E4M3: return launch<E4M3, D>(a, s);
    case KDA_CACHE_INT8: return launch<Int8, D>(a, s);
    default: return launch<float, D>(a, s);
  }
}

}  // namespace

Split attn_general_split(const AttnArgs& a) { return split_of(a, kRows, kTile, 1, 2); }

// The join's blocks may be placed while the last of the main kernel's still run.
template <typename T, int D>
static cudaError_t join(const AttnArgs& a, const Split& s) {
  const int rows = a.T * a.rep;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)s.blocks, rows < s.rows ? rows : s.rows);
  c.blockDim = dim3(32 * kJoinWarps);
  c.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, attn_join_kernel<T, D>, a, s);
}
cudaError_t launch_attn_join(const AttnArgs& a, const Split& s) {
  using bf = __nv_bfloat16;
  if (a.d == 128) return a.bf16 ? join<bf, 128>(a, s) : join<float, 128>(a, s);
  return a.bf16 ? join<bf, 64>(a, s) : join<float, 64>(a, s);
}

cudaError_t launch_attn_general(const AttnArgs& a) {
  Split s = attn_general_split(a);
  split_place(s, a.ws);
  cudaError_t e = a.d == 128 ? by_cache<128>(a, s) : by_cache<64>(a, s);
  return e != cudaSuccess ? e : launch_attn_join(a, s);
}

size_t attn_workspace(const AttnArgs& a) {
  return split_bytes(a.bf16 ? attn_mma_split(a) : attn_general_split(a));
}

cudaError_t launch_attn(const AttnArgs& a) {
  if (a.B == 0) return cudaMemsetAsync(a.ws, 0, 4, a.stream);
  return a.bf16 ? launch_attn_mma(a) : launch_attn_general(a);
}

}  // namespace attn
}  // namespace kda
