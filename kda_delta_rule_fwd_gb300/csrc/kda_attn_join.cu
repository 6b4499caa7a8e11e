// Attention of new tokens: the join of the parts that the main kernel's blocks leave of an item.
#include "kda_attn_split.cuh"

namespace kda {
namespace attn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// A part's sum, weighted; one that is not finite stays so, as its own weights made it, though w may be 0.
__device__ __forceinline__ float plus(float o, float x, float w) { return isfinite(x) ? fmaf(x, w, o) : o + x; }

// For each cut item and row: the parts' outputs weighted by 2^(m - the largest m), over the sum of
// their sums.  A lane has four channels.  Few rows (long items in many parts): a block per row, whose
// four warps take every fourth part; many rows: a warp per row (32 rows of 304 cuts, mostly of two
// parts, take 14 us with a block each).
constexpr int kJoinWarps = 4;
template <typename T, int D, int WAYS>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(AttnArgs a, Split s) {
  __shared__ float4 fold[WAYS][32];
  __shared__ float sums[WAYS], tops[WAYS];
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, way = WAYS == 1 ? 0 : warp;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    unsigned int bad = 0;
    for (int64_t b = tid; b < s.blocks; b += blockDim.x) bad |= s.verdict[b];
    bad = __syncthreads_or(bad);
    if (tid == 0) *s.status = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
  }
  const int64_t b0 = blockIdx.x, item = s.cut[b0], b1 = s.last[b0];
  if (item < 0) return;
  const int64_t each = (int64_t)a.hk * s.chunks;
  const int n = (int)(item / each), head = (int)(item % each) / s.chunks;
  const int r = blockIdx.y * (kJoinWarps / WAYS) + (WAYS == 1 ? warp : 0);
  const int row = (int)(item % s.chunks) * s.rows + r;
  if (r >= s.rows || row >= a.T * a.rep) return;  // whole warps, or the whole block
  float m = -INFINITY;
  for (int64_t b = b0 + lane + 32 * way; b <= b1; b += 32 * WAYS) m = fmaxf(m, part_of(s, b, b == b0)[r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (WAYS > 1) {
    if (lane == 0) tops[way] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAYS; ++i) m = fmaxf(m, tops[i]);
  }
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int64_t b = b0 + way; b <= b1; b += WAYS) {
    const float* p = part_of(s, b, b == b0);
    const float w = exp2f(p[r] - base);
    l = fmaf(p[s.rows + r], w, l);
    if (lane * 4 < D) {
      const float4 x = *reinterpret_cast<const float4*>(p + 2 * s.rows + r * D + lane * 4);
      o.x = plus(o.x, x.x, w);
      o.y = plus(o.y, x.y, w);
      o.z = plus(o.z, x.z, w);
      o.w = plus(o.w, x.w, w);
    }
  }
  if constexpr (WAYS > 1) {
    fold[way][lane] = o;
    if (lane == 0) sums[way] = l;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int i = 1; i < WAYS; ++i) {
      const float4 x = fold[i][lane];
      o.x += x.x;
      o.y += x.y;
      o.z += x.z;
      o.w += x.w;
      l += sums[i];
    }
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

// Short tables: what the main kernel's blocks meet, places past the table and pages not in the pool.
constexpr int kTableThreads = 512;
__global__ void __launch_bounds__(kTableThreads) attn_table_kernel(AttnArgs a, Split s) {
  const int entries = a.B * a.t.max_pages;
  int bad = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < entries; i += kTableThreads) {
    const int n = i / a.t.max_pages;
    const int64_t from = (int64_t)(i - n * a.t.max_pages) << a.t.shift;
    const Keys k = keys_of(a, s.tile, n);
    if (from < k.hi && from + (1 << a.t.shift) > k.first) bad |= (unsigned)a.t.pages[i] >= (unsigned)a.t.num_pages;
    bad |= a.t.lens[n] > (int64_t)a.t.max_pages << a.t.shift;
  }
  bad = __syncthreads_or(bad);
  cudaGridDependencySynchronize();
  if (threadIdx.x == 0) *s.status = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
}

// Blocks of a kernel behind the main one may be placed while the last of its still run.
template <class F>
cudaError_t launch_behind(F kernel, dim3 grid, int threads, const AttnArgs& a, const Split& s) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a, s);
}
template <typename T, int D, int WAYS>
cudaError_t launch(const AttnArgs& a, const Split& s) {
  const int rows = a.T * a.rep < s.rows ? a.T * a.rep : s.rows, per = kJoinWarps / WAYS;
  return launch_behind(attn_join_kernel<T, D, WAYS>, dim3((unsigned)s.blocks, (rows + per - 1) / per), 32 * kJoinWarps, a, s);
}
template <typename T, int D>
cudaError_t join(const AttnArgs& a, const Split& s) {
  return s.rows > 8 ? launch<T, D, 1>(a, s) : launch<T, D, kJoinWarps>(a, s);
}

}  // namespace

cudaError_t launch_attn_table(const AttnArgs& a, const Split& s) {
  return launch_behind(attn_table_kernel, dim3(1), kTableThreads, a, s);
}
cudaError_t launch_attn_join(const AttnArgs& a, const Split& s) {
  using bf = __nv_bfloat16;
  if (a.d == 128) return a.bf16 ? join<bf, 128>(a, s) : join<float, 128>(a, s);
  return a.bf16 ? join<bf, 64>(a, s) : join<float, 64>(a, s);
}

}  // namespace attn
}  // namespace kda
