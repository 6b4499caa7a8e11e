// Verification of drafted tokens: the kept prefix, then one token from max(p - q, 0) or p.
//
// Probabilities are whole multiples of 2^-44 in 64 bits, so their sums are exact in any order,
// and with fewer than 2^19 of them below 2^63.  The token drawn is the first whose running sum
// exceeds floor(m total / 2^24), m the 24 bits of the random number.
//
// One pass over the row (or, after a refusal, the two rows) of the place where the token is drawn.  What
// bounds it is the fixed-point arithmetic, which both rows get for every token, also where no q is read:
// 256 sequences of 131072 tokens take 45 us in float32 with 43% refusals (192 MB, 28 us at a copy's rate),
// 48 with certain drafts (134 MB), 44 in bf16 (96 MB).  A cluster of blocks per sequence, each with a
// stretch of the vocabulary, keeps the sum of every run of a warp's 16-byte loads in shared memory; the
// blocks' totals meet in the cluster, and the block that holds the place reads that one run again.
#include <cooperative_groups.h>

#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

namespace cg = cooperative_groups;
using layer::Raw;
using layer::fetch;
using layer::open;

// 256 sequences of 131072 tokens take 46 us with 8 blocks of 128 threads to an SM, 51 to 56 with 4 of
// 256 and 59 with 2 of 512: a block waits three times for loads before its row's, so many small ones
// hide it.
constexpr int kThreads = 128, kPerSm = 8, kWarps = kThreads / 32;
using u64 = unsigned long long;

// A probability as hi 2^22 + lo: hi = p 2^22 to the nearest, lo = what is left to the nearest 2^-44,
// both read off the mantissas of sums with a number so large that its last bit counts one (hi 2^22
// is even, so ties of lo go to the even whole; a conversion to 64 bits issues at a quarter of this).
struct Fixed {
  int hi, lo;  // with the large numbers' own bits, which differences lose
};
__device__ __forceinline__ Fixed fixed(float p) {
  const float x = __saturatef(p) * 4194304.f;  // NaN and below 0: 0
  const float h = x + 8388608.f;
  const float l = fmaf(x - (h - 8388608.f), 4194304.f, 12582912.f);
  return {__float_as_int(h), __float_as_int(l)};
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// inclusive running sums over a warp's lanes
__device__ __forceinline__ u64 warp_scan(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Weights of a lane's tokens in a batch: VEC in a row (aligned rows), else lane, lane + 32, ...
// A run is kBatches of them, requested together and added up before the warp's sum.
constexpr int kBatches = 4;
template <typename T, bool kWide>
struct Weights {
  static constexpr int VEC = 16 / sizeof(T), kRun = 32 * VEC;
  const T *p, *q;  // rows; q may be null
  int V, certain;  // certain: the token that the draft was sure of, or -1
  struct Held { Raw<T, VEC> p, q; };
  __device__ __forceinline__ int token(int r, int e) const {
    const int lane = threadIdx.x & 31;
    return r * kRun + (kWide ? lane * VEC + e : e * 32 + lane);
  }
  __device__ __forceinline__ void request(int r, Held& h) const {
    T* hp = reinterpret_cast<T*>(&h.p);
    T* hq = reinterpret_cast<T*>(&h.q);
    if (kWide) {  // V is a multiple of VEC
      const int i = token(r, 0);
      h.p = h.q = Raw<T, VEC>{};
      if (i < V) {
        h.p = fetch<T, VEC>(p + i);
        if (q) h.q = fetch<T, VEC>(q + i);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = token(r, e);
        hp[e] = i < V ? p[i] : from_f32<T>(0.f);
        hq[e] = q && i < V ? q[i] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void weigh(int r, const Held& h, u64 (&w)[VEC]) const {
    float x[VEC], y[VEC];
    open<T, VEC>(h.p, x);
    open<T, VEC>(h.q, y);  // zeros without q
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Fixed f = fixed(x[e]), g = fixed(y[e]);
      const long long d = (long long)(f.hi - g.hi) * (1 << 22) + (f.lo - g.lo);
      w[e] = d > 0 ? (u64)d : 0;
    }
    if (certain >= 0 && certain / kRun == r) {  // q = 1 there, p at most that
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (token(r, e) == certain) w[e] = 0;
    }
  }
};

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kPerSm) verify_kernel(VerifyArgs a, int per) {
  using W = Weights<T, kWide>;
  extern __shared__ u64 run[];  // sums of this block's runs [0, per)
  __shared__ u64 total_of[kWarps], total_here[2];
  __shared__ int kept_of, have_of;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int b = blockIdx.x / blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* p = static_cast<const T*>(a.p) + (int64_t)b * (a.K + 1) * a.V;
  const T* q = a.q ? static_cast<const T*>(a.q) + (int64_t)b * a.K * a.V : nullptr;
  const int32_t* drafts = a.drafts + (int64_t)b * a.K;
  const float* u = a.u + (int64_t)b * (a.K + 1);
  int32_t* tokens = a.tokens + (int64_t)b * (a.K + 1);
  if (warp == 0) {  // lane i judges draft i
    int have = a.counts ? a.counts[b] : a.K;
    if (have < -1 || have > a.K) {
      if (lane == 0) latch_status(a.status, KDA_ERR_INVALID_ARG);
      have = -1;
    }
    bool keep = false;
    int d = -1;
    if (lane < have) {
      d = drafts[lane];
      if (d >= 0 && d < a.V) {
        const double pd = to_f32(p[(int64_t)lane * a.V + d]);
        const double qd = q ? (double)to_f32(q[(int64_t)lane * a.V + d]) : 1.0;
        keep = (double)u[lane] * qd < pd;  // 24 bits times 24: exact
      } else {
        latch_status(a.status, KDA_ERR_INVALID_ARG);
      }
    }
    const int kept = __ffs(~__ballot_sync(0xffffffffu, keep)) - 1;  // K < 32: a lane is 0
    if (rank == 0 && lane <= a.K) tokens[lane] = lane < kept ? d : -1;
    if (lane == 0) {
      if (rank == 0) a.commit[b] = have < 0 ? 0 : kept + 1;
      kept_of = kept;
      have_of = have;
    }
  }
  __syncthreads();
  const int kept = kept_of, have = have_of;
  if (have < 0) return;  // the whole cluster's
  W w{p + (int64_t)kept * a.V, nullptr, a.V, -1};
  if (kept < have) {
    if (q) w.q = q + (int64_t)kept * a.V;
    else w.certain = drafts[kept];
  }
  const int first = rank * per, runs = min(per, (a.V + W::kRun * kBatches - 1) / (W::kRun * kBatches) - first);  // may be below 0
  const u64 m = (u64)(fminf(fmaxf(u[a.K], 0.f), 0.99999994f) * 16777216.f);
  for (int turn = 0;; ++turn) {
    u64 sum = 0;
    for (int r = warp; r < runs; r += kWarps) {
      typename W::Held h[kBatches];
#pragma unroll
      for (int i = 0; i < kBatches; ++i) w.request((first + r) * kBatches + i, h[i]);
      u64 s = 0;
#pragma unroll
      for (int i = 0; i < kBatches; ++i) {
        u64 x[W::VEC];
        w.weigh((first + r) * kBatches + i, h[i], x);
#pragma unroll
        for (int e = 0; e < W::VEC; ++e) s += x[e];
      }
      s = warp_sum(s);
      if (lane == 0) run[r] = s;
      sum += s;
    }
    if (lane == 0) total_of[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 t = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) t += total_of[i];
      total_here[turn] = t;
    }
    cluster.sync();
    u64 total = 0, before = 0, mine = 0;
    for (int i = 0; i < blocks; ++i) {
      const u64 t = *cluster.map_shared_rank(&total_here[turn], i);
      if (i < rank) before += t;
      if (i == rank) mine = t;
      total += t;
    }
    if (total == 0 && turn == 0 && (w.q || w.certain >= 0)) {  // nothing left of p - q: p itself
      w.q = nullptr;
      w.certain = -1;
      continue;
    }
    if (total == 0) {
      if (rank == 0 && threadIdx.x == 0) latch_status(a.status, KDA_ERR_INVALID_ARG);
      break;  // -1 stays
    }
    u64 left = m * (total >> 24) + ((m * (total & 0xffffffu)) >> 24);
    if (warp != 0 || left < before || left >= before + mine) break;
    left -= before;
    int at = 0;
    for (int base = 0; base < runs; base += 32) {
      const u64 x = base + lane < runs ? run[base + lane] : 0;
      const u64 up = warp_scan(x);
      const unsigned past = __ballot_sync(0xffffffffu, up > left);
      if (past) {
        const int i = __ffs(past) - 1;
        at = base + i;
        left -= __shfl_sync(0xffffffffu, up - x, i);
        break;
      }
      left -= __shfl_sync(0xffffffffu, up, 31);
    }
    bool found = false;
    for (int k = 0; k < kBatches && !found; ++k) {
      const int batch = (first + at) * kBatches + k;
      typename W::Held h;
      u64 x[W::VEC];
      w.request(batch, h);
      w.weigh(batch, h, x);
      if (kWide) {
        u64 s = 0;
#pragma unroll
        for (int e = 0; e < W::VEC; ++e) s += x[e];
        const u64 up = warp_scan(s);
        u64 past = up - s;
        int token = -1;
#pragma unroll
        for (int e = 0; e < W::VEC; ++e) {
          past += x[e];
          if (token < 0 && past > left) token = w.token(batch, e);
        }
        const unsigned who = __ballot_sync(0xffffffffu, token >= 0);
        if (who && lane == __ffs(who) - 1) tokens[kept] = token;
        found = who != 0;
        left -= __shfl_sync(0xffffffffu, up, 31);
      } else {
#pragma unroll
        for (int e = 0; e < W::VEC; ++e) {
          const u64 up = warp_scan(x[e]);
          const unsigned past = __ballot_sync(0xffffffffu, up > left);
          if (!found && past && lane == __ffs(past) - 1) tokens[kept] = w.token(batch, e);
          found |= past != 0;
          if (found) break;
          left -= __shfl_sync(0xffffffffu, up, 31);
        }
      }
    }
    break;
  }
  cluster.sync();  // nobody leaves while its total may be read; the place's -1 came before the token
}

template <typename T, bool kWide>
cudaError_t launch(const VerifyArgs& a) {
  using W = Weights<T, kWide>;
  // Blocks per sequence: half as many as are resident on the device, with a run for every warp (the
  // same 256 sequences: 46 us, 49 with twice as many, 57 with half)
  const int runs = (a.V + W::kRun * kBatches - 1) / (W::kRun * kBatches);
  int blocks = 1;
  while (blocks < 8 && (int64_t)a.B * blocks < 4 * a.sms && runs >= kWarps * blocks) blocks *= 2;
  const int per = (runs + blocks - 1) / blocks;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)a.B * blocks);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = per * sizeof(u64);
  c.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, verify_kernel<T, kWide>, a, per);
}
template <typename T>
cudaError_t by_alignment(const VerifyArgs& a) {
  const bool wide = (uintptr_t)a.p % 16 == 0 && (uintptr_t)a.q % 16 == 0 && a.V % (16 / (int)sizeof(T)) == 0;
  return wide ? launch<T, true>(a) : launch<T, false>(a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a) {
  if (a.B == 0) return cudaSuccess;
  return a.bf16 ? by_alignment<__nv_bfloat16>(a) : by_alignment<float>(a);
}

}  // namespace attn
}  // namespace kda
