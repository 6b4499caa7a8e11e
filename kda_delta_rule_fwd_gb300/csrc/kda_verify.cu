// Verification of drafted tokens: the kept prefix, then one token from max(p - q, 0) or p.
//
// Probabilities are whole multiples of 2^-44 in 64 bits, so their sums are exact in any order,
// and with fewer than 2^19 of them below 2^63.  The token drawn is the first whose running sum
// exceeds floor(m total / 2^24), m the 24 bits of the random number.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

using namespace layer;

constexpr int kThreads = 512, kWarps = kThreads / 32, kRun = 128;  // kRun: tokens of a warp's turn
constexpr int kRuns = (1 << 19) / kRun;
using u64 = unsigned long long;

__device__ __forceinline__ long long fixed(float p) {
  p = p > 0.f ? fminf(p, 1.f) : 0.f;  // NaN: 0
  return __float2ll_rn(p * 17592186044416.f);
}

// the weight of token i
template <typename T>
struct Weights {
  const T *p, *q;  // rows; q may be null
  int certain;     // the token that the draft was certain of, or -1
  __device__ __forceinline__ u64 at(int i) const {
    long long w = fixed(to_f32(p[i]));
    if (q) w -= fixed(to_f32(q[i]));
    if (i == certain) w -= 1ll << 44;
    return w > 0 ? (u64)w : 0;
  }
};

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

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
  __shared__ u64 run[kRuns];
  __shared__ u64 total_of[kWarps];
  __shared__ int kept_of, have_of;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    if (lane <= a.K) tokens[lane] = lane < kept ? d : -1;
    if (lane == 0) {
      a.commit[b] = have < 0 ? 0 : kept + 1;
      kept_of = kept;
      have_of = have;
    }
  }
  __syncthreads();
  const int kept = kept_of, have = have_of;
  if (have < 0) return;
  Weights<T> w{p + (int64_t)kept * a.V, nullptr, -1};
  if (kept < have) {
    if (q) w.q = q + (int64_t)kept * a.V;
    else w.certain = drafts[kept];
  }
  const int runs = (a.V + kRun - 1) / kRun;
  const u64 m = (u64)(fminf(fmaxf(u[a.K], 0.f), 0.99999994f) * 16777216.f);
  for (;;) {
    u64 sum = 0;
    for (int r = warp; r < runs; r += kWarps) {
      u64 s = 0;
#pragma unroll
      for (int e = 0; e < kRun / 32; ++e) {
        const int i = r * kRun + e * 32 + lane;
        if (i < a.V) s += w.at(i);
      }
      s = warp_sum(s);
      if (lane == 0) run[r] = s;
      sum += s;
    }
    if (lane == 0) total_of[warp] = sum;
    __syncthreads();
    u64 total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += total_of[i];
    if (total == 0 && (w.q || w.certain >= 0)) {  // nothing left of p - q: p itself
      w.q = nullptr;
      w.certain = -1;
      __syncthreads();
      continue;
    }
    if (warp == 0) {
      if (total == 0) {
        if (lane == 0) latch_status(a.status, KDA_ERR_INVALID_ARG);
        return;  // -1 stays
      }
      u64 left = m * (total >> 24) + ((m * (total & 0xffffffu)) >> 24);
      int at = 0;
      for (int base = 0; base < runs; base += 32) {
        const u64 mine = base + lane < runs ? run[base + lane] : 0;
        const u64 up = warp_scan(mine);
        const unsigned past = __ballot_sync(0xffffffffu, up > left);
        if (past) {
          const int i = __ffs(past) - 1;
          at = base + i;
          left -= __shfl_sync(0xffffffffu, up - mine, i);
          break;
        }
        left -= __shfl_sync(0xffffffffu, up, 31);
      }
      for (int e = 0; e < kRun / 32; ++e) {
        const int i = at * kRun + e * 32 + lane;
        const u64 up = warp_scan(i < a.V ? w.at(i) : 0);
        const unsigned past = __ballot_sync(0xffffffffu, up > left);
        if (past) {
          if (lane == 0) tokens[kept] = at * kRun + e * 32 + __ffs(past) - 1;
          return;
        }
        left -= __shfl_sync(0xffffffffu, up, 31);
      }
    }
    return;
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a) {
  if (a.B == 0) return cudaSuccess;
  if (a.bf16) verify_kernel<__nv_bfloat16><<<a.B, kThreads, 0, a.stream>>>(a);
  else verify_kernel<float><<<a.B, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
