// Norms of queries and keys per head with the position's rotation, and their gradient.
//
//     n = x k w,  k = 1 / sqrt(mean(x^2) + eps);   (a, b) -> (a cos f - b sin f, a sin f + b cos f)
//     backward:  g = the rotation by -f of dy,  dw = sum of g x k,  p = g w,
//                dx = k (p - n0 mean(p n0)),  n0 = x k      (dx = g without a weight)
//
// Angles.  f / 2 pi per position is a fraction of a turn in 64-bit fixed point, and position
// times it modulo 2^64 is the place on the circle: whole turns fall off the top, exactly, for
// positions of either sign.  The top 32 bits then go to sincospi.
#include "kda_attn.cuh"

namespace kda {
namespace attn {
namespace {

using namespace layer;

__device__ __forceinline__ unsigned long long turn_of(double freq) {
  const double t = freq * 0.15915494309189533577;  // turns per position
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 angle(unsigned long long turn, int pos) {  // (cos, sin)
  const unsigned long long f = turn * (unsigned long long)(long long)pos;
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
  unsigned long long turn[kPairs];
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

constexpr int kPerSm = 4;  // blocks of a part

cudaError_t run(QKArgs& a, bool bwd) {
  int most = 0;
  for (QKPart& p : a.p) {
    p.ctas = (int)qknorm_bwd_ctas(a.tokens, p.heads, a.sms);
    most = p.ctas > most ? p.ctas : most;
  }
  if (most == 0) return cudaSuccess;
  const dim3 grid(most, a.p[1].heads > 0 ? 2 : 1), block(32 * kNarrowWarps);
  using bf = __nv_bfloat16;
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
