// RMS norms with gate and residual scale: the forward (see kda_norm.cuh).
#include "kda_norm.cuh"

namespace kda {
namespace layer {
namespace {

using namespace norm;

// threads per SM: what the registers of one row allow
template <int NC, int TPR, bool kFull> constexpr int resident() {
  return TPR > 512 ? TPR : kFull ? 512 : NC > 1 ? 640 : 1024;
}

// kFull: with a residual, a per-channel scale or an outer norm; otherwise r = scale m alone
template <typename T, typename TR, int VEC, int NC, int TPR, int PLACE, bool kFull>
__global__ void __launch_bounds__(block_of<TPR>(), resident<NC, TPR, kFull>() / block_of<TPR>())
norm_fwd_kernel(NormArgs a) {
  constexpr int kRows = block_of<TPR>() / TPR;  // rows per block
  constexpr bool kKeep = TPR <= 32;             // parameters stay in registers
  __shared__ float2 scratch[2][32];
  int flip = 0;
  const int64_t rows = a.tokens * a.heads, step = (int64_t)gridDim.x * kRows;
  const int lane = threadIdx.x % TPR;
  const bool silu = a.gate_act == KDA_GATE_SILU;
  float w[NC][VEC], ls[NC][VEC], ow[NC][VEC];
  auto params = [&]() {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (c < a.d) {
        param<VEC>(a.w, c, kFull ? 1.f : a.scale, w[i]);
        if (kFull) param<VEC>(a.ls, c, a.scale, ls[i]);
        if (kFull && a.ow) param<VEC>(a.ow, c, 1.f, ow[i]);
      }
    }
  };
  if (kKeep) params();
  RowIn<T, TR, VEC, NC, false> in;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  request<T, TR, VEC, NC, TPR, PLACE, false>(a, row, lane, in);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < rows; base += step, row += step) {
    const bool on = row < rows;
    float v[NC][VEC], z[NC][VEC], rs[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      open<T, VEC>(in.x[i], v[i]);
      if (PLACE != kNoGate) open<T, VEC>(in.g[i], z[i]);
      open<TR, VEC>(in.res[i], rs[i]);
    }
    request<T, TR, VEC, NC, TPR, PLACE, false>(a, row + step, lane, in);
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (PLACE != kNoGate) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[i][e] = gate_of(z[i][e], sigmoid(z[i][e]), silu);
      }
      if (PLACE == kFirst) mul_v(v[i], z[i]);
      dot_v(v[i], v[i], ss);
    }
    float k = 1.f;
    if (a.w) k = rsqrtf(fmaf(row_sum<TPR>(ss.x + ss.y, scratch, flip), a.inv_d, a.eps));
    if (!kKeep) params();
    ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (c < a.d) {
        mul_v(v[i], k);
        mul_v(v[i], w[i]);
        if (PLACE == kAfter) mul_v(v[i], z[i]);
        if (kFull) {
          fma_v(ls[i], v[i], rs[i]);
          copy_v(rs[i], v[i]);
          dot_v(v[i], v[i], ss);
        }
        if (a.r && on) store<VEC>(static_cast<TR*>(a.r) + row * a.d + c, v[i]);
      }
    }
    if (!kFull || !a.ow) continue;
    k = rsqrtf(fmaf(row_sum<TPR>(ss.x + ss.y, scratch, flip), a.inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (on && c < a.d) {
        mul_v(v[i], k);
        mul_v(v[i], ow[i]);
        store<VEC>(static_cast<T*>(a.y) + row * a.d + c, v[i]);
      }
    }
  }
}

template <bool kFull>
struct Kind {
  template <typename T, typename TR, int VEC, int NC, int TPR, int PLACE>
  struct Forward {
    static constexpr bool kPairs = !kFull;
    static cudaError_t run(const NormArgs& a) {
      constexpr int kRows = block_of<TPR>() / TPR;
      const int threads = threads_of<VEC, NC, TPR>(a.d);
      const int64_t rows = a.tokens * a.heads;
      const int64_t blocks = (rows + kRows - 1) / kRows, most = a.sms * (resident<NC, TPR, kFull>() / threads);
      if (blocks == 0) return cudaSuccess;
      norm_fwd_kernel<T, TR, VEC, NC, TPR, PLACE, kFull>
          <<<(unsigned)(blocks < most ? blocks : most), threads, 0, a.stream>>>(a);
      return cudaGetLastError();
    }
  };
};

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a) {
  return a.res || a.ls || a.ow ? by_type<Kind<true>::Forward>(a) : by_type<Kind<false>::Forward>(a);
}

}  // namespace layer
}  // namespace kda
