// RMS norms before and after a block, fused with the block's gate and residual
// scale, and their gradients.  Per row of d channels:
//
//     z = act(gate);  v = x z (gate first) or x;  m = v k w,  k = 1 / rms(v)
//     b = m z (gate after) or m;  r = residual + scale ls b;  y = r k' w'
//
// One pass: a row stays in registers between its reductions, so each input is read
// once and each output written once, and the work is bound by memory traffic.  A row
// of d channels is held by up to TPR threads with NC chunks of VEC channels each; rows
// of up to 32 threads reduce by shuffles alone, longer ones have a block of their own
// with as many warps as they fill.  Blocks are persistent: as many as are resident
// together, each walks rows and requests the next one's inputs before it works on the
// present one, so that the reductions' latency is covered; the parameters are loaded
// once where a row's chunks leave room for them (up to 32 threads per row).
//
// One GB300, bf16: 16384 x 32 gated rows of 128 take 64 us forward (6.3 TB/s, 92% of a copy's
// rate); the gradient through both norms, gate and residual scale over 16384 rows of 4096 takes
// 283 us (3.8 TB/s): three sums over a row's 512 threads follow each other, with half the
// issue slots used and no registers left for a second row.
#pragma once

#include <type_traits>

#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace norm {

// the warps of a long row's block, up to a power of two
template <int TPR> constexpr int warps_of() { return TPR > 512 ? 32 : TPR / 32; }

// sum over the threads of a row; every thread gets it.  With TPR above 32 the row is
// the whole block: two alternating scratch rows leave one barrier per sum.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float2 (*scratch)[32], int& flip) {
  constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = warps_of<TPR>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, at = lane % kWarps;
    if (lane == 0) scratch[flip][warp].x = v;
    __syncthreads();
    v = at * 32 < blockDim.x ? scratch[flip][at].x : 0.f;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    flip ^= 1;
  }
  return v;
}

// the same for two sums at once
template <int TPR>
__device__ __forceinline__ float2 row_sums(float a, float b, float2 (*scratch)[32], int& flip) {
  constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = warps_of<TPR>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, at = lane % kWarps;
    if (lane == 0) scratch[flip][warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = at * 32 < blockDim.x ? scratch[flip][at] : make_float2(0.f, 0.f);
    a = v.x;
    b = v.y;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    flip ^= 1;
  }
  return make_float2(a, b);
}

// The most threads of a block, and those of a call: long rows leave out the warps that
// their d does not need.  Chunk i of a thread follows chunk i - 1 by the row's threads.
template <int TPR> constexpr int block_of() { return TPR < 128 ? 128 : TPR; }
template <int VEC, int NC, int TPR> int threads_of(int d) {
  return TPR > 32 ? (d + VEC * NC * 32 - 1) / (VEC * NC * 32) * 32 : block_of<TPR>();
}
template <int TPR> __device__ __forceinline__ int row_threads() { return TPR > 32 ? blockDim.x : TPR; }

// where the gate sits
enum Place { kNoGate = 0, kAfter = 1, kFirst = 2 };

// the gate z and its slope from s = sigmoid(g)
__device__ __forceinline__ float gate_of(float g, float s, bool silu) { return silu ? g * s : s; }
__device__ __forceinline__ float gate_slope(float g, float s, bool silu) {
  return s * (silu ? fmaf(g, 1.f - s, 1.f) : 1.f - s);
}

// a row's inputs as they come from memory
template <typename T, typename TR, int VEC, int NC, bool kBwd>
struct RowIn {
  Raw<T, VEC> x[NC], g[NC], dy[kBwd ? NC : 1];
  Raw<TR, VEC> res[NC], dr[kBwd ? NC : 1];
};

template <typename T, typename TR, int VEC, int NC, int TPR, int PLACE, bool kBwd>
__device__ __forceinline__ void request(const NormArgs& a, int64_t row, int lane,
                                        RowIn<T, TR, VEC, NC, kBwd>& in) {
  int64_t xo = row * a.d, go = xo;
  // chunks past the row (and rows past the last) are zeros
  const bool on = row < a.tokens * a.heads;
  if (on && !a.dense) {
    const int64_t tok = row / a.heads;
    const int64_t head = (row - tok * a.heads) * a.d;
    xo = tok * a.ldx + head;
    go = tok * a.ldg + head;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * row_threads<TPR>()) * VEC;
    const bool in_row = on && c < a.d;
    auto get = [&](auto& raw, const auto* p, int64_t o, bool have) {
      using E = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
      if (in_row && have) raw = fetch<E, VEC>(p + o + c);
      else raw = Raw<E, VEC>{};
    };
    get(in.x[i], static_cast<const T*>(a.x), xo, true);
    if (PLACE != kNoGate) get(in.g[i], static_cast<const T*>(a.gate), go, true);
    // the gradient needs the residual only to form y's norm again
    get(in.res[i], static_cast<const TR*>(a.res), row * a.d, a.res && (!kBwd || a.ow));
    if constexpr (kBwd) {
      get(in.dr[i], static_cast<const TR*>(a.dr), row * a.d, a.dr != nullptr);
      get(in.dy[i], static_cast<const T*>(a.dy), row * a.d, a.dy != nullptr);
    }
  }
}

// VEC parameters times `scale`, or the scale alone where there are none
template <int VEC>
__device__ __forceinline__ void param(const float* p, int c, float scale, float (&v)[VEC]) {
  if (p) {
    load<VEC>(p + c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] *= scale;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = scale;
  }
}

inline bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }
inline bool wide_ok(const NormArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  const void* ptrs[] = {a.x, a.gate, a.res, a.dr, a.dy, a.w, a.ls, a.ow, a.r,
                        a.y, a.dx, a.dgate, a.dres};
  bool wide = a.d % v == 0 && a.ldx % v == 0 && a.ldg % v == 0;
  for (const void* p : ptrs) wide = wide && al16(p);
  return wide;
}

// Threads per row by the row's chunks: up to 32 chunks the row stays inside a warp, with two
// chunks per thread (F::kPairs) up to 64.  Eight threads for rows of up to 8 chunks leave few
// lanes idle: rows of 64 bf16 channels, 128 MB of them with a gate, take 69 us forward against
// 96 with 16 lanes per row.  Two chunks per thread where their registers allow it: rows of 128
// take 65 us, with one chunk 69.  `F<T, TR, VEC, NC, TPR, PLACE>::run` is the launch.
template <template <typename, typename, int, int, int, int> class F, typename T, typename TR, int VEC, int PLACE>
cudaError_t by_size(const NormArgs& a) {
  const int chunks = (a.d + VEC - 1) / VEC;
  if constexpr (VEC == 1) {
    if (chunks <= 128) return F<T, TR, 1, 4, 32, PLACE>::run(a);
    if (chunks <= 1024) return F<T, TR, 1, 4, 256, PLACE>::run(a);
    return F<T, TR, 1, 8, 1024, PLACE>::run(a);
  } else {
    if (chunks <= 8) return F<T, TR, VEC, 1, 8, PLACE>::run(a);
    if constexpr (F<T, TR, VEC, 1, 32, PLACE>::kPairs) {
      if (chunks <= 16) return F<T, TR, VEC, 2, 8, PLACE>::run(a);
      if (chunks <= 32) return F<T, TR, VEC, 2, 16, PLACE>::run(a);
      if (chunks <= 64) return F<T, TR, VEC, 2, 32, PLACE>::run(a);
    } else {
      if (chunks <= 16) return F<T, TR, VEC, 1, 16, PLACE>::run(a);
      if (chunks <= 32) return F<T, TR, VEC, 1, 32, PLACE>::run(a);
    }
    if (chunks <= 128) return F<T, TR, VEC, 1, 128, PLACE>::run(a);
    if (chunks <= 256) return F<T, TR, VEC, 1, 256, PLACE>::run(a);
    if (chunks <= 512) return F<T, TR, VEC, 1, 512, PLACE>::run(a);
    if (chunks <= 768) return F<T, TR, VEC, 1, 768, PLACE>::run(a);
    if constexpr (VEC == 4) {  // float32 rows past 4096 channels
      if (chunks > 1024) return F<T, TR, VEC, 2, 1024, PLACE>::run(a);
    }
    return F<T, TR, VEC, 1, 1024, PLACE>::run(a);
  }
}
template <template <typename, typename, int, int, int, int> class F, typename T, typename TR, int VEC>
cudaError_t by_place(const NormArgs& a) {
  if (!a.gate_act) return by_size<F, T, TR, VEC, kNoGate>(a);
  return a.gate_first ? by_size<F, T, TR, VEC, kFirst>(a) : by_size<F, T, TR, VEC, kAfter>(a);
}
template <template <typename, typename, int, int, int, int> class F>
cudaError_t by_type(const NormArgs& a) {
  using bf = __nv_bfloat16;
  const bool wide = wide_ok(a);
  if (!a.bf16) return wide ? by_place<F, float, float, 4>(a) : by_place<F, float, float, 1>(a);
  if (a.res_bf16) return wide ? by_place<F, bf, bf, 8>(a) : by_place<F, bf, bf, 1>(a);
  return wide ? by_place<F, bf, float, 8>(a) : by_place<F, bf, float, 1>(a);
}

}  // namespace norm
}  // namespace layer
}  // namespace kda
