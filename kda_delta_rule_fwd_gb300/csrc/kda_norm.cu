// RMS norms before and after a block, fused with the block's gate and residual
// scale, and their gradients.  Per row of d channels:
//
//     z = act(gate);  v = x z (gate first) or x;  m = v k w,  k = 1 / rms(v)
//     b = m z (gate after) or m;  r = residual + scale ls b;  y = r k' w'
//
// One pass: a row stays in registers between its two reductions, so each input
// is read once and each output written once, and the work is bound by memory
// traffic.  A row of d channels is held by TPR threads with NC chunks of VEC
// channels each; rows of up to 32 chunks reduce by shuffles alone.
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace {

// sum over the TPR threads of a row; every thread gets it.  Above 32 threads the
// row is the whole block: two alternating scratch rows leave one barrier per sum.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[32], int& flip) {
  constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) scratch[flip][warp] = v;
    __syncthreads();
    v = lane < kWarps ? scratch[flip][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    flip ^= 1;
  }
  return v;
}

template <int TPR> constexpr int block_of() { return TPR < 128 ? 128 : TPR; }

// act(g) and, where wanted, its derivative
__device__ __forceinline__ float gate_of(float g, int act) {
  const float s = sigmoid(g);
  return act == KDA_GATE_SIGMOID ? s : g * s;
}
__device__ __forceinline__ float gate_slope(float g, int act) {
  const float s = sigmoid(g);
  return act == KDA_GATE_SIGMOID ? s * (1.f - s) : s * fmaf(g, 1.f - s, 1.f);
}

template <typename T, typename TR, int VEC, int NC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>())
norm_fwd_kernel(NormArgs a) {
  constexpr int kRows = block_of<TPR>() / TPR;  // rows per block
  __shared__ float scratch[2][32];
  int flip = 0;
  const int64_t rows = a.tokens * a.heads;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const bool on = row < rows;
  const int lane = threadIdx.x % TPR;
  const int64_t tok = on ? row / a.heads : 0;
  const int head = on ? (int)(row - tok * a.heads) : 0;
  const T* x = static_cast<const T*>(a.x) + tok * a.ldx + (int64_t)head * a.d;
  const T* g = static_cast<const T*>(a.gate) + tok * a.ldg + (int64_t)head * a.d;
  const TR* res = static_cast<const TR*>(a.res) + row * a.d;
  float v[NC][VEC], z[NC][VEC], rs[NC][VEC];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * VEC;
    const bool in = on && c < a.d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i][e] = z[i][e] = rs[i][e] = 0.f;
    if (in) {
      load<VEC>(x + c, v[i]);
      if (a.gate_act) load<VEC>(g + c, z[i]);
      if (a.res) load<VEC>(res + c, rs[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (a.gate_act) {
        z[i][e] = gate_of(z[i][e], a.gate_act);
        if (a.gate_first) v[i][e] *= z[i][e];
      }
      ss = fmaf(v[i][e], v[i][e], ss);
    }
  float k = 1.f;
  if (a.w) k = rsqrtf(row_sum<TPR>(ss, scratch, flip) / a.d + a.eps);
  const bool after = a.gate_act && !a.gate_first;
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * VEC;
    if (c < a.d) {
      float w[VEC], ls[VEC];
      if (a.w) load<VEC>(a.w + c, w);
      if (a.ls) load<VEC>(a.ls + c, ls);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float m = a.w ? v[i][e] * k * w[e] : v[i][e];
        if (after) m *= z[i][e];
        const float s = a.ls ? a.scale * ls[e] : a.scale;
        v[i][e] = fmaf(s, m, rs[i][e]);
        ss = fmaf(v[i][e], v[i][e], ss);
      }
      if (a.r && on) store<VEC>(static_cast<TR*>(a.r) + row * a.d + c, v[i]);
    }
  }
  if (!a.ow) return;
  k = rsqrtf(row_sum<TPR>(ss, scratch, flip) / a.d + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * VEC;
    if (on && c < a.d) {
      float w[VEC];
      load<VEC>(a.ow + c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] *= v[i][e] * k;
      store<VEC>(static_cast<T*>(a.y) + row * a.d + c, w);
    }
  }
}

// Gradients.  For n = v k, y = n w:  dv = k (p - n mean(p n)) with p = dy w, and
// dw = sum over rows of dy n.  Each block walks the rows blockIdx, blockIdx +
// grid, ... and keeps its sums for the parameters in registers; they go to
// part[block][3][d] and are added in the order of the blocks.
template <typename T, typename TR, int VEC, int NC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>())
norm_bwd_kernel(NormArgs a) {
  constexpr int kRows = block_of<TPR>() / TPR;
  __shared__ float scratch[2][32];
  int flip = 0;
  const int64_t rows = a.tokens * a.heads;
  const int lane = threadIdx.x % TPR;
  const bool after = a.gate_act && !a.gate_first;
  float sw[NC][VEC], sl[NC][VEC], so[NC][VEC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sw[i][e] = sl[i][e] = so[i][e] = 0.f;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < rows; base += (int64_t)gridDim.x * kRows) {
    const int64_t row = base + threadIdx.x / TPR;
    const bool on = row < rows;
    const int64_t tok = on ? row / a.heads : 0;
    const int head = on ? (int)(row - tok * a.heads) : 0;
    const T* x = static_cast<const T*>(a.x) + tok * a.ldx + (int64_t)head * a.d;
    const T* g = static_cast<const T*>(a.gate) + tok * a.ldg + (int64_t)head * a.d;
    float xv[NC][VEC], gv[NC][VEC], rs[NC][VEC], dr[NC][VEC], dy[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * TPR) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) xv[i][e] = gv[i][e] = rs[i][e] = dr[i][e] = dy[i][e] = 0.f;
      if (on && c < a.d) {
        load<VEC>(x + c, xv[i]);
        if (a.gate_act) load<VEC>(g + c, gv[i]);
        if (a.dr) load<VEC>(static_cast<const TR*>(a.dr) + row * a.d + c, dr[i]);
        if (a.ow) {
          if (a.res) load<VEC>(static_cast<const TR*>(a.res) + row * a.d + c, rs[i]);
          if (a.dy) load<VEC>(static_cast<const T*>(a.dy) + row * a.d + c, dy[i]);
        }
      }
    }
    auto value = [&](int i, int e) {  // v: the norm's input
      return a.gate_act && a.gate_first ? xv[i][e] * gate_of(gv[i][e], a.gate_act) : xv[i][e];
    };
    float k = 1.f, ss = 0.f;
    if (a.w) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(value(i, e), value(i, e), ss);
      k = rsqrtf(row_sum<TPR>(ss, scratch, flip) / a.d + a.eps);
    }
    // the branch before its scale, b = m z, and then the sum r (in rs)
    auto branch = [&](int i, int e, float w) {
      float m = a.w ? value(i, e) * k * w : value(i, e);
      return after ? m * gate_of(gv[i][e], a.gate_act) : m;
    };
    if (a.ow) {
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (lane + i * TPR) * VEC;
        if (c < a.d) {
          float w[VEC], ls[VEC];
          if (a.w) load<VEC>(a.w + c, w);
          if (a.ls) load<VEC>(a.ls + c, ls);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float s = a.ls ? a.scale * ls[e] : a.scale;
            rs[i][e] = fmaf(s, branch(i, e, w[e]), rs[i][e]);
            ss = fmaf(rs[i][e], rs[i][e], ss);
          }
        }
      }
      const float ko = rsqrtf(row_sum<TPR>(ss, scratch, flip) / a.d + a.eps);
      float pn = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (lane + i * TPR) * VEC;
        if (c < a.d) {
          float ow[VEC];
          load<VEC>(a.ow + c, ow);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            rs[i][e] *= ko;  // n
            so[i][e] = fmaf(dy[i][e], rs[i][e], so[i][e]);
            dy[i][e] *= ow[e];  // p
            pn = fmaf(dy[i][e], rs[i][e], pn);
          }
        }
      }
      pn = row_sum<TPR>(pn, scratch, flip) / a.d;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          dr[i][e] = fmaf(ko, dy[i][e] - rs[i][e] * pn, dr[i][e]);
    }
    // through the residual sum and the branch
    float pn = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * TPR) * VEC;
      if (c < a.d) {
        float w[VEC], ls[VEC];
        if (a.w) load<VEC>(a.w + c, w);
        if (a.ls) load<VEC>(a.ls + c, ls);
        if (a.dres && on) store<VEC>(static_cast<TR*>(a.dres) + row * a.d + c, dr[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float s = a.ls ? a.scale * ls[e] : a.scale;
          const float v = value(i, e), n = v * k;
          const float m = a.w ? n * w[e] : v;
          const float z = a.gate_act ? gate_of(gv[i][e], a.gate_act) : 1.f;
          if (a.ls) sl[i][e] = fmaf(a.scale * dr[i][e], after ? m * z : m, sl[i][e]);
          float db = s * dr[i][e];
          if (after) {
            rs[i][e] = db * m * gate_slope(gv[i][e], a.gate_act);  // dgate
            db *= z;
          }
          if (a.w) {
            sw[i][e] = fmaf(db, n, sw[i][e]);
            db *= w[e];  // p
            pn = fmaf(db, n, pn);
          }
          dr[i][e] = db;
        }
      }
    }
    if (a.w) pn = row_sum<TPR>(pn, scratch, flip) / a.d;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * TPR) * VEC;
      if (on && c < a.d) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float dv = a.w ? k * (dr[i][e] - value(i, e) * k * pn) : dr[i][e];
          if (a.gate_act && a.gate_first) {
            rs[i][e] = dv * xv[i][e] * gate_slope(gv[i][e], a.gate_act);
            dv *= gate_of(gv[i][e], a.gate_act);
          }
          dr[i][e] = dv;
        }
        if (a.dx) store<VEC>(static_cast<T*>(a.dx) + row * a.d + c, dr[i]);
        if (a.dgate) store<VEC>(static_cast<T*>(a.dgate) + row * a.d + c, rs[i]);
      }
    }
  }
  // the block's sums: with several rows per block, its row groups are added first
  float* part = a.part + (int64_t)blockIdx.x * 3 * a.d;
  if constexpr (kRows > 1) {
    __shared__ float fold[kRows][TPR * VEC];
    auto put = [&](float (&s)[NC][VEC], int which) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) fold[threadIdx.x / TPR][lane * VEC + e] = s[i][e];
        __syncthreads();
        for (int j = threadIdx.x; j < TPR * VEC; j += blockDim.x) {
          float t = 0.f;
#pragma unroll
          for (int q = 0; q < kRows; ++q) t += fold[q][j];
          const int c = i * TPR * VEC + j;
          if (c < a.d) part[(int64_t)which * a.d + c] = t;
        }
      }
    };
    if (a.dw) put(sw, 0);
    if (a.dls) put(sl, 1);
    if (a.dow) put(so, 2);
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * TPR) * VEC;
      if (c < a.d) {
        if (a.dw) store<VEC>(part + c, sw[i]);
        if (a.dls) store<VEC>(part + a.d + c, sl[i]);
        if (a.dow) store<VEC>(part + 2 * (int64_t)a.d + c, so[i]);
      }
    }
  }
}

// one warp row per 32 columns: 8 warps take every 8th block's sums, then fold
__global__ void __launch_bounds__(256) norm_reduce_kernel(NormArgs a) {
  __shared__ float fold[8][33];
  const int which = blockIdx.y;
  float* out = which == 0 ? a.dw : which == 1 ? a.dls : a.dow;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.d) {
#pragma unroll 8
    for (int64_t b = warp; b < a.ctas; b += 8) s += a.part[(b * 3 + which) * a.d + c];
  }
  fold[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += fold[q][lane];
    out[c] = s;
  }
}

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }
bool wide_ok(const NormArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  const void* ptrs[] = {a.x, a.gate, a.res, a.dr, a.dy, a.w, a.ls, a.ow, a.r,
                        a.y, a.dx, a.dgate, a.dres};
  bool wide = a.d % v == 0 && a.ldx % v == 0 && a.ldg % v == 0;
  for (const void* p : ptrs) wide = wide && al16(p);
  return wide;
}

template <typename T, typename TR, int VEC, int NC, int TPR>
cudaError_t run(const NormArgs& a, bool bwd) {
  constexpr int kRows = block_of<TPR>() / TPR;
  const int64_t rows = a.tokens * a.heads;
  if (bwd) {
    norm_bwd_kernel<T, TR, VEC, NC, TPR><<<(unsigned)a.ctas, block_of<TPR>(), 0, a.stream>>>(a);
  } else {
    const int64_t grid = (rows + kRows - 1) / kRows;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    norm_fwd_kernel<T, TR, VEC, NC, TPR><<<(unsigned)grid, block_of<TPR>(), 0, a.stream>>>(a);
  }
  return cudaGetLastError();
}

// threads per row by the row's chunks: up to 32 the row stays inside a warp
template <typename T, typename TR, int VEC>
cudaError_t by_size(const NormArgs& a, bool bwd) {
  const int chunks = (a.d + VEC - 1) / VEC;
  if constexpr (VEC == 1) {
    if (chunks <= 128) return run<T, TR, 1, 4, 32>(a, bwd);
    if (chunks <= 1024) return run<T, TR, 1, 4, 256>(a, bwd);
    return run<T, TR, 1, 8, 1024>(a, bwd);
  } else {
    if (chunks <= 8) return run<T, TR, VEC, 1, 8>(a, bwd);
    if (chunks <= 16) return run<T, TR, VEC, 1, 16>(a, bwd);
    if (chunks <= 32) return run<T, TR, VEC, 1, 32>(a, bwd);
    if (chunks <= 128) return run<T, TR, VEC, 1, 128>(a, bwd);
    if (chunks <= 256) return run<T, TR, VEC, 1, 256>(a, bwd);
    if (chunks <= 512) return run<T, TR, VEC, 1, 512>(a, bwd);
    if (chunks <= 1024) return run<T, TR, VEC, 1, 1024>(a, bwd);
    return run<T, TR, VEC, 2, 1024>(a, bwd);  // float32 rows past 4096 channels
  }
}
cudaError_t by_type(const NormArgs& a, bool bwd) {
  const bool wide = wide_ok(a);
  if (!a.bf16)
    return wide ? by_size<float, float, 4>(a, bwd) : by_size<float, float, 1>(a, bwd);
  using bf = __nv_bfloat16;
  if (a.res_bf16)
    return wide ? by_size<bf, bf, 8>(a, bwd) : by_size<bf, bf, 1>(a, bwd);
  return wide ? by_size<bf, float, 8>(a, bwd) : by_size<bf, float, 1>(a, bwd);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a) { return by_type(a, false); }

int64_t norm_bwd_ctas(int64_t rows, int d, bool bf16, int64_t sms) {
  (void)d; (void)bf16;
  const int64_t most = 4 * sms;
  return rows < 1 ? 1 : rows < most ? rows : most;
}

cudaError_t launch_norm_bwd(const NormArgs& a) {
  cudaError_t e = by_type(a, true);
  if (e != cudaSuccess) return e;
  if (!a.dw && !a.dls && !a.dow) return cudaSuccess;
  norm_reduce_kernel<<<dim3((unsigned)((a.d + 31) / 32), 3), 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace kda
