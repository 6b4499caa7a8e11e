// RMS norms with gate and residual scale: the gradient (see kda_norm.cuh).
//
// For n = v k, y = n w:  dv = k (p - n mean(p n)) with p = dy w, and dw = sum over rows
// of dy n.  Each block keeps its rows' sums for the parameters in registers; they go to
// part[block][3][d] and are added in the order of the blocks, so that the results do not
// depend on scheduling.
#include <algorithm>

#include "kda_norm.cuh"

namespace kda {
namespace layer {
namespace {

using namespace norm;

// threads per SM: what the registers of one row allow (rows inside a warp take more of them:
// 128 MB in rows of 128 take 161 us with 384 threads, 166 with 512, which spill)
constexpr int resident(bool long_row) { return long_row ? 512 : 384; }

template <typename T, typename TR, int VEC, int NC, int TPR, int PLACE>
__global__ void __launch_bounds__(block_of<TPR>(), TPR > 256 ? 1 : resident(TPR > 32) / block_of<TPR>())
norm_bwd_kernel(NormArgs a) {
  constexpr int kRows = block_of<TPR>() / TPR;
  __shared__ float2 scratch[2][32];
  int flip = 0;
  const int64_t rows = a.tokens * a.heads, step = (int64_t)gridDim.x * kRows;
  const int lane = threadIdx.x % TPR;
  const bool silu = a.gate_act == KDA_GATE_SILU;
  float sw[NC][VEC], sl[NC][VEC], so[NC][VEC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sw[i][e] = sl[i][e] = so[i][e] = 0.f;
  RowIn<T, TR, VEC, NC, true> in;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  request<T, TR, VEC, NC, TPR, PLACE, true>(a, row, lane, in);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < rows; base += step, row += step) {
    const bool on = row < rows;
    // n: the norm's input v, then v k;  z, sz: the gate and (x's factor in) its slope;
    // r: residual, then n of the outer norm;  dr: gradient of r, then of the branch
    float n[NC][VEC], z[NC][VEC], sz[NC][VEC], r[NC][VEC], dr[NC][VEC], dy[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      open<T, VEC>(in.x[i], n[i]);
      if (PLACE != kNoGate) open<T, VEC>(in.g[i], z[i]);
      open<TR, VEC>(in.res[i], r[i]);
      open<TR, VEC>(in.dr[i], dr[i]);
      open<T, VEC>(in.dy[i], dy[i]);
    }
    request<T, TR, VEC, NC, TPR, PLACE, true>(a, row + step, lane, in);
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (PLACE != kNoGate) {
        float s[VEC];
        sigmoid_v(z[i], s);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          sz[i][e] = gate_slope(z[i][e], s[e], silu);
          z[i][e] = gate_of(z[i][e], s[e], silu);
        }
      }
      if (PLACE == kFirst) {
        mul_v(sz[i], n[i]);
        mul_v(n[i], z[i]);
      }
      dot_v(n[i], n[i], ss);
    }
    // A place without a row holds zeros, of which 1 / rms is infinite with eps = 0: it gets 0, so that
    // the sums over rows take nothing from it.
    float k = 1.f;
    if (a.w) {
      k = rsqrtf(fmaf(row_sum<TPR>(ss.x + ss.y, scratch, flip), a.inv_d, a.eps));
      if (!on) k = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) mul_v(n[i], k);
    }
    if (a.ow) {
      float2 rr = make_float2(0.f, 0.f), pr = rr;  // r . r and p . r: p . n is k2 times the second
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (lane + i * row_threads<TPR>()) * VEC;
        if (c < a.d) {
          float w[VEC], ls[VEC], p[VEC];
          param<VEC>(a.w, c, 1.f, w);
          param<VEC>(a.ls, c, a.scale, ls);
          param<VEC>(a.ow, c, 1.f, p);
          mul_v(w, n[i]);
          if (PLACE == kAfter) mul_v(w, z[i]);
          fma_v(ls, w, r[i]);
          dot_v(r[i], r[i], rr);
          mul_v(p, dy[i]);
          dot_v(p, r[i], pr);
        }
      }
      const float2 s = row_sums<TPR>(rr.x + rr.y, pr.x + pr.y, scratch, flip);
      const float k2 = on ? rsqrtf(fmaf(s.x, a.inv_d, a.eps)) : 0.f, mean = k2 * k2 * s.y * a.inv_d;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (lane + i * row_threads<TPR>()) * VEC;
        if (c < a.d) {
          float p[VEC], t[VEC];
          param<VEC>(a.ow, c, 1.f, p);
          mul_v(p, dy[i]);
          fma_v(r[i], -mean, p);
          fma_v(p, k2, dr[i]);
          copy_v(r[i], t);
          mul_v(t, k2);
          fma_v(dy[i], t, so[i]);
        }
      }
    }
    // through the residual sum and the branch; dgate (gate after) in sz
    float2 pn = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (c < a.d) {
        float w[VEC], db[VEC], b[VEC];
        param<VEC>(a.w, c, 1.f, w);
        param<VEC>(a.ls, c, a.scale, db);
        if (a.dres && on) store<VEC>(static_cast<TR*>(a.dres) + row * a.d + c, dr[i]);
        mul_v(db, dr[i]);
        copy_v(n[i], b);
        mul_v(b, w);
        if (PLACE == kAfter) {
          mul_v(sz[i], b);
          mul_v(sz[i], db);
          mul_v(b, z[i]);
          mul_v(db, z[i]);
        }
        fma_v(dr[i], b, sl[i]);  // times the scale at the end
        fma_v(db, n[i], sw[i]);
        mul_v(db, w);  // p
        dot_v(db, n[i], pn);
        copy_v(db, dr[i]);
      }
    }
    const float mean = a.w ? row_sum<TPR>(pn.x + pn.y, scratch, flip) * a.inv_d : 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (on && c < a.d) {
        fma_v(n[i], -mean, dr[i]);
        mul_v(dr[i], k);
        if (PLACE == kFirst) {
          mul_v(sz[i], dr[i]);
          mul_v(dr[i], z[i]);
        }
        store<VEC>(static_cast<T*>(a.dx) + row * a.d + c, dr[i]);
        if (PLACE != kNoGate && a.dgate) store<VEC>(static_cast<T*>(a.dgate) + row * a.d + c, sz[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sl[i][e] *= a.scale;
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
      const int c = (lane + i * row_threads<TPR>()) * VEC;
      if (c < a.d) {
        if (a.dw) store<VEC>(part + c, sw[i]);
        if (a.dls) store<VEC>(part + a.d + c, sl[i]);
        if (a.dow) store<VEC>(part + 2 * (int64_t)a.d + c, so[i]);
      }
    }
  }
}

// 32 columns per block: its warps take every kWarps-th block's sums, then fold
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) norm_reduce_kernel(NormArgs a) {
  __shared__ float fold[kWarps][33];
  const int which = blockIdx.y;
  float* out = which == 0 ? a.dw : which == 1 ? a.dls : a.dow;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.d) {
#pragma unroll 8
    for (int64_t b = warp; b < a.ctas; b += kWarps) s += a.part[(b * 3 + which) * a.d + c];
  }
  fold[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
#pragma unroll
    for (int q = 1; q < kWarps; ++q) s += fold[q][lane];
    out[c] = s;
  }
}

template <typename T, typename TR, int VEC, int NC, int TPR, int PLACE>
struct Backward {
  static constexpr bool kPairs = false;
  static cudaError_t run(const NormArgs& a) {
    norm_bwd_kernel<T, TR, VEC, NC, TPR, PLACE>
        <<<(unsigned)a.ctas, threads_of<VEC, NC, TPR>(a.d), 0, a.stream>>>(a);
    return cudaGetLastError();
  }
};

}  // namespace

// Blocks of the backward: those that are resident together, no more than there are rows for.
// It follows by_size; without the alignment for wide accesses a row takes more threads.
static int64_t blocks_of(int64_t rows, int d, bool bf16, bool wide, int64_t sms) {
  const int chunks = (d + (bf16 ? 8 : 4) - 1) / (bf16 ? 8 : 4);
  int per, threads;  // rows and threads of a block
  if (wide) {
    per = chunks <= 8 ? 16 : chunks <= 16 ? 8 : chunks <= 32 ? 4 : 1;
    threads = per > 1 ? 128 : (chunks + 31) / 32 * 32;
  } else {
    const int part = d <= 1024 ? 128 : 256;  // elements of a warp
    per = d <= 128 ? 4 : 1;
    threads = per > 1 ? 128 : (d + part - 1) / part * 32;
  }
  const int64_t most = threads > 512 ? sms : resident(per == 1) / threads * sms;
  const int64_t blocks = (rows + per - 1) / per;
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

int64_t norm_bwd_ctas(int64_t rows, int d, bool bf16, int64_t sms) {
  return std::max(blocks_of(rows, d, bf16, true, sms), blocks_of(rows, d, bf16, false, sms));
}

cudaError_t launch_norm_bwd(NormArgs a) {
  a.ctas = blocks_of(a.tokens * a.heads, a.d, a.bf16, wide_ok(a), a.sms);
  cudaError_t e = by_type<Backward>(a);
  if (e != cudaSuccess) return e;
  if (!a.dw && !a.dls && !a.dow) return cudaSuccess;
  const dim3 grid((unsigned)((a.d + 31) / 32), 3);
  // with few columns the sums' latency counts, with many the blocks' number: 2048 rows of 512 take
  // 9.4 us on the GPU with 32 warps and 10.4 with 16, 256 rows of 4096 9.5 and 8.4
  if (a.d <= 2048) norm_reduce_kernel<32><<<grid, 1024, 0, a.stream>>>(a);
  else norm_reduce_kernel<16><<<grid, 512, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace kda
