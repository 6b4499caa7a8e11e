// Short causal convolution over the tokens of each channel: prompts, single
// tokens and the gradient.
//
//     u[t] = bias + sum_{j < W} w[j] x[t - (W - 1) + j],   y = silu(u) or u
//
// Every input and output is touched once and there are W multiply-adds per
// element: the work is bound by memory traffic.  A thread owns VEC channels (16
// bytes) and walks a tile of tokens with the window of W - 1 earlier inputs in
// registers, so a tile re-reads only the W - 1 tokens before it; the loads of
// kAhead tokens are issued together, ahead of their use.  Sequence boundaries
// of a packed batch are found once per tile by bisection and then followed.
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // tokens whose loads are in flight together

// the window of W - 1 inputs before token t of sequence n, whose tokens start at s0
template <int VEC, int W, typename T>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* init, int64_t t,
                                            int64_t s0, int n, int D, int c, float (&win)[W - 1][VEC]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int64_t p = t - (W - 1) + i;
    if (p >= s0) {
      load<VEC>(x + p * ldx + c, win[i]);
    } else if (init) {  // row p - s0 + W - 1 of the start state
      load<VEC>(init + ((int64_t)n * (W - 1) + (p - s0 + W - 1)) * D + c, win[i]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[i][e] = 0.f;
    }
  }
}

template <int VEC, int W>
__device__ __forceinline__ void load_params(const float* w, const float* b, int c,
                                            float (&wr)[W][VEC], float (&br)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    br[e] = b ? b[c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) wr[j][e] = w[(int64_t)(c + e) * W + j];
  }
}

template <int VEC, int W>
__device__ __forceinline__ void shift_in(float (&win)[W - 1][VEC], const float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < W - 2; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) win[i][e] = win[i + 1][e];
#pragma unroll
  for (int e = 0; e < VEC; ++e) win[W - 2][e] = x[e];
}

// Blocks [0, cblocks * tiles): one tile of tokens and kThreads * VEC channels
// each; the rest: the final state of one sequence.
template <typename T, int VEC, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(ConvArgs a, int cblocks) {
  const T* x = static_cast<const T*>(a.x);
  const T* init = static_cast<const T*>(a.init);
  const int cb = blockIdx.x % cblocks;
  const int64_t job = blockIdx.x / cblocks;
  if (blockIdx.x == 0) check_seqlens(a.q, a.status);
  const int c = (cb * kThreads + threadIdx.x) * VEC;
  if (c >= a.D) return;
  if (job >= a.tiles) {
    const int n = (int)(job - a.tiles);
    int64_t s0, s1;
    a.q.range(n, s0, s1);
    float win[W - 1][VEC];
    load_window<VEC, W>(x, a.ldx, init, s1, s0, n, a.D, c, win);
    T* f = static_cast<T*>(a.fin) + (int64_t)n * (W - 1) * a.D + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store<VEC>(f + (int64_t)i * a.D, win[i]);
    return;
  }
  float wr[W][VEC], br[VEC], win[W - 1][VEC];
  load_params<VEC, W>(a.w, a.b, c, wr, br);
  const int64_t t0 = job * a.tile;
  const int64_t t1 = t0 + a.tile < a.q.total ? t0 + a.tile : a.q.total;
  int n = a.q.find(t0);
  int64_t s0, s1;
  a.q.range(n, s0, s1);
  load_window<VEC, W>(x, a.ldx, init, t0, s0, n, a.D, c, win);
  T* y = static_cast<T*>(a.y) + c;
  for (int64_t t = t0; t < t1; t += kAhead) {
    float xa[kAhead][VEC];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < t1) load<VEC>(x + (t + i) * a.ldx + c, xa[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i >= t1) break;
      if (t + i >= s1 && n + 1 < a.q.N) {  // the next sequence with tokens starts here
        do a.q.range(++n, s0, s1);
        while (t + i >= s1 && n + 1 < a.q.N);
        load_window<VEC, W>(x, a.ldx, init, t + i, s0, n, a.D, c, win);
      }
      float u[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[e] = fmaf(wr[W - 1][e], xa[i][e], br[e]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) u[e] = fmaf(wr[j][e], win[j][e], u[e]);
        if (kSilu) u[e] *= sigmoid(u[e]);
      }
      store<VEC>(y + (t + i) * a.D, u);
      shift_in<VEC, W>(win, xa[i]);
    }
  }
}

// One block row per sequence: T tokens in order, the state in registers.
template <typename T, int VEC, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(ConvArgs a, int cblocks) {
  const T* x = static_cast<const T*>(a.x);
  const int cb = blockIdx.x % cblocks, n = blockIdx.x / cblocks;
  if (blockIdx.x == 0) check_counts(a.counts, a.q.N, a.T, a.status);
  const int c = (cb * kThreads + threadIdx.x) * VEC;
  if (c >= a.D) return;
  T* st = static_cast<T*>(a.state) + (int64_t)n * (W - 1) * a.D + c;
  float wr[W][VEC], br[VEC], win[W - 1][VEC];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) load<VEC>(st + (int64_t)i * a.D, win[i]);
  load_params<VEC, W>(a.w, a.b, c, wr, br);
  int keep = a.T;
  if (a.counts) {
    keep = a.counts[n];
    if (keep < 0 || keep > a.T) keep = 0;
  }
  for (int t = 0; t < a.T; ++t) {
    float xt[VEC], u[VEC];
    load<VEC>(x + ((int64_t)n * a.T + t) * a.ldx + c, xt);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      u[e] = fmaf(wr[W - 1][e], xt[e], br[e]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) u[e] = fmaf(wr[j][e], win[j][e], u[e]);
      if (kSilu) u[e] *= sigmoid(u[e]);
    }
    if (a.y) store<VEC>(static_cast<T*>(a.y) + ((int64_t)n * a.T + t) * a.D + c, u);
    shift_in<VEC, W>(win, xt);
    if (t + 1 == keep) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i) store<VEC>(st + (int64_t)i * a.D, win[i]);
    }
  }
}

// Gradient.  With du = dy silu'(u): dx[s] = sum_k w[W-1-k] du[s+k] over the
// sequence's tokens, dw[j] = sum_t du[t] x[t-(W-1)+j], dbias = sum_t du[t].
// A thread walks its tile and the W - 1 tokens after it (recomputing their du),
// keeping the dx of the last W - 1 tokens unfinished in registers; the tile's
// sums for dw and dbias go to part[tile][W + 1][D] and are added in the order of
// the tiles by conv_reduce_kernel, so the results do not depend on scheduling.
template <typename T, int VEC, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads)
conv_bwd_kernel(ConvArgs a, int cblocks) {
  const T* x = static_cast<const T*>(a.x);
  const T* init = static_cast<const T*>(a.init);
  const T* dy = static_cast<const T*>(a.dy);
  const T* dfin = static_cast<const T*>(a.dfinal);
  const int cb = blockIdx.x % cblocks;
  const int64_t job = blockIdx.x / cblocks;
  if (blockIdx.x == 0) check_seqlens(a.q, a.status);
  const int c = (cb * kThreads + threadIdx.x) * VEC;
  if (c >= a.D) return;
  float wr[W][VEC], br[VEC], win[W - 1][VEC];
  load_params<VEC, W>(a.w, a.b, c, wr, br);
  auto grad_u = [&](const float (&xt)[VEC], const float (&g)[VEC], float (&du)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (kSilu) {
        float u = fmaf(wr[W - 1][e], xt[e], br[e]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) u = fmaf(wr[j][e], win[j][e], u);
        const float s = sigmoid(u);
        du[e] = g[e] * s * fmaf(u, 1.f - s, 1.f);
      } else {
        du[e] = g[e];
      }
    }
  };
  if (job >= a.tiles) {  // gradient of the start state of one sequence
    const int n = (int)(job - a.tiles);
    int64_t s0, s1;
    a.q.range(n, s0, s1);
    const int len = s1 - s0 < W - 1 ? (int)(s1 - s0) : W - 1;
    load_window<VEC, W>(x, a.ldx, init, s0, s0, n, a.D, c, win);
    float dst[W - 1][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dst[i][e] = 0.f;
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      if (t < len) {
        float xt[VEC], g[VEC], du[VEC];
        load<VEC>(x + (s0 + t) * a.ldx + c, xt);
        load<VEC>(dy + (s0 + t) * a.D + c, g);
        grad_u(xt, g, du);
#pragma unroll
        for (int i = t; i < W - 1; ++i)  // row i meets token t at tap i - t
#pragma unroll
          for (int e = 0; e < VEC; ++e) dst[i][e] = fmaf(wr[i - t][e], du[e], dst[i][e]);
        shift_in<VEC, W>(win, xt);
      }
    }
    T* o = static_cast<T*>(a.dinit) + (int64_t)n * (W - 1) * a.D + c;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      if (dfin && i >= len) {  // a short sequence hands these rows on to its final state
        float g[VEC];
        load<VEC>(dfin + ((int64_t)n * (W - 1) + i - len) * a.D + c, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dst[i][e] += g[e];
      }
      store<VEC>(o + (int64_t)i * a.D, dst[i]);
    }
    return;
  }
  float dw[W][VEC], db[VEC], pend[W - 1][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) pend[k][e] = 0.f;
  }
  const int64_t t0 = job * a.tile;
  const int64_t t1 = t0 + a.tile < a.q.total ? t0 + a.tile : a.q.total;
  int n = a.q.find(t0);
  int64_t s0, s1;
  a.q.range(n, s0, s1);
  load_window<VEC, W>(x, a.ldx, init, t0, s0, n, a.D, c, win);
  T* dx = static_cast<T*>(a.dx) + c;
  // the dx of the last tokens before `end` of sequence n (pend[k]: token end-1-k),
  // which no later token of the sequence adds to
  auto flush = [&](int64_t end) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int64_t s = end - 1 - k;
      if (s >= t0 && s >= s0 && s < t1) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = pend[k][e];
        if (dfin) {
          float g[VEC];
          load<VEC>(dfin + ((int64_t)n * (W - 1) + (W - 2 - k)) * a.D + c, g);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] += g[e];
        }
        store<VEC>(dx + s * a.D, o);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) pend[k][e] = 0.f;
    }
  };
  int64_t stop = t1 + W - 1 < a.q.total ? t1 + W - 1 : a.q.total;
  bool ended = false;  // the walk stops at a sequence's end at or after t1
  for (int64_t t = t0; t < stop && !ended; t += kAhead) {
    float xa[kAhead][VEC], ga[kAhead][VEC];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < stop) {
        load<VEC>(x + (t + i) * a.ldx + c, xa[i]);
        load<VEC>(dy + (t + i) * a.D + c, ga[i]);
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = t + i;
      if (p >= stop || ended) break;
      if (p >= s1 && n + 1 < a.q.N) {
        flush(s1);
        if (p >= t1) {
          ended = true;
          break;
        }
        do a.q.range(++n, s0, s1);
        while (p >= s1 && n + 1 < a.q.N);
        load_window<VEC, W>(x, a.ldx, init, p, s0, n, a.D, c, win);
      }
      float du[VEC];
      grad_u(xa[i], ga[i], du);
      const int64_t s = p - (W - 1);
      if (s >= t0 && s >= s0) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(wr[0][e], du[e], pend[W - 2][e]);
        store<VEC>(dx + s * a.D, o);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int k = W - 2; k > 0; --k) pend[k][e] = fmaf(wr[W - 1 - k][e], du[e], pend[k - 1][e]);
        pend[0][e] = wr[W - 1][e] * du[e];
        if (p < t1) {
          db[e] += du[e];
          dw[W - 1][e] = fmaf(du[e], xa[i][e], dw[W - 1][e]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(du[e], win[j][e], dw[j][e]);
        }
      }
      shift_in<VEC, W>(win, xa[i]);
    }
  }
  if (!ended && s1 <= stop) flush(s1);
  float* pt = a.part + job * (W + 1) * (int64_t)a.D + c;
#pragma unroll
  for (int j = 0; j < W; ++j) store<VEC>(pt + (int64_t)j * a.D, dw[j]);
  store<VEC>(pt + (int64_t)W * a.D, db);
}

__global__ void __launch_bounds__(256) conv_reduce_kernel(ConvArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = (int64_t)(a.W + 1) * a.D;
  if (i >= per) return;
  float sum = 0.f;
#pragma unroll 8
  for (int64_t t = 0; t < a.tiles; ++t) sum += a.part[t * per + i];
  const int j = (int)(i / a.D), c = (int)(i % a.D);
  if (j < a.W) a.dw[(int64_t)c * a.W + j] = sum;
  else if (a.db) a.db[c] = sum;
}

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <typename T, int VEC, int W>
cudaError_t run(const ConvArgs& a, int what) {
  const int cblocks = (a.D + kThreads * VEC - 1) / (kThreads * VEC);
  const int64_t extra = what == 0 ? (a.fin ? a.q.N : 0) : what == 2 ? (a.dinit ? a.q.N : 0) : 0;
  const int64_t jobs = what == 1 ? a.q.N : a.tiles + extra;
  const int64_t grid = jobs * cblocks;
  if (grid == 0)  // nothing to check or to compute
    return a.status ? cudaMemsetAsync(a.status, 0, sizeof(unsigned int), a.stream) : cudaSuccess;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
#define KDA_CONV(KERNEL)                                                             \
  (a.silu ? KERNEL<T, VEC, W, true><<<(unsigned)grid, kThreads, 0, a.stream>>>(a, cblocks) \
          : KERNEL<T, VEC, W, false><<<(unsigned)grid, kThreads, 0, a.stream>>>(a, cblocks))
  if (what == 0) KDA_CONV(conv_fwd_kernel);
  else if (what == 1) KDA_CONV(conv_step_kernel);
  else KDA_CONV(conv_bwd_kernel);
#undef KDA_CONV
  return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t by_width(const ConvArgs& a, int what) {
  switch (a.W) {
    case 2: return run<T, VEC, 2>(a, what);
    case 3: return run<T, VEC, 3>(a, what);
    default: return run<T, VEC, 4>(a, what);
  }
}
// wide loads where every row of every operand starts on a 16-byte boundary
cudaError_t by_type(const ConvArgs& a, int what) {
  const int v = what == 2 ? 4 : (a.bf16 ? 8 : 4);
  const void* ptrs[] = {a.x, a.init, a.dy, a.dfinal, a.y, a.fin, a.dx, a.dinit, a.state};
  bool wide = a.D % v == 0 && a.ldx % v == 0;
  for (const void* p : ptrs) wide = wide && al16(p);
  if (what == 2)
    return a.bf16 ? (wide ? by_width<__nv_bfloat16, 4>(a, what) : by_width<__nv_bfloat16, 1>(a, what))
                  : (wide ? by_width<float, 4>(a, what) : by_width<float, 1>(a, what));
  if (a.bf16)
    return wide ? by_width<__nv_bfloat16, 8>(a, what) : by_width<__nv_bfloat16, 1>(a, what);
  return wide ? by_width<float, 4>(a, what) : by_width<float, 1>(a, what);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a0) {
  ConvArgs a = a0;
  // tiles of 64 tokens re-read 5% of x at W = 4; short inputs take smaller ones, for more blocks
  const int64_t per = kThreads * (a.bf16 ? 8 : 4);
  const int64_t cb = (a.D + per - 1) / per;
  a.tile = 64;
  while (a.tile > 8 && cb * ((a.q.total + a.tile - 1) / a.tile) < 4 * 152) a.tile /= 2;
  a.tiles = (a.q.total + a.tile - 1) / a.tile;
  return by_type(a, 0);
}

cudaError_t launch_conv_step(const ConvArgs& a) { return by_type(a, 1); }

int64_t conv_bwd_tile(int64_t tokens, int D, int64_t sms) {
  const int64_t cb = (D + kThreads * 4 - 1) / (kThreads * 4);
  int64_t tile = 256;
  while (tile > 16 && cb * ((tokens + tile - 1) / tile) < 8 * sms) tile /= 2;
  return tile;
}

cudaError_t launch_conv_bwd(const ConvArgs& a) {
  cudaError_t e = by_type(a, 2);
  if (e != cudaSuccess) return e;
  const int64_t per = (int64_t)(a.W + 1) * a.D;
  conv_reduce_kernel<<<(unsigned)((per + 255) / 256), 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace kda
