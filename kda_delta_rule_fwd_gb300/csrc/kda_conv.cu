// Short causal convolution over the tokens of each channel: prompts, single
// tokens and the gradient.
//
//     u[t] = bias + sum_{j < W} w[j] x[t - (W - 1) + j],   y = silu(u) or u
//
// Every input and output is touched once and there are W multiply-adds per
// element: the work is bound by memory traffic.  A thread owns VEC channels (16
// bytes) and walks a tile of tokens with the window of
// W - 1 earlier inputs in registers, so a tile re-reads only the W - 1 tokens
// before it.  The wide path keeps the next tokens' inputs in flight into shared
// memory (cp.async, each thread for itself, so that no barrier is needed): bytes in
// flight then cost no registers.  Sequence boundaries of a packed batch are found
// once per tile by bisection and then followed.
//
// 12288 channels of width 4 in bf16 on one GB300: 58511 packed tokens take 433 us (6.6 TB/s,
// a copy's rate); one token of each of 1024 sequences 37 us (5.4 TB/s; the
// floor is 30 us, and 33 us pass on the GPU when the launch is replayed from a graph); the
// gradient of 16384 tokens 246 us (4.9 TB/s): 32 instructions per element, for which 12 warps per SM
// (168 registers) fill 65% of the issue slots.
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 128;
constexpr int kStepBlocks = 4, kBwdBlocks = 3;  // resident per SM, by their registers
// A thread's own ring of kSlots vectors in shared memory, filled ahead by cp.async.
// Narrow elements (VEC = 1) are below the copy's smallest size: they are loaded in place.
template <typename T, int VEC, int kSlots>
struct Ring {
  Raw<T, VEC>* mine;  // this thread's slot 0
  __device__ __forceinline__ Raw<T, VEC>& slot(int64_t i) const { return mine[(i % kSlots) * kThreads]; }
  __device__ __forceinline__ void request(int64_t i, const T* src) const {
    if constexpr (VEC > 1) {
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(&slot(i));
      static_assert(sizeof(Raw<T, VEC>) == 16, "one copy per vector");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    } else {
      slot(i) = fetch<T, VEC>(src);
    }
  }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The window of W - 1 inputs before token t of sequence n, whose tokens start at s0.  Offsets
// that do not begin with 0 leave tokens before the first sequence (t < s0): they have neither
// inputs nor a row of the start state before them, and get zeros.
template <int VEC, int W, typename T>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* init, int64_t t,
                                            int64_t s0, int n, int D, int c, float (&win)[W - 1][VEC]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int64_t p = t - (W - 1) + i;
    if (p >= s0) {
      load<VEC>(x + p * ldx + c, win[i]);
    } else if (init && p - s0 + W - 1 >= 0) {  // that row of the start state
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
    if constexpr (W == 4 && VEC > 1) {  // 16-byte aligned where the wide path is taken
      const float4 v = *reinterpret_cast<const float4*>(w + (int64_t)(c + e) * 4);
      wr[0][e] = v.x; wr[1][e] = v.y; wr[2][e] = v.z; wr[3][e] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) wr[j][e] = w[(int64_t)(c + e) * W + j];
    }
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

// u of one token from its window
template <int VEC, int W>
__device__ __forceinline__ void taps(const float (&wr)[W][VEC], const float (&br)[VEC],
                                     const float (&win)[W - 1][VEC], const float (&x)[VEC],
                                     float (&u)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) u[e] = br[e];
  fma_v(wr[W - 1], x, u);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) fma_v(wr[j], win[j], u);
}

// Blocks [0, cblocks * tiles): one tile of tokens and kThreads * VEC channels
// each; the rest: the final state of one sequence.
template <typename T, int VEC, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads, 5)
conv_fwd_kernel(ConvArgs a, int cblocks) {
  constexpr int kGroup = 4, kGroups = 4;  // tokens per group of copies, groups in the ring
  __shared__ __align__(16) Raw<T, VEC> ring_mem[kGroup * kGroups * kThreads];
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
  auto token = [&](int64_t t, const Raw<T, VEC>& raw) {
    float xt[VEC], u[VEC];
    open<T, VEC>(raw, xt);
    taps<VEC, W>(wr, br, win, xt, u);
    if (kSilu) {
      float s[VEC];
      sigmoid_v(u, s);
      mul_v(u, s);
    }
    store<VEC>(y + t * a.D, u);
    shift_in<VEC, W>(win, xt);
  };
  const Ring<T, VEC, kGroup * kGroups> ring{ring_mem + threadIdx.x};
  const int count = (int)(t1 - t0);
  const T* src = x + t0 * a.ldx + c;
  auto request = [&](int i0) {  // the group of copies that starts at the tile's token i0
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (i0 + i < count) ring.request(i0 + i, src + (i0 + i) * a.ldx);
    ring_commit();
  };
#pragma unroll
  for (int g = 0; g < kGroups - 1; ++g) request(g * kGroup);
  for (int i0 = 0; i0 < count; i0 += kGroup) {
    request(i0 + (kGroups - 1) * kGroup);
    ring_wait<kGroups - 1>();
    const int64_t t = t0 + i0;
    if (i0 + kGroup <= count && t + kGroup <= s1) {  // inside one sequence
#pragma unroll
      for (int i = 0; i < kGroup; ++i) token(t + i, ring.slot(i0 + i));
    } else {
#pragma unroll 1
      for (int i = i0; i < i0 + kGroup && i < count; ++i) {
        if (t0 + i >= s1 && n + 1 < a.q.N) {  // the next sequence with tokens starts here
          do a.q.range(++n, s0, s1);
          while (t0 + i >= s1 && n + 1 < a.q.N);
          load_window<VEC, W>(x, a.ldx, init, t0 + i, s0, n, a.D, c, win);
        }
        token(t0 + i, ring.slot(i));
      }
    }
  }
}

// Single tokens.  A block owns kThreads * VEC channels, loads their taps once and
// walks sequences j, j + jobs, ...; the state and the first token of the next kSeqs
// sequences are in flight into shared memory meanwhile.  T tokens in order, the state
// in registers.
template <typename T, int VEC, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads, kStepBlocks)
conv_step_kernel(ConvArgs a, int cblocks) {
  constexpr int kSeqs = 4;
  __shared__ __align__(16) Raw<T, VEC> ring_mem[kSeqs * W * kThreads];
  const Ring<T, VEC, kSeqs * W> ring{ring_mem + threadIdx.x};
  const T* x = static_cast<const T*>(a.x);
  const int cb = blockIdx.x % cblocks;
  const int64_t jobs = gridDim.x / cblocks;
  if (blockIdx.x == 0) check_counts(a.counts, a.q.N, a.T, a.status);
  const int c = (cb * kThreads + threadIdx.x) * VEC;
  if (c >= a.D) return;
  const int64_t n0 = blockIdx.x / cblocks;
  auto request = [&](int64_t k) {  // this block's k-th sequence
    const int64_t n = n0 + k * jobs;
    if (n < a.q.N) {
      const T* st = static_cast<const T*>(a.state) + n * (W - 1) * a.D + c;
#pragma unroll
      for (int i = 0; i < W - 1; ++i) ring.request(k * W + i, st + (int64_t)i * a.D);
      ring.request(k * W + W - 1, x + n * a.T * a.ldx + c);
    }
    ring_commit();
  };
#pragma unroll
  for (int k = 0; k < kSeqs - 1; ++k) request(k);
  float wr[W][VEC], br[VEC];
  load_params<VEC, W>(a.w, a.b, c, wr, br);
#pragma unroll 1
  for (int64_t k = 0, n = n0; n < a.q.N; ++k, n += jobs) {
    request(k + kSeqs - 1);
    ring_wait<kSeqs - 1>();
    T* st = static_cast<T*>(a.state) + n * (W - 1) * a.D + c;
    float win[W - 1][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) open<T, VEC>(ring.slot(k * W + i), win[i]);
    int keep = a.counts ? a.counts[n] : a.T;
    if (keep < 0 || keep > a.T) keep = 0;
#pragma unroll 1
    for (int t = 0; t < a.T; ++t) {
      float xt[VEC], u[VEC];
      if (t == 0) open<T, VEC>(ring.slot(k * W + W - 1), xt);
      else load<VEC>(x + (n * a.T + t) * a.ldx + c, xt);
      taps<VEC, W>(wr, br, win, xt, u);
      if (kSilu) {
        float s[VEC];
        sigmoid_v(u, s);
        mul_v(u, s);
      }
      if (a.y) store<VEC>(static_cast<T*>(a.y) + (n * a.T + t) * a.D + c, u);
      shift_in<VEC, W>(win, xt);
      if (t + 1 == keep) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) store<VEC>(st + (int64_t)i * a.D, win[i]);
      }
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
__global__ void __launch_bounds__(kThreads, kBwdBlocks)
conv_bwd_kernel(ConvArgs a, int cblocks) {
  // W - 1 tokens per group: after as many shifts the window holds new values only, and no
  // register has to move
  constexpr int kGroup = W - 1, kGroups = 8 / (W - 1) + 1;
  __shared__ __align__(16) Raw<T, VEC> ring_x[kGroup * kGroups * kThreads];
  __shared__ __align__(16) Raw<T, VEC> ring_g[kGroup * kGroups * kThreads];
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
    if (kSilu) {
      float u[VEC];
      taps<VEC, W>(wr, br, win, xt, u);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float s = sigmoid(u[e]);
        du[e] = g[e] * s * fmaf(u[e], 1.f - s, 1.f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) du[e] = g[e];
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
  const int64_t stop = t1 + W - 1 < a.q.total ? t1 + W - 1 : a.q.total;
  bool ended = false;  // the walk stops at a sequence's end at or after t1
  // one token; emit: the dx W - 1 tokens back is finished by it; sum: it counts for this tile
  auto token = [&](int64_t p, const Raw<T, VEC>& xr, const Raw<T, VEC>& gr, bool emit, bool sum) {
    float xt[VEC], g[VEC], du[VEC];
    open<T, VEC>(xr, xt);
    open<T, VEC>(gr, g);
    grad_u(xt, g, du);
    if (emit) {
      fma_v(wr[0], du, pend[W - 2]);
      store<VEC>(dx + (p - (W - 1)) * a.D, pend[W - 2]);
    }
#pragma unroll
    for (int k = W - 2; k > 0; --k) {
      fma_v(wr[W - 1 - k], du, pend[k - 1]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) pend[k][e] = pend[k - 1][e];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) pend[0][e] = wr[W - 1][e] * du[e];
    if (sum) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) db[e] += du[e];
      fma_v(du, xt, dw[W - 1]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) fma_v(du, win[j], dw[j]);
    }
    shift_in<VEC, W>(win, xt);
  };
  const Ring<T, VEC, kGroup * kGroups> rx{ring_x + threadIdx.x}, rg{ring_g + threadIdx.x};
  const int count = (int)(stop - t0);
  const T* px = x + t0 * a.ldx + c;
  const T* pg = dy + t0 * a.D + c;
  auto request = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (i0 + i < count) {
        rx.request(i0 + i, px + (i0 + i) * a.ldx);
        rg.request(i0 + i, pg + (i0 + i) * (int64_t)a.D);
      }
    ring_commit();
  };
#pragma unroll
  for (int g = 0; g < kGroups - 1; ++g) request(g * kGroup);
  for (int i0 = 0; i0 < count && !ended; i0 += kGroup) {
    request(i0 + (kGroups - 1) * kGroup);
    ring_wait<kGroups - 1>();
    const int64_t t = t0 + i0;
    if (t + kGroup <= t1 && t + kGroup <= s1 && t - (W - 1) >= t0 && t - (W - 1) >= s0) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) token(t + i, rx.slot(i0 + i), rg.slot(i0 + i), true, true);
    } else {
#pragma unroll 1
      for (int i = i0; i < i0 + kGroup && i < count; ++i) {
        const int64_t p = t0 + i;
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
        token(p, rx.slot(i), rg.slot(i), p - (W - 1) >= t0 && p - (W - 1) >= s0, p < t1);
      }
    }
  }
  if (!ended && s1 <= stop) flush(s1);
  float* pt = a.part + job * (W + 1) * (int64_t)a.D + c;
#pragma unroll
  for (int j = 0; j < W; ++j) store<VEC>(pt + (int64_t)j * a.D, dw[j]);
  store<VEC>(pt + (int64_t)W * a.D, db);
}

// 32 columns per block: its warps take every kWarps-th tile's sums, then fold in a fixed order
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) conv_reduce_kernel(ConvArgs a) {
  __shared__ float fold[kWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = (int64_t)(a.W + 1) * a.D;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (i < per) {
#pragma unroll 8
    for (int64_t t = warp; t < a.tiles; t += kWarps) sum += a.part[t * per + i];
  }
  fold[warp][lane] = sum;
  __syncthreads();
  if (warp > 0 || i >= per) return;
#pragma unroll
  for (int q = 1; q < kWarps; ++q) sum += fold[q][lane];
  const int j = (int)(i / a.D), c = (int)(i % a.D);
  if (j < a.W) a.dw[(int64_t)c * a.W + j] = sum;
  else if (a.db) a.db[c] = sum;
}

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <typename T, int VEC, int W>
cudaError_t run(const ConvArgs& a, int what) {
  const int cblocks = (a.D + kThreads * VEC - 1) / (kThreads * VEC);
  const int64_t extra = what == 0 ? (a.fin ? a.q.N : 0) : what == 2 ? (a.dinit ? a.q.N : 0) : 0;
  // single tokens: no more blocks than are resident together, each with its share of sequences
  const int64_t fill = a.sms * kStepBlocks / cblocks > 0 ? a.sms * kStepBlocks / cblocks : 1;
  const int64_t jobs = what == 1 ? (a.q.N < fill ? a.q.N : fill) : a.tiles + extra;
  const int64_t grid = jobs * cblocks;
  if (grid == 0)  // nothing to check or to compute
    return a.status ? cudaMemsetAsync(a.status, 0, sizeof(unsigned int), a.stream) : cudaSuccess;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  auto go = [&](auto* kernel) {
    kernel<<<(unsigned)grid, kThreads, 0, a.stream>>>(a, cblocks);
    return cudaGetLastError();
  };
  if (what == 0)
    return a.silu ? go(conv_fwd_kernel<T, VEC, W, true>) : go(conv_fwd_kernel<T, VEC, W, false>);
  if (what == 1)
    return a.silu ? go(conv_step_kernel<T, VEC, W, true>) : go(conv_step_kernel<T, VEC, W, false>);
  return a.silu ? go(conv_bwd_kernel<T, VEC, W, true>) : go(conv_bwd_kernel<T, VEC, W, false>);
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
  const void* ptrs[] = {a.x, a.init, a.dy, a.dfinal, a.y, a.fin, a.dx, a.dinit, a.state};
  const int v = a.bf16 ? 8 : 4;
  bool wide = a.D % v == 0 && a.ldx % v == 0 && al16(a.w);
  for (const void* p : ptrs) wide = wide && al16(p);
  if (!a.bf16) return wide ? by_width<float, 4>(a, what) : by_width<float, 1>(a, what);
  if (!wide) return by_width<__nv_bfloat16, 1>(a, what);
  return by_width<__nv_bfloat16, 8>(a, what);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a0) {
  ConvArgs a = a0;
  // tiles of 64 tokens re-read 5% of x at W = 4; short inputs take smaller ones, for more blocks:
  // 256 tokens of 12288 channels run 6.4 us on the GPU, with tiles of 64 13.6, 1024 tokens 16.7
  // and 16.9
  const int64_t per = kThreads * (a.bf16 ? 8 : 4);
  const int64_t cb = (a.D + per - 1) / per;
  a.tile = 64;
  while (a.tile > 8 && cb * ((a.q.total + a.tile - 1) / a.tile) < 8 * a.sms) a.tile /= 2;
  a.tiles = (a.q.total + a.tile - 1) / a.tile;
  return by_type(a, 0);
}

cudaError_t launch_conv_step(const ConvArgs& a) { return by_type(a, 1); }

// One tile for each block that is resident: all of them end together, and there are few sums to
// add up.  16384 tokens of 12288 channels: 250 us with 38 tiles, 254 with two rounds of blocks,
// 266 with four, 281 with tiles of 128 tokens.
int64_t conv_bwd_tile(int64_t tokens, int D, bool bf16, int64_t sms) {
  const int64_t per = kThreads * (bf16 ? 8 : 4);
  const int64_t cb = (D + per - 1) / per;
  const int64_t tiles = kBwdBlocks * sms / cb;
  const int64_t tile = tiles > 0 ? (tokens + tiles - 1) / tiles : 0;
  return tile < 16 ? 16 : tile;
}

cudaError_t launch_conv_bwd(const ConvArgs& a) {
  cudaError_t e = by_type(a, 2);
  if (e != cudaSuccess) return e;
  const int64_t per = (int64_t)(a.W + 1) * a.D;
  const unsigned blocks = (unsigned)((per + 31) / 32);
  // many tiles (of few channels): more warps, for their latency.  16384 tokens of 264 channels take
  // 23 us on the GPU with 32 warps and 35 with 8, 2048 tokens of 12288 channels 55 and 41
  if (a.tiles >= 128) conv_reduce_kernel<32><<<blocks, 1024, 0, a.stream>>>(a);
  else conv_reduce_kernel<8><<<blocks, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace layer
}  // namespace kda
