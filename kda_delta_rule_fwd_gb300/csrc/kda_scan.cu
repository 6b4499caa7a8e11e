// Selective state-space scan, token by token on the CUDA cores: float32 prompts
// and the single-token step over resident states.
//
//     S <- exp(delta_t A) S + delta_t B_t x_t^T;   y_t = S^T C_t + D x_t
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace {

// ---------------------------------------------------------------------------
// Prompts.  One block of 128 threads per (sequence, head, COLS state columns): a
// thread owns one column and DS * COLS / 128 of its rows, in registers.  kTile tokens
// are staged in shared memory as float32 at a time, two tiles in turn: the next tile's
// inputs are requested before this one's tokens are worked on and stored after.  Four
// tokens' parts of y are reduced together, each exchange between lanes halving the
// tokens that a lane still holds; the warps' parts meet once per tile.
// With many blocks it is bound by issue (2 multiply-adds per state element and token) and
// shared memory reads, and 32 columns share each read of B and C best; with few, by the
// chain of tokens, which 8 columns per block keep short.  512 tokens, state 64 x 64: 8
// chains take 37 us with 8 columns and 60 with 32, 512 chains 390 and 230.
// ---------------------------------------------------------------------------
constexpr int kTile = 16;
constexpr int kStep = 4;  // tokens whose parts of y are reduced together

template <typename T, typename TO, int DS, int COLS>
__global__ void __launch_bounds__(128)
scan_recurrent_kernel(ScanArgs a) {
  constexpr int R = DS * COLS / 128;       // rows per thread
  constexpr int kB = kTile * DS / 128;     // elements of B (and C) a thread stages
  constexpr int kX = kTile * COLS / 128;
  // groups of tokens per trip, as measured for 8 chains of 512 tokens: 8 columns take 37 us with 4
  // and 47 with 2, 32 columns 86 with 4 and 60 with 2
  constexpr int kUnroll = COLS == 8 ? 4 : 2;
  __shared__ __align__(16) float s_b[2][kTile][DS], s_c[2][kTile][DS];
  __shared__ float s_x[2][kTile][COLS], s_y[2][kTile][4][COLS], s_a[2][kTile], s_d[2][kTile];
  if (blockIdx.x == 0) check_seqlens(a.q, a.status);
  const int slices = a.dx / COLS;
  const int sl = blockIdx.x % slices;
  const int64_t chain = blockIdx.x / slices;
  const int h = (int)(chain % a.H), n = (int)(chain / a.H), g = h / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cl = lane % COLS;                              // column in the slice
  const int row0 = (warp * (32 / COLS) + lane / COLS) * R;
  int64_t s0, s1;
  a.q.range(n, s0, s1);
  const int64_t base = (chain * DS + row0) * (int64_t)a.dx + sl * COLS + cl;
  float2 S[R / 2];  // rows in pairs
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const float* p = a.h0 + base + (int64_t)(2 * i) * a.dx;
    S[i] = a.h0 ? make_float2(p[0], p[a.dx]) : make_float2(0.f, 0.f);
  }
  const float decay = a.A[h], skip = a.D ? a.D[h] : 0.f, bias = a.dtb ? a.dtb[h] : 0.f;
  const T* x = static_cast<const T*>(a.x) + (int64_t)h * a.dx + sl * COLS;
  const T* dt = static_cast<const T*>(a.dt) + h;
  const T* Bm = static_cast<const T*>(a.Bm) + (int64_t)g * DS;
  const T* Cm = static_cast<const T*>(a.Cm) + (int64_t)g * DS;
  TO* y = static_cast<TO*>(a.y) + (int64_t)h * a.dx + sl * COLS;
  const int64_t ldy = (int64_t)a.H * a.dx;
  // tokens past the end enter as zeros with a decay of 1
  T rb[kB], rc[kB], rx[kX], rd;
  auto request = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int t = (i * 128 + tid) / DS, c = (i * 128 + tid) % DS;
      const bool in = t0 + t < s1;
      rb[i] = in ? Bm[(t0 + t) * a.ldb + c] : from_f32<T>(0.f);
      rc[i] = in ? Cm[(t0 + t) * a.ldc + c] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      const int t = (i * 128 + tid) / COLS, c = (i * 128 + tid) % COLS;
      rx[i] = t0 + t < s1 ? x[(t0 + t) * a.ldx + c] : from_f32<T>(0.f);
    }
    if (tid < kTile && t0 + tid < s1) rd = dt[(t0 + tid) * a.lddt];
  };
  auto stage = [&](int64_t t0, int b) {
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int t = (i * 128 + tid) / DS, c = (i * 128 + tid) % DS;
      s_b[b][t][c] = to_f32(rb[i]);
      s_c[b][t][c] = to_f32(rc[i]);
    }
#pragma unroll
    for (int i = 0; i < kX; ++i)
      s_x[b][(i * 128 + tid) / COLS][(i * 128 + tid) % COLS] = to_f32(rx[i]);
    if (tid < kTile) {
      const float d = t0 + tid < s1 ? step_size(to_f32(rd), bias, a.softplus) : 0.f;
      s_d[b][tid] = d;
      s_a[b][tid] = expf(d * decay);
    }
  };
  if (s0 < s1) {
    request(s0);
    stage(s0, 0);
  }
  __syncthreads();
  int b = 0;
  for (int64_t t0 = s0; t0 < s1; t0 += kTile, b ^= 1) {
    if (t0 + kTile < s1) request(t0 + kTile);
#pragma unroll kUnroll
    for (int tt = 0; tt < kTile; tt += kStep) {
      float v[kStep];
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        const int t = tt + k;
        const float at = s_a[b][t], xw = s_d[b][t] * s_x[b][t][cl];
        const float2 at2 = make_float2(at, at), xw2 = make_float2(xw, xw);
        float2 p = make_float2(row0 == 0 ? skip * s_x[b][t][cl] : 0.f, 0.f), q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R / 2; i += 2) {
          const float4 bv = *reinterpret_cast<const float4*>(&s_b[b][t][row0 + 2 * i]);
          const float4 cv = *reinterpret_cast<const float4*>(&s_c[b][t][row0 + 2 * i]);
          S[i] = fma2(at2, S[i], mul2(make_float2(bv.x, bv.y), xw2));
          S[i + 1] = fma2(at2, S[i + 1], mul2(make_float2(bv.z, bv.w), xw2));
          p = fma2(make_float2(cv.x, cv.y), S[i], p);
          q = fma2(make_float2(cv.z, cv.w), S[i + 1], q);
        }
        v[k] = (p.x + p.y) + (q.x + q.y);
      }
      // the row groups' parts meet, and every group ends up with tokens of its own
      int t = tt;
      int n = kStep;
#pragma unroll
      for (int o = 16; o >= COLS; o >>= 1) {
        n >>= 1;
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < kStep / 2; ++k)
          if (k < n) {
            const float mine = up ? v[n + k] : v[k], other = up ? v[k] : v[n + k];
            v[k] = mine + __shfl_xor_sync(0xffffffffu, other, o);
          }
        if (up) t += n;
      }
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (k < kStep * COLS / 32) s_y[b][t + k][warp][cl] = v[k];
    }
    if (t0 + kTile < s1) stage(t0 + kTile, b ^ 1);
    __syncthreads();
    for (int i = tid; i < kTile * COLS; i += 128) {
      const int t = i / COLS, c = i % COLS;
      const float v = (s_y[b][t][0][c] + s_y[b][t][1][c]) + (s_y[b][t][2][c] + s_y[b][t][3][c]);
      if (t0 + t < s1) y[(t0 + t) * ldy + c] = from_f32<TO>(v);
    }
  }
  if (a.hT) {
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
      float* p = a.hT + base + (int64_t)(2 * i) * a.dx;
      p[0] = S[i].x;
      p[a.dx] = S[i].y;
    }
  }
}

// ---------------------------------------------------------------------------
// Single tokens.  One block of 256 threads per (sequence, head): the state is
// read once with 16-byte loads (a warp covers whole rows), kept in registers for
// the step's tokens and written once.  Bound by the state's traffic: 1024 sequences of
// 32 heads of 128 x 128 take 641 us (6.7 TB/s, 99% of a copy's rate).
// ---------------------------------------------------------------------------
constexpr int kMaxStep = 8;

template <typename T, typename TO, int DS, int DX, bool kCommit>
__global__ void __launch_bounds__(256, 2)
scan_step_kernel(ScanArgs a) {
  constexpr int CQ = DX / 4;        // threads per state row
  constexpr int RG = 256 / CQ;      // rows per pass
  constexpr int R = DS / RG;        // rows per thread
  constexpr int YP = 8;             // y parts: one per warp
  __shared__ __align__(16) float s_b[kMaxStep][DS], s_c[kMaxStep][DS], s_x[kMaxStep][DX];
  __shared__ __align__(16) float s_y[kMaxStep][YP][DX];
  __shared__ float s_a[kMaxStep], s_d[kMaxStep];
  if (blockIdx.x == 0) check_counts(a.counts, a.q.N, a.T, a.status);
  const int64_t chain = blockIdx.x;
  const int h = (int)(chain % a.H), n = (int)(chain / a.H), g = h / (a.H / a.G);
  const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
  float* st = a.state + chain * (int64_t)(DS * DX) + cq * 4;
  float4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = *reinterpret_cast<const float4*>(st + (int64_t)(rg + i * RG) * DX);
  const T* x = static_cast<const T*>(a.x) + (int64_t)h * DX;
  const T* Bm = static_cast<const T*>(a.Bm) + (int64_t)g * DS;
  const T* Cm = static_cast<const T*>(a.Cm) + (int64_t)g * DS;
  const int64_t tok = (int64_t)n * a.T;
  for (int i = tid; i < a.T * DS; i += 256) {
    s_b[i / DS][i % DS] = to_f32(Bm[(tok + i / DS) * a.ldb + i % DS]);
    s_c[i / DS][i % DS] = to_f32(Cm[(tok + i / DS) * a.ldc + i % DS]);
  }
  for (int i = tid; i < a.T * DX; i += 256) s_x[i / DX][i % DX] = to_f32(x[(tok + i / DX) * a.ldx + i % DX]);
  if (tid < a.T) {
    const float d = step_size(to_f32(static_cast<const T*>(a.dt)[(tok + tid) * a.lddt + h]),
                              a.dtb ? a.dtb[h] : 0.f, a.softplus);
    s_d[tid] = d;
    s_a[tid] = expf(d * a.A[h]);
  }
  int keep = a.T;
  if (kCommit) {
    keep = a.counts[n];
    if (keep < 0 || keep > a.T) keep = 0;
  }
  __syncthreads();
  for (int t = 0; t < a.T; ++t) {
    const float at = s_a[t], d = s_d[t];
    const float4 xv = *reinterpret_cast<const float4*>(&s_x[t][cq * 4]);
    const float4 xw = make_float4(d * xv.x, d * xv.y, d * xv.z, d * xv.w);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float b = s_b[t][rg + i * RG], c = s_c[t][rg + i * RG];
      S[i].x = fmaf(at, S[i].x, b * xw.x);
      S[i].y = fmaf(at, S[i].y, b * xw.y);
      S[i].z = fmaf(at, S[i].z, b * xw.z);
      S[i].w = fmaf(at, S[i].w, b * xw.w);
      acc.x = fmaf(c, S[i].x, acc.x);
      acc.y = fmaf(c, S[i].y, acc.y);
      acc.z = fmaf(c, S[i].z, acc.z);
      acc.w = fmaf(c, S[i].w, acc.w);
    }
    if constexpr (CQ < 32) {  // two rows per warp pass
      acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
      acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
      acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
      acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    }
    if (CQ == 32 || (tid & 31) < 16)
      *reinterpret_cast<float4*>(&s_y[t][tid >> 5][cq * 4]) = acc;
    if (kCommit && t + 1 == keep) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        *reinterpret_cast<float4*>(st + (int64_t)(rg + i * RG) * DX) = S[i];
    }
  }
  if (!kCommit) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      *reinterpret_cast<float4*>(st + (int64_t)(rg + i * RG) * DX) = S[i];
  }
  if (!a.y) return;
  __syncthreads();
  const float skip = a.D ? a.D[h] : 0.f;
  TO* y = static_cast<TO*>(a.y) + (int64_t)h * DX;
  for (int i = tid; i < a.T * DX; i += 256) {
    const int t = i / DX, c = i % DX;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < YP; ++w) v += s_y[t][w][c];
    y[(tok + t) * (int64_t)a.H * DX + c] = from_f32<TO>(fmaf(skip, s_x[t][c], v));
  }
}

template <typename T, typename TO, int DS, int COLS>
cudaError_t recurrent_cols(const ScanArgs& a) {
  const int64_t grid = (int64_t)a.q.N * a.H * (a.dx / COLS);
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  scan_recurrent_kernel<T, TO, DS, COLS><<<(unsigned)grid, 128, 0, a.stream>>>(a);
  return cudaGetLastError();
}
template <typename T, typename TO, int DS>
cudaError_t recurrent(const ScanArgs& a) {
  // 8 columns per block while there are up to two such blocks per SM (512 tokens, 128 x 64: 32
  // chains take 56 us against 89 with 32 columns, 64 chains 105 against 89)
  return (int64_t)a.q.N * a.H * (a.dx / 8) <= 2 * a.sms ? recurrent_cols<T, TO, DS, 8>(a)
                                                        : recurrent_cols<T, TO, DS, 32>(a);
}
template <typename T, typename TO>
cudaError_t recurrent_ds(const ScanArgs& a) {
  return a.ds == 64 ? recurrent<T, TO, 64>(a) : recurrent<T, TO, 128>(a);
}

template <typename T, typename TO, int DS, int DX>
cudaError_t step(const ScanArgs& a) {
  const int64_t grid = (int64_t)a.q.N * a.H;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (a.counts) scan_step_kernel<T, TO, DS, DX, true><<<(unsigned)grid, 256, 0, a.stream>>>(a);
  else scan_step_kernel<T, TO, DS, DX, false><<<(unsigned)grid, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}
template <typename T, typename TO>
cudaError_t step_size_of(const ScanArgs& a) {
  if (a.ds == 64) return a.dx == 64 ? step<T, TO, 64, 64>(a) : step<T, TO, 64, 128>(a);
  return a.dx == 64 ? step<T, TO, 128, 64>(a) : step<T, TO, 128, 128>(a);
}

}  // namespace

using bf = __nv_bfloat16;
cudaError_t launch_scan_recurrent(const ScanArgs& a) {
  if ((int64_t)a.q.N * a.H == 0)
    return a.status ? cudaMemsetAsync(a.status, 0, sizeof(unsigned int), a.stream) : cudaSuccess;
  if (a.bf16) return a.out_bf16 ? recurrent_ds<bf, bf>(a) : recurrent_ds<bf, float>(a);
  return a.out_bf16 ? recurrent_ds<float, bf>(a) : recurrent_ds<float, float>(a);
}
cudaError_t launch_scan_step(const ScanArgs& a) {
  if (a.q.N == 0)
    return a.status ? cudaMemsetAsync(a.status, 0, sizeof(unsigned int), a.stream) : cudaSuccess;
  if (a.bf16) return a.out_bf16 ? step_size_of<bf, bf>(a) : step_size_of<bf, float>(a);
  return a.out_bf16 ? step_size_of<float, bf>(a) : step_size_of<float, float>(a);
}

}  // namespace layer
}  // namespace kda
