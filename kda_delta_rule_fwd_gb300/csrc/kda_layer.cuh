// Declarations shared by the translation units of the operators around the
// recurrence (convolution, scan, norms): wide loads and stores as float32, the
// activations, packed-batch lookups and the launchers' argument structs.
#pragma once

#include "kda_internal.cuh"
#include "kda_layer.h"

namespace kda {
namespace layer {

// VEC consecutive elements (whole 16-byte words, or one element) as float32
template <int VEC>
__device__ __forceinline__ void load(const float* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else if constexpr (VEC == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = p[e];
  }
}
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int VEC>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    unpack2(u.x, x[0], x[1]); unpack2(u.y, x[2], x[3]);
    unpack2(u.z, x[4], x[5]); unpack2(u.w, x[6], x[7]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = __bfloat162float(p[e]);
  }
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4)
      *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[e] = x[e];
  }
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[e] = __float2bfloat16_rn(x[e]);
  }
}

// VEC consecutive elements as they lie in memory, to be held while in flight
template <typename T, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };
template <> struct Raw<float, 8> { float4 v, w; };
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 v; };
template <> struct Raw<float, 1> { float v; };
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> fetch(const T* p) {
  return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void open(const Raw<T, VEC>& r, float (&x)[VEC]) {
  load<VEC>(reinterpret_cast<const T*>(&r), x);
}

// sigmoid on the special-function unit: 2^(-x log2 e), then the reciprocal (a few ulp; 0
// below x ~ -88, 1 above 17)
__device__ __forceinline__ float sigmoid(float x) {
  float e, y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + e));
  return y;
}
// Element-wise work on VEC values, two per instruction where they come in pairs:
// c += a b;  c += a s;  a *= b;  a *= s;  acc += a . b (two partial sums)
template <int VEC>
__device__ __forceinline__ void fma_v(const float (&a)[VEC], const float (&b)[VEC], float (&c)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 r = fma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]),
                            make_float2(c[e], c[e + 1]));
      c[e] = r.x;
      c[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = fmaf(a[e], b[e], c[e]);
  }
}
template <int VEC>
__device__ __forceinline__ void fma_v(const float (&a)[VEC], float s, float (&c)[VEC]) {
  float b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) b[e] = s;
  fma_v(a, b, c);
}
template <int VEC>
__device__ __forceinline__ void mul_v(float (&a)[VEC], const float (&b)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 r = mul2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
      a[e] = r.x;
      a[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) a[e] *= b[e];
  }
}
template <int VEC>
__device__ __forceinline__ void mul_v(float (&a)[VEC], float s) {
  float b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) b[e] = s;
  mul_v(a, b);
}
template <int VEC>
__device__ __forceinline__ void dot_v(const float (&a)[VEC], const float (&b)[VEC], float2& acc) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      acc = fma2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), acc);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc.x = fmaf(a[e], b[e], acc.x);
  }
}
// s = sigmoid(x), as sigmoid()
template <int VEC>
__device__ __forceinline__ void sigmoid_v(const float (&x)[VEC], float (&s)[VEC]) {
  float one[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    s[e] = x[e];
    one[e] = 1.f;
  }
  mul_v(s, -1.4426950408889634f);
#pragma unroll
  for (int e = 0; e < VEC; ++e) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s[e]) : "f"(s[e]));
  fma_v(s, 1.f, one);
#pragma unroll
  for (int e = 0; e < VEC; ++e) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[e]) : "f"(one[e]));
}
template <int VEC>
__device__ __forceinline__ void copy_v(const float (&a)[VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) b[e] = a[e];
}

// delta = softplus(dt + bias), or dt as given
__device__ __forceinline__ float step_size(float dt, float bias, bool softplus) {
  if (!softplus) return dt;
  const float x = dt + bias;
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// The sequence that holds flat token t (fixed: t / T; packed: the last n with
// cu[n] <= t, found by bisection), and its token range [start, end).
// Malformed offsets give some sequence in [0, N) and a range inside [0, total).
struct Seqs {
  const int32_t* cu;  // nullptr: fixed length
  int64_t T, total;   // tokens per sequence (fixed) and in all
  int N;
  __device__ __forceinline__ void range(int n, int64_t& start, int64_t& end) const {
    if (!cu) {
      start = (int64_t)n * T;
      end = start + T;
      return;
    }
    const int64_t a = cu[n], b = cu[n + 1];
    start = a < 0 ? 0 : (a > total ? total : a);
    end = b < start ? start : (b > total ? total : b);
  }
  __device__ __forceinline__ int find(int64_t t) const {
    if (!cu) return (int)(t / T);
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
};

// One block's check of cu_seqlens: non-decreasing from 0 to total.  The verdict
// is written, not latched: no earlier clearing of the word is needed.
__device__ __forceinline__ void check_seqlens(const Seqs& q, unsigned int* status) {
  if (!status) return;
  int bad = 0;
  if (q.cu)
    for (int n = threadIdx.x; n <= q.N; n += blockDim.x) {
      const int64_t v = q.cu[n];
      if ((n == 0 && v != 0) || (n == q.N && v != q.total) || (n > 0 && v < q.cu[n - 1])) bad = 1;
    }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
}
__device__ __forceinline__ void check_counts(const int32_t* counts, int B, int T,
                                             unsigned int* status) {
  if (!status) return;
  int bad = 0;
  if (counts)
    for (int n = threadIdx.x; n < B; n += blockDim.x) bad |= counts[n] < 0 || counts[n] > T;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? KDA_ERR_INVALID_ARG : KDA_OK;
}

struct ConvArgs {
  const void *x, *init, *dy, *dfinal;
  const float *w, *b;
  const int32_t* counts;  // step: commit counts, or nullptr
  void *y, *fin, *dx, *dinit, *state;
  float *dw, *db, *part;  // part: the backward's per-tile sums
  Seqs q;
  int D, W, T;            // T: tokens per step
  int64_t ldx;
  bool bf16, silu;
  int64_t tile, tiles;
  int64_t sms;
  unsigned int* status;
  cudaStream_t stream;
};
cudaError_t launch_conv_fwd(const ConvArgs& a);
cudaError_t launch_conv_step(const ConvArgs& a);
int64_t conv_bwd_tile(int64_t tokens, int D, bool bf16, int64_t sms);
cudaError_t launch_conv_bwd(const ConvArgs& a);

struct ScanArgs {
  const void *x, *dt, *Bm, *Cm;
  const float *A, *D, *dtb, *h0;
  const int32_t* counts;
  void* y;
  float *hT, *state;
  Seqs q;
  int H, G, ds, dx, T;
  int64_t ldx, lddt, ldb, ldc;
  bool bf16, out_bf16, softplus;
  unsigned int* status;
  int64_t sms;
  void* ws;          // the workspace past its header, or nullptr
  cudaStream_t stream;
};
cudaError_t launch_scan_recurrent(const ScanArgs& a);
cudaError_t launch_scan_step(const ScanArgs& a);
// the tensor-core path of bf16 prompts: whether the operands' alignment allows it, what it
// needs of the workspace past the header, and the call
bool scan_bf16_ok(const ScanArgs& a);
size_t scan_bf16_workspace(bool packed, int64_t N, int64_t T, int64_t total, int H, int G, int ds,
                           int dx, int64_t sms);
cudaError_t launch_scan_bf16(const ScanArgs& a);

struct NormArgs {
  const void *x, *gate, *res, *dr, *dy;
  const float *w, *ls, *ow;
  void *r, *y, *dx, *dgate, *dres;
  float *dw, *dls, *dow, *part;
  int64_t tokens, ldx, ldg;
  int heads, d, gate_act;
  bool bf16, res_bf16, gate_first;
  float scale, eps, inv_d;
  bool dense;    // x and gate rows lie d apart
  int64_t sms;
  int64_t ctas;  // backward: CTAs, each with its own row of partial sums
  cudaStream_t stream;
};
cudaError_t launch_norm_fwd(const NormArgs& a);
cudaError_t launch_norm_bwd(NormArgs a);
int64_t norm_bwd_ctas(int64_t rows, int d, bool bf16, int64_t sms);  // the most of a call

}  // namespace layer
int64_t device_sms();  // SMs of the current device (152 when there is none)
}  // namespace kda
