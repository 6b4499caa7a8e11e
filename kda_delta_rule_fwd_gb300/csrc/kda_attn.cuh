// Declarations shared by the translation units of the attention layers' operators
// (norms of queries and keys with rotation, paged cache, attention of new tokens,
// verification of drafts): argument structs, launchers, places in the paged cache.
#pragma once

#include <cuda_fp16.h>

#include "kda_attn.h"
#include "kda_layer.cuh"

namespace kda {
namespace attn {

using layer::Seqs;

// ---------------------------------------------------------------------------
// norms of queries and keys with the position's rotation
// ---------------------------------------------------------------------------
struct QKPart {  // q or k
  const void *x, *dy;
  const float* w;
  void *y, *dx;
  float *dw, *part;  // part: the backward's sums, [ctas][d]
  int64_t ld;
  int heads, ctas;
};
struct QKArgs {
  QKPart p[2];
  const int32_t* pos;
  const double* freqs;
  int64_t tokens;
  int d, rot;
  bool bf16, interleaved;
  float eps, inv_d;
  int64_t sms;
  cudaStream_t stream;
};
cudaError_t launch_qknorm_fwd(QKArgs a);
cudaError_t launch_qknorm_bwd(QKArgs a);
// the most blocks of the backward's part (0: q, 1: k), each with a row of sums
int64_t qknorm_bwd_ctas(int64_t tokens, int heads, int64_t sms);

// ---------------------------------------------------------------------------
// paged cache
// ---------------------------------------------------------------------------
// 2^(b - 127) from a row's byte; 255 gives an infinity, which turns its codes (0) into NaN
__device__ __forceinline__ float power(unsigned b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

struct Table {
  const int32_t* pages;  // [N][max_pages]
  const int32_t* lens;   // [N]
  int max_pages, num_pages, shift;  // page = 1 << shift
};
// The page that holds place p >= 0 of sequence n; -1 past the table or outside the pool.
__device__ __forceinline__ int page_of(const Table& t, int n, int64_t p) {
  const int64_t col = p >> t.shift;
  if (col >= t.max_pages) return -1;
  const int id = t.pages[(int64_t)n * t.max_pages + col];
  return id >= 0 && id < t.num_pages ? id : -1;
}

struct CacheArgs {
  const void *k, *v;  // written
  void *ko, *vo;      // read
  void *kc, *vc;
  uint8_t *ks, *vs;
  Seqs q;
  Table t;
  int heads, d, cache;
  bool bf16;
  int64_t ldk, ldv, ldpage;
  unsigned int* status;
  int64_t sms;
  cudaStream_t stream;
};
cudaError_t launch_cache_write(const CacheArgs& a);
cudaError_t launch_cache_read(const CacheArgs& a);

// ---------------------------------------------------------------------------
// attention of new tokens
// ---------------------------------------------------------------------------
struct AttnArgs {
  const void *q, *kc, *vc;
  const uint8_t *ks, *vs;
  Table t;
  void* out;
  float* lse;
  int B, T, hq, hk, rep, d, cache, window;
  bool bf16;
  float scale;
  int64_t ldq, ldpage;
  void* ws;
  int64_t sms;
  cudaStream_t stream;
};
size_t attn_workspace(const AttnArgs& a);
cudaError_t launch_attn(const AttnArgs& a);

// ---------------------------------------------------------------------------
// verification of drafts
// ---------------------------------------------------------------------------
struct VerifyArgs {
  const void *p, *q;
  const int32_t *drafts, *counts;
  const float* u;
  int32_t *tokens, *commit;
  int B, K, V;
  bool bf16;
  unsigned int* status;
  int64_t sms;
  cudaStream_t stream;
};
cudaError_t launch_verify(const VerifyArgs& a);

}  // namespace attn
}  // namespace kda
