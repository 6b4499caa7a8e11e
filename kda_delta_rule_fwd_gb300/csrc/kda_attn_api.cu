// C ABI of the attention layers' operators: argument checks, workspace carving and
// dispatch.  Every check that can be made on the host is made before anything is
// launched; nothing here allocates memory.
#include "kda_attn.cuh"

using namespace kda;
using namespace kda::attn;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
size_t dsize(kda_dtype t) { return t == KDA_F32 ? 4 : 2; }
bool cache_ok(kda_cache_dtype t) {
  return t == KDA_CACHE_F32 || t == KDA_CACHE_BF16 || t == KDA_CACHE_E4M3 || t == KDA_CACHE_INT8;
}
bool coded(kda_cache_dtype t) { return t == KDA_CACHE_E4M3 || t == KDA_CACHE_INT8; }
size_t csize(kda_cache_dtype t) { return t == KDA_CACHE_F32 ? 4 : t == KDA_CACHE_BF16 ? 2 : 1; }
constexpr int64_t kMaxElems = (int64_t)1 << 40;  // elements of one tensor

// every pointer of the list (NULLs aside) a multiple of `a`
template <int N>
bool all_aligned(const void* const (&p)[N], size_t a) {
  for (const void* q : p)
    if (q && !aligned(q, a)) return false;
  return true;
}
bool stride_ok(int64_t& ld, int64_t row) {
  if (ld == 0) ld = row;
  return ld >= row && ld <= kMaxElems;
}
kda_status check_status_ws(const void* ws, size_t bytes) {
  if (!ws) return KDA_OK;
  return aligned(ws, 256) && bytes >= kWsHeader ? KDA_OK : KDA_ERR_WORKSPACE;
}
kda_status launched(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
// the word in which kernels latch what they find, cleared in stream order
cudaError_t clear_status(void* ws, void* stream) {
  return ws ? cudaMemsetAsync(ws, 0, 4, static_cast<cudaStream_t>(stream)) : cudaSuccess;
}

kda_status check_qknorm(const kda_qknorm_shape* s, QKArgs& a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->tokens < 0 || s->q_heads < 1 || s->k_heads < 0 || s->q_heads > 65536 || s->k_heads > 65536 || s->d < 2 || s->d % 2 || s->rot < 0 ||
      s->rot % 2 || s->rot > s->d || !dtype_ok(s->dtype) || !(s->eps >= 0.f))
    return KDA_ERR_INVALID_ARG;
  if (s->d > 256) return KDA_ERR_UNSUPPORTED;
  a.p[0].ld = s->ldq;
  a.p[1].ld = s->ldk;
  if (!stride_ok(a.p[0].ld, (int64_t)s->q_heads * s->d) ||
      !stride_ok(a.p[1].ld, (int64_t)s->k_heads * s->d))
    return KDA_ERR_INVALID_ARG;
  const int64_t widest = a.p[0].ld > a.p[1].ld ? a.p[0].ld : a.p[1].ld;
  if (s->tokens > kMaxElems / widest) return KDA_ERR_INVALID_ARG;
  a.p[0].heads = s->q_heads;
  a.p[1].heads = s->k_heads;
  a.tokens = s->tokens;
  a.d = s->d; a.rot = s->rot;
  a.bf16 = s->dtype == KDA_BF16;
  a.interleaved = s->interleaved != 0;
  a.eps = s->eps;
  a.inv_d = 1.f / (float)s->d;
  a.sms = device_sms();
  return KDA_OK;
}

kda_status check_table(int32_t page, int32_t max_pages, int32_t num_pages, Table& t) {
  if (page < 1 || max_pages < 1 || num_pages < 1) return KDA_ERR_INVALID_ARG;
  if ((page & (page - 1)) || page > 65536) return KDA_ERR_UNSUPPORTED;
  t.max_pages = max_pages;
  t.num_pages = num_pages;
  t.shift = 0;
  while ((1 << t.shift) < page) ++t.shift;
  return KDA_OK;
}
// the stride between pages: at least a page, whole 16-byte words, the pool within limits
bool page_stride_ok(int64_t& ld, int64_t page_elems, int32_t num_pages, kda_cache_dtype c) {
  return stride_ok(ld, page_elems) && ld * csize(c) % 16 == 0 && num_pages <= kMaxElems / ld;
}

kda_status check_cache(const kda_cache_shape* s, bool packed, CacheArgs& a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->T < 0 || s->heads < 1 || s->heads > 65536 || s->d < 1 || !dtype_ok(s->dtype) ||
      !cache_ok(s->cache))
    return KDA_ERR_INVALID_ARG;
  if (packed ? (s->B != 1 || s->num_seqs < 0 || (s->num_seqs == 0 && s->T > 0)) : s->B < 0)
    return KDA_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return KDA_ERR_UNSUPPORTED;
  kda_status st = check_table(s->page, s->max_pages, s->num_pages, a.t);
  if (st != KDA_OK) return st;
  const int64_t row = (int64_t)s->heads * s->d;
  a.ldk = s->ldk; a.ldv = s->ldv; a.ldpage = s->ldpage;
  if (!stride_ok(a.ldk, row) || !stride_ok(a.ldv, row) ||
      !page_stride_ok(a.ldpage, row * s->page, s->num_pages, s->cache))
    return KDA_ERR_INVALID_ARG;
  if ((int64_t)s->B * s->T > kMaxElems / (a.ldk > a.ldv ? a.ldk : a.ldv)) return KDA_ERR_INVALID_ARG;
  a.heads = s->heads; a.d = s->d; a.cache = s->cache;
  a.bf16 = s->dtype == KDA_BF16;
  a.sms = device_sms();
  return KDA_OK;
}

kda_status check_attn(const kda_attn_shape* s, AttnArgs& a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->B < 0 || s->q_heads < 1 || s->kv_heads < 1 || s->q_heads % s->kv_heads ||
      s->q_heads > 65536 || s->d < 1 || !dtype_ok(s->dtype) || !cache_ok(s->cache) ||
      !(s->scale == s->scale) || s->window < 0)
    return KDA_ERR_INVALID_ARG;
  if (s->T < 1 || s->T > 8 || (s->d != 64 && s->d != 128)) return KDA_ERR_UNSUPPORTED;
  if (!coded(s->cache) && csize(s->cache) != dsize(s->dtype)) return KDA_ERR_UNSUPPORTED;
  kda_status st = check_table(s->page, s->max_pages, s->num_pages, a.t);
  if (st != KDA_OK) return st;
  a.ldq = s->ldq; a.ldpage = s->ldpage;
  if (!stride_ok(a.ldq, (int64_t)s->q_heads * s->d) ||
      !page_stride_ok(a.ldpage, (int64_t)s->kv_heads * s->d * s->page, s->num_pages, s->cache))
    return KDA_ERR_INVALID_ARG;
  if ((int64_t)s->B * s->T > kMaxElems / a.ldq) return KDA_ERR_INVALID_ARG;
  a.B = s->B; a.T = s->T;
  a.hq = s->q_heads; a.hk = s->kv_heads; a.rep = s->q_heads / s->kv_heads;
  a.d = s->d; a.cache = s->cache;
  a.window = s->window;
  a.bf16 = s->dtype == KDA_BF16;
  a.scale = s->scale;
  a.sms = device_sms();
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_qknorm_fwd(const kda_qknorm_shape* s, const void* q, const void* k,
                          const int32_t* positions, const double* freqs, const float* q_weight,
                          const float* k_weight, void* q_out, void* k_out, void* stream) {
  QKArgs a{};
  kda_status st = check_qknorm(s, a);
  if (st != KDA_OK) return st;
  const bool any = s->tokens > 0;
  if (any && (!q || !q_out || (s->k_heads > 0 && (!k || !k_out)) || (s->rot > 0 && (!positions || !freqs))))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({q, k, (const void*)q_out, (const void*)k_out}, dsize(s->dtype)) ||
      !all_aligned({(const void*)positions, (const void*)q_weight, (const void*)k_weight}, 4) ||
      !aligned(freqs, 8))
    return KDA_ERR_INVALID_ARG;
  a.p[0].x = q; a.p[0].w = q_weight; a.p[0].y = q_out;
  a.p[1].x = k; a.p[1].w = k_weight; a.p[1].y = k_out;
  a.pos = positions; a.freqs = freqs;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_qknorm_fwd(a));
}

size_t kda_qknorm_bwd_workspace_size(const kda_qknorm_shape* s) {
  if (!s || s->tokens < 0 || s->q_heads < 1 || s->k_heads < 0 || s->d < 1) return 0;
  const int64_t sms = device_sms();
  return kWsHeader + (size_t)(qknorm_bwd_ctas(s->tokens, s->q_heads, sms) +
                              qknorm_bwd_ctas(s->tokens, s->k_heads, sms)) * s->d * sizeof(float);
}

kda_status kda_qknorm_bwd(const kda_qknorm_shape* s, const void* q, const void* k,
                          const void* dq_out, const void* dk_out, const int32_t* positions,
                          const double* freqs, const float* q_weight, const float* k_weight,
                          void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                          size_t workspace_bytes, void* stream) {
  QKArgs a{};
  kda_status st = check_qknorm(s, a);
  if (st != KDA_OK) return st;
  const bool any = s->tokens > 0, keys = s->k_heads > 0;
  if (any && (!q || !dq_out || !dq || (keys && (!k || !dk_out || !dk)) ||
              (s->rot > 0 && (!positions || !freqs))))
    return KDA_ERR_INVALID_ARG;
  // a gradient is asked for only where its operand is there
  if ((dq_weight && !q_weight) || (dk_weight && (!k_weight || !keys))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({q, k, dq_out, dk_out, (const void*)dq, (const void*)dk}, dsize(s->dtype)) ||
      !all_aligned({(const void*)positions, (const void*)q_weight, (const void*)k_weight,
                    (const void*)dq_weight, (const void*)dk_weight}, 4) ||
      !aligned(freqs, 8))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda_qknorm_bwd_workspace_size(s))
    return KDA_ERR_WORKSPACE;
  a.p[0].x = q; a.p[0].dy = dq_out; a.p[0].w = q_weight; a.p[0].dx = dq; a.p[0].dw = dq_weight;
  a.p[1].x = k; a.p[1].dy = dk_out; a.p[1].w = k_weight; a.p[1].dx = dk; a.p[1].dw = dk_weight;
  a.p[0].part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeader);
  a.p[1].part = a.p[0].part + qknorm_bwd_ctas(s->tokens, s->q_heads, a.sms) * s->d;
  a.pos = positions; a.freqs = freqs;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_qknorm_bwd(a));
}

kda_status kda_cache_write(const kda_cache_shape* s, const void* k, const void* v,
                           const int32_t* cu_seqlens, const int32_t* pages, const int32_t* lens,
                           void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  CacheArgs a{};
  kda_status st = check_cache(s, packed, a);
  if (st != KDA_OK) return st;
  const int64_t tokens = (int64_t)s->B * s->T;
  if (tokens > 0 && (!k || !v || !pages || !lens || !k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
  if (coded(s->cache) ? tokens > 0 && (!k_scale || !v_scale) : k_scale || v_scale)
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({k, v}, dsize(s->dtype)) ||
      !all_aligned({(const void*)cu_seqlens, (const void*)pages, (const void*)lens}, 4) ||
      !all_aligned({(const void*)k_cache, (const void*)v_cache, (const void*)k_scale, (const void*)v_scale}, 16))
    return KDA_ERR_INVALID_ARG;
  if ((st = check_status_ws(workspace, workspace_bytes)) != KDA_OK) return st;
  a.k = k; a.v = v;
  a.kc = k_cache; a.vc = v_cache; a.ks = k_scale; a.vs = v_scale;
  a.q = Seqs{cu_seqlens, s->T, tokens, packed ? s->num_seqs : s->B};
  a.t.pages = pages; a.t.lens = lens;
  a.status = static_cast<unsigned int*>(workspace);
  a.stream = static_cast<cudaStream_t>(stream);
  if (clear_status(workspace, stream) != cudaSuccess) return KDA_ERR_CUDA;
  return launched(launch_cache_write(a));
}

kda_status kda_cache_read(const kda_cache_shape* s, const int32_t* cu_seqlens,
                          const int32_t* pages, const int32_t* lens, const void* k_cache,
                          const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                          void* k, void* v, void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  CacheArgs a{};
  kda_status st = check_cache(s, packed, a);
  if (st != KDA_OK) return st;
  const int64_t tokens = (int64_t)s->B * s->T;
  if (tokens > 0 && (!pages || !lens || !k_cache || !v_cache || (!k && !v))) return KDA_ERR_INVALID_ARG;
  if (coded(s->cache) ? tokens > 0 && (!k_scale || !v_scale) : k_scale || v_scale)
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({(const void*)k, (const void*)v}, dsize(s->dtype)) ||
      !all_aligned({(const void*)cu_seqlens, (const void*)pages, (const void*)lens}, 4) ||
      !all_aligned({k_cache, v_cache, (const void*)k_scale, (const void*)v_scale}, 16))
    return KDA_ERR_INVALID_ARG;
  if ((st = check_status_ws(workspace, workspace_bytes)) != KDA_OK) return st;
  a.ko = k; a.vo = v;
  a.kc = const_cast<void*>(k_cache); a.vc = const_cast<void*>(v_cache);
  a.ks = const_cast<uint8_t*>(k_scale); a.vs = const_cast<uint8_t*>(v_scale);
  a.q = Seqs{cu_seqlens, s->T, tokens, packed ? s->num_seqs : s->B};
  a.t.pages = pages; a.t.lens = lens;
  a.status = static_cast<unsigned int*>(workspace);
  a.stream = static_cast<cudaStream_t>(stream);
  if (clear_status(workspace, stream) != cudaSuccess) return KDA_ERR_CUDA;
  return launched(launch_cache_read(a));
}

size_t kda_attn_workspace_size(const kda_attn_shape* s) {
  AttnArgs a{};
  return check_attn(s, a) == KDA_OK ? attn_workspace(a) : 0;
}

kda_status kda_attn_step(const kda_attn_shape* s, const void* q, const void* k_cache,
                         const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                         const int32_t* pages, const int32_t* lens, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  AttnArgs a{};
  kda_status st = check_attn(s, a);
  if (st != KDA_OK) return st;
  if (s->B > 0 && (!q || !out || !pages || !lens || !k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
  if (coded(s->cache) ? s->B > 0 && (!k_scale || !v_scale) : k_scale || v_scale)
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({q, (const void*)out}, dsize(s->dtype)) ||
      !all_aligned({(const void*)pages, (const void*)lens, (const void*)lse}, 4) ||
      !all_aligned({k_cache, v_cache, (const void*)k_scale, (const void*)v_scale}, 16))
    return KDA_ERR_INVALID_ARG;
  const size_t need = attn_workspace(a);  // the status alone may be left out
  if ((workspace || workspace_bytes || need > kWsHeader) &&
      (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return KDA_ERR_WORKSPACE;
  a.q = q; a.kc = k_cache; a.vc = v_cache; a.ks = k_scale; a.vs = v_scale;
  a.t.pages = pages; a.t.lens = lens;
  a.out = out; a.lse = lse;
  a.ws = workspace;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_attn(a));
}

kda_status kda_draft_verify(const kda_verify_shape* s, const void* p, const void* q,
                            const int32_t* drafts, const int32_t* num_draft, const float* u,
                            int32_t* tokens, int32_t* num_commit, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->B < 0 || s->K < 0 || s->V < 1 || !dtype_ok(s->dtype)) return KDA_ERR_INVALID_ARG;
  if (s->K > 31 || s->V >= 1 << 19) return KDA_ERR_UNSUPPORTED;
  if (s->B > 0 && (!p || !u || !tokens || !num_commit || (s->K > 0 && !drafts)))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({p, q}, dsize(s->dtype)) ||
      !all_aligned({(const void*)drafts, (const void*)num_draft, (const void*)u,
                    (const void*)tokens, (const void*)num_commit}, 4))
    return KDA_ERR_INVALID_ARG;
  kda_status st = check_status_ws(workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  VerifyArgs a{};
  a.p = p; a.q = q; a.drafts = drafts; a.counts = num_draft; a.u = u;
  a.tokens = tokens; a.commit = num_commit;
  a.B = s->B; a.K = s->K; a.V = s->V;
  a.bf16 = s->dtype == KDA_BF16;
  a.status = static_cast<unsigned int*>(workspace);
  a.sms = device_sms();
  a.stream = static_cast<cudaStream_t>(stream);
  if (clear_status(workspace, stream) != cudaSuccess) return KDA_ERR_CUDA;
  return launched(launch_verify(a));
}

}  // extern "C"
