// C ABI of the operators around the recurrence: argument checks, workspace
// carving and dispatch.  Every check that can be made on the host is made before
// anything is launched; nothing here allocates memory.
#include "kda_layer.cuh"

using namespace kda;
using namespace kda::layer;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
size_t dsize(kda_dtype t) { return t == KDA_F32 ? 4 : 2; }
constexpr int64_t kMaxElems = (int64_t)1 << 40;  // elements of one tensor
constexpr int kMaxChannels = 0x7fffffff - 1023;  // a block's last channel stays below 2^31

// every pointer of the list (NULLs aside) a multiple of `a`
template <int N>
bool all_aligned(const void* const (&p)[N], size_t a) {
  for (const void* q : p)
    if (q && !aligned(q, a)) return false;
  return true;
}

// the optional workspace: absent, or aligned and large enough for the status word
kda_status check_status_ws(const void* ws, size_t bytes) {
  if (!ws) return KDA_OK;
  return aligned(ws, 256) && bytes >= kWsHeader ? KDA_OK : KDA_ERR_WORKSPACE;
}

kda_status check_tokens(int32_t B, int32_t T, int32_t num_seqs, bool packed) {
  if (T < 0) return KDA_ERR_INVALID_ARG;
  if (packed ? (B != 1 || num_seqs < 0) : B < 0) return KDA_ERR_INVALID_ARG;
  // tokens of a packed batch belong to some sequence
  if (packed && num_seqs == 0 && T > 0) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}
// a token stride of 0 is the dense one; rows may not overlap
bool stride_ok(int64_t& ld, int64_t row) {
  if (ld == 0) ld = row;
  return ld >= row && ld <= kMaxElems;
}

kda_status check_conv(const kda_conv_shape* s, bool packed, int64_t& ldx) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->D < 1 || s->D > kMaxChannels || !dtype_ok(s->dtype)) return KDA_ERR_INVALID_ARG;
  kda_status st = check_tokens(s->B, s->T, s->num_seqs, packed);
  if (st != KDA_OK) return st;
  if (s->W < 2 || s->W > 4) return KDA_ERR_UNSUPPORTED;
  ldx = s->ldx;
  if (!stride_ok(ldx, s->D)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)s->B * s->T > kMaxElems / ldx) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

ConvArgs conv_args(const kda_conv_shape* s, bool packed, const int32_t* cu, int64_t ldx,
                   const void* x, const float* w, const float* b, void* ws, void* stream) {
  ConvArgs a{};
  a.x = x; a.w = w; a.b = b;
  a.q = Seqs{cu, s->T, (int64_t)s->B * s->T, packed ? s->num_seqs : s->B};
  a.D = s->D; a.W = s->W; a.T = s->T;
  a.ldx = ldx;
  a.bf16 = s->dtype == KDA_BF16;
  a.silu = s->silu != 0;
  a.sms = device_sms();
  a.status = static_cast<unsigned int*>(ws);
  a.stream = static_cast<cudaStream_t>(stream);
  return a;
}

int64_t conv_tiles(const kda_conv_shape* s, int64_t& tile) {
  const int64_t tokens = (int64_t)s->B * s->T;
  tile = conv_bwd_tile(tokens, s->D, s->dtype == KDA_BF16, device_sms());
  return (tokens + tile - 1) / tile;
}

kda_status check_scan(const kda_scan_shape* s, bool packed, ScanArgs& a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->H < 1 || s->G < 1 || s->H % s->G != 0 || s->ds < 1 || s->dx < 1) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(s->in_dtype) || !dtype_ok(s->out_dtype)) return KDA_ERR_INVALID_ARG;
  kda_status st = check_tokens(s->B, s->T, s->num_seqs, packed);
  if (st != KDA_OK) return st;
  if ((s->ds != 64 && s->ds != 128) || (s->dx != 64 && s->dx != 128)) return KDA_ERR_UNSUPPORTED;
  a.ldx = s->ldx; a.lddt = s->lddt; a.ldb = s->ldb; a.ldc = s->ldc;
  const int64_t gd = (int64_t)s->G * s->ds;
  if (!stride_ok(a.ldx, (int64_t)s->H * s->dx) || !stride_ok(a.lddt, s->H) ||
      !stride_ok(a.ldb, gd) || !stride_ok(a.ldc, gd))
    return KDA_ERR_INVALID_ARG;
  int64_t widest = a.ldx;
  for (int64_t l : {a.lddt, a.ldb, a.ldc}) widest = l > widest ? l : widest;
  if ((int64_t)s->B * s->T > kMaxElems / widest) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

size_t scan_bytes(const kda_scan_shape* s, bool packed) {
  if (!s || s->B < 0 || s->T < 0 || s->H < 1 || s->G < 1 || (packed && s->num_seqs < 0) ||
      (s->ds != 64 && s->ds != 128) || (s->dx != 64 && s->dx != 128))
    return 0;
  if (s->in_dtype != KDA_BF16) return kWsHeader;
  return kWsHeader + scan_bf16_workspace(packed, packed ? s->num_seqs : s->B, s->T,
                                         (int64_t)s->B * s->T, s->H, s->G, s->ds, s->dx,
                                         device_sms());
}

void fill_scan(const kda_scan_shape* s, ScanArgs& a, bool packed, const int32_t* cu, const void* x,
               const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
               const float* dtb, void* y, void* ws, void* stream) {
  a.x = x; a.dt = dt; a.Bm = Bm; a.Cm = Cm;
  a.A = A; a.D = D; a.dtb = dtb;
  a.y = y;
  a.q = Seqs{cu, s->T, (int64_t)s->B * s->T, packed ? s->num_seqs : s->B};
  a.H = s->H; a.G = s->G; a.ds = s->ds; a.dx = s->dx; a.T = s->T;
  a.bf16 = s->in_dtype == KDA_BF16;
  a.out_bf16 = s->out_dtype == KDA_BF16;
  a.softplus = s->dt_softplus != 0;
  a.status = static_cast<unsigned int*>(ws);
  a.sms = device_sms();
  a.stream = static_cast<cudaStream_t>(stream);
}

kda_status check_norm(const kda_norm_shape* s, NormArgs& a) {
  if (!s) return KDA_ERR_INVALID_ARG;
  if (s->tokens < 0 || s->heads < 1 || s->d < 1 || !dtype_ok(s->dtype)) return KDA_ERR_INVALID_ARG;
  if (s->res_dtype != s->dtype && s->res_dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
  if (s->gate != KDA_GATE_NONE && s->gate != KDA_GATE_SIGMOID && s->gate != KDA_GATE_SILU)
    return KDA_ERR_INVALID_ARG;
  if (!(s->scale == s->scale) || !(s->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (s->d > 8192) return KDA_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)s->heads * s->d;
  a.ldx = s->ldx; a.ldg = s->ldgate;
  if (!stride_ok(a.ldx, row) || !stride_ok(a.ldg, row)) return KDA_ERR_INVALID_ARG;
  if (s->tokens > kMaxElems / (a.ldx > a.ldg ? a.ldx : a.ldg)) return KDA_ERR_INVALID_ARG;
  a.tokens = s->tokens; a.heads = s->heads; a.d = s->d;
  a.bf16 = s->dtype == KDA_BF16;
  a.res_bf16 = s->res_dtype == KDA_BF16;
  a.gate_act = s->gate;
  a.gate_first = s->gate_first != 0;
  a.scale = s->scale; a.eps = s->eps;
  a.inv_d = 1.f / (float)s->d;
  a.sms = device_sms();
  a.dense = a.ldx == row && a.ldg == row;
  return KDA_OK;
}

kda_status launched(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

kda_status kda_conv_fwd(const kda_conv_shape* s, const void* x, const float* weight,
                        const float* bias, const int32_t* cu_seqlens, const void* init_state,
                        void* y, void* final_state, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int64_t ldx;
  kda_status st = check_conv(s, packed, ldx);
  if (st != KDA_OK) return st;
  if (!weight || ((int64_t)s->B * s->T > 0 && (!x || !y))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, init_state, (const void*)y, (const void*)final_state}, dsize(s->dtype)) ||
      !all_aligned({(const void*)weight, (const void*)bias, (const void*)cu_seqlens}, 4))
    return KDA_ERR_INVALID_ARG;
  if ((st = check_status_ws(workspace, workspace_bytes)) != KDA_OK) return st;
  ConvArgs a = conv_args(s, packed, cu_seqlens, ldx, x, weight, bias, workspace, stream);
  a.init = init_state;
  a.y = y;
  a.fin = final_state;
  return launched(launch_conv_fwd(a));
}

kda_status kda_conv_step(const kda_conv_shape* s, const void* x, const float* weight,
                         const float* bias, const int32_t* num_commit, void* state, void* y,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int64_t ldx;
  kda_status st = check_conv(s, false, ldx);
  if (st != KDA_OK) return st;
  if (s->T < 1 || s->T > 8) return KDA_ERR_UNSUPPORTED;
  if (!weight || (s->B > 0 && (!x || !state || (!y && !num_commit)))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, (const void*)state, (const void*)y}, dsize(s->dtype)) ||
      !all_aligned({(const void*)weight, (const void*)bias, (const void*)num_commit}, 4))
    return KDA_ERR_INVALID_ARG;
  if ((st = check_status_ws(workspace, workspace_bytes)) != KDA_OK) return st;
  ConvArgs a = conv_args(s, false, nullptr, ldx, x, weight, bias, workspace, stream);
  a.counts = num_commit;
  a.state = state;
  a.y = y;
  return launched(launch_conv_step(a));
}

size_t kda_conv_bwd_workspace_size(const kda_conv_shape* s) {
  if (!s || s->B < 0 || s->T < 0 || s->D < 1 || s->W < 2 || s->W > 4) return 0;
  int64_t tile;
  return kWsHeader + (size_t)conv_tiles(s, tile) * (s->W + 1) * s->D * sizeof(float);
}

kda_status kda_conv_bwd(const kda_conv_shape* s, const void* x, const float* weight,
                        const float* bias, const int32_t* cu_seqlens, const void* init_state,
                        const void* dy, const void* dfinal, void* dx, float* dweight,
                        float* dbias, void* dinit, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int64_t ldx;
  kda_status st = check_conv(s, packed, ldx);
  if (st != KDA_OK) return st;
  if (!weight || !dweight || ((int64_t)s->B * s->T > 0 && (!x || !dy || !dx)))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, init_state, dy, dfinal, (const void*)dx, (const void*)dinit},
                   dsize(s->dtype)) ||
      !all_aligned({(const void*)weight, (const void*)bias, (const void*)cu_seqlens,
                    (const void*)dweight, (const void*)dbias}, 4))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda_conv_bwd_workspace_size(s))
    return KDA_ERR_WORKSPACE;
  ConvArgs a = conv_args(s, packed, cu_seqlens, ldx, x, weight, bias, workspace, stream);
  a.init = init_state;
  a.dy = dy; a.dfinal = dfinal;
  a.dx = dx; a.dw = dweight; a.db = dbias; a.dinit = dinit;
  a.tiles = conv_tiles(s, a.tile);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeader);
  return launched(launch_conv_bwd(a));
}

size_t kda_scan_workspace_size(const kda_scan_shape* s) {
  // a fixed-length call ignores num_seqs, which may hold anything: enough for either call
  const size_t fixed = scan_bytes(s, false);
  const size_t packed = s && s->B == 1 && s->num_seqs > 0 ? scan_bytes(s, true) : 0;
  return fixed > packed ? fixed : packed;
}

kda_status kda_scan_fwd(const kda_scan_shape* s, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                        const int32_t* cu_seqlens, const float* h0, void* y, float* hT,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  ScanArgs a{};
  kda_status st = check_scan(s, packed, a);
  if (st != KDA_OK) return st;
  if (!A || (dt_bias && !s->dt_softplus) ||
      ((int64_t)s->B * s->T > 0 && (!x || !dt || !Bm || !Cm || !y)))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, dt, Bm, Cm}, dsize(s->in_dtype)) || !aligned(y, dsize(s->out_dtype)) ||
      !all_aligned({(const void*)A, (const void*)D, (const void*)dt_bias,
                    (const void*)cu_seqlens}, 4) ||
      !all_aligned({(const void*)h0, (const void*)hT}, 16))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < scan_bytes(s, packed))
    return KDA_ERR_WORKSPACE;
  fill_scan(s, a, packed, cu_seqlens, x, dt, A, Bm, Cm, D, dt_bias, y, workspace, stream);
  a.h0 = h0;
  a.hT = hT;
  a.ws = static_cast<char*>(workspace) + kWsHeader;
  return launched(scan_bf16_ok(a) ? launch_scan_bf16(a) : launch_scan_recurrent(a));
}

kda_status kda_scan_step(const kda_scan_shape* s, const void* x, const void* dt, const float* A,
                         const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                         const int32_t* num_commit, float* state, void* y, void* workspace,
                         size_t workspace_bytes, void* stream) {
  ScanArgs a{};
  kda_status st = check_scan(s, false, a);
  if (st != KDA_OK) return st;
  if (s->T < 1 || s->T > 8) return KDA_ERR_UNSUPPORTED;
  if (!A || (dt_bias && !s->dt_softplus) ||
      (s->B > 0 && (!x || !dt || !Bm || !Cm || !state || (!y && !num_commit))))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, dt, Bm, Cm}, dsize(s->in_dtype)) || !aligned(y, dsize(s->out_dtype)) ||
      !all_aligned({(const void*)A, (const void*)D, (const void*)dt_bias,
                    (const void*)num_commit}, 4) ||
      !aligned(state, 16))
    return KDA_ERR_INVALID_ARG;
  if ((st = check_status_ws(workspace, workspace_bytes)) != KDA_OK) return st;
  fill_scan(s, a, false, nullptr, x, dt, A, Bm, Cm, D, dt_bias, y, workspace, stream);
  a.counts = num_commit;
  a.state = state;
  return launched(launch_scan_step(a));
}

kda_status kda_norm_fwd(const kda_norm_shape* s, const void* x, const float* weight,
                        const void* gate, const void* residual, const float* res_scale,
                        const float* out_weight, void* r, void* y, void* stream) {
  NormArgs a{};
  kda_status st = check_norm(s, a);
  if (st != KDA_OK) return st;
  if ((s->gate != KDA_GATE_NONE) != (gate != nullptr) && s->tokens > 0) return KDA_ERR_INVALID_ARG;
  if ((out_weight != nullptr) != (y != nullptr) && s->tokens > 0) return KDA_ERR_INVALID_ARG;
  if (s->tokens > 0 && (!x || (!r && !y))) return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, gate, (const void*)y}, dsize(s->dtype)) ||
      !all_aligned({residual, (const void*)r}, dsize(s->res_dtype)) ||
      !all_aligned({(const void*)weight, (const void*)res_scale, (const void*)out_weight}, 4))
    return KDA_ERR_INVALID_ARG;
  a.x = x; a.w = weight; a.gate = gate; a.res = residual; a.ls = res_scale; a.ow = out_weight;
  a.r = r; a.y = y;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_norm_fwd(a));
}

size_t kda_norm_bwd_workspace_size(const kda_norm_shape* s) {
  if (!s || s->tokens < 0 || s->heads < 1 || s->d < 1) return 0;
  return kWsHeader + (size_t)norm_bwd_ctas(s->tokens * s->heads, s->d, s->dtype == KDA_BF16,
                                           device_sms()) * 3 * s->d * sizeof(float);
}

kda_status kda_norm_bwd(const kda_norm_shape* s, const void* x, const float* weight,
                        const void* gate, const void* residual, const float* res_scale,
                        const float* out_weight, const void* dr, const void* dy, void* dx,
                        void* dgate, void* dresidual, float* dweight, float* dres_scale,
                        float* dout_weight, void* workspace, size_t workspace_bytes,
                        void* stream) {
  NormArgs a{};
  kda_status st = check_norm(s, a);
  if (st != KDA_OK) return st;
  const bool any = s->tokens > 0;
  if ((s->gate != KDA_GATE_NONE) != (gate != nullptr) && any) return KDA_ERR_INVALID_ARG;
  if ((dy && !out_weight) || (any && !dr && !dy)) return KDA_ERR_INVALID_ARG;
  if (any && (!x || !dx)) return KDA_ERR_INVALID_ARG;
  // a gradient is asked for only where its operand is there
  if ((dgate && !gate && any) || (dresidual && !residual && any) || (dweight && !weight) ||
      (dres_scale && !res_scale) || (dout_weight && !out_weight))
    return KDA_ERR_INVALID_ARG;
  if (!all_aligned({x, gate, dy, (const void*)dx, (const void*)dgate}, dsize(s->dtype)) ||
      !all_aligned({residual, dr, (const void*)dresidual}, dsize(s->res_dtype)) ||
      !all_aligned({(const void*)weight, (const void*)res_scale, (const void*)out_weight,
                    (const void*)dweight, (const void*)dres_scale, (const void*)dout_weight}, 4))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kda_norm_bwd_workspace_size(s))
    return KDA_ERR_WORKSPACE;
  a.x = x; a.w = weight; a.gate = gate; a.res = residual; a.ls = res_scale; a.ow = out_weight;
  a.dr = dr; a.dy = dy; a.dx = dx; a.dgate = dgate; a.dres = dresidual;
  a.dw = dweight; a.dls = dres_scale; a.dow = dout_weight;
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeader);
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_norm_bwd(a));
}

}  // extern "C"
