// Selective state-space scan of bf16 prompts on the tcgen05 tensor cores, 64
// tokens (a chunk) at a time.  With c_i the running sum of delta A over the chunk
// (in log2 units) and S the state at its start:
//
//     y_i = 2^c_i S^T C_i + sum_{j <= i} M_ij x_j + D x_i,   M_ij = 2^(c_i - c_j) delta_j (C_i . B_j)
//     S  <- 2^c_last S + sum_j B_j (w_j x_j)^T,              w_j = 2^(c_last - c_j) delta_j
//
// Every exponent is a sum over the tokens between two others, at most 0: nothing overflows.  It is
// never the rounded difference of two long sums, of which a token that forgets nearly everything
// (c far below -1000) would leave few digits: w and the factors of M's lower left block are summed
// from their own ends, and the c of M's diagonal blocks start with each block and are exact in
// steps of 2^-9, with what is left summed apart (with c in one float the outputs after a step of
// 300 at A = -1e4 were off by up to 1.8 of their rms).  A token's own exponent is not let below
// -1024, which is nothing in float32 too, so that the sums stay finite.
// Per chunk and 128 state columns (one head of 128 channels or two
// neighbouring heads of 64 that share B and C) the products are, as D[lane][column]
// in tensor memory:
//     G  [token i][token j]   = C B^T      (rows 64.. of its M = 128 are unused)
//     U  [channel][state row] = (w x)^T B
//     Yi [channel][token]     = Sb C^T     (Sb: S^T, A operand in tensor memory)
//     Yx [channel][token]     = x^T M^T    (one per head)
// B, C and x are bf16 as given; Sb and M enter as bf16 hi + lo (16 bits: 2.4e-6 of the outputs' rms,
// below what bf16 outputs keep), w x in three parts (24 bits, as S is kept in float32).  D sits on M's diagonal.  S itself stays float32 in the
// registers of the state warps.
//
// One persistent CTA per SM; its warps are specialised and hand chunks on through
// mbarriers, so that the tensor core works on one chunk while other warps prepare the next
// one's operands and write the last one's outputs:
//     warps 0-7    state: S = 2^c_last S + U in registers (columns split in two), Sb
//     warps 8-11   outputs: y = 2^c Yi + Yx to global memory
//     warps 12,13,17   M from G (the three 32 x 32 blocks on and below the diagonal)
//     warps 14,15,18,19,24-27  w x in parts from the x tile; zero rows past the sequence's end
//     warps 21, 23, 16 tcgen05.mma: G and U; Yi; Yx (one thread each)
//     warp 22      work items, tile loads (TMA, 128-byte swizzle)
//     warp 20      per-token factors (delta, running sums, weights)
// The code of one chunk's steady state has to stay inside the SM's instruction cache with
// all roles at work: loops that need no register arrays are kept rolled, and items are decoded
// once, by warp 22.
// U does not depend on S, so the chain from chunk to chunk is one multiply-add per state
// element; every product is off it.  The state warps take registers from the others.
//
// Long sequences are cut into segments that run as items of their own: a first
// launch forms each segment's own end state (all but the last; no outputs) and its
// total decay, the second starts each segment from the decayed sum of those before.
//
// One GB300: 4 x 4096 tokens of 32 heads of 128 (4 groups, state 128) take 131 us, 16 packed
// sequences (58511 tokens) of 64 heads of 64 take 635 us, 131071 tokens of 32 heads 1.44 ms.
// A chunk takes about 3900 cycles (5100 for two heads): no unit is full (tensor pipe 40%, issue
// 50%, shared memory about 390 KB or 3000 cycles per chunk, half of them operands of the
// products), and the longest turn is M's: wait for the products with the last M, form it, hand
// it to the tensor core.
#include <cudaTypedefs.h>

#include "kda_layer.cuh"
#include "kda_prefill_common.cuh"

namespace kda {
namespace layer {
namespace {

using namespace sm100;
using pf::bf16_hi;
using pf::bf16_lo;
using pf::ex2;
using pf::pack2;

constexpr int Q = 64;              // tokens per chunk
constexpr int kScanThreads = 896;  // 28 warps
constexpr int kRing = 4;           // chunks of per-token factors
constexpr int kItems = 4;          // items handed out ahead
constexpr int kFlags = 2 * kRing;  // flags of chunks: w x is at most kRing ahead of the outputs
// the roles are spread so that the SM's four schedulers (warp % 4) get about the same work
constexpr int kFactorWarp = 20, kStateMmaWarp = 21, kLoadWarp = 22, kYiMmaWarp = 23, kYxMmaWarp = 16;
constexpr int kTile = 8192;        // 64 tokens x 64 channels of bf16, 128-byte rows
// Exponents in [-1024, 0]: (x + kGrid) - kGrid rounds to a multiple of 2^-9, of which float32 holds
// every sum over 32 tokens exactly
constexpr float kFloor = -1024.f, kGrid = 24576.f;

// tensor memory columns: U, Sb hi and lo, G, then Yi and Yx.  One head of 128 channels
// leaves room for two Yi; two heads have a Yx each.
constexpr uint32_t TM_U = 0, TM_SB = 128, TM_G = 256, TM_YI = 320, TM_YX = 448, TM_ALL = 512;
constexpr uint32_t TM_YX2 = 384;  // two heads: the second one's Yx
// of 72 at launch: 2 * 120 + 72 + 4 * 48 <= 7 * 72
constexpr int kStateRegs = 120, kOutRegs = 72, kOtherRegs = 48;

// per-token factors of one head and chunk, in shared memory
struct Factors {
  // running log2 decay since token 0 or 32 in steps of 2^-9; 2^(what that leaves out), and the step
  // sizes (0 past the end) over it: 2^(c_i - c_j) delta_j = r_i 2^(c[i] - c[j]) delta[j]
  float c[Q], r[Q], delta[Q];
  float w[Q];      // weights of the state update
  float e[Q];      // 2^(running decay since token 0)
  float u[32];     // 2^(c_i - c_31), i = 32 ..
  float v[32];     // 2^(c_31 - c_j) delta_j, j = .. 31
  float alpha;     // 2^c_last
  float pad[3];
};

template <int DS, int HPC>
struct Layout {
  static constexpr int kStages = HPC == 1 ? 3 : 2;   // tile stages, as many as fit
  static constexpr int kB = DS / 64 * kTile;         // bytes of a B or C tile
  static constexpr int kStage = 2 * kB + 2 * kTile;  // C, B, x
  static constexpr int kC = 0, kBt = kB, kX = 2 * kB;
  static constexpr int kWx = kStages * kStage;       // [3 parts][2 tiles]
  static constexpr int kM = kWx + 6 * kTile;         // [HPC][hi, lo]
  static constexpr int kY = kM + 2 * HPC * kTile;    // 32 tokens of y
  static constexpr int kF = kY + kTile;              // Factors [kRing][HPC]
  static constexpr int kBars = kF + kRing * HPC * (int)sizeof(Factors);
  static constexpr int kBytes = kBars + 768 + 1024;  // + alignment of the base to 1024
};

// mbarriers.  A phase is waited for by its parity, so that a barrier may not complete the phase
// after the next before every one of its waiters has seen this one: where the waiters do not
// hold each other up, there is one barrier per stage or per parity of the chunk.
enum Bar {
  B_FULL = 0,               // [stages] B and C tiles have landed
  B_FULLX = 3,              // [stages] the x tile has
  B_EMPTY = 6,              // [stages] the chunk's products are done
  B_FFULL = 9,              // [kRing] factors written
  B_FEMPTY = 13,            // [kRing] factors read
  B_IFULL = 17,             // [kItems] item published
  B_IEMPTY = 21,            // [kItems] item read by every warp that takes items
  B_G = 25,                 // G complete
  B_M = 26,                 // M written (and G read)
  B_X = 27,                 // [stages][2] w x written, tokens 0-31 and 32-63
  B_WX = 33,                // [2] those w x free
  B_U = 35,                 // U complete
  B_UFREE = 36,             // U read
  B_S = 37,                 // Sb written
  B_YI = 38,                // [2] Yi complete (and Sb free)
  B_YX = 40,                // Yx complete (and M free)
  B_YFREE = 41,             // [2] Yi and Yx read
  B_DRAIN = 43,
  B_COUNT = 44
};

struct ScanParams {
  Seqs q;
  const __nv_bfloat16 *x, *dt;
  const float *A, *D, *dtb, *h0;
  void* y;
  float* hT;
  int H, G, hpg, tpg;        // heads, groups, heads and 128-column tiles per group
  int64_t ldx, lddt;
  int softplus, out_bf16;
  // segments: tokens each (0: none); the states before segments 1 .. of split
  // sequences, [slot][H][DS][dx], and their decays [slot][H]
  int64_t seg;
  int nseg;                  // fixed length: segments per sequence
  float *seg_s, *seg_a;
  const int32_t* plan;       // packed: counts, then the items (see plan_kernel), or nullptr
  int64_t plan_most;         // bound on the items of either launch
  unsigned int* status;
  int first;                 // this launch clears the status word
};

// packed plan: [0] output items, [1] state items, then at 4: output items (sequence, segment),
// state items, and per sequence its first slot
struct PlanView {
  const int32_t* p;
  int64_t most;
  __device__ const int2* out() const { return reinterpret_cast<const int2*>(p + 4); }
  __device__ const int2* st() const { return out() + most; }
  __device__ const int32_t* slot() const { return reinterpret_cast<const int32_t*>(st() + most); }
};

struct Item {
  int64_t t0;             // first flat token
  int64_t slot;           // the sequence's first state slot
  int n, h0, nh, g;       // sequence, first head, heads in the tile, group
  int len, chunks;        // tokens and chunks
  int seg, last;          // segment and whether it ends the sequence
  int valid;              // 0: no more items
  int pad[3];
};

template <int HPC, bool kState>
__device__ __forceinline__ int64_t item_count(const ScanParams& p) {
  const int64_t tiles = (int64_t)p.G * p.tpg;
  if (p.plan) return (int64_t)p.plan[kState ? 1 : 0] * tiles;
  return (int64_t)p.q.N * (kState ? p.nseg - 1 : p.nseg) * tiles;
}

template <int HPC, bool kState>
__device__ __forceinline__ Item get_item(const ScanParams& p, int64_t i) {
  const int64_t tiles = (int64_t)p.G * p.tpg;
  const int64_t k = i / tiles;
  const int tile = (int)(i - k * tiles);
  Item it;
  it.g = tile / p.tpg;
  const int in = (tile - it.g * p.tpg) * HPC;  // first head of the tile within its group
  it.h0 = it.g * p.hpg + in;
  it.nh = p.hpg - in < HPC ? p.hpg - in : HPC;
  if (p.plan) {
    const PlanView v{p.plan, p.plan_most};
    const int2 e = kState ? v.st()[k] : v.out()[k];
    it.n = e.x;
    it.seg = e.y;
    it.slot = v.slot()[it.n];
  } else {
    const int per = kState ? p.nseg - 1 : p.nseg;
    it.n = (int)(k / per);
    it.seg = (int)(k - (int64_t)it.n * per);
    it.slot = (int64_t)it.n * (p.nseg - 1);
  }
  int64_t s0, s1;
  p.q.range(it.n, s0, s1);
  it.last = 1;
  if (p.seg > 0) {
    s0 += it.seg * p.seg;
    if (s0 > s1) s0 = s1;
    if (s1 - s0 > p.seg) {
      s1 = s0 + p.seg;
      it.last = 0;
    }
  }
  it.t0 = s0;
  it.len = (int)(s1 - s0);
  it.valid = 1;
  it.chunks = (int)((it.len + Q - 1) / Q);
  return it;
}
// items of a CTA, in snake order: longest first in every round, alternating direction
__device__ __forceinline__ int64_t item_at(int64_t round) {
  const int64_t b = (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  return round * gridDim.x + b;
}

// softplus(x) = max(x, 0) + log1p(y), y = e^-|x|: with s = y / (2 + y) <= 1/3, log1p(y) =
// 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...), cut after s^12/13 (2e-8 of the sum).  In few
// instructions, and a few 1e-7 of the result for small results too.
__device__ __forceinline__ float step_size_fast(float dt, float bias, bool softplus) {
  if (!softplus) return dt;
  const float x = dt + bias;
  const float y = ex2(-fabsf(x) * 1.4426950408889634f);
  const float s = __fdividef(y, 2.f + y), q = s * s;
  float v = 1.f / 13.f;
  v = fmaf(v, q, 1.f / 11.f);
  v = fmaf(v, q, 1.f / 9.f);
  v = fmaf(v, q, 1.f / 7.f);
  v = fmaf(v, q, 1.f / 5.f);
  v = fmaf(v, q, 1.f / 3.f);
  v = fmaf(v, q, 1.f);
  return fmaf(2.f * s, v, fmaxf(x, 0.f));
}

// bf16 parts of two values, packed (first value in the low half); each remainder is exact
__device__ __forceinline__ float2 part_of(float2 v, uint32_t& p) {
  p = pack2(v.x, v.y);
  return fma2(make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)), make_float2(-1.f, -1.f), v);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const float2 r = part_of(make_float2(a, b), hi);
  lo = pack2(r.x, r.y);
}
__device__ __forceinline__ void split3(float2 v, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  const float2 r = part_of(part_of(v, p0), p1);
  p2 = pack2(r.x, r.y);
}

// whether one of four pairs of bf16 is a NaN
__device__ __forceinline__ bool any_nan(const uint4& v) {
  const auto h = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 t = __hadd2(__hadd2(h(v.x), h(v.y)), __hadd2(h(v.z), h(v.w)));
  return !__hbeq2(t, t);
}
// a pair of bf16 with zeros for what is not finite
__device__ __forceinline__ uint32_t finite_part(uint32_t u) {
  if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
  return u;
}

// Wait for the phase of a barrier with the given parity; 0 when it does not come.  Each try
// suspends the thread for a while (about half a microsecond); the limit is between 20 ms and a
// second.  In few instructions: there are many waits, and the code has to stay small.
__device__ __forceinline__ uint32_t wait_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n"
      "TRY:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.and.u32 q, n, 0x100000, !p;\n\t"
      "@q bra TRY;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}

__device__ __forceinline__ uint32_t try_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}

struct Ctx {
  uint32_t bars;             // shared address of the barriers
  volatile uint32_t* abort;  // raised when a wait ran out
  uint32_t lane;
  __device__ __forceinline__ bool wait_one(int bar, uint32_t parity) const {
    if (wait_phase(bars + 8 * bar, parity)) return true;
    *abort = 1u;
    return false;
  }
  // up to three phases, whose first tries overlap (a try alone takes about 200 cycles)
  __device__ __forceinline__ bool wait_all(int bar, uint32_t parity, int bar2, uint32_t parity2, int bar3 = -1,
                                           uint32_t parity3 = 0) const {
    const uint32_t a = try_phase(bars + 8 * bar, parity);
    const uint32_t b = bar2 < 0 ? 1u : try_phase(bars + 8 * bar2, parity2);
    const uint32_t d = bar3 < 0 ? 1u : try_phase(bars + 8 * bar3, parity3);
    return (a || wait_one(bar, parity)) && (b || wait_one(bar2, parity2)) && (d || wait_one(bar3, parity3));
  }
  // the same by a whole warp, which stays converged
  __device__ __forceinline__ bool wait(int bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait_one(bar, parity));
  }
  __device__ __forceinline__ bool wait(int bar, uint32_t parity, int bar2, uint32_t parity2, int bar3 = -1,
                                       uint32_t parity3 = 0) const {
    return __all_sync(0xffffffffu, wait_all(bar, parity, bar2, parity2, bar3, parity3));
  }
  // by the warps of a group, which meet at named barrier `id`: its first warp waits (every waiting
  // warp takes issue slots from the working ones) and all of them get the same answer, so that
  // none leaves while another stays.
  __device__ __forceinline__ bool wait_group(int id, int count, bool first, int bar, uint32_t parity,
                                             int bar2 = -1, uint32_t parity2 = 0, int bar3 = -1,
                                             uint32_t parity3 = 0) const {
    int ok = 1;
    if (first) {
      ok = wait_all(bar, parity, bar2, parity2, bar3, parity3);
      __syncwarp();
    }
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(ok), "r"(id), "r"(count)
        : "memory");
    return all != 0;
  }
  __device__ __forceinline__ void arrive_warp(int bar) const {  // one arrival per warp
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.eq.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bars + 8 * bar),
        "r"(lane)
        : "memory");
  }
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  uint32_t u[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
        "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}
// 128-byte-swizzle operands.  K-major (rows of 64 K elements): 8-row groups 1024 bytes
// apart, the next 64 K elements one tile further.  MN-major (rows are K, 64 M/N elements
// each): 8-row groups 1024 bytes apart, the next 64 M/N elements one tile (the leading
// offset) further.  The descriptors' high word is the same for all of them.
__device__ __forceinline__ uint64_t op_desc(uint32_t lo) {
  constexpr uint32_t hi = (1024 >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 apart, version 1, swizzle 128
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint32_t op_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// Products and commits by one lane of a converged warp: the whole warp runs the code around them,
// so that descriptors are formed in uniform registers.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss_by(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_by(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_by(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// 32 columns of 16 lanes as 8 x 8 matrix fragments: r[4 q ..] holds columns 8 q + 2 (lane % 4)
// + {0, 1} of rows lane / 4 and lane / 4 + 8
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&r)[16]) {
  uint32_t u[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]),
        "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int DS, int HPC, bool kState>
__global__ void __launch_bounds__(kScanThreads, 1)
scan_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_c, const ScanParams p) {
  using L = Layout<DS, HPC>;
  constexpr int kStages = L::kStages;
  constexpr int DX = 128 / HPC;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile uint32_t* s_abort = s_tmem + 1;
  Item* s_items = reinterpret_cast<Item*>(s_tmem + 4);
  // [kFlags] set by the w x warps: the chunk has an x that is not finite; cleared by the outputs' warps
  volatile int* s_odd = reinterpret_cast<volatile int*>(s_items + kItems);
  static_assert(B_COUNT * 8 + 16 + kItems * sizeof(Item) + kFlags * 4 <= 768, "barrier area");
  Factors* factors = reinterpret_cast<Factors*>(sm + L::kF);
  // The shuffle tells the compiler that a warp's role is the same for all its lanes: addresses and
  // descriptors then go through the uniform registers (4 x 4096 tokens of 32 heads: 132 us, 167 without).
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int quad = warp & 3;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;

  if (threadIdx.x == 0) {
    if (p.first && p.status && blockIdx.x == 0) *p.status = KDA_OK;
    auto init = [&](int b, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(bars + b + i, count);
    };
    init(B_FULL, 6, 1);
    init(B_EMPTY, 3, kState ? 1 : 3);
    init(B_FFULL, kRing, 1);
    init(B_FEMPTY, kRing, kState ? 16 : 23);  // state 8, w x 8, outputs 4, M 3
    init(B_IFULL, kItems, 1);
    init(B_IEMPTY, kItems, kState ? 18 : 27);  // those, the products' warps, the factors'
    init(B_G, 1, 1);
    init(B_M, 1, 3);
    init(B_X, 6, 8);
    init(B_WX, 2, 1);
    init(B_U, 1, 1);
    init(B_UFREE, 1, 8);
    init(B_S, 1, 8);
    init(B_YI, 2, 1);
    init(B_YX, 1, 1);
    init(B_YFREE, 2, 4);
    init(B_DRAIN, 1, kState ? 1 : 3);
    *s_abort = 0;
    for (int i = 0; i < kFlags; ++i) s_odd[i] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_b);
    if (!kState) tma_prefetch_desc(&tm_c);
  }
  if (warp == 0) {
    tmem_alloc(s_tmem, TM_ALL);
    tmem_relinquish();
  }
  // M's block above the diagonal is never written: zero
  for (int i = threadIdx.x; i < 2 * HPC * kTile / 16; i += kScanThreads)
    reinterpret_cast<uint4*>(sm + L::kM)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *s_tmem;
  const uint32_t sbase = smem_u32(sm);
  const Ctx cx{smem_u32(bars), s_abort, (uint32_t)lane};

  // the next item, for the warps of a group; false when there is none (or the CTA gives up)
  auto next_item = [&](int id, int count, bool first, uint32_t& m, Item& it) {
    if (!cx.wait_group(id, count, first, B_IFULL + m % kItems, (m / kItems) & 1)) return false;
    it = s_items[m % kItems];
    cx.arrive_warp(B_IEMPTY + m % kItems);
    ++m;
    return it.valid != 0;
  };
  auto next_item_alone = [&](uint32_t& m, Item& it) {  // for one warp
    if (!cx.wait(B_IFULL + m % kItems, (m / kItems) & 1)) return false;
    it = s_items[m % kItems];
    cx.arrive_warp(B_IEMPTY + m % kItems);
    ++m;
    return it.valid != 0;
  };
  uint32_t m = 0, c = 0;  // items and chunks taken so far
  Item it;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
    // ---- state: S of lane's channel, columns [half * DS/2, + DS/2), in registers
    constexpr int kCols = DS / 2;
    const int half = warp >> 2;
    const int ch = quad * 32 + lane;         // channel of the tile
    const int k = HPC == 2 ? ch >> 6 : 0;    // its head in the tile
    const uint32_t tu = tb + lane_base + TM_U + half * kCols;
    const uint32_t tsb = tb + lane_base + TM_SB + half * (kCols / 2);
    bool alive = true;
    while (alive && next_item(2, 256, warp == 0, m, it)) {
      const bool on = k < it.nh;
      const int head = it.h0 + k;
      const int64_t at = ((int64_t)head * DS + half * kCols) * DX + (HPC == 2 ? ch & 63 : ch);
      const int64_t per = (int64_t)p.H * DS * DX;  // one sequence's or slot's states
      // start state: h0, or the decayed sum of the segments before this one, newest first
      float S[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) S[e] = 0.f;
      const float* src = it.seg == 0 ? (p.h0 ? p.h0 + it.n * per + at : nullptr)
                         : kState ? nullptr : p.seg_s + (it.slot + it.seg - 1) * per + at;
      if (on && src) {
        float f = 1.f;
#pragma unroll 1
        for (int j = it.seg - 1;; --j) {
#pragma unroll
          for (int e = 0; e < kCols; ++e) S[e] = fmaf(f, src[e * DX], S[e]);
          if (j < 1) break;
          f *= p.seg_a[(it.slot + j) * p.H + head];
          if (f == 0.f) break;
          src -= per;
        }
      }
      float alpha = 1.f, decay = 1.f;
#pragma unroll 1
      for (int ci = 0; ci <= it.chunks; ++ci) {
        if (ci > 0) {  // S = alpha S + U of the chunk before
          if (!cx.wait_group(2, 256, warp == 0, B_U, (c - 1) & 1)) { alive = false; break; }
          tc_fence_after();
          const float2 al = make_float2(alpha, alpha);
#pragma unroll
          for (int col = 0; col < kCols; col += 32) {
            float u[32];
            tmem_ld32(tu + col, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 s = fma2(al, make_float2(S[col + e], S[col + e + 1]), make_float2(u[e], u[e + 1]));
              S[col + e] = s.x;
              S[col + e + 1] = s.y;
            }
          }
          tc_fence_before();
          cx.arrive_warp(B_UFREE);
          if (ci == it.chunks) break;
        } else if (it.chunks == 0) {
          break;
        }
        // the factors; Sb may be rewritten once the last product with it is done
        if (!cx.wait_group(2, 256, warp == 0, B_FFULL + c % kRing, (c / kRing) & 1,
                           !kState && c > 0 ? B_YI + (int)((c - 1) & 1) : -1, ((c - 1) >> 1) & 1)) {
          alive = false;
          break;
        }
        alpha = factors[(c % kRing) * HPC + k].alpha;
        decay *= alpha;
        cx.arrive_warp(B_FEMPTY + c % kRing);
        if (!kState) {
          tc_fence_after();
#pragma unroll
          for (int col = 0; col < kCols; col += 32) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) split2(S[col + 2 * e], S[col + 2 * e + 1], hi[e], lo[e]);
            tmem_st16(tsb + col / 2, hi);
            tmem_st16(tsb + DS / 2 + col / 2, lo);
          }
          tmem_wait_st();
          tc_fence_before();
          cx.arrive_warp(B_S);
        }
        ++c;
      }
      if (!alive) break;
      // end state
      float* dst = nullptr;
      if (kState) dst = p.seg_s + (it.slot + it.seg) * per + at;
      else if (it.last && p.hT) dst = p.hT + it.n * per + at;
      if (dst && on) {
#pragma unroll
        for (int e = 0; e < kCols; ++e) dst[e * DX] = S[e];
      }
      if (kState && on && half == 0 && (HPC == 2 ? (ch & 63) : ch) == 0)
        p.seg_a[(it.slot + it.seg) * p.H + head] = decay;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }

  if (warp >= 8 && warp < 12 && !kState) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    // ---- outputs
    const int64_t ldy = (int64_t)p.H * DX;
    bool alive = true;
    while (alive && next_item(1, 128, warp == 8, m, it)) {
#pragma unroll 1
      for (int ci = 0; ci < it.chunks; ++ci, ++c) {
        const int left = it.len - ci * Q;
        const int n = left < Q ? left : Q;
        const int k = HPC == 2 ? quad >> 1 : 0;
        const Factors& f = factors[(c % kRing) * HPC + k];
        if (!cx.wait_group(1, 128, warp == 8, B_FFULL + c % kRing, (c / kRing) & 1, B_YI + (c & 1),
                           (c >> 1) & 1, B_YX, c & 1)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t ti = tb + lane_base + TM_YI + (HPC == 1 ? (c & 1) * 64 : 0);
        const uint32_t tx = tb + lane_base + (HPC == 2 && k ? TM_YX2 : TM_YX);
        const int64_t row0 = it.t0 + ci * Q;
        if (p.out_bf16) {
          // y^T fragments, transposed into a [token][channel] tile (128-byte swizzle) and out,
          // 32 tokens at a time
          const uint32_t ys = sbase + L::kY + (quad >> 1) * (kTile / 2);
          const int u = threadIdx.x - 256;  // 16-byte unit within 8 rows of both halves
          const int hf = (u >> 3) & 1, ck = u & 7;
          uint16_t* y = static_cast<uint16_t*>(p.y) + row0 * ldy + (int64_t)it.h0 * DX + hf * 64 + ck * 8;
          const int most = HPC == 1 || hf < it.nh ? n : 0;
          uint32_t w[4][8];  // both halves leave tensor memory first
#pragma unroll
          for (int part = 0; part < 4; ++part) {
            const int rows = (part & 1) * 16, j = (part >> 1) * 32;
            float a[16], b[16];
            tmem_ld_frag(ti + ((uint32_t)rows << 16) + j, a);
            tmem_ld_frag(tx + ((uint32_t)rows << 16) + j, b);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 e = *reinterpret_cast<const float2*>(&f.e[j + 8 * q + 2 * (lane & 3)]);
              const float2 y0 = fma2(e, make_float2(a[4 * q], a[4 * q + 1]), make_float2(b[4 * q], b[4 * q + 1]));
              const float2 y1 = fma2(e, make_float2(a[4 * q + 2], a[4 * q + 3]), make_float2(b[4 * q + 2], b[4 * q + 3]));
              w[part][2 * q] = pack2(y0.x, y0.y);
              w[part][2 * q + 1] = pack2(y1.x, y1.y);
            }
          }
          tc_fence_before();
          cx.arrive_warp(B_YFREE + (c & 1));
          cx.arrive_warp(B_FEMPTY + c % kRing);
          // matrices (token block, channel block) in the order (q, 0), (q, 1), (q + 1, 0), (q + 1, 1)
          const int tok = ((lane >> 4) << 3) + (lane & 7);
          const int chunk = ((quad & 1) << 2) + ((lane >> 3) & 1);
          const uint32_t ad = ys + tok * 128;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t o = ((chunk + 2 * r) ^ (tok & 7)) << 4;
              const uint32_t(&v)[8] = w[2 * j + r];
              stmatrix4_trans(ad + o, v[0], v[1], v[2], v[3]);
              stmatrix4_trans(ad + o + 16 * 128, v[4], v[5], v[6], v[7]);
            }
            pf::named_bar_sync(1, 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = (u >> 4) + 8 * i;
              if (32 * j + r < most)
                *reinterpret_cast<uint4*>(y + (32 * j + r) * ldy) = *reinterpret_cast<const uint4*>(
                    sm + L::kY + hf * (kTile / 2) + r * 128 + ((ck ^ (r & 7)) << 4));
            }
            pf::named_bar_sync(1, 128);
          }
        } else {
          const int ch = quad * 32 + lane;
          float* y = static_cast<float*>(p.y) + row0 * ldy + (int64_t)it.h0 * DX + ch;
          const int most = k < it.nh ? n : 0;
#pragma unroll 1
          for (int j = 0; j < Q; j += 8) {
            float a[8], b[8];
            tmem_ld8(ti + j, a);
            tmem_ld8(tx + j, b);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (j + e < most) *y = fmaf(f.e[j + e], a[e], b[e]);
              y += ldy;
            }
          }
          tc_fence_before();
          cx.arrive_warp(B_YFREE + (c & 1));
          cx.arrive_warp(B_FEMPTY + c % kRing);
        }
        // A channel's outputs from its first x on that is not finite are NaN (its 16 upper bits here)
        if (s_odd[c % kFlags]) {
          if (HPC == 1 || k < it.nh) {
            const int64_t ch = (int64_t)it.h0 * DX + quad * 32 + lane;
            const __nv_bfloat16* x = p.x + row0 * p.ldx + ch;
            const int step = p.out_bf16 ? 1 : 2;
            uint16_t* y = static_cast<uint16_t*>(p.y) + (row0 * ldy + ch) * step + (step - 1);
            bool nan = false;
#pragma unroll 1
            for (int i = 0; i < n; ++i, x += p.ldx, y += ldy * step) {
              nan |= !isfinite(to_f32(*x));
              if (nan) asm volatile("st.global.u16 [%0], %1;" ::"l"(y), "h"((uint16_t)0x7fff) : "memory");
            }
          }
          pf::named_bar_sync(1, 128);
          s_odd[c % kFlags] = 0;
        }
      }
    }
  } else if (warp == 12 || warp == 13 || warp == 17) {
    // ---- M = decayed G, the blocks on and below the diagonal
    const int jb = warp >= 16 ? 32 : 0;  // first column
    if (!kState) {
      const int row = quad * 32 + lane;
      const bool diag = quad * 32 == jb;
      bool alive = true;
      while (alive && next_item_alone(m, it)) {
        float skip[HPC];
#pragma unroll
        for (int k = 0; k < HPC; ++k) skip[k] = p.D && k < it.nh ? p.D[it.h0 + k] : 0.f;
#pragma unroll 1
        for (int ci = 0; ci < it.chunks; ++ci, ++c) {
          if (!cx.wait(B_FFULL + c % kRing, (c / kRing) & 1, B_G, c & 1)) {
            alive = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 32 && alive; j += 8) {
            float g[8];
            tmem_ld8(tb + lane_base + TM_G + jb + j, g);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < HPC; ++k) {
              const Factors& f = factors[(c % kRing) * HPC + k];
              unsigned char* mt = sm + L::kM + k * 2 * kTile + row * 128;
              float v[8];
              if (diag) {
                const int at = lane - j;
                const float ci_ = f.c[row], ri = f.r[row];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float x = fmaf(g[e] * ri, ex2(ci_ - f.c[jb + j + e]) * f.delta[jb + j + e], e == at ? skip[k] : 0.f);
                  v[e] = e <= at ? x : 0.f;
                }
              } else {
                const float u = f.u[lane];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  const float2 r = mul2(make_float2(g[e], g[e + 1]), mul2(make_float2(u, u), make_float2(f.v[j + e], f.v[j + e + 1])));
                  v[e] = r.x;
                  v[e + 1] = r.y;
                }
              }
              uint4 hi, lo;
              split2(v[0], v[1], hi.x, lo.x);
              split2(v[2], v[3], hi.y, lo.y);
              split2(v[4], v[5], hi.z, lo.z);
              split2(v[6], v[7], hi.w, lo.w);
              const int o = (((jb + j) >> 3) ^ (row & 7)) << 4;
              // the products that read the last M are done
              if (k == 0 && j == 0 && c > 0 && !cx.wait(B_YX, (c - 1) & 1)) { alive = false; break; }
              *reinterpret_cast<uint4*>(mt + o) = hi;
              *reinterpret_cast<uint4*>(mt + kTile + o) = lo;
            }
          }
          if (!alive) break;
          fence_proxy_async_smem();
          tc_fence_before();
          cx.arrive_warp(B_M);
          cx.arrive_warp(B_FEMPTY + c % kRing);
        }
      }
    }
  } else if (warp == 14 || warp == 15 || warp == 18 || warp == 19 || warp >= 24) {
    // ---- w x in three parts, in the x tile's own layout
    const int xw = warp >= 24 ? warp - 20 : ((warp - 14) >> 2) * 2 + (warp & 1);
    const int xt = xw * 32 + lane;  // 0 .. 255
    uint32_t st = 0, ph = 0;
    bool alive = true;
    while (alive && next_item_alone(m, it)) {
#pragma unroll 1
      for (int ci = 0; ci < it.chunks; ++ci, ++c) {
        const int left = it.len - ci * Q;
        const int n = left < Q ? left : Q;
        unsigned char* x = sm + st * L::kStage + L::kX + xt * 16;
        unsigned char* wx = sm + L::kWx + xt * 16;
        const Factors* f = factors + (c % kRing) * HPC;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        // 32 tokens at a time: the state update takes the first while the others are formed
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!(h == 0 ? cx.wait(B_FULLX + st, ph, B_FFULL + c % kRing, (c / kRing) & 1, c > 0 ? B_WX : -1, (c - 1) & 1)
                       : c == 0 || cx.wait(B_WX + 1, (c - 1) & 1))) {
            alive = false;
            break;
          }
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {  // tiles of 64 channels; this thread's 16 bytes of a row
            const int o = q * kTile + h * (kTile / 2);
            const int tok = h * 32 + (xt >> 3);
            uint4 a = zero, b = zero, d = zero;
            if (tok < n) {
              const float w = f[HPC == 2 ? q : 0].w[tok];
              const float2 w2 = make_float2(w, w);
              const uint4 v = *reinterpret_cast<const uint4*>(x + o);
              split3(mul2(w2, make_float2(bf16_lo(v.x), bf16_hi(v.x))), a.x, b.x, d.x);
              split3(mul2(w2, make_float2(bf16_lo(v.y), bf16_hi(v.y))), a.y, b.y, d.y);
              split3(mul2(w2, make_float2(bf16_lo(v.z), bf16_hi(v.z))), a.z, b.z, d.z);
              split3(mul2(w2, make_float2(bf16_lo(v.w), bf16_hi(v.w))), a.w, b.w, d.w);
              // The third part of what is not finite is NaN.  M's zeros above the diagonal would carry
              // x to earlier tokens: the tile gets a zero, and the outputs' warps write the NaN.
              if (!kState && any_nan(d)) {
                *reinterpret_cast<uint4*>(x + o) =
                    make_uint4(finite_part(v.x), finite_part(v.y), finite_part(v.z), finite_part(v.w));
                s_odd[c % kFlags] = 1;
              }
            } else {  // what follows the sequence may hold anything
              *reinterpret_cast<uint4*>(x + o) = zero;
            }
            *reinterpret_cast<uint4*>(wx + o) = a;
            *reinterpret_cast<uint4*>(wx + 2 * kTile + o) = b;
            *reinterpret_cast<uint4*>(wx + 4 * kTile + o) = d;
          }
          if (n < Q && h == 0) {  // B's rows past the end, before either half is used
            if (!cx.wait(B_FULL + st, ph)) { alive = false; break; }
            unsigned char* bt = sm + st * L::kStage + L::kBt;
#pragma unroll 1
            for (int idx = xt; idx < L::kB / 16; idx += 256)
              if (((idx >> 3) & 63) >= n) *reinterpret_cast<uint4*>(bt + idx * 16) = zero;
          }
          fence_proxy_async_smem();
          cx.arrive_warp(B_X + 2 * st + h);
        }
        if (!alive) break;
        cx.arrive_warp(B_FEMPTY + c % kRing);
        if (++st == kStages) { st = 0; ph ^= 1; }
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- items and tile loads
    if (lane == 0) {
      const int64_t items = item_count<HPC, kState>(p);
      bool alive = true;
      auto publish = [&](const Item& v) {
        if (m >= kItems && !cx.wait_one(B_IEMPTY + m % kItems, ((m / kItems) - 1) & 1)) return false;
        s_items[m % kItems] = v;
        mbar_arrive(bars + B_IFULL + m % kItems);
        ++m;
        return true;
      };
#pragma unroll 1
      for (int64_t r = 0; alive && r * gridDim.x < items; ++r) {
        const int64_t i = item_at(r);
        if (i >= items) continue;
        it = get_item<HPC, kState>(p, i);
        if (!publish(it)) { alive = false; break; }
#pragma unroll 1
        for (int ci = 0; ci < it.chunks; ++ci, ++c) {
          const uint32_t st = c % kStages;
          if (c >= kStages && !cx.wait_one(B_EMPTY + st, ((c / kStages) - 1) & 1)) { alive = false; break; }
          unsigned char* s = sm + st * L::kStage;
          uint64_t* bar = bars + B_FULL + st;
          const int y = (int)(it.t0 + ci * Q);
          mbar_arrive_expect_tx(bars + B_FULLX + st, 2 * kTile);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_2d(s + L::kX + j * kTile, &tm_x, it.h0 * DX + j * 64, y, bars + B_FULLX + st);
          mbar_arrive_expect_tx(bar, kState ? L::kB : 2 * L::kB);
#pragma unroll
          for (int j = 0; j < DS / 64; ++j) {
            if (!kState) tma_load_2d(s + L::kC + j * kTile, &tm_c, it.g * DS + j * 64, y, bar);
            tma_load_2d(s + L::kBt + j * kTile, &tm_b, it.g * DS + j * 64, y, bar);
          }
        }
      }
      if (alive) {
        it.valid = 0;
        publish(it);
      }
      if (*s_abort)  // what was requested lands before the memory goes away
        for (uint32_t k = c > kStages ? c - kStages : 0; k < c; ++k) {
          const long long t0 = clock64();
          while ((!mbar_try_wait(bars + B_FULL + k % kStages, (k / kStages) & 1) ||
                  !mbar_try_wait(bars + B_FULLX + k % kStages, (k / kStages) & 1)) &&
                 clock64() - t0 < 20000000ll) {}
        }
    }
    __syncwarp();
  } else if (warp == kStateMmaWarp || (!kState && (warp == kYiMmaWarp || warp == kYxMmaWarp))) {
    // ---- products: G and U, Yi, or Yx (what arrives last is waited for last)
    constexpr uint32_t id_g = idesc_bf16(128, 64, 0, 0);
    constexpr uint32_t id_x = idesc_bf16(128, 64, 1, 0);
    constexpr uint32_t id_u = idesc_bf16(128, DS, 1, 1);
    const uint32_t lead = elect_lane();
    const uint32_t kmaj = op_lo(sbase, 0), mnmaj = op_lo(sbase, kTile);
    uint32_t st = 0, ph = 0;
    bool alive = true;
    while (alive) {
      if (!cx.wait(B_IFULL + m % kItems, (m / kItems) & 1)) break;
      const int chunks = __shfl_sync(0xffffffffu, s_items[m % kItems].chunks, 0);
      const int valid = __shfl_sync(0xffffffffu, s_items[m % kItems].valid, 0);
      cx.arrive_warp(B_IEMPTY + m % kItems);
      ++m;
      if (!valid) break;
#pragma unroll 1
      for (int ci = 0; ci < chunks; ++ci, ++c) {
        const uint32_t so = st * (L::kStage >> 4);
        const uint32_t now = c & 1, last = now ^ 1;  // parities of this chunk's and the last one's phases
        if (warp == kStateMmaWarp) {
          if (!cx.wait(B_FULL + st, ph, !kState && c > 0 ? B_M : -1, last)) { alive = false; break; }
          if (!kState) {
            tc_fence_after();
            uint32_t a = kmaj + so + (L::kC >> 4), b = kmaj + so + (L::kBt >> 4);
#pragma unroll
            for (uint32_t kk = 0; kk < DS / 16; kk += 2) {  // 32 K elements, 64 bytes
              mma_ss_by(lead, tb + TM_G, op_desc(a), op_desc(b), id_g, kk);
              mma_ss_by(lead, tb + TM_G, op_desc(a + 2), op_desc(b + 2), id_g, 1);
              const uint32_t d = kk & 2 ? (kTile >> 4) - 4 : 4;
              a += d;
              b += d;
            }
            commit_by(lead, cx.bars + 8 * B_G);
          }
          if (c > 0 && !cx.wait(B_UFREE, last)) { alive = false; break; }
          uint32_t a = mnmaj + (L::kWx >> 4), b = mnmaj + so + (L::kBt >> 4);
#pragma unroll 1
          for (uint32_t h = 0; h < 2; ++h, a += kTile >> 5, b += kTile >> 5) {
            if (!cx.wait(B_X + 2 * st + h, ph)) { alive = false; break; }
            tc_fence_after();
            uint32_t w = a;
#pragma unroll
            for (uint32_t part = 0; part < 3; ++part, w += 2 * kTile >> 4) {
              mma_ss_by(lead, tb + TM_U, op_desc(w), op_desc(b), id_u, h + part);
              mma_ss_by(lead, tb + TM_U, op_desc(w + 128), op_desc(b + 128), id_u, 1);
            }
            commit_by(lead, cx.bars + 8 * (B_WX + h));
          }
          if (!alive) break;
          commit_by(lead, cx.bars + 8 * B_U);
        } else if (warp == kYiMmaWarp) {
          // the Yi used last time has been read: two chunks ago, or the last with two heads' one Yi
          const uint32_t back = HPC == 1 ? 2 : 1;
          if (!cx.wait(B_S, now, B_FULL + st, ph, c >= back ? B_YFREE + (int)((c - back) & 1) : -1,
                       ((c - back) >> 1) & 1)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t yi = tb + TM_YI + (HPC == 1 ? now * 64 : 0);
          uint32_t s = tb + TM_SB, b = kmaj + so + (L::kC >> 4);
#pragma unroll
          for (uint32_t kk = 0; kk < DS / 8; kk += 2, s += 16) {  // hi, then lo
            mma_ts_by(lead, yi, s, op_desc(b), id_g, kk);
            mma_ts_by(lead, yi, s + 8, op_desc(b + 2), id_g, 1);
            b += kk & 2 ? (kTile >> 4) - 4 : 4;
            if (kk == DS / 16 - 2) b = kmaj + so + (L::kC >> 4);
          }
          commit_by(lead, cx.bars + 8 * (B_YI + now));
        } else {
          // x with zeros past the end and for what is not finite (B_X's second phase follows the first)
          if (!cx.wait(B_M, now, B_X + 2 * st + 1, ph, c > 0 ? B_YFREE + (int)last : -1, ((c - 1) >> 1) & 1)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = mnmaj + so + (L::kX >> 4);
          uint32_t b = kmaj + (L::kM >> 4);
#pragma unroll 1
          for (uint32_t h = 0; h < 2 * HPC; ++h, b += kTile >> 4) {
            const uint32_t d = tb + (h >= 2 ? TM_YX2 : TM_YX);
            mma_ss_by(lead, d, op_desc(a), op_desc(b), id_x, h & 1);
#pragma unroll
            for (int kk = 1; kk < Q / 16; ++kk)
              mma_ss_by(lead, d, op_desc(a + kk * 128), op_desc(b + 2 * kk), id_x, 1);
          }
          commit_by(lead, cx.bars + 8 * B_YX);
        }
        commit_by(lead, cx.bars + 8 * (B_EMPTY + st));
        if (++st == kStages) { st = 0; ph ^= 1; }
      }
    }
    // every product is done before the memory goes away
    commit_by(lead, cx.bars + 8 * B_DRAIN);
    wait_phase(cx.bars + 8 * B_DRAIN, 0);
    __syncwarp();
  } else if (warp == kFactorWarp) {
    // ---- per-token factors
    bool alive = true;
    while (alive && next_item_alone(m, it)) {
      float rate[HPC], bias[HPC];
#pragma unroll
      for (int k = 0; k < HPC; ++k) {
        const bool on = k < it.nh;
        rate[k] = on ? p.A[it.h0 + k] : 0.f;
        bias[k] = on && p.dtb ? p.dtb[it.h0 + k] : 0.f;
      }
#pragma unroll 1
      for (int ci = 0; ci < it.chunks; ++ci, ++c) {
        const int left = it.len - ci * Q;
        const __nv_bfloat16* src = p.dt + (it.t0 + ci * Q) * p.lddt + it.h0;
        float raw[HPC][2];
#pragma unroll
        for (int k = 0; k < HPC; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = h * 32 + lane;
            raw[k][h] = k < it.nh && t < left ? to_f32(src[t * p.lddt + k]) : 0.f;
          }
        if (c >= kRing && !cx.wait(B_FEMPTY + c % kRing, ((c / kRing) - 1) & 1)) { alive = false; break; }
#pragma unroll 1
        for (int k = 0; k < HPC; ++k) {
          const bool on = k < it.nh;
          float d[2], pre[2], err[2], suf[2];  // the running sum is pre + err
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float v = step_size_fast(k == 0 ? raw[0][h] : raw[HPC - 1][h], k == 0 ? bias[0] : bias[HPC - 1], p.softplus);
            d[h] = on && h * 32 + lane < left ? v : 0.f;
            float x = d[h] * (k == 0 ? rate[0] : rate[HPC - 1]) * 1.4426950408889634f;
            x = x < kFloor ? kFloor : x;  // (a NaN stays one)
            suf[h] = x;
            pre[h] = (x + kGrid) - kGrid;
            err[h] = x - pre[h];
          }
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float a = __shfl_up_sync(0xffffffffu, pre[h], o);
              const float ae = __shfl_up_sync(0xffffffffu, err[h], o);
              const float b = __shfl_down_sync(0xffffffffu, suf[h], o);
              if (lane >= o) {
                pre[h] += a;
                err[h] += ae;
              }
              if (lane + o < 32) suf[h] += b;
            }
          const float low = __shfl_sync(0xffffffffu, pre[0] + err[0], 31);   // the sum over tokens 0 .. 31
          const float high = __shfl_sync(0xffffffffu, suf[1], 0);   // over tokens 32 .. 63
          // the sum after a token, exclusive: each from its own end, where it is small
          float aft[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float n = __shfl_down_sync(0xffffffffu, suf[h], 1);
            aft[h] = lane < 31 ? n : 0.f;
          }
          Factors& f = factors[(c % kRing) * HPC + k];
          f.c[lane] = pre[0];
          f.c[32 + lane] = pre[1];
          f.r[lane] = ex2(err[0]);
          f.r[32 + lane] = ex2(err[1]);
          f.delta[lane] = ex2(-err[0]) * d[0];
          f.delta[32 + lane] = ex2(-err[1]) * d[1];
          f.w[lane] = ex2(aft[0] + high) * d[0];
          f.w[32 + lane] = ex2(aft[1]) * d[1];
          f.e[lane] = ex2(pre[0] + err[0]);
          f.e[32 + lane] = ex2(low + (pre[1] + err[1]));
          f.u[lane] = ex2(pre[1] + err[1]);
          f.v[lane] = ex2(aft[0]) * d[0];
          if (lane == 0) f.alpha = ex2(low + high);
        }
        cx.arrive_warp(B_FFULL + c % kRing);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) latch_status(p.status, KDA_ERR_DEVICE_TIMEOUT);
  if (warp == 0) tmem_dealloc(tb, TM_ALL);
}

// Items of a packed batch, one block: checks the offsets, counts each sequence's
// segments and lists them, the longest sequences first (up to 1024 sequences; with
// more, in their own order), and gives split sequences their state slots.
__global__ void __launch_bounds__(1024) scan_plan_kernel(Seqs q, int64_t seg, int32_t* plan,
                                                         int64_t most, unsigned int* status) {
  __shared__ int s_len[1024];
  __shared__ int s_out, s_st;
  check_seqlens(q, status);
  int2* out = reinterpret_cast<int2*>(plan + 4);
  int2* st = out + most;
  int32_t* slot = reinterpret_cast<int32_t*>(st + most);
  const int tid = threadIdx.x;
  auto length = [&](int n) {
    int64_t a, b;
    q.range(n, a, b);
    return (int)(b - a);
  };
  auto segments = [&](int len) { return seg > 0 && len > seg ? (int)((len + seg - 1) / seg) : 1; };
  if (q.N <= 1024) {
    const int mine = tid < q.N ? length(tid) : 0;
    s_len[tid] = mine;
    __syncthreads();
    if (tid < q.N) {
      int before = 0, split = 0;  // segments and slots of the sequences listed before this one
      for (int m = 0; m < q.N; ++m) {
        const int l = s_len[m];
        if (l > mine || (l == mine && m < tid)) {
          before += segments(l);
          split += segments(l) - 1;
        }
      }
      const int ns = segments(mine);
      slot[tid] = split;
      for (int s = 0; s < ns && before + s < most; ++s) out[before + s] = make_int2(tid, s);
      for (int s = 0; s < ns - 1 && split + s < most; ++s) st[split + s] = make_int2(tid, s);
    }
    if (tid == 0) {
      int no = 0, ns = 0;
      for (int m = 0; m < q.N; ++m) {
        no += segments(s_len[m]);
        ns += segments(s_len[m]) - 1;
      }
      plan[0] = no < most ? no : (int)most;
      plan[1] = ns < most ? ns : (int)most;
    }
    return;
  }
  // many sequences: blocks of 1024, each thread's place from a running count
  if (tid == 0) s_out = s_st = 0;
  __syncthreads();
  for (int base = 0; base < q.N; base += 1024) {
    const int n = base + tid;
    const int ns = n < q.N ? segments(length(n)) : 0;
    s_len[tid] = ns;
    __syncthreads();
    int before = s_out, split = s_st;
    for (int m = 0; m < tid; ++m) {
      before += s_len[m];
      split += s_len[m] > 0 ? s_len[m] - 1 : 0;
    }
    if (n < q.N) {
      slot[n] = split;
      for (int s = 0; s < ns && before + s < most; ++s) out[before + s] = make_int2(n, s);
      for (int s = 0; s < ns - 1 && split + s < most; ++s) st[split + s] = make_int2(n, s);
    }
    __syncthreads();
    if (tid == 1023) {
      s_out = before + ns;
      s_st = split + (ns > 0 ? ns - 1 : 0);
    }
    __syncthreads();
  }
  if (tid == 0) {
    plan[0] = s_out < most ? s_out : (int)most;
    plan[1] = s_st < most ? s_st : (int)most;
  }
}

bool make_map(CUtensorMap* m, const void* base, int64_t tokens, int64_t cols, int64_t ld) {
  auto enc = pf::get_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)tokens};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, Q};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DS, int HPC, bool kState>
cudaError_t launch(const CUtensorMap (&m)[3], const ScanParams& p, int64_t most, int64_t sms,
                   cudaStream_t stream) {
  constexpr int bytes = Layout<DS, HPC>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(scan_chunk_kernel<DS, HPC, kState>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = most < sms ? most : sms;
  scan_chunk_kernel<DS, HPC, kState><<<(unsigned)grid, kScanThreads, bytes, stream>>>(m[0], m[1], m[2], p);
  return cudaGetLastError();
}

template <int DS, int HPC>
cudaError_t run(const ScanArgs& a, const CUtensorMap (&m)[3], ScanParams p, int64_t out_items,
                int64_t state_items) {
  if (state_items > 0) {
    cudaError_t e = launch<DS, HPC, true>(m, p, state_items, a.sms, a.stream);
    if (e != cudaSuccess) return e;
    p.first = 0;
  }
  return launch<DS, HPC, false>(m, p, out_items, a.sms, a.stream);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// What a call needs past the workspace's header.
struct Sizes {
  int64_t seg = 0;        // tokens per segment, 0: sequences run whole
  int64_t slots = 0;      // states of segments
  int64_t most = 0;       // packed: bound on the list's entries
  size_t plan = 0, states = 0, decays = 0;
  size_t h0 = 0;          // a copy of the start states, for calls whose hT is their h0
  size_t total() const { return plan + states + decays + h0; }
};

// Segment length in tokens.  Fixed length: the number of segments that a model of the
// two launches favours, in chunk-steps on `sms` CTAs: the state launch runs all segments
// but the last at kStateCost of a full chunk's time, the output launch all of them, each
// item pays kStart chunk-steps to fill its pipeline, and a segment's start state sums up
// those before it (kJoin each; the times are flat around these constants).  Packed: a
// sequence may be as long as the SMs' mean share of the batch's work; longer ones are cut to
// that length.  Segments have at least kMinSeg chunks.  On the GPU, in segments and whole:
// 131071 tokens of 32 heads 1.39 and 3.75 ms, 16384 tokens of one head 39 and 484 us, 2048 of 8
// heads 30 and 65, 700 of two heads 23 and 27 (with 8 chunks at least 40 and 27 for the last two).
constexpr double kStateCost = 0.8, kStart = 4.0, kJoin = 0.4;
constexpr int64_t kMinSeg = 2, kMaxSegs = 64;
Sizes plan_sizes(const Seqs& q, bool packed, int64_t tiles, int H, int ds, int dx, int64_t sms) {
  Sizes s;
  if (q.total == 0 || q.N == 0) return s;
  auto waves = [&](int64_t n) { return (double)((n + sms - 1) / sms); };
  auto cost = [&](int64_t chains, int64_t chunks, int64_t ns) {
    const double len = (double)((chunks + ns - 1) / ns) + kStart;
    return ns == 1 ? waves(chains) * len
                   : (kStateCost * waves(chains * (ns - 1)) + waves(chains * ns)) * len + kJoin * (double)ns;
  };
  if (packed) {
    const int64_t chunks = (q.total + Q - 1) / Q;
    int64_t share = (chunks * tiles + sms - 1) / sms;
    // with few tiles the share is short: no more segments than the model would take of one
    // sequence as long as the batch
    int64_t best = 1;
    for (int64_t ns = 2; ns <= kMaxSegs && chunks / ns >= kMinSeg; ++ns)
      if (cost(tiles, chunks, ns) < cost(tiles, chunks, best)) best = ns;
    if (share < (chunks + best - 1) / best) share = (chunks + best - 1) / best;
    if (chunks > share) s.seg = share * Q;
    s.slots = s.seg > 0 ? q.total / s.seg : 0;
    s.most = s.slots + q.N;
    s.plan = round256(16 + 2 * (size_t)s.most * 8 + (size_t)q.N * 4);
  } else {
    const int64_t chunks = (q.T + Q - 1) / Q, chains = q.N * tiles;
    double best = 0.95 * cost(chains, chunks, 1);
    int64_t nseg = 1;
    for (int64_t ns = 2; ns <= kMaxSegs && chunks / ns >= kMinSeg; ++ns) {
      const double t = cost(chains, chunks, ns);
      if (t < best) {
        best = t;
        const int64_t len = (chunks + ns - 1) / ns;
        nseg = (chunks + len - 1) / len;
        s.seg = len * Q;
      }
    }
    s.slots = q.N * (nseg - 1);
  }
  s.states = round256((size_t)s.slots * H * ds * dx * 4);
  s.decays = round256((size_t)s.slots * H * 4);
  if (s.slots > 0) s.h0 = (size_t)q.N * H * ds * dx * 4;
  return s;
}
int64_t tiles_of(int H, int G, int dx) {
  const int hpc = 128 / dx, hpg = H / G;
  return (int64_t)G * ((hpg + hpc - 1) / hpc);
}

}  // namespace

size_t scan_bf16_workspace(bool packed, int64_t N, int64_t T, int64_t total, int H, int G, int ds,
                           int dx, int64_t sms) {
  const Seqs q{nullptr, T, total, (int)N};
  return plan_sizes(q, packed, tiles_of(H, G, dx), H, ds, dx, sms).total();
}

// TMA and the output rows need 16-byte alignment, and coordinates of 31 bits
bool scan_bf16_ok(const ScanArgs& a) {
  const void* ptrs[] = {a.x, a.Bm, a.Cm, a.y};
  for (const void* p : ptrs)
    if ((uintptr_t)p % 16) return false;
  return a.bf16 && a.q.T < (1 << 30) && a.ldx % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0 &&
         (int64_t)a.H * a.dx < 0x7fffffffll && (int64_t)a.G * a.ds < 0x7fffffffll &&
         a.q.total > 0 && a.q.total < 0x7fffffffll - Q;
}

cudaError_t launch_scan_bf16(const ScanArgs& a) {
  const int hpc = 128 / a.dx;
  CUtensorMap m[3];
  if (!make_map(&m[0], a.x, a.q.total, (int64_t)a.H * a.dx, a.ldx) ||
      !make_map(&m[1], a.Bm, a.q.total, (int64_t)a.G * a.ds, a.ldb) ||
      !make_map(&m[2], a.Cm, a.q.total, (int64_t)a.G * a.ds, a.ldc))
    return cudaErrorInvalidValue;
  ScanParams p{};
  p.q = a.q;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.dt = static_cast<const __nv_bfloat16*>(a.dt);
  p.A = a.A; p.D = a.D; p.dtb = a.dtb; p.h0 = a.h0;
  p.y = a.y; p.hT = a.hT;
  p.H = a.H; p.G = a.G;
  p.hpg = a.H / a.G;
  p.tpg = (p.hpg + hpc - 1) / hpc;
  p.ldx = a.ldx;
  p.lddt = a.lddt;
  p.softplus = a.softplus;
  p.out_bf16 = a.out_bf16;
  p.status = a.status;
  p.first = 1;
  const int64_t tiles = (int64_t)p.G * p.tpg;
  const bool packed = a.q.cu != nullptr;  // the workspace was checked for this form
  const Sizes z = plan_sizes(a.q, packed, tiles, a.H, a.ds, a.dx, a.sms);
  char* w = static_cast<char*>(a.ws);
  p.seg = z.seg;
  p.seg_s = reinterpret_cast<float*>(w + z.plan);
  p.seg_a = reinterpret_cast<float*>(w + z.plan + z.states);
  if (z.slots > 0 && a.h0 && a.h0 == a.hT) {  // a last segment may end before a first one starts
    float* copy = reinterpret_cast<float*>(w + z.plan + z.states + z.decays);
    cudaError_t e = cudaMemcpyAsync(copy, a.h0, z.h0, cudaMemcpyDeviceToDevice, a.stream);
    if (e != cudaSuccess) return e;
    p.h0 = copy;
  }
  p.nseg = z.seg > 0 ? (int)((a.q.T + z.seg - 1) / z.seg) : 1;
  int64_t out_items = (int64_t)a.q.N * p.nseg * tiles;
  int64_t state_items = (int64_t)a.q.N * (p.nseg - 1) * tiles;
  if (packed) {
    p.plan = reinterpret_cast<const int32_t*>(w);
    p.plan_most = z.most;
    scan_plan_kernel<<<1, 1024, 0, a.stream>>>(a.q, z.seg, reinterpret_cast<int32_t*>(w), z.most, a.status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.first = 0;
    out_items = z.most * tiles;
    state_items = z.slots * tiles;
  }
  if (a.ds == 128)
    return hpc == 1 ? run<128, 1>(a, m, p, out_items, state_items)
                    : run<128, 2>(a, m, p, out_items, state_items);
  return hpc == 1 ? run<64, 1>(a, m, p, out_items, state_items)
                  : run<64, 2>(a, m, p, out_items, state_items);
}

}  // namespace layer
}  // namespace kda
