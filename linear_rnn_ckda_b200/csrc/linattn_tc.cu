// linattn_tc.cu -- linear attention with a decay for each head on the tensor cores (bf16 inputs):
// forward and gradients, sm_100a (tcgen05 / TMEM / TMA).
//
// One recurrence serves all: with roles X (queries), Y (keys), Z (values),
//   out_i = rowf_i M x_i + sum_j P_ij z_j,   P_ij = e^{+-(G_i - G_j)} (x_i . y_j) over the causal side,
//   M    <- e^{G_C} M + sum_j tokf_j z_j y_j^T,        M the state with lane = z channel,
// run forwards (rowf = e^{G_i}, tokf = e^{G_C - G_i}, j <= i) or backwards in time (rowf =
// e^{G_C - G_i}, tokf = e^{G_i}, j >= i):
//   o  : X q,  Y k,  Z v   forwards       dq : X dO, Y v,  Z k   forwards (M = S)
//   dv : X k,  Y q,  Z dO  backwards      dk : X v,  Y dO, Z q   backwards (M = X_grad)
// and for the decays' gradients dq's and dk's passes also write q_i . dq_i and k_j . dk_j.
//
// Raw bf16 tiles go from TMA into the products as they are: a per-token decay multiplies a row
// or a column of a product, so it is applied in fp32 to scores, to outputs as they leave, and
// for the state to Z alone.  Per chunk of 64 tokens (all M = 128, fp32 accumulation in TMEM):
//   scores  X Y^T            [64 x 64]   A, B from shared memory
//   O       M X^T + Z^T P^T  [z x 64]    M in bf16 terms from TMEM, P in bf16 terms through shared memory
//   D       (tokf Z)^T Y     [z x x]     tokf Z in three bf16 terms
// While a chunk decays by no more than 2^-72, a row's factor is common to both parts of O: P is
// formed as colb_j (x_i . y_j) and O is scaled once as it leaves.  So that no value can leave fp32's
// range on the way, M is held times 2^-72 and so is colb, whose 1 / rowf_i <= 2^72 it makes up for:
// nothing is larger than what it stands for.  Small values pay: states and x . y are held to about
// 2^-126 2^72 = 2^-54 absolutely.  (With 2^-64 decays of 2^(-1/2) a token, a usual slope, already take
// the form by blocks: B8 T8192 H16 with one such head 444 us, with 72 411.)  A chunk that decays faster
// takes its weights block by block, and one that decays faster still pair by pair; then the second
// part has its own accumulator.
//
// M is held in fp32: in registers, or (dq and dk, whose operand M is wanted in three terms, which
// are an fp32 value's 24 bits) as those terms in tensor memory.  tokf Z is split into three terms, so
// M carries fp32 accuracy over any length.  M and P go into o and dv in two terms, 2^-18 of a value
// off: what is left is the rounding of the output (1.66e-3; in one term each 2.35e-3, and 172 us were
// 156, 395 us 336).  Where row dots are wanted (decay gradients, which cancel) M and P go into O in
// three terms (two leave dg 2.7e-5 off).
// The tensor cores truncate the accumulator at every addition (dq came out 4.4e-7 too small), so
// terms are added from the lowest up, and the many additions of lower terms truncate a small sum
// only: dg 1.8e-6 -> 1.0e-6 off, final states 2.3e-7 -> 1.1e-7 (B4 T4096 H16), for 4 % of the
// gradients' time.  (D's lower terms of both halves of a chunk first, as the gradients take them, cost
// the forward 10 %: there each half is added by itself.)
//
// One CTA per (segment, head), 28 warps: 0-3 and 24-27 state (112 registers a thread where they hold
// M), 4-11 outputs, 12, 13 and one of 16, 17 scores (a 32 x 32 block each), 14 TMA loads and decays, 15
// issue of O, 23 issue of scores and D (two issuers: one thread's products take 50 cycles or
// more each to issue), the rest tokf Z.  The roles run the chunks at their own pace through
// mbarriers.  Unrolled loops cost more than they save: the warps share what is left of L1, and waiting
// for code is the second largest stall.  (Four state warps, each with twice the code: 178, 434 and
// 550 us where eight take 169, 395 and 521.)
//
// Measured (B200): B4 T4096 H16 128 x 128 forward 172 us, B8 T8192 H16 395 to 420 us (1090 MB, 2.7 TB/s),
// gradients of the first 535 us.  Bound by the latency of a chunk's chain (TMA -> tokf Z -> D -> M -> O ->
// rows), not by bytes or tensor cycles: DRAM 26 %, tensor pipe 29 % of the time.
//
// A sequence may be cut into segments: a first launch computes every segment's own state, an
// elementwise walk over a sequence's segments gives each its incoming state (the decay is a
// scalar, so a segment's state map is one factor), and the main launch runs all segments side
// by side.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "internal.h"
#include "linattn_common.cuh"
#include "sm100.cuh"

namespace ckda {
namespace lin {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ bf16 products
__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// kind::f16 instruction descriptor: bf16 operands, f32 accumulation
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 16 lanes x 16 columns as 8 x 8 blocks: registers 4 k, 4 k + 1 hold lane t / 4, columns 8 k + 2 (t % 4)
// and the next; 4 k + 2, 4 k + 3 the same of lane t / 4 + 8
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16 lanes x 16 columns of words: registers 2 k, 2 k + 1 are lane t / 4 and t / 4 + 8, column 4 k + t % 4
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// four 8 x 8 blocks of 16-bit values, transposed: lane t's register i is column t / 4, rows 2 (t % 4)
// and the next, of block i; lane 8 i + r gives the address of block i's row r
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
// a * b + c on two fp32 values
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// two fp32 values rounded to bf16 (first in the low half), and back
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  float a, b;
  f2up(v, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t unpack_bf16(uint32_t u) {
  return f2pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint64_t f2bits(uint32_t a, uint32_t b) {
  return f2pk(__uint_as_float(a), __uint_as_float(b));
}

// ------------------------------------------------------------------ shapes
enum : int { kStates = 0, kOut = 1, kGrad = 2 };   // what a launch computes
enum : int { kWhole = 0, kBlocks = 1, kPairs = 2 };   // how a chunk's weights are formed
constexpr int kThreads = 896;
// M is held times 2^-kShift; a chunk's weights have one reference while it decays by 2^-kShift at most
constexpr int kShift = 72;
constexpr float kUp = 4722366482869645213696.f, kDown = 1.f / kUp;
// (a reset is held as 2^-201.9, and its row factor, times 2^kShift, has to be 0: below 2^-126)
static_assert(kShift <= 75, "resets");
constexpr uint32_t kPanel = 8192;                  // 64 tokens x 64 channels of bf16, 128-byte swizzle
constexpr uint32_t kTileB = 2 * kPanel;            // 64 tokens x 128 channels
// The causal side of P in 32 x 32 blocks of 64-byte rows (64-byte swizzle): the two blocks that share
// their columns (keys), one above the other, and the other diagonal block behind them
constexpr uint32_t kPBig = 4096, kPTerm = 6144;
constexpr uint32_t kTokB = 3 * kPanel;             // tokf Z of 32 tokens: three terms x two panels of 4 KB
// Registers a thread by role where the state role holds M: 256 x 112 + 640 x 56 = 64,512, the
// launch's 896 x 72.
constexpr int kRegsState = 112, kRegsOther = 56;

template <int KIND>
struct Cfg {
  static constexpr int kTiles = KIND == kStates ? 2 : KIND == kOut ? 3 : 4;   // Y Z | X Y Z | X Y Z W
  static constexpr int kStages = KIND == kGrad ? 2 : 3;
  static constexpr int kTerms = KIND == kGrad ? 3 : 2;                        // of M and P
  static constexpr int kTokBufs = KIND == kStates ? 4 : 2;                    // half chunks of tokf Z
  static constexpr uint32_t kStage = kTiles * kTileB;
  static constexpr uint32_t oX = 0;
  static constexpr uint32_t oY = KIND == kStates ? 0 : kTileB;
  static constexpr uint32_t oZ = oY + kTileB;
  [[maybe_unused]] static constexpr uint32_t oW = oZ + kTileB;                // kGrad
  static constexpr uint32_t offTok = kStages * kStage;
  static constexpr uint32_t offP = offTok + kTokBufs * kTokB;
  static constexpr uint32_t kP = KIND == kStates ? 0 : kTerms * kPTerm;
  static constexpr uint32_t offOut = offP + kP;
  static constexpr uint32_t offGate = offOut + (KIND == kStates ? 0 : 8 * 2048);
  static constexpr uint32_t kGate = 7 * 64 * 4 + 16;                          // one stage's decays
  static constexpr uint32_t offDot = offGate + kStages * kGate;               // kGrad: 2 x 4 x 64 floats
  static constexpr uint32_t offBar = offDot + (KIND == kGrad ? 512 * 4 : 0);
  static constexpr int kBars = 3 * kStages + 2 * kTokBufs + (KIND == kStates ? 22 : 26);
  static constexpr uint32_t kSmem = offBar + kBars * 8 + 64 + 1024;           // + slack to align
  // TMEM columns: scores, M, O twice, D (twice where there is room)
  static constexpr int kDBufs = KIND == kStates ? 2 : 1;
  static constexpr uint32_t cSc = 0, cM = 64, cO = cM + 64 * kTerms, cD = 512 - 128 * kDBufs;
};
static_assert(Cfg<kGrad>::cO + 128 <= Cfg<kGrad>::cD && Cfg<kOut>::cO + 128 <= Cfg<kOut>::cD, "tensor memory");
static_assert(Cfg<kOut>::kSmem <= 232448 && Cfg<kGrad>::kSmem <= 232448 && Cfg<kStates>::kSmem <= 232448,
              "shared memory");

struct Pass {
  int ix, iy, iz, iw;             // tensor maps (iw: kGrad's row dots)
  int hx, hy, hz, hw;             // their heads
  int dx, dz;                     // channels of X and Y, of Z
  int rev;
  const float *init;              // [N, H, dk, dv] or NULL (used without seg_in)
  const float *seg_in;            // [slots, H, dk, dv] incoming states, or NULL
  float *end;                     // [N, H, dk, dv]: the last segment's end state, or NULL
  float *end_slot;                // [slots, H, ..]: end state of every segment (kStates), or of the
                                  // last to the sequence's spare slot (kGrad; kOut for dv), or NULL
  float *decay;                   // kStates: [slots, H] the segment's whole decay
  void *out;                      // [rows, H, dz]
  int part;                       // out is fp32 per-head shares of a shared head's gradient
  float *dots;                    // kGrad: [H, rows] row dots
};
struct Params {
  CUtensorMap maps[4];            // q, k, v, dO
  CUtensorMap outs[3];            // the passes' outputs (bf16)
  Pass pass[3];
  const float *g;
  int H, g_fixed, elems, no_dO;
  long rows;
  Slots slots;
  int *status;
  int inject_chunk;               // test hook: chunk of a segment whose loads wait for nothing (-1: off)
  uint64_t inject_wait_ns;        // that wait's bound
};

// Waits are bounded by a count of tries, 110 ns each as measured, so 2 s in all, after which every role
// ends and the status word says so.  (Reading the clock in every wait instead is so much more code that
// calls take 5 to 8 % longer.)
constexpr uint32_t kTries = 20000000;
constexpr uint64_t kDrainNs = 2000000000ull;
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  uint32_t n = 0;
  while (!mbar_try_wait(bar, parity & 1u))
    if (*abort || ++n > kTries) return false;
  return true;
}
__device__ __forceinline__ void give_up(volatile int *abort, int *status) {
  *abort = 1;
  set_status(status, CKDA_ERR_TIMEOUT);
}

template <int KIND>
__device__ __forceinline__ void lin_tc(const Params &p) {
  using C = Cfg<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const Pass &ps = p.pass[blockIdx.z];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y;
  const bool rev = ps.rev != 0;
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  // a segment whose own state nothing reads: the last in the direction of the walk
  const bool last_seg = rev ? u.piece == 0 : u.piece == u.pieces - 1;
  if (KIND == kStates && last_seg) return;
  const int nc = pieces_of(u.len, kC);

  // Warps by role (the scores' off-diagonal block lies in the TMEM lanes of a quarter that goes
  // with the direction: 17 forwards, 16 backwards; the other of the two takes part in tokf Z)
  const int off_warp = rev ? 16 : 17;
  const int tok_warps = KIND == kStates ? 16 : 6;
  const int tok_index = KIND == kStates ? (warp < 14 ? warp - 4 : warp - 6) : warp >= 18 ? warp - 17 : 0;
  const bool is_score = KIND != kStates && (warp == 12 || warp == 13 || warp == off_warp);
  const bool is_tok = KIND == kStates ? (warp >= 4 && warp < 14) || (warp >= 16 && warp < 22) : warp >= 16 && warp < 23 && warp != off_warp;

  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::offBar);
  uint64_t *b_full = bars, *b_empty = bars + C::kStages, *b_gate = bars + 2 * C::kStages;
  uint64_t *b_w = bars + 3 * C::kStages, *b_wfree = b_w + C::kTokBufs;
  uint64_t *bx = b_wfree + C::kTokBufs;
  uint64_t *b_zeroed = bx, *b_sc = bx + 1, *b_p = bx + 2, *b_s = bx + 21 /* 4, kOut and kGrad */, *b_o = bx + 4 /* 2 */,
           *b_ofree = bx + 6 /* 2 */, *b_d = bx + 8 /* 2 */, *b_dfree = bx + 16 /* 2 */, *b_drain = bx + 10 /* 2 */,
           *b_red = bx + 12 /* 2 */, *b_o1 = bx + 14, *b_never = bx + (KIND == kStates ? 21 : 25);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bx + 18);
  volatile int *s_abort = reinterpret_cast<volatile int *>(bx + 19);
  volatile int *s_issued = reinterpret_cast<volatile int *>(bx + 20);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full + s, 1);
      // state 8, tokf Z, a commit; beside outputs 8, scores 3 and a second commit
      mbar_init(b_empty + s, 8 + tok_warps + 1 + (KIND == kStates ? 0 : 12));
      mbar_init(b_gate + s, 1);
    }
    for (int s = 0; s < C::kTokBufs; ++s) {
      mbar_init(b_w + s, tok_warps);
      mbar_init(b_wfree + s, 1);
    }
    mbar_init(b_zeroed, tok_warps);
    mbar_init(b_sc, 1);
    mbar_init(b_p, 3);
    for (int s = 0; s < (KIND == kStates ? 0 : 4); ++s) mbar_init(b_s + s, 4);
    mbar_init(b_o1, 1);
    mbar_init(b_never, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(b_o + s, 1);
      mbar_init(b_d + s, 1);
      mbar_init(b_dfree + s, 8);
      mbar_init(b_ofree + s, 8);
      mbar_init(b_red + s, 8);
      mbar_init(b_drain + s, 1);
    }
    *s_abort = 0;
    *s_issued = 0;
    mbar_fence_init();
  }
  if (warp == 15) tmem_alloc(s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;    // all 512 columns are this CTA's (one CTA an SM)

  // chunk c of the walk: its index in the segment, its valid rows
  auto chunk_at = [&](int c) { return rev ? nc - 1 - c : c; };
  auto rows_of = [&](int ci) { return min(kC, u.len - ci * kC); };
  // Matrix descriptors: a low word over one common high word (8-row groups 1024 bytes apart,
  // version, 128-byte swizzle); K-major tiles, or MN-major ones of two panels.
  const uint32_t sb = smem_u32(sm);
  constexpr uint64_t kHi = (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32;
  auto kmajor = [&](uint32_t at) { return kHi | (((sb + at) >> 4) | (1u << 16)); };
  constexpr uint64_t kHi64 = (uint64_t)((512u >> 4) | (1u << 14) | (4u << 29)) << 32;   // 64-byte swizzle: P
  auto mnmajor = [&](uint32_t at, uint32_t panel) { return kHi | (((sb + at) >> 4) | ((panel >> 4) << 16)); };
  auto gates = [&](int st) { return reinterpret_cast<float *>(sm + C::offGate + st * C::kGate); };
  // gates (floats): [0] rowf 2^72, [64] tokf 2^-72, [128] colb, [192] rowb, [256] cross, [320] G (64-bit
  // fixed point), [448] e^{G_C}, [449] mode, [450] G_C.  P_ij is (x_i . y_j) times
  //   kWhole : colb_j 2^-72, its row's factor left to rowf (the chunk decays by at most 2^-72)
  //   kBlocks: rowb_i colb_j on the diagonal 32 x 32 blocks, cross_i cross_j (through token 31) off
  //            them (each half decays by at most 2^-100)
  //   kPairs : each pair's own weight on the diagonal blocks, cross_i cross_j off them
  // a warp's wait (all lanes agree on the outcome) and a single thread's
  auto wait = [&](uint64_t *b, uint32_t ph) { return __all_sync(0xffffffffu, bar_wait(b, ph, s_abort)) != 0; };
  auto need = [&](uint64_t *b, uint32_t ph) { return bar_wait(b, ph, s_abort); };
  // Phases: chunk c's completion of a barrier used once a chunk has parity c & 1; of one used
  // every other chunk (c >> 1) & 1; of a stage's, `ph`, which the roles carry along with `st`.
  auto next = [&](int &st, uint32_t &ph) {
    if (++st == C::kStages) {
      st = 0;
      ph ^= 1u;
    }
  };
  int c = 0, st = 0;
  uint32_t ph = 0;
  bool ok = true;

  // State: the warps of group 0 (0-3) and 1 (24-27) take turns at blocks of 32 x channels
  const bool is_state = warp < 4 || warp >= 24;
  const int quad_warp = warp & 3, group = warp >= 24;
  if (KIND == kGrad && is_state) {
    // ---------------------------------------------------------------- state (warps 0-3, 24-27)
    // M is its operand: three bf16 terms hold an fp32 value's 24 bits, and O1 wants them anyway.
    // So M lives in tensor memory only, and a chunk's M <- e^{G_C} M + D is one short loop (held in
    // registers as in the other kinds, the unrolled splitting into three terms kept the warps waiting for
    // code).
    const uint32_t quarter = tmem + ((uint32_t)(32 * quad_warp) << 16), lanes = quarter + C::cM;
    auto split = [&](const uint64_t (&m)[8], uint32_t (&r)[3][8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[0][i] = pack_bf16(m[i]);
        uint64_t x = f2sub(m[i], unpack_bf16(r[0][i]));
        r[1][i] = pack_bf16(x);
        x = f2sub(x, unpack_bf16(r[1][i]));
        r[2][i] = pack_bf16(x);
      }
    };
    auto whole = [&](const uint32_t (&r)[3][8], int i) {
      return f2add(f2add(unpack_bf16(r[0][i]), unpack_bf16(r[1][i])), unpack_bf16(r[2][i]));
    };
    // Stored states are rows of x channels: a warp reads and writes 8 of them (32-byte pieces) at a
    // time, in the layout that puts a row into a lane (B4 T4096 H16 582 -> 515 us against a lane's own
    // row, 4 or 16 bytes at a time).
    const size_t state = ((size_t)blockIdx.x * p.H + h) * p.elems;
    const int z0 = 32 * quad_warp + (lane >> 2), x0 = 2 * (lane & 3);
    auto at = [&](int b, int y, int i) {             // where word i of 16 lanes and channels 32 b .. is stored
      return (size_t)(z0 + 16 * y + 8 * (i & 1)) * ps.dx + 32 * b + 8 * (i >> 1) + x0;
    };
    auto have = [&](int b, int y, int i) { return z0 + 16 * y + 8 * (i & 1) < ps.dz && 32 * b + 8 * (i >> 1) < ps.dx; };
    auto ready = [&](int b) {                        // 32 x channels of the operand (O1 need not wait for all)
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_s + b);
    };
#pragma unroll 1
    for (int b = group; 32 * b < ps.dx; b += 2) {
      uint64_t m[2][8];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int y = i >> 3, w = i & 7;
        m[y][w] = have(b, y, w) ? *reinterpret_cast<const uint64_t *>(ps.seg_in + state + at(b, y, w)) : 0;
      }
      __syncwarp();                                  // (all loads are in flight)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t r[3][8];
#pragma unroll
        for (int w = 0; w < 8; ++w) m[y][w] = f2mul(f2pk(kDown, kDown), m[y][w]);
        split(m[y], r);
#pragma unroll
        for (int t = 0; t < 3; ++t) tmem_st_rows(lanes + ((16u * y) << 16) + 64 * t + 16 * b, r[t]);
      }
      ready(b);
    }
    for (; c < nc; ++c, next(st, ph)) {
      if (!(ok = wait(b_gate + st, ph))) break;
      const float a = gates(st)[448];
      const uint64_t a2 = f2pk(a, a);
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty + st);
      // (D is there, and O1 of this chunk has read the operand)
      if (!(ok = wait(b_o1, c) && wait(b_d, c))) break;
      tc_fence_after();
#pragma unroll 1
      for (int b = 2 * group; 16 * b < ps.dx; b += b & 1 ? 3 : 1) {
        uint32_t d[16], r[3][8];
        uint64_t m[8];
        tmem_ld16(quarter + C::cD + 16 * b, d);
#pragma unroll
        for (int t = 0; t < 3; ++t) tmem_ld8(lanes + 64 * t + 8 * b, r[t]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = f2fma(a2, whole(r, i), f2bits(d[2 * i], d[2 * i + 1]));
        split(m, r);
#pragma unroll
        for (int t = 0; t < 3; ++t) tmem_st8(lanes + 64 * t + 8 * b, r[t]);
        if ((b & 1) || ps.dx == 16) ready(b >> 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_dfree);
    }
    if (ok && last_seg && ps.end_slot) {
      float *dst = ps.end_slot + state + (size_t)p.H * p.elems;      // the next slot
#pragma unroll 1
      for (int b = group; 32 * b < ps.dx; b += 2) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t r[3][8];
#pragma unroll
          for (int t = 0; t < 3; ++t) tmem_ld_rows(lanes + ((16u * y) << 16) + 64 * t + 16 * b, r[t]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (have(b, y, i)) *reinterpret_cast<uint64_t *>(dst + at(b, y, i)) = f2mul(f2pk(kUp, kUp), whole(r, i));
        }
      }
    }
  } else if (KIND != kGrad && is_state) {
    // ---------------------------------------------------------------- state (warps 0-3, 24-27)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
    const int z = 32 * quad_warp + lane;            // this thread's value channel (TMEM lane)
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad_warp) << 16);
    const bool live = z < ps.dz;
    uint64_t M[32];                                 // times 2^-72: x channels x_of(i) and the next
    auto block = [&](int j) { return 2 * j + group; };              // the j-th of this group's blocks
    auto x_of = [&](int i) { return 32 * block(i >> 4) + 2 * (i & 15); };
    {
      const float *src = nullptr;
      if (KIND != kStates) {
        if (ps.seg_in) src = ps.seg_in + ((size_t)blockIdx.x * p.H + h) * p.elems;
        else if (ps.init) src = ps.init + ((size_t)u.n * p.H + h) * p.elems;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const bool in = src && live && x_of(i) < ps.dx;
        M[i] = f2pk(in ? src[x_of(i) * ps.dz + z] : 0.f, in ? src[(x_of(i) + 1) * ps.dz + z] : 0.f);
      }
      __syncwarp();                                 // (all loads are in flight)
#pragma unroll
      for (int i = 0; i < 32; ++i) M[i] = f2mul(f2pk(kDown, kDown), M[i]);
    }
    // a block of M as the next chunk's operand
    auto put_state = [&](int j) {
      const uint32_t at = lanes + C::cM + 16 * block(j);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t r[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t m = M[16 * j + 8 * t + i];
          r[0][i] = pack_bf16(m);
          r[1][i] = pack_bf16(f2sub(m, unpack_bf16(r[0][i])));
        }
        tmem_st8(at + 8 * t, r[0]);
        tmem_st8(at + 64 + 8 * t, r[1]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_s + block(j));
    };
    if (KIND != kStates) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (32 * block(j) < ps.dx) put_state(j);
    }
    long long whole = 0;                            // kStates: the segment's decay
    for (; c < nc; ++c, next(st, ph)) {
      if (!(ok = wait(b_gate + st, ph))) break;
      const float a = gates(st)[448];
      if (KIND == kStates) whole = max(whole + *reinterpret_cast<const long long *>(gates(st) + 450), -(1ll << 52));
      const uint64_t a2 = f2pk(a, a);
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty + st);
      const int db = c & (C::kDBufs - 1);
      // (O1 of this chunk has read the operand)
      const bool put = KIND != kStates && c + 1 < nc;
      if (!(ok = wait(b_d + db, c / C::kDBufs) && (!put || wait(b_o1, c)))) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (32 * block(j) >= ps.dx) break;
        uint32_t r[32];
        tmem_ld32(lanes + C::cD + 128 * (c & (C::kDBufs - 1)) + 32 * block(j), r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) M[16 * j + i] = f2fma(a2, M[16 * j + i], f2bits(r[2 * i], r[2 * i + 1]));
        if (put) put_state(j);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_dfree + db);
    }
    // (a backward walk's segments but the last belong to the forward walk too, which writes theirs)
    if (KIND == kStates && ok && tid == 0 && (!rev || u.piece == u.pieces - 1))
      ps.decay[(size_t)blockIdx.x * p.H + h] = exp2_fixed(whole);
    if (ok && live) {
      auto store = [&](float *dst) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float a, b;
          f2up(f2mul(f2pk(kUp, kUp), M[i]), a, b);
          if (x_of(i) >= ps.dx) break;
          dst[x_of(i) * ps.dz + z] = a;
          dst[(x_of(i) + 1) * ps.dz + z] = b;
        }
      };
      if (KIND == kStates) store(ps.end_slot + ((size_t)blockIdx.x * p.H + h) * p.elems);
      else if (last_seg) {
        if (ps.end) store(ps.end + ((size_t)u.n * p.H + h) * p.elems);
        if (ps.end_slot) store(ps.end_slot + ((size_t)(blockIdx.x - u.piece + u.pieces) * p.H + h) * p.elems);
      }
    }
  } else {
    if (KIND != kGrad) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 14 || (KIND == kStates && warp == 22)) {
      // -------------------------------------------------------------- loads (14) and decays
      // (kStates, whose chunks are short: 14 and 22 take turns at the chunks' decays, which take a
      // warp some 2,000 cycles)
      const int px = (ps.dx + 63) / 64, pz = (ps.dz + 63) / 64;
      const uint32_t bytes = kPanel * ((KIND != kStates ? px : 0) + px + pz + (KIND == kGrad ? pz : 0));
      // lane 2 t + q loads panel q of tile t (Y Z, X Y Z, or X Y Z W)
      const int tile = (lane >> 1) + (KIND == kStates ? 1 : 0);
      const bool load = lane < 2 * C::kTiles && (lane & 1) < (tile < 2 ? px : pz);
      const int map = tile == 0 ? ps.ix : tile == 1 ? ps.iy : tile == 2 ? ps.iz : ps.iw;
      const int head = load ? head_of(h, p.H, tile == 0 ? ps.hx : tile == 1 ? ps.hy : tile == 2 ? ps.hz : ps.hw) : 0;
      for (; c < nc; ++c, next(st, ph)) {
        const int ci = chunk_at(c), len = rows_of(ci);
        const bool turn = KIND != kStates || (c & 1) == (warp == 14 ? 0 : 1);
        float g0 = 0.f, g1 = 0.f;
        if (turn) {                                  // (in flight while the stage is waited for)
          const size_t r = (size_t)(u.row0 + ci * kC) + 2 * lane;
          if (2 * lane < len) g0 = p.g[p.g_fixed ? (size_t)h : r * p.H + h];
          if (2 * lane + 1 < len) g1 = p.g[p.g_fixed ? (size_t)h : (r + 1) * p.H + h];
        }
        if (c >= C::kStages && (turn || warp == 14) && !(ok = wait(b_empty + st, ph ^ 1u))) break;
        if (warp == 14) {
          // test hook: a wait that runs out (ckda_debug_wait_injection)
          if (c == p.inject_chunk && !(ok = mbar_wait(b_never, 0, p.inject_wait_ns))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(b_full + st, bytes);
            *s_issued = c + 1;
          }
          __syncwarp();
          if (load) {
            // (no dO: its loads start past the tensor's end, where TMA reads 0)
            const int row = map == 3 && p.no_dO ? 1 << 30 : (int)(u.row0 + ci * kC);
            tma_load_3d(sm + st * C::kStage + lane * kPanel, &p.maps[map], b_full + st, 64 * (lane & 1), head, row);
          }
        }
        if (!turn) continue;
        // (fixed decays: a stage that held as many rows holds the same decays)
        if (!p.g_fixed || c < C::kStages || rows_of(chunk_at(c - C::kStages)) != len) {
          const long long x0 = 2 * lane < len ? fixed_log2(g0) : 0;
          const long long x1 = 2 * lane + 1 < len ? fixed_log2(g1) : 0;
          const long long sum = scan_pairs(x0, x1);
          const long long all = __shfl_sync(0xffffffffu, sum, 31);
          const long long mid = __shfl_sync(0xffffffffu, sum, 15);      // up to token 31
          const long long lim = 100ll << 32, shift = (long long)kShift << 32;
          const int mode = all >= -shift ? kWhole : mid >= -lim && all - mid >= -lim ? kBlocks : kPairs;
          // where a block's factors start from: forwards its first token's past, backwards its end
          const long long ref = mode == kWhole ? (rev ? all + shift : -shift) : (lane < 16) == rev ? mid : rev ? all : 0;
          float *gt = gates(st);
          float2 rf, tf, cb, rb, cr;
          auto one = [&](long long G, int i, float &r, float &t, float &c, float &b, float &x) {
            const long long row = rev ? all - G : G, tok = rev ? G : all - G;
            r = exp2_fixed(row + shift);
            t = i < len ? exp2_fixed(tok - shift) : 0.f;
            if (KIND == kStates) return;
            c = exp2_fixed(rev ? G - ref : ref - G);
            if (mode == kWhole) return;
            b = exp2_fixed(rev ? ref - G : G - ref);
            x = exp2_fixed(i < 32 ? mid - G : G - mid);
          };
          one(sum - x1, 2 * lane, rf.x, tf.x, cb.x, rb.x, cr.x);
          one(sum, 2 * lane + 1, rf.y, tf.y, cb.y, rb.y, cr.y);
          const bool bad = chunk_is_nan(g0, g1);
          if (bad) rf.x = rf.y = tf.x = tf.y = cb.x = cb.y = rb.x = rb.y = cr.x = cr.y = nanf("");
          reinterpret_cast<float2 *>(gt + 64)[lane] = tf;
          if (KIND != kStates) {
            reinterpret_cast<float2 *>(gt)[lane] = rf;
            reinterpret_cast<float2 *>(gt + 128)[lane] = cb;
            if (mode != kWhole) {
              reinterpret_cast<float2 *>(gt + 192)[lane] = rb;
              reinterpret_cast<float2 *>(gt + 256)[lane] = cr;
              reinterpret_cast<longlong2 *>(gt + 320)[lane] = make_longlong2(sum - x1, sum);
            }
          }
          if (lane == 0) {
            gt[448] = bad ? nanf("") : exp2_fixed(all);
            gt[449] = (float)mode;
            *reinterpret_cast<long long *>(gt + 450) = all;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_gate + st);
      }
    } else if (warp == 15) {
      // -------------------------------------------------------------- issue of O
      if (KIND != kStates && lane == 0) {
        const uint32_t id1 = idesc_bf16(128, 64, false, false), id2 = idesc_bf16(128, 64, true, false), id3 = idesc_bf16(128, 32, true, false);
        // M's columns times X^T, 16 channels at a time
        auto out1 = [&](uint32_t d, uint32_t m, uint64_t b, bool more) {
          mma_bf16_ts(d, m, b, id1, more);
          if (ps.dx >= 64) {
#pragma unroll
            for (int k = 1; k < 4; ++k) mma_bf16_ts(d, m + 8 * k, b + 2 * k, id1, true);
            if (ps.dx == 128) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_bf16_ts(d, m + 32 + 8 * k, b + (kPanel >> 4) + 2 * k, id1, true);
            }
          } else if (ps.dx == 32) {
            mma_bf16_ts(d, m + 8, b + 2, id1, true);
          }
        };
        bool both = false;             // the chunk before took both buffers
        for (; ok && c < nc; ++c, next(st, ph)) {
          // (the outputs that were in this buffer have been read; X is there, for the scores read it)
          const int ob = c & 1;
          if (!(ok = (c < 2 || need(b_ofree + ob, (c >> 1) - 1)))) break;
          if (!(ok = need(b_full + st, ph) && need(b_gate + st, ph) && (!both || need(b_ofree + (ob ^ 1), (c - 1) >> 1)))) break;
          tc_fence_after();
          const uint64_t x = kmajor(st * C::kStage + C::oX);
          const uint32_t d = tmem + C::cO + 64 * ob;
          // 32 channels of M at a time, as they are updated: of the gradients' the lower terms, and
          // all first terms at the end
#pragma unroll 1
          for (int b = 0; 32 * b < ps.dx; ++b) {
            if (!(ok = need(b_s + b, c))) break;
            tc_fence_after();
            const uint64_t xb = x + (b >> 1) * (kPanel >> 4) + 4 * (b & 1);
#pragma unroll
            for (int t = C::kTerms - 1; t >= C::kTerms - 2; --t) {
              mma_bf16_ts(d, tmem + C::cM + 64 * t + 16 * b, xb, id1, b > 0 || t < C::kTerms - 1);
              if (ps.dx > 16) mma_bf16_ts(d, tmem + C::cM + 64 * t + 16 * b + 8, xb + 2, id1, true);
            }
          }
          if (!ok) break;
          if (KIND == kGrad) out1(d, tmem + C::cM, x, true);
          mma_commit(b_o1);
          // the second part on top, or (weights not over the whole chunk) in the other buffer
          const bool apart = gates(st)[449] != (float)kWhole;
          if (!(ok = need(b_p, c) && (!apart || c == 0 || need(b_ofree + (ob ^ 1), (c - 1) >> 1)))) break;
          tc_fence_after();
          // (P's terms, the last first: its two blocks of common keys for all tokens, then the other)
          const uint64_t dz = mnmajor(st * C::kStage + C::oZ, kPanel) + (rev ? 256 : 0), dp = kHi64 | ((sb + C::offP) >> 4) | (1u << 16);
          const uint64_t dz2 = mnmajor(st * C::kStage + C::oZ, kPanel) + (rev ? 0 : 256);
          const uint32_t d2 = apart ? tmem + C::cO + 64 * (ob ^ 1) : d;
          both = apart;
#pragma unroll
          for (int t = C::kTerms - 1; t >= 0; --t) {
            const uint64_t dt = dp + t * (kPTerm >> 4);
            mma_bf16_ss(d2, dz, dt, id2, t < C::kTerms - 1 || !apart);
            mma_bf16_ss(d2, dz + 128, dt + 2, id2, true);
            mma_bf16_ss(d2 + (rev ? 0 : 32), dz2, dt + (kPBig >> 4), id3, true);
            mma_bf16_ss(d2 + (rev ? 0 : 32), dz2 + 128, dt + (kPBig >> 4) + 2, id3, true);
          }
          mma_commit(b_o + ob);
          mma_commit(b_empty + st);
        }
        // every product issued has completed before the tensor memory is released
        mma_commit(b_drain);
        mbar_wait(b_drain, 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp == 23) {
      // -------------------------------------------------------------- issue of scores and D
      if (lane == 0) {
        const uint32_t id_s = idesc_bf16(128, 64, false, false), id_d = idesc_bf16(128, ps.dx, true, true);
        for (; ok && c < nc; ++c, next(st, ph)) {
          if (KIND != kStates) {
            // (tiles landed, rows past a ragged end 0, the scores before read)
            if (!(ok = need(b_full + st, ph) && (rows_of(chunk_at(c)) == kC || need(b_zeroed, 0)) &&
                       (c == 0 || need(b_p, c - 1))))
              break;
            tc_fence_after();
            const uint64_t a = kmajor(st * C::kStage + C::oX), b = kmajor(st * C::kStage + C::oY);
            mma_bf16_ss(tmem + C::cSc, a, b, id_s, false);
            if (ps.dx >= 64) {
#pragma unroll
              for (int k = 1; k < 4; ++k) mma_bf16_ss(tmem + C::cSc, a + 2 * k, b + 2 * k, id_s, true);
              if (ps.dx == 128) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16_ss(tmem + C::cSc, a + (kPanel >> 4) + 2 * k, b + (kPanel >> 4) + 2 * k, id_s, true);
              }
            } else if (ps.dx == 32) {
              mma_bf16_ss(tmem + C::cSc, a + 2, b + 2, id_s, true);
            }
            mma_commit(b_sc);
          }
          // tokf Z's terms from the lowest up: in the gradients the lower ones of both halves of the
          // chunk first, else of each half, whose room is free the sooner
          const int db = c & (C::kDBufs - 1);
          const uint32_t d = tmem + C::cD + 128 * db;
          constexpr bool kBoth = KIND == kGrad;
#pragma unroll 1
          for (int step = 0; step < (kBoth ? 4 : 2); ++step) {
            const int half = step & 1, hh = 2 * c + half, slot = hh % C::kTokBufs;
            const uint64_t dy = mnmajor(st * C::kStage + C::oY, kPanel) + 256 * half;
            const uint64_t dw = mnmajor(C::offTok + slot * kTokB, kPanel / 2);
            if (step < 2) {
              if (!(ok = need(b_w + slot, hh / C::kTokBufs) && (half || c < C::kDBufs || need(b_dfree + db, c / C::kDBufs - 1)))) break;
              tc_fence_after();
#pragma unroll
              for (int m = 5; m >= 2; --m)           // (m >> 1)-th term, 16 tokens
                mma_bf16_ss(d, dw + (m >> 1) * (kPanel >> 4) + 128 * (m & 1), dy + 128 * (m & 1), id_d, step > 0 || m < 5);
            }
            if (step >= 2 || !kBoth) {
              mma_bf16_ss(d, dw, dy, id_d, true);
              mma_bf16_ss(d, dw + 128, dy + 128, id_d, true);
              mma_commit(b_wfree + slot);
            }
          }
          if (!ok) break;
          mma_commit(b_d + db);
          mma_commit(b_empty + st);
        }
        mma_commit(b_drain + 1);
        mbar_wait(b_drain + 1, 0, kDrainNs);
      }
      __syncwarp();
    } else if (is_tok) {
      // -------------------------------------------------------------- tokf Z in three bf16 terms
      const int kT = 32 * tok_warps;
      const int t = 32 * tok_index + lane, n = 256 * ((ps.dz + 63) / 64);   // 16-byte pieces of half a tile
      for (; c < nc; ++c, next(st, ph)) {
        const int len = rows_of(chunk_at(c));
        uint8_t *base = sm + st * C::kStage;
        if (!(ok = wait(b_full + st, ph))) break;
        if (len < kC) {
          // a ragged end: the rows that follow belong to another sequence
          for (int i = t; i < (int)(C::kStage / 16); i += kT)
            if ((i >> 3 & 63) >= len) reinterpret_cast<uint4 *>(base)[i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_zeroed);
          if (!(ok = wait(b_zeroed, 0))) break;
        }
        if (!(ok = wait(b_gate + st, ph))) break;
        const float *tokf = gates(st) + 64;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int hh = 2 * c + half, slot = hh % C::kTokBufs;
          if (hh >= C::kTokBufs && !(ok = wait(b_wfree + slot, hh / C::kTokBufs - 1))) break;
          const uint4 *src = reinterpret_cast<const uint4 *>(base + C::oZ) + 256 * half;
          uint4 *dst = reinterpret_cast<uint4 *>(sm + C::offTok + slot * kTokB);
#pragma unroll 1
          for (int v = t; v < n; v += kT) {
            const float f = tokf[32 * half + (v >> 3 & 31)];
            const uint64_t w = f2pk(f, f);
            const uint4 z = src[v + (v & 256)];                              // panel v / 256, this half's rows
            const uint32_t zi[4] = {z.x, z.y, z.z, z.w};
            uint32_t r[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint64_t x = f2mul(unpack_bf16(zi[e]), w);
              r[0][e] = pack_bf16(x);
              x = f2sub(x, unpack_bf16(r[0][e]));
              r[1][e] = pack_bf16(x);
              x = f2sub(x, unpack_bf16(r[1][e]));
              r[2][e] = pack_bf16(x);
            }
#pragma unroll
            for (int t3 = 0; t3 < 3; ++t3)
              dst[t3 * (kPanel / 16) + v] = make_uint4(r[t3][0], r[t3][1], r[t3][2], r[t3][3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_w + slot);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(b_empty + st);
      }
    } else if (is_score) {
      // -------------------------------------------------------------- scores, a 32 x 32 block each
      const int rb = warp & 3, row = 32 * rb + lane;               // rows (TMEM lanes) of the block
      const int cb = warp < 16 ? rb : 1 - rb;                      // its columns: the diagonal, or the causal other
      const uint32_t lanes = tmem + ((uint32_t)(32 * rb) << 16);
      uint8_t *P = sm + C::offP + (cb == (rev ? 1 : 0) ? row * 64 : kPBig + lane * 64);
      const uint32_t mask = cb != rb ? ~0u : rev ? ~0u << lane : ~0u >> (31 - lane);   // the causal columns
      for (; c < nc; ++c, next(st, ph)) {
        if (!(ok = wait(b_gate + st, ph))) break;
        const float *gt = gates(st);
        const int mode = (int)gt[449];
        if (!(ok = wait(b_sc, c))) break;
        if (c > 0 && !(ok = wait(b_o + ((c - 1) & 1), (c - 1) >> 1))) break;   // (the scores before have been read)
        tc_fence_after();
        if (mode == kPairs && cb == rb) {                          // every weight from its own difference of sums
          const long long *G = reinterpret_cast<const long long *>(gt + 320);
          const long long me = G[row];
#pragma unroll 1
          for (int j = 0; j < 32; ++j) {
            uint32_t s1;
            tmem_ld1(lanes + C::cSc + 32 * cb + j, s1);
            tmem_wait_ld();
            const long long o = G[32 * cb + j];
            float x = mask >> j & 1 ? __uint_as_float(s1) * exp2_fixed(rev ? o - me : me - o) : 0.f;
#pragma unroll
            for (int t = 0; t < C::kTerms; ++t) {
              const __nv_bfloat16 v = __float2bfloat16_rn(x);
              *reinterpret_cast<__nv_bfloat16 *>(P + t * kPTerm + ((j / 8 ^ (lane >> 1 & 3)) << 4) + 2 * (j & 7)) = v;
              x -= __bfloat162float(v);
            }
          }
        } else {
          const float *col = gt + (mode == kWhole || cb == rb ? 128 : 256);
          const float scale = mode == kWhole ? 1.f : cb == rb ? gt[192 + row] : gt[256 + row];
          const uint64_t mine = f2pk(scale, scale);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int j0 = 32 * cb + 8 * q;
            const uint32_t m = mask >> (8 * q);
            uint32_t s[8];
            tmem_ld8(lanes + C::cSc + j0, s);
            const float4 f0 = *reinterpret_cast<const float4 *>(col + j0);
            const float4 f1 = *reinterpret_cast<const float4 *>(col + j0 + 4);
            const uint64_t f[4] = {f2pk(f0.x, f0.y), f2pk(f0.z, f0.w), f2pk(f1.x, f1.y), f2pk(f1.z, f1.w)};
            tmem_wait_ld();
            uint32_t r[C::kTerms][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // (the mask selects, so that whatever stands on the acausal side vanishes)
              float a, b;
              f2up(f2mul(f2bits(s[2 * j], s[2 * j + 1]), f2mul(f[j], mine)), a, b);
              uint64_t x = f2pk(m & (1u << (2 * j)) ? a : 0.f, m & (2u << (2 * j)) ? b : 0.f);
#pragma unroll
              for (int t = 0; t < C::kTerms; ++t) {
                r[t][j] = pack_bf16(x);
                x = f2sub(x, unpack_bf16(r[t][j]));
              }
            }
            uint8_t *at = P + ((q ^ (lane >> 1 & 3)) << 4);
#pragma unroll
            for (int t = 0; t < C::kTerms; ++t)
              *reinterpret_cast<uint4 *>(at + t * kPTerm) = make_uint4(r[t][0], r[t][1], r[t][2], r[t][3]);
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p);
          mbar_arrive(b_empty + st);
        }
      }
    } else if (KIND != kStates && warp < 12) {
      // -------------------------------------------------------------- outputs (warps 4-11)
      // A warp holds 32 channels of 32 tokens.  It reads O in 8 x 8 blocks, which are bf16 matrix
      // fragments once two tokens are packed into a register, so four transposing stores put 32
      // channels of 8 tokens into rows.  Whole chunks leave as one TMA store a warp (read out of
      // shared memory only when the loads issued before it have been, some 2,800 cycles later:
      // still within a chunk's time).
      const int quad = warp & 3, g = (warp >> 2) - 1;
      const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + 32 * g;
      float *red = reinterpret_cast<float *>(sm + C::offDot) + 32 * g;   // [2][4 quads][64]
      const uint32_t mine = C::offOut + (warp - 4) * 2048;   // 32 tokens x 32 channels
      const int ch = 32 * quad + (lane >> 2), tk = 2 * (lane & 3);  // this lane's first channel and token in a block
      const bool any = 32 * quad < ps.dz && ps.out;
      for (; c < nc; ++c, next(st, ph)) {
        const int ci = chunk_at(c), len = rows_of(ci) - 32 * g, ob = c & 1;
        const float *gt = gates(st);
        const bool tma = len >= 32 && any && !(ps.part);
        const long row0 = u.row0 + ci * kC + 32 * g;
        if (!(ok = wait(b_gate + st, ph))) break;
        const bool apart = gt[449] != (float)kWhole;
        float *rd = red + ob * 256 + quad * 64;
        if (!(ok = wait(b_o + ob, c >> 1))) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {                      // 16 tokens, two blocks
          const int t0 = 16 * half + tk;
          uint64_t f[2], d[2];                                      // rowf of this lane's two tokens a block; dots
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 x = *reinterpret_cast<const float2 *>(gt + 32 * g + t0 + 8 * k);
            f[k] = f2pk(x.x, x.y);
            d[k] = 0;
          }
          uint32_t pk[2][4];                                        // [y][2 k + m]: block k, channel ch + 16 y + 8 m
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t r[8];
            tmem_ld_blocks(lanes + ((16u * y) << 16) + C::cO + 64 * ob + 16 * half, r);
            tmem_wait_ld();
            uint64_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2mul(f[i >> 1], f2bits(r[2 * i], r[2 * i + 1]));
            if (apart) {
              tmem_ld_blocks(lanes + ((16u * y) << 16) + C::cO + 64 * (ob ^ 1) + 16 * half, r);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = f2add(v[i], f2bits(r[2 * i], r[2 * i + 1]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) pk[y][i] = pack_bf16(v[i]);
            if (!tma && any) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int t = t0 + 8 * (i >> 1), z = ch + 16 * y + 8 * (i & 1);
                float a, b;
                f2up(v[i], a, b);
                const size_t step = (size_t)p.H * ps.dz, at = ((size_t)(row0 + t) * p.H + h) * ps.dz + z;
                if (z >= ps.dz) continue;
                if (ps.part) {
                  if (t < len) static_cast<float *>(ps.out)[at] = a;
                  if (t + 1 < len) static_cast<float *>(ps.out)[at + step] = b;
                } else {
                  if (t < len) static_cast<__nv_bfloat16 *>(ps.out)[at] = __float2bfloat16_rn(a);
                  if (t + 1 < len) static_cast<__nv_bfloat16 *>(ps.out)[at + step] = __float2bfloat16_rn(b);
                }
              }
            }
            if constexpr (KIND == kGrad) {
              // products with W, the two blocks of two channel groups
              const uint32_t wt = sb + st * C::kStage + C::oW + (quad >> 1) * kPanel;
              const int row = 32 * g + 16 * half + 8 * (lane >> 4) + (lane & 7);
              uint32_t w[4];
              ldmatrix4_t(wt + row * 128 + (((4 * (quad & 1) + 2 * y + (lane >> 3 & 1)) ^ (row & 7)) << 4), w);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (32 * quad + 16 * y < ps.dz) d[e >> 1] = f2fma(v[e], unpack_bf16(w[e]), d[e >> 1]);
            }
          }
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_ofree + ob);
          }
          if (tma) {
            if (half == 0) {
              if (lane == 0) bulk_wait_read();                     // (the last store has been read)
              __syncwarp();
            }
            // rows of 64 bytes, 16-byte pieces permuted by row / 2 % 4 (64-byte swizzle)
            const int row = 16 * half + (lane & 7);
            const uint32_t at = sb + mine + row * 64 + (((lane >> 3) ^ (row >> 1 & 3)) << 4);
#pragma unroll
            for (int k = 0; k < 2; ++k) stmatrix4_t(at + 512 * k, pk[0][2 * k], pk[0][2 * k + 1], pk[1][2 * k], pk[1][2 * k + 1]);
          }
          if constexpr (KIND == kGrad) {
            // four tokens' sums over this lane's channels, then over the lanes that hold the same
            // tokens (bits 2-4): two of them end up with one token
            float s4[4];
            f2up(d[0], s4[0], s4[1]);
            f2up(d[1], s4[2], s4[3]);
#pragma unroll
            for (int step = 2; step >= 1; step >>= 1) {
              const bool up = lane & (8 * step);
#pragma unroll
              for (int i = 0; i < step; ++i) {
                const float send = up ? s4[i] : s4[i + step], keep = up ? s4[i + step] : s4[i];
                s4[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8 * step);
              }
            }
            s4[0] += __shfl_xor_sync(0xffffffffu, s4[0], 4);
            if (!(lane & 4)) rd[t0 + 8 * (lane >> 4) + (lane >> 3 & 1)] = s4[0];
          }
        }
        if (tma) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&p.outs[blockIdx.z], sm + mine, 32 * quad, h, (int)row0);
            bulk_commit();
          }
        }
        if constexpr (KIND == kGrad) {
          __syncwarp();
          // (two barriers: a warp may be a chunk ahead of another that waits for its store)
          if (lane == 0) mbar_arrive(b_red + ob);
          if (quad == 0) {
            if (!(ok = wait(b_red + ob, c >> 1))) break;
            if (lane < len)
              ps.dots[(size_t)h * p.rows + row0 + lane] = (rd[lane] + rd[64 + lane]) + (rd[128 + lane] + rd[192 + lane]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_empty + st);
      }
      if (lane == 0) bulk_wait_all();
    }
  }
  if (!ok) give_up(s_abort, p.status);
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    // loads that a role which gave up did not wait for have landed
    for (int i = max(0, *s_issued - C::kStages); i < *s_issued; ++i)
      mbar_wait(b_full + i % C::kStages, (i / C::kStages) & 1, kDrainNs);
  }
  __syncthreads();
  if (warp == 15) {
    tc_fence_after();
    tmem_dealloc(*s_tmem, 512);
  }
}
template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ Params p) {
  // (kGrad is dq and dk; dv, which has no row dots, is what kOut computes: 3.9 -> 2.4 us a chunk)
  if (KIND == kGrad && blockIdx.z == 2) lin_tc<kOut>(p);
  else lin_tc<KIND>(p);
}

// ------------------------------------------------------------------ walk over the segments
// Replaces every segment's own state by the state it starts from (walked in its direction).
// blockIdx: (sequence, head, direction x block of 4 x 128 entries).
struct JoinParams {
  float *seg[2];
  const float *init[2];
  const float *decay;
  float *end[2];          // a sequence without tokens: its end state
  int H, elems, blocks;
  Slots slots;
};
__global__ void __launch_bounds__(128) lin_join_kernel(const JoinParams p) {
  if (p.slots.cu && *p.slots.status) return;
  const int n = blockIdx.x, h = blockIdx.y, back = blockIdx.z / p.blocks;
  const int e = ((blockIdx.z % p.blocks) * 128 + threadIdx.x) * 4;
  if (e >= p.elems) return;
  const int len = p.slots.cu ? p.slots.cu[n + 1] - p.slots.cu[n] : p.slots.T;
  const int m = pieces_of(len, p.slots.L);
  const long base = p.slots.base(n);
  const size_t own = ((size_t)n * p.H + h) * p.elems + e;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.init[back]) S = *reinterpret_cast<const float4 *>(p.init[back] + own);
  constexpr int kAhead = 4;
  for (int c0 = 0; c0 < m; c0 += kAhead) {
    float4 d[kAhead];
    float a[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (c0 + x >= m - 1) continue;
      const size_t at = (size_t)(base + (back ? m - 1 - c0 - x : c0 + x)) * p.H + h;
      d[x] = *reinterpret_cast<const float4 *>(p.seg[back] + at * p.elems + e);
      a[x] = p.decay[at];
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (c0 + x >= m) continue;
      const size_t at = (size_t)(base + (back ? m - 1 - c0 - x : c0 + x)) * p.H + h;
      *reinterpret_cast<float4 *>(p.seg[back] + at * p.elems + e) = S;
      if (c0 + x == m - 1) continue;
      S.x = fmaf(a[x], S.x, d[x].x); S.y = fmaf(a[x], S.y, d[x].y);
      S.z = fmaf(a[x], S.z, d[x].z); S.w = fmaf(a[x], S.w, d[x].w);
    }
  }
  if (m == 0 && p.end[back]) *reinterpret_cast<float4 *>(p.end[back] + own) = S;
}

// ------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}
// [rows, heads, d] bf16 as (channel, head, token): loads take boxes of 64 x 1 x 64, 128-byte
// swizzle (channels past d and tokens past rows read as 0), stores of 32 x 1 x 32, 64-byte swizzle
bool make_map(CUtensorMap *map, const void *base, int heads, long rows, int d, bool store = false) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
  const cuuint32_t side = store ? 32 : 64;
  cuuint32_t box[3] = {side, 1, side}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             store ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             store ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSMs = 148;

// Tokens per segment.  Unpacked: the cut into m segments that a model in chunk times finds
// shortest.  Forwards: main launch = waves x (segment + 3 chunks' worth of start), first launch
// half a chunk time per chunk, 8 for the extra launches (B1 T4096 H32: 16 chunks 94 us, 64 150;
// B4 T4096 H16: 32 or 64 chunks 155, 22 185).  Backwards, where two units on the SMs of a pair run
// at two thirds of one's speed: all units' chunks over all SMs, 1.2 times a unit's own for the last
// ones, 0.6 a chunk for the first launch (B1 T4096 H32: 16 chunks 311 us, 64 463; B2 T2048 H16:
// 8 chunks 190, 32 253).  Packed: lengths are on the device, so a segment is half an SM's share of
// all chunks (backwards a quarter), between 8 and 64 chunks, a multiple of 4 so that even lengths
// are cut evenly (14 sequences, 42,992 tokens, H16 forward: 32 chunks 416 us, 16 433, 34 436, 64
// 445; 11 sequences, 7,923 tokens, H16 backward: 12 chunks 390 us, 24 422).  (Taken when o and dv had one
// term of M and P each; all are some 10 % more since.)
int segment_tokens(bool packed, int B, int T, int H, bool back) {
  const long nch = ((long)T + kC - 1) / kC;
  const long units1 = (long)B * H * (back ? 3 : 1), local1 = (long)B * H * (back ? 2 : 1);
  if (nch <= 1) return kC;
  if (packed) return (int)(std::min(std::max(nch * units1 / kSMs / (back ? 4 : 2), 8L), 64L) & ~3L) * kC;
  long best = -1, best_c = nch;
  for (long m = 1; m <= nch && m <= 64; ++m) {
    const long c = (nch + m - 1) / m, mm = (nch + c - 1) / c;
    long cost;
    if (back) {
      cost = units1 * mm * (c + 3) * 10 / kSMs + 12 * (c + 3);
      if (mm > 1) cost += local1 * (mm - 1) * (c + 3) * 6 / kSMs + 30;
    } else {
      cost = 2 * ((units1 * mm + kSMs - 1) / kSMs) * (c + 3);
      if (mm > 1) cost += ((local1 * (mm - 1) + kSMs - 1) / kSMs) * (c + 3) + 16;
    }
    if (best < 0 || cost < best) { best = cost; best_c = c; }
  }
  return (int)best_c * kC;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace past the header.
struct TcLayout {
  int L;
  bool seg;                 // some sequence may have several segments
  long slots;
  size_t table, decay, S, X, rho, kappa, pq, pk, pv, dg, total;
};
TcLayout tc_layout(bool packed, int N, int B, int T, int H, int Hq, int Hk, int Hv, int dk, int dv,
                   bool g_fixed, bool back) {
  TcLayout l = {};
  l.L = segment_tokens(packed, B, T, H, back);
  l.seg = packed || T > l.L;
  l.slots = slot_count(packed, N, T, l.L, back ? 1 : 0);
  const size_t rows = (size_t)B * T, state = (size_t)l.slots * H * dk * dv * 4;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += round256(bytes); return r; };
  l.table = take(packed ? (size_t)l.slots * 4 : 0);
  l.decay = take(l.seg ? (size_t)l.slots * H * 4 : 0);
  l.S = take(l.seg || back ? state : 0);
  l.X = take(back ? state : 0);
  l.rho = take(back ? rows * H * 4 : 0);
  l.kappa = take(back ? rows * H * 4 : 0);
  l.pq = take(back && Hq < H ? rows * H * dk * 4 : 0);
  l.pk = take(back && Hk < H ? rows * H * dk * 4 : 0);
  l.pv = take(back && Hv < H ? rows * H * dv * 4 : 0);
  l.dg = take(back && g_fixed ? rows * H * 4 : 0);
  l.total = at;
  return l;
}

template <int KIND>
bool launch(const Params &p, dim3 grid, cudaStream_t s) {
  auto kern = lin_tc_kernel<KIND>;
  const uint32_t smem = KIND == kGrad ? std::max(Cfg<kGrad>::kSmem, Cfg<kOut>::kSmem) : Cfg<KIND>::kSmem;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  kern<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace

size_t tc_workspace(bool packed, int N, int B, int T, int H, int Hq, int Hk, int Hv, int dk, int dv,
                    bool g_fixed, bool back) {
  return tc_layout(packed, N, B, T, H, Hq, Hk, Hv, dk, dv, g_fixed, back).total;
}

int launch_tc(const LinArgs &a, const LinBwdArgs *b, cudaStream_t s) {
  const TcLayout l = tc_layout(a.cu != nullptr, a.N, a.B, a.T, a.H, a.Hq, a.Hk, a.Hv, a.dk, a.dv,
                               a.g_fixed, b != nullptr);
  const long rows = (long)a.B * a.T;
  Params p = {};
  if (rows > 0) {
    if (!make_map(&p.maps[0], a.q, a.Hq, rows, a.dk) || !make_map(&p.maps[1], a.k, a.Hk, rows, a.dk) ||
        !make_map(&p.maps[2], a.v, a.Hv, rows, a.dv) ||
        (b && !(b->dO ? make_map(&p.maps[3], b->dO, a.H, rows, a.dv) : make_map(&p.maps[3], a.q, 1, 1, 16))))
      return CKDA_ERR_CUDA;
    p.no_dO = b && !b->dO;
  }
  p.g = a.g; p.H = a.H; p.g_fixed = a.g_fixed; p.elems = a.dk * a.dv; p.rows = rows;
  p.status = a.status;
  p.inject_chunk = wait_injection(&p.inject_wait_ns);
  if (p.inject_wait_ns == 0) p.inject_wait_ns = kDrainNs;
  p.slots = Slots{a.cu, reinterpret_cast<const int *>(a.ws + l.table), a.status, a.N, a.T, l.L, b ? 1 : 0};
  if (a.cu) {
    const PlanTable t{reinterpret_cast<int *>(a.ws + l.table), l.L, b ? 1 : 0, l.slots};
    const int rc = launch_plan(a.cu, a.N, a.T, t, a.status, s);
    if (rc != CKDA_OK) return rc;
  }
  float *segS = reinterpret_cast<float *>(a.ws + l.S), *segX = reinterpret_cast<float *>(a.ws + l.X);
  float *decay = reinterpret_cast<float *>(a.ws + l.decay);
  const unsigned slots = (unsigned)l.slots, H = (unsigned)a.H;
  const bool joined = l.seg || b || rows == 0;      // incoming states are in the segments' slots
  if (l.seg && slots > 0) {
    Params w = p;
    Pass &f = w.pass[0];
    f.iy = 1; f.iz = 2; f.hy = a.Hk; f.hz = a.Hv; f.dx = a.dk; f.dz = a.dv;
    f.end_slot = segS; f.decay = decay;
    Pass &r = w.pass[1];
    r = f;
    r.iy = 0; r.iz = 3; r.hy = a.Hq; r.hz = a.H; r.rev = 1; r.end_slot = segX;
    if (!launch<kStates>(w, dim3(slots, H, b ? 2 : 1), s)) return CKDA_ERR_CUDA;
  }
  if (joined) {
    JoinParams j = {};
    j.seg[0] = segS; j.seg[1] = segX;
    j.init[0] = a.S0; j.init[1] = b ? b->dS_T : nullptr;
    j.end[0] = a.S_T; j.end[1] = b ? b->dS0 : nullptr;
    j.decay = decay; j.H = a.H; j.elems = p.elems; j.blocks = (p.elems / 4 + 127) / 128;
    j.slots = p.slots;
    lin_join_kernel<<<dim3((unsigned)a.N, H, (unsigned)(j.blocks * (b ? 2 : 1))), 128, 0, s>>>(j);
  }
  if (slots == 0 || rows == 0) return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
  if (!b) {
    if (!a.o && !a.S_T) return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
    Pass &f = p.pass[0];
    f.ix = 0; f.iy = 1; f.iz = 2;
    f.hx = a.Hq; f.hy = a.Hk; f.hz = a.Hv; f.dx = a.dk; f.dz = a.dv;
    f.init = a.S0; f.seg_in = l.seg ? segS : nullptr; f.end = a.S_T; f.out = a.o;
    if (a.o && !make_map(&p.outs[0], a.o, a.H, rows, a.dv, true)) return CKDA_ERR_CUDA;
    return launch<kOut>(p, dim3(slots, H, 1), s) ? CKDA_OK : CKDA_ERR_CUDA;
  }
  const bool part_q = a.Hq < a.H, part_k = a.Hk < a.H, part_v = a.Hv < a.H;
  float *rho = reinterpret_cast<float *>(a.ws + l.rho), *kappa = reinterpret_cast<float *>(a.ws + l.kappa);
  Pass &pq = p.pass[0];
  pq.ix = 3; pq.iy = 2; pq.iz = 1; pq.iw = 0;
  pq.hx = a.H; pq.hy = a.Hv; pq.hz = a.Hk; pq.hw = a.Hq; pq.dx = a.dv; pq.dz = a.dk;
  pq.seg_in = segS; pq.end_slot = segS;
  pq.part = part_q; pq.out = part_q ? a.ws + l.pq : static_cast<uint8_t *>(b->dq);
  pq.dots = rho;
  Pass &pk = p.pass[1];
  pk = pq;
  pk.ix = 2; pk.iy = 3; pk.iz = 0; pk.iw = 1;
  pk.hx = a.Hv; pk.hy = a.H; pk.hz = a.Hq; pk.hw = a.Hk; pk.rev = 1;
  pk.seg_in = segX; pk.end_slot = nullptr;
  pk.part = part_k; pk.out = part_k ? a.ws + l.pk : static_cast<uint8_t *>(b->dk);
  pk.dots = kappa;
  Pass &pv = p.pass[2];
  pv = pk;
  pv.ix = 1; pv.iy = 0; pv.iz = 3;
  pv.hx = a.Hk; pv.hy = a.Hq; pv.hz = a.H; pv.dx = a.dk; pv.dz = a.dv;
  pv.end = b->dS0; pv.end_slot = a.S0 ? segX : nullptr;
  pv.part = part_v; pv.out = part_v ? a.ws + l.pv : static_cast<uint8_t *>(b->dv);
  pv.dots = nullptr;
  for (int i = 0; i < 3; ++i)      // (a shared head's gradient goes through fp32 sums instead)
    if (!p.pass[i].part && !make_map(&p.outs[i], p.pass[i].out, a.H, rows, p.pass[i].dz, true)) return CKDA_ERR_CUDA;
  if (!launch<kGrad>(p, dim3(slots, H, 3), s)) return CKDA_ERR_CUDA;
  DecayParams d = {};
  d.S = segS; d.X = segX; d.rho = rho; d.kappa = kappa; d.g = a.g; d.g_fixed = a.g_fixed; d.has_S0 = a.S0 != nullptr; d.slices = 1;
  d.dg = a.g_fixed ? reinterpret_cast<float *>(a.ws + l.dg) : b->dg;
  d.H = a.H; d.elems = p.elems; d.rows = rows; d.slots = p.slots;
  launch_decay(d, l.slots, s);
  if (part_q) launch_share(pq.out, b->dq, rows, a.H, a.Hq, a.dk, true, a.status, s);
  if (part_k) launch_share(pk.out, b->dk, rows, a.H, a.Hk, a.dk, true, a.status, s);
  if (part_v) launch_share(pv.out, b->dv, rows, a.H, a.Hv, a.dv, true, a.status, s);
  if (a.g_fixed) launch_fixed(d.dg, b->dg, rows, a.H, a.status, s);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // namespace lin
}  // namespace ckda
