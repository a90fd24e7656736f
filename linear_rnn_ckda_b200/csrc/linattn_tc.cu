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
//   O1      M X^T            [z x 64]    A = M as bf16 from TMEM
//   O2      Z^T P^T          [z x 64]    P as bf16 through shared memory
//   D       (tokf Z)^T Y     [z x x]     tokf Z in three bf16 terms
// M is kept in fp32 registers.  Roundings to bf16: P, M as an operand of O1 (each 2^-9 of a
// term in the mean, the size of the output's own rounding); tokf Z is split into three terms
// (24 bits), so M itself carries fp32 accuracy over any length.  Where row dots are wanted
// (decay gradients, which cancel) M goes into O1 in three terms and the scores' part of the dot
// is summed in fp32 from unrounded scores.
//
// One CTA per (segment, head), 16 warps: 0-7 state and output, 8-9 scores (TMEM lanes 0-63),
// 10 TMA loads and decays, 11 MMA issue (one thread), 12-15 tokf Z.  The roles run the chunks
// at their own pace through mbarriers.  A sequence may be cut into segments: a first launch
// computes every segment's own state, an elementwise walk over a sequence's segments gives each
// its incoming state (the decay is a scalar, so a segment's state map is one factor), and the
// main launch runs all segments side by side.
#include <cuda.h>
#include <cudaTypedefs.h>

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
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
// two fp32 values rounded to bf16 (first in the low half), and back
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// ------------------------------------------------------------------ shapes
enum : int { kStates = 0, kOut = 1, kGrad = 2 };   // what a launch computes
constexpr int kThreads = 512;
constexpr uint32_t kPanel = 8192;                  // 64 tokens x 64 channels of bf16, 128-byte swizzle
constexpr uint32_t kTileB = 2 * kPanel;            // 64 tokens x 128 channels

template <int KIND>
struct Cfg {
  static constexpr int kTiles = KIND == kStates ? 2 : KIND == kOut ? 3 : 4;   // Y Z | X Y Z | X Y Z W
  static constexpr int kStages = KIND == kStates ? 4 : KIND == kOut ? 3 : 2;
  static constexpr int kTerms = KIND == kGrad ? 3 : 1;                        // of M in O1
  static constexpr int kPBufs = KIND == kStates ? 0 : KIND == kOut ? 2 : 1;
  static constexpr uint32_t kStage = kTiles * kTileB;
  static constexpr uint32_t oX = 0;
  static constexpr uint32_t oY = KIND == kStates ? 0 : kTileB;
  static constexpr uint32_t oZ = oY + kTileB;
  static constexpr uint32_t oW = oZ + kTileB;                                 // kGrad
  static constexpr uint32_t offTok = kStages * kStage;                        // tokf Z, three terms
  static constexpr uint32_t offP = offTok + 3 * kTileB;
  static constexpr uint32_t offGate = offP + kPBufs * kPanel;
  static constexpr uint32_t kGate = 6 * 64 * 4 + 16;                          // one stage's decays
  static constexpr uint32_t offDot = offGate + kStages * kGate;               // kGrad: 2 x 64 + 2 x 2 x 4 x 32 floats
  static constexpr uint32_t offBar = offDot + (KIND == kGrad ? 2 * 64 * 4 + 512 * 4 : 0);
  static constexpr int kBars = 3 * kStages + 19;
  static constexpr uint32_t kSmem = offBar + kBars * 8 + 64 + 1024;           // + slack to align
  // TMEM columns
  static constexpr uint32_t cSc = 0, cSc2 = 64, cO2 = KIND == kGrad ? 0 : 64;
  static constexpr uint32_t cM = 128, cO1 = cM + 64 * kTerms, cD = KIND == kStates ? 0 : 384;
  static constexpr uint32_t kCols = KIND == kStates ? 128 : 512;
};
static_assert(Cfg<kOut>::kSmem <= 232448 && Cfg<kGrad>::kSmem <= 232448 && Cfg<kStates>::kSmem <= 232448,
              "shared memory");
static_assert(Cfg<kGrad>::cO1 + 64 <= Cfg<kGrad>::cD, "tensor memory");

struct Pass {
  int ix, iy, iz, iw;             // tensor maps (iw < 0: no row dots)
  int hx, hy, hz, hw;             // their heads
  int dx, dz;                     // channels of X and Y, of Z
  int rev;
  int sz, sx;                     // strides of z and x channels in a stored state [dk][dv]
  const float *init;              // [N, H, dk, dv] or NULL (used without seg_in)
  const float *seg_in;            // [slots, H, dk, dv] incoming states, or NULL
  float *end;                     // [N, H, dk, dv]: the last segment's end state, or NULL
  float *end_slot;                // [slots, H, ..]: end state of every segment (kStates), or of the
                                  // last to the slot after it (kGrad), or NULL
  float *decay;                   // kStates: [slots, H] the segment's whole decay
  void *out;                      // [rows, ho, dz]
  int ho, part;                   // part: fp32 per-head sums, [rows, H, dz]
  float *dots;                    // [H, rows] row dots, or NULL
};
struct Params {
  CUtensorMap maps[4];            // q, k, v, dO
  Pass pass[3];
  const float *g;
  int H, g_fixed, elems, no_dO;
  long rows;
  Slots slots;
  int *status;
};

constexpr uint64_t kWaitNs = 2000000000ull;

// A role's wait: all lanes agree on the outcome; a wait that runs out ends every role.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *status) {
  const bool ok = mbar_wait_or_abort(bar, parity & 1u, kWaitNs, abort);
  if (__all_sync(0xffffffffu, ok)) return true;
  *abort = 1;
  if ((threadIdx.x & 31) == 0) set_status(status, CKDA_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool thread_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *status) {
  if (mbar_wait_or_abort(bar, parity & 1u, kWaitNs, abort)) return true;
  *abort = 1;
  set_status(status, CKDA_ERR_TIMEOUT);
  return false;
}

// The sum over the warp's lanes of d[t], t < 16: lane l returns token l % 16's.
__device__ __forceinline__ float lane_sums16(float (&d)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 8; step >= 1; step >>= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int i = 0; i < step; ++i) {
      const float send = up ? d[i] : d[i + step], keep = up ? d[i + step] : d[i];
      d[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
    }
  }
  return d[0] + __shfl_xor_sync(0xffffffffu, d[0], 16);
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ Params p) {
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
  const int nc = (u.len + kC - 1) / kC;

  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::offBar);
  uint64_t *b_full = bars, *b_empty = bars + C::kStages, *b_gate = bars + 2 * C::kStages;
  uint64_t *bx = bars + 3 * C::kStages;
  uint64_t *b_zeroed = bx, *b_sc = bx + 1, *b_p = bx + 2, *b_s = bx + 3, *b_o = bx + 4 /* 2 */,
           *b_ofree = bx + 6, *b_d = bx + 7, *b_dfree = bx + 8, *b_drain = bx + 9, *b_red = bx + 10 /* 2 */,
           *b_w = bx + 12 /* 2 */, *b_wfree = bx + 14 /* 2 */;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bx + 16);
  volatile int *s_abort = reinterpret_cast<volatile int *>(bx + 17);
  volatile int *s_issued = reinterpret_cast<volatile int *>(bx + 18);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full + s, 1);
      // the MMA's commit, warps 0-7, 12-15 and the scores' two
      mbar_init(b_empty + s, KIND == kStates ? 13 : 15);
      mbar_init(b_gate + s, 1);
    }
    mbar_init(b_zeroed, 4);
    mbar_init(b_sc, 1);
    mbar_init(b_p, 2);
    mbar_init(b_s, 8);
    mbar_init(b_o, 1);
    mbar_init(b_o + 1, 1);
    mbar_init(b_ofree, 8);
    for (int s = 0; s < 2; ++s) {
      mbar_init(b_w + s, 4);
      mbar_init(b_wfree + s, 1);
    }
    mbar_init(b_d, 1);
    mbar_init(b_dfree, 8);
    mbar_init(b_drain, 1);
    mbar_init(b_red, 4);
    mbar_init(b_red + 1, 4);
    *s_abort = 0;
    *s_issued = 0;
    mbar_fence_init();
  }
  if (warp == 11) tmem_alloc(s_tmem, C::kCols);
  // (scores on the acausal side are never written: they stay 0)
  for (int i = tid; i < (int)(C::kPBufs * kPanel / 16); i += kThreads)
    reinterpret_cast<uint4 *>(sm + C::offP)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // chunk c of the walk: its index in the segment, its valid rows
  auto chunk_at = [&](int c) { return rev ? nc - 1 - c : c; };
  auto rows_of = [&](int ci) { return min(kC, u.len - ci * kC); };
  auto gates = [&](int st) { return reinterpret_cast<float *>(sm + C::offGate + st * C::kGate); };
  // gates (floats): [0] rowf, [64] tokf, [128] rowa, [192] colb, [256] G (64-bit fixed point),
  // [384] e^{G_C}, [385] whether P_ij is formed as rowa_i (colb_j x_i . y_j)

  if (warp == 10) {
    // ---------------------------------------------------------------- loads and decays
    const int px = (ps.dx + 63) / 64, pz = (ps.dz + 63) / 64;
    const bool has_w = KIND == kGrad && ps.iw >= 0;
    const uint32_t bytes = kPanel * ((KIND != kStates ? px : 0) + px + pz + (has_w ? pz : 0));
    // lane 2 t + q loads panel q of tile t (Y Z, X Y Z, or X Y Z W)
    const int tile = (lane >> 1) + (KIND == kStates ? 1 : 0);
    const bool load = lane < 2 * C::kTiles && (lane & 1) < (tile < 2 ? px : pz) && (tile < 3 || has_w);
    const int map = tile == 0 ? ps.ix : tile == 1 ? ps.iy : tile == 2 ? ps.iz : ps.iw;
    const int head = h * (tile == 0 ? ps.hx : tile == 1 ? ps.hy : tile == 2 ? ps.hz : ps.hw) / p.H;
    long long whole = 0, all = 0;
    float gv[2];
    auto load_g = [&](int c) {
      const int ci = chunk_at(c), len = rows_of(ci);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        gv[e] = i < len ? p.g[p.g_fixed ? (size_t)h : (size_t)(u.row0 + ci * kC + i) * p.H + h] : 0.f;
      }
    };
    load_g(0);
    for (int c = 0; c < nc; ++c) {
      const int st = c % C::kStages, ci = chunk_at(c), len = rows_of(ci);
      if (c >= C::kStages && !warp_wait(b_empty + st, c / C::kStages - 1, s_abort, p.status)) break;
      // one lane per panel
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
      // (fixed decays: a stage that held as many rows holds the same decays)
      if (!p.g_fixed || c < C::kStages || rows_of(chunk_at(c - C::kStages)) != len) {
        const long long x0 = 2 * lane < len ? fixed_log2(gv[0]) : 0;
        const long long x1 = 2 * lane + 1 < len ? fixed_log2(gv[1]) : 0;
        if (c + 1 < nc) load_g(c + 1);
        const long long sum = scan_pairs(x0, x1);
        all = __shfl_sync(0xffffffffu, sum, 31);
        const long long mid = __shfl_sync(0xffffffffu, sum, 15);      // up to token 31
        // weights as one product about token 31 while neither half decays by more than 2^-60
        const long long lim = 60ll << 32;
        const bool plain = mid >= -lim && all - mid >= -lim;
        float *gt = gates(st);
        float2 rf, tf, ra, cb;
        auto one = [&](long long G, int i, float &r, float &t, float &a, float &b) {
          const float since = exp2_fixed(G), until = exp2_fixed(all - G);
          r = rev ? until : since;
          t = i < len ? (rev ? since : until) : 0.f;
          if (KIND == kStates) return;
          const float up = exp2_fixed(G - mid), down = exp2_fixed(mid - G);
          a = plain ? (rev ? down : up) : 1.f;
          b = plain ? (rev ? up : down) : i < 32 ? down : up;   // (to / from token 31)
        };
        one(sum - x1, 2 * lane, rf.x, tf.x, ra.x, cb.x);
        one(sum, 2 * lane + 1, rf.y, tf.y, ra.y, cb.y);
        reinterpret_cast<float2 *>(gt)[lane] = rf;
        reinterpret_cast<float2 *>(gt + 64)[lane] = tf;
        if (KIND != kStates) {
          reinterpret_cast<float2 *>(gt + 128)[lane] = ra;
          reinterpret_cast<float2 *>(gt + 192)[lane] = cb;
          reinterpret_cast<longlong2 *>(gt + 256)[lane] = make_longlong2(sum - x1, sum);
        }
        if (lane == 0) {
          gt[384] = exp2_fixed(all);
          gt[385] = plain ? 1.f : 0.f;
        }
      }
      whole = max(whole + all, -(1ll << 52));
      __syncwarp();
      if (lane == 0) mbar_arrive(b_gate + st);
    }
    // (a backward walk's segments but the last belong to the forward walk too, which writes theirs)
    if (KIND == kStates && lane == 0 && (!rev || u.piece == u.pieces - 1)) {
      ps.decay[(size_t)blockIdx.x * p.H + h] = exp2_fixed(whole);
    }
  } else if (warp == 11) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t sb = smem_u32(sm);
      const int kx = ps.dx / 16;
      const uint32_t id_sc = idesc_bf16(128, 64, false, false), id_o2 = idesc_bf16(128, 64, true, false),
                     id_d = idesc_bf16(128, ps.dx, true, true);
      auto kmajor = [&](uint32_t at) { return smem_desc_sw128(sb + at, 16, 1024); };
      auto mnmajor = [&](uint32_t at) { return smem_desc_sw128(sb + at, kPanel, 1024); };
      // wait helper: false ends the role
      auto need = [&](uint64_t *b, int ph) { return thread_wait(b, (uint32_t)ph, s_abort, p.status); };
      auto tiles = [&](int c) {      // chunk c's tiles have landed (and rows past a ragged end are 0)
        if (!need(b_full + c % C::kStages, c / C::kStages)) return false;
        return rows_of(chunk_at(c)) == kC || need(b_zeroed, 0);
      };
      auto scores = [&](int c) {
        const uint32_t st = (c % C::kStages) * C::kStage;
        for (int kk = 0; kk < kx; ++kk) {
          const uint32_t pan = (kk >> 2) * kPanel;
          mma_bf16_ss(tmem + C::cSc, kmajor(st + C::oX + pan) + 2 * (kk & 3),
                      kmajor(st + C::oY + pan) + 2 * (kk & 3), id_sc, kk > 0);
        }
        if (KIND == kGrad && ps.iw >= 0)
          for (int kk = 0; kk < ps.dz / 16; ++kk) {
            const uint32_t pan = (kk >> 2) * kPanel;
            mma_bf16_ss(tmem + C::cSc2, kmajor(st + C::oW + pan) + 2 * (kk & 3),
                        kmajor(st + C::oZ + pan) + 2 * (kk & 3), id_sc, kk > 0);
          }
        mma_commit(b_sc);
      };
      // D from the tokens of one half of the chunk
      auto state = [&](int c, int half) {
        const uint32_t st = (c % C::kStages) * C::kStage;
        const uint64_t dy = mnmajor(st + C::oY);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const uint64_t dw = mnmajor(C::offTok + t * kTileB);
#pragma unroll
          for (int kk = 2 * half; kk < 2 * half + 2; ++kk)
            mma_bf16_ss(tmem + C::cD, dw + 128 * kk, dy + 128 * kk, id_d, half + t + (kk & 1) > 0);
        }
        mma_commit(b_wfree + half);
        if (half) mma_commit(b_d);
      };
      auto out1 = [&](int c) {
        const uint32_t st = (c % C::kStages) * C::kStage;
        const int terms = KIND == kGrad && ps.iw >= 0 ? C::kTerms : 1;
        for (int t = 0; t < terms; ++t)
          for (int kk = 0; kk < kx; ++kk)
            mma_bf16_ts(tmem + C::cO1, tmem + C::cM + 64 * t + 8 * kk,
                        kmajor(st + C::oX + (kk >> 2) * kPanel) + 2 * (kk & 3), id_sc, t + kk > 0);
      };
      auto out2 = [&](int c) {
        const uint32_t st = (c % C::kStages) * C::kStage;
        const uint64_t dz = mnmajor(st + C::oZ), dp = kmajor(C::offP + (C::kPBufs > 1 ? (c & 1) * kPanel : 0));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16_ss(tmem + C::cO2, dz + 128 * kk, dp + 2 * kk, id_o2, kk > 0);
        mma_commit(b_o + (c & 1));
      };
      bool ok = true;
      if (KIND == kOut) {
        ok = tiles(0);
        if (ok) { tc_fence_after(); scores(0); }
      }
      for (int c = 0; ok && c < nc; ++c) {
        if (KIND != kOut && !(ok = tiles(c))) break;
        if (KIND == kGrad) {
          if (!(ok = c == 0 || need(b_ofree, c - 1))) break;
          tc_fence_after();
          scores(c);
        }
        if (!(ok = need(b_w, c) && (c == 0 || need(b_dfree, c - 1)))) break;
        tc_fence_after();
        state(c, 0);
        if (KIND == kOut) {
          if (!(ok = need(b_p, c) && (c + 1 >= nc || tiles(c + 1)))) break;
          tc_fence_after();
          if (c + 1 < nc) scores(c + 1);
        }
        if (!(ok = need(b_w + 1, c))) break;
        tc_fence_after();
        state(c, 1);
        if (KIND != kStates) {
          if (!(ok = need(b_s, c) && (KIND == kGrad || c == 0 || need(b_ofree, c - 1)))) break;
          tc_fence_after();
          out1(c);
          if (KIND == kGrad) {
            if (!(ok = need(b_p, c))) break;
            tc_fence_after();
          }
          out2(c);
        }
        mma_commit(b_empty + c % C::kStages);
      }
      // every product issued has completed before the tensor memory is released
      mma_commit(b_drain);
      mbar_wait(b_drain, 0, kWaitNs);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- tokf Z in three bf16 terms
    const int t = tid - 12 * 32, pz = (ps.dz + 63) / 64;
    for (int c = 0; c < nc; ++c) {
      const int st = c % C::kStages, len = rows_of(chunk_at(c));
      uint8_t *base = sm + st * C::kStage;
      if (!warp_wait(b_full + st, c / C::kStages, s_abort, p.status)) break;
      if (len < kC) {
        // a ragged end: the rows that follow belong to another sequence
        for (uint32_t i = t; i < C::kStage / 16; i += 128)
          if ((int)(i >> 3 & 63) >= len) reinterpret_cast<uint4 *>(base)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_zeroed);
        if (!warp_wait(b_zeroed, 0, s_abort, p.status)) break;
      }
      if (!warp_wait(b_gate + st, c / C::kStages, s_abort, p.status)) break;
      const float *tokf = gates(st) + 64;
      const uint4 *src = reinterpret_cast<const uint4 *>(base + C::oZ);
      uint4 *dst = reinterpret_cast<uint4 *>(sm + C::offTok);
      bool ok = true;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (c > 0 && !(ok = warp_wait(b_wfree + half, c - 1, s_abort, p.status))) break;
        for (int q = 0; q < pz; ++q) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int i = 512 * q + 256 * half + 128 * v + t;
            const float w = tokf[i >> 3 & 63];
            const uint4 z = src[i];
            uint4 r[3];
            const uint32_t *zi = &z.x;
            uint32_t *r0 = &r[0].x, *r1 = &r[1].x, *r2 = &r[2].x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a = lo_f32(zi[e]) * w, b = hi_f32(zi[e]) * w;
              r0[e] = pack_bf16(a, b);
              a -= lo_f32(r0[e]); b -= hi_f32(r0[e]);
              r1[e] = pack_bf16(a, b);
              a -= lo_f32(r1[e]); b -= hi_f32(r1[e]);
              r2[e] = pack_bf16(a, b);
            }
            dst[i] = r[0];
            dst[kTileB / 16 + i] = r[1];
            dst[2 * kTileB / 16 + i] = r[2];
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_w + half);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(b_empty + st);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- scores (warps 8, 9)
    if (KIND != kStates) {
      const int wr = warp - 8, row = 32 * wr + lane;
      const uint32_t lanes = tmem + ((uint32_t)(32 * wr) << 16);
      const bool dots = KIND == kGrad && ps.iw >= 0;
      float *row_dot = reinterpret_cast<float *>(sm + C::offDot);
      const int other = rev ? 1 : 0;               // the column block a causal off-diagonal block has
      for (int c = 0; wr < 2 && c < nc; ++c) {
        const int st = c % C::kStages;
        if (!warp_wait(b_gate + st, c / C::kStages, s_abort, p.status)) break;
        if (!warp_wait(b_sc, c, s_abort, p.status)) break;
        tc_fence_after();
        // (the scores two chunks back, or one, have been read)
        if (c >= C::kPBufs && !warp_wait(b_o + ((c - C::kPBufs) & 1), (c - C::kPBufs) >> 1, s_abort, p.status))
          break;
        const float *gt = gates(st);
        uint8_t *P = sm + C::offP + (C::kPBufs > 1 ? (c & 1) * kPanel : 0) + row * 128;
        const bool plain = gt[385] != 0.f;
        const float mine = gt[192 + row];
        const long long *G = reinterpret_cast<const long long *>(gt + 256);
        float dot = 0.f;
#pragma unroll 1
        for (int b = wr == other ? wr : 0; b < (wr == other ? wr + 1 : 2); ++b) {
          if (!plain && b == wr) {                  // every weight from its own difference of sums
            const long long me = G[row];
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
              uint32_t s1, w1 = 0;
              tmem_ld1(lanes + C::cSc + 32 * b + j, s1);
              if (dots) tmem_ld1(lanes + C::cSc2 + 32 * b + j, w1);
              tmem_wait_ld();
              const long long o = G[32 * b + j];
              const float x = (rev ? j >= lane : j <= lane) ? __uint_as_float(s1) * exp2_fixed(rev ? o - me : me - o) : 0.f;
              if (dots && j != lane) dot = (rev ? j > lane : j < lane) ? fmaf(x, __uint_as_float(w1), dot) : dot;
              *reinterpret_cast<__nv_bfloat16 *>(P + (((4 * b + j / 8) ^ (row & 7)) << 4) + 2 * (j & 7)) =
                  __float2bfloat16_rn(x);
            }
            continue;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int j0 = 32 * b + 16 * half;
            uint32_t s[16], w2[16];
            tmem_ld16(lanes + C::cSc + j0, s);
            if (dots) tmem_ld16(lanes + C::cSc2 + j0, w2);
            float f[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(f + 4 * j) = *reinterpret_cast<const float4 *>(gt + 192 + j0 + 4 * j);
            if (!plain) {                           // (off the diagonal block: through token 31)
#pragma unroll
              for (int j = 0; j < 16; ++j) f[j] *= mine;
            }
            tmem_wait_ld();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(s[j]) * f[j];
            if (b == wr) {                          // the diagonal block: mask, and no diagonal in the dot
              const uint32_t m = (rev ? ~0u << lane : ~0u >> (31 - lane)) >> (16 * half);
              const uint32_t m1 = m & ~((1u << lane) >> (16 * half));
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                v[j] = m & (1u << j) ? v[j] : 0.f;
                if (dots) dot = m1 & (1u << j) ? fmaf(v[j], __uint_as_float(w2[j]), dot) : dot;
              }
            } else if (dots) {
#pragma unroll
              for (int j = 0; j < 16; ++j) dot = fmaf(v[j], __uint_as_float(w2[j]), dot);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint4 pk;
              pk.x = pack_bf16(v[8 * q], v[8 * q + 1]);
              pk.y = pack_bf16(v[8 * q + 2], v[8 * q + 3]);
              pk.z = pack_bf16(v[8 * q + 4], v[8 * q + 5]);
              pk.w = pack_bf16(v[8 * q + 6], v[8 * q + 7]);
              *reinterpret_cast<uint4 *>(P + (((j0 / 8 + q) ^ (row & 7)) << 4)) = pk;
            }
          }
        }
        dot *= gt[128 + row];
        if (dots) row_dot[(c & 1) * 64 + row] = dot;
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p);
          mbar_arrive(b_empty + st);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- state and output (warps 0-7)
    const int quad = warp & 3, hf = warp >> 2;
    const int z = 32 * quad + lane;                 // this thread's value channel (TMEM lane)
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const bool live = z < ps.dz && 64 * hf < ps.dx;
    const bool dots = KIND == kGrad && ps.iw >= 0;
    const int ncol = min(64, ps.dx - 64 * hf);      // state columns of this half (<= 0: none)
    float M[64];
    {
      const float *src = nullptr;
      if (KIND != kStates) {
        if (ps.seg_in) src = ps.seg_in + ((size_t)blockIdx.x * p.H + h) * p.elems;
        else if (ps.init) src = ps.init + ((size_t)u.n * p.H + h) * p.elems;
      }
      if (src) src += (size_t)z * ps.sz + (size_t)(64 * hf) * ps.sx;
      const bool have = src && live;
      if (ps.sx == 1) {
#pragma unroll
        for (int i = 0; i < 64; i += 4)
          *reinterpret_cast<float4 *>(M + i) = have && i < ncol ? *reinterpret_cast<const float4 *>(src + i)
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) M[i] = have && i < ncol ? src[(size_t)i * ps.sx] : 0.f;
      }
    }
    // M as the next chunk's operand
    auto put_state = [&]() {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t r[C::kTerms][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = M[16 * b + 2 * i], y = M[16 * b + 2 * i + 1];
          r[0][i] = pack_bf16(x, y);
          if constexpr (KIND == kGrad) {
            if (!dots) continue;
#pragma unroll
            for (int t = 1; t < 3; ++t) {
              x -= lo_f32(r[t - 1][i]);
              y -= hi_f32(r[t - 1][i]);
              r[t][i] = pack_bf16(x, y);
            }
          }
        }
        tmem_st8(lanes + C::cM + 32 * hf + 8 * b, r[0]);
        if constexpr (KIND == kGrad) {
          if (dots) {
            tmem_st8(lanes + C::cM + 64 + 32 * hf + 8 * b, r[1]);
            tmem_st8(lanes + C::cM + 128 + 32 * hf + 8 * b, r[2]);
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_s);
    };
    bool ok = true;
    if (KIND != kStates) put_state();
    float *row_dot = reinterpret_cast<float *>(sm + C::offDot);
    float *red = row_dot + 128;                     // [2][2 halves][4 quads][32]
    for (int c = 0; c < nc; ++c) {
      const int st = c % C::kStages, ci = chunk_at(c), len = rows_of(ci);
      if (!(ok = warp_wait(b_gate + st, c / C::kStages, s_abort, p.status))) break;
      const float *gt = gates(st);
      const float a = gt[384];
      if (!(ok = warp_wait(b_d, c, s_abort, p.status))) break;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t r[16];
        tmem_ld16(lanes + C::cD + 64 * hf + 16 * b, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) M[16 * b + i] = fmaf(a, M[16 * b + i], __uint_as_float(r[i]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_dfree);
      if (KIND != kStates) {
        if (!(ok = warp_wait(b_o + (c & 1), c >> 1, s_abort, p.status))) break;
        // (the scores' row dots; waited for here, before b_ofree lets the next phase complete)
        if (dots && !(ok = warp_wait(b_p, c, s_abort, p.status))) break;
        tc_fence_after();
        if (KIND == kOut && c + 1 < nc) put_state();
        // outputs of 32 tokens, 16 at a time
        const size_t ostr = (size_t)(ps.part ? p.H : ps.ho) * ps.dz;
        const size_t o0 = (size_t)(u.row0 + ci * kC + 32 * hf) * ostr + (size_t)h * ps.dz + z;
        const int lim = z < ps.dz && ps.out ? len - 32 * hf : 0;
        const uint8_t *wt = sm + st * C::kStage + C::oW + (z >> 6) * kPanel + (32 * hf) * 128;
        float sums = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t r1[16], r2[16];
          tmem_ld16(lanes + C::cO1 + 32 * hf + 16 * b, r1);
          tmem_ld16(lanes + C::cO2 + 32 * hf + 16 * b, r2);
          tmem_wait_ld();
          if (b == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_ofree);
          }
          const float4 *rf = reinterpret_cast<const float4 *>(gt + 32 * hf + 16 * b);
          const float4 *ra = reinterpret_cast<const float4 *>(gt + 128 + 32 * hf + 16 * b);
          float x[16], v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = rf[i], e = ra[i];
            x[4 * i] = f.x * __uint_as_float(r1[4 * i]);
            x[4 * i + 1] = f.y * __uint_as_float(r1[4 * i + 1]);
            x[4 * i + 2] = f.z * __uint_as_float(r1[4 * i + 2]);
            x[4 * i + 3] = f.w * __uint_as_float(r1[4 * i + 3]);
            v[4 * i] = fmaf(e.x, __uint_as_float(r2[4 * i]), x[4 * i]);
            v[4 * i + 1] = fmaf(e.y, __uint_as_float(r2[4 * i + 1]), x[4 * i + 1]);
            v[4 * i + 2] = fmaf(e.z, __uint_as_float(r2[4 * i + 2]), x[4 * i + 2]);
            v[4 * i + 3] = fmaf(e.w, __uint_as_float(r2[4 * i + 3]), x[4 * i + 3]);
          }
          if (ps.part) {
            float *o = static_cast<float *>(ps.out) + o0 + (size_t)(16 * b) * ostr;
#pragma unroll
            for (int i = 0; i < 16; ++i, o += ostr)
              if (16 * b + i < lim) *o = v[i];
          } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(ps.out) + o0 + (size_t)(16 * b) * ostr;
#pragma unroll
            for (int i = 0; i < 16; ++i, o += ostr)
              if (16 * b + i < lim) *o = __float2bfloat16_rn(v[i]);
          }
          if (dots) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int t = 16 * b + i;
              const float w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
                  wt + t * 128 + (((z & 63) * 2) ^ ((t & 7) << 4))));
              x[i] = z < ps.dz ? x[i] * w : 0.f;
            }
            const float s = lane_sums16(x);
            if ((lane >> 4) == b) sums = s;         // lane t holds token t of this half
          }
        }
        if (KIND == kGrad && c + 1 < nc) put_state();
        if (dots) {
          float *rd = red + ((c & 1) * 2 + hf) * 128;
          rd[quad * 32 + lane] = sums;
          __syncwarp();
          if (lane == 0) mbar_arrive(b_red + hf);
          if (quad == 0 && !(ok = warp_wait(b_red + hf, c, s_abort, p.status))) break;
          if (quad == 0 && 32 * hf + lane < len)
            ps.dots[(size_t)h * p.rows + u.row0 + ci * kC + 32 * hf + lane] =
                (rd[lane] + rd[32 + lane]) + (rd[64 + lane] + rd[96 + lane]) + row_dot[(c & 1) * 64 + 32 * hf + lane];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty + st);
    }
    if (ok && live) {
      auto store = [&](float *dst) {
        dst += (size_t)z * ps.sz + (size_t)(64 * hf) * ps.sx;
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i < ncol) dst[(size_t)i * ps.sx] = M[i];
      };
      if (KIND == kStates) store(ps.end_slot + ((size_t)blockIdx.x * p.H + h) * p.elems);
      else if (last_seg) {
        if (ps.end) store(ps.end + ((size_t)u.n * p.H + h) * p.elems);
        if (ps.end_slot) store(ps.end_slot + ((size_t)(blockIdx.x + 1) * p.H + h) * p.elems);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    // loads that a role which gave up did not wait for have landed
    for (int c = max(0, *s_issued - C::kStages); c < *s_issued; ++c)
      mbar_wait(b_full + c % C::kStages, (c / C::kStages) & 1, kWaitNs);
  }
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
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
  const int m = (len + p.slots.L - 1) / p.slots.L;
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

// ------------------------------------------------------------------ decay gradients
// dg_t = <S_out, X> + sum_{s >= t} (q_s . dq_s - k_s . dk_s) over a segment, S_out the state
// after it and X its gradient.  One block per (segment, head).
struct DecayParams {
  const float *S, *X;       // [slots, H, elems]: incoming states (and the last's end), gradients
  const float *rho, *kappa; // [H, rows]
  float *dg;                // [rows, H]
  int H, elems;
  long rows;
  Slots slots;
};
__global__ void __launch_bounds__(256) lin_decay_kernel(const DecayParams p) {
  __shared__ double s_sum[8];
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float4 *S = reinterpret_cast<const float4 *>(p.S + ((size_t)(blockIdx.x + 1) * p.H + h) * p.elems);
  const float4 *X = reinterpret_cast<const float4 *>(p.X + ((size_t)blockIdx.x * p.H + h) * p.elems);
  float part = 0.f;
  for (int e = tid; e < p.elems / 4; e += 256) {
    const float4 a = S[e], b = X[e];
    part = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, part))));
  }
  double dot = part;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  if (lane == 0) s_sum[warp] = dot;
  __syncthreads();
  double run = 0.0;                              // <S_out, X> plus the blocks after this one
#pragma unroll
  for (int w = 0; w < 8; ++w) run += s_sum[w];
  const float *rho = p.rho + (size_t)h * p.rows + u.row0, *kap = p.kappa + (size_t)h * p.rows + u.row0;
  // 256 tokens at a time from the end; thread 0 takes the last of them
  for (int top = u.len; top > 0; top -= 256) {
    const int i = top - 1 - tid;
    double x = i >= 0 ? (double)rho[i] - (double)kap[i] : 0.0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (i >= 0) p.dg[(size_t)(u.row0 + i) * p.H + h] = (float)(run + before + x);
    run += all;
  }
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
// [rows, heads, d] bf16 as (channel, head, token), box 64 x 1 x 64, 128-byte swizzle; channels
// past d and tokens past rows read as 0
bool make_map(CUtensorMap *map, const void *base, int heads, long rows, int d) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
  cuuint32_t box[3] = {64, 1, 64}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSMs = 148;

// Tokens per segment.  Unpacked: the cut into m segments that the model below finds shortest, in
// chunk times: main launch = waves x (segment + 3 chunks' worth of start), first launch half a
// chunk time per chunk, 8 for the extra launches.  Packed: lengths are on the device, so a
// segment is a quarter of an SM's share of all chunks, between 8 and 64 chunks.
int segment_tokens(bool packed, int N, int B, int T, int H, int passes) {
  const long nch = ((long)T + kC - 1) / kC;
  if (nch <= 1) return kC;
  if (packed) {
    long c = nch * H * passes / kSMs / 4;
    c = c < 8 ? 8 : c > 64 ? 64 : c;
    return (int)c * kC;
  }
  long best = -1, best_c = nch;
  for (long m = 1; m <= nch && m <= 64; ++m) {
    const long c = (nch + m - 1) / m, mm = (nch + c - 1) / c;
    const long units = (long)B * H * passes * mm;
    long cost = 2 * ((units + kSMs - 1) / kSMs) * (c + 3);
    if (mm > 1) cost += (((long)B * H * (passes > 1 ? 2 : 1) * (mm - 1) + kSMs - 1) / kSMs) * (c + 3) + 16;
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
  l.L = segment_tokens(packed, N, B, T, H, back ? 3 : 1);
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
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<KIND>::kSmem) != cudaSuccess)
    return false;
  kern<<<grid, kThreads, Cfg<KIND>::kSmem, s>>>(p);
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
  p.slots = Slots{a.cu, reinterpret_cast<const int *>(a.ws + l.table), a.status, a.N, a.T, l.L, b ? 1 : 0};
  if (a.cu) {
    const PlanTable t{reinterpret_cast<int *>(a.ws + l.table), l.L, b ? 1 : 0, l.slots};
    const int rc = launch_plan(a.cu, a.N, a.T, &t, 1, a.status, s);
    if (rc != CKDA_OK) return rc;
  }
  float *segS = reinterpret_cast<float *>(a.ws + l.S), *segX = reinterpret_cast<float *>(a.ws + l.X);
  float *decay = reinterpret_cast<float *>(a.ws + l.decay);
  const unsigned slots = (unsigned)l.slots, H = (unsigned)a.H;
  const bool joined = l.seg || b || rows == 0;      // incoming states are in the segments' slots
  if (l.seg && slots > 0) {
    Params w = p;
    Pass &f = w.pass[0];
    f.iy = 1; f.iz = 2; f.hy = a.Hk; f.hz = a.Hv; f.dx = a.dk; f.dz = a.dv; f.sz = 1; f.sx = a.dv;
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
    f.ix = 0; f.iy = 1; f.iz = 2; f.iw = -1;
    f.hx = a.Hq; f.hy = a.Hk; f.hz = a.Hv; f.dx = a.dk; f.dz = a.dv; f.sz = 1; f.sx = a.dv;
    f.init = a.S0; f.seg_in = l.seg ? segS : nullptr; f.end = a.S_T; f.out = a.o; f.ho = a.H;
    return launch<kOut>(p, dim3(slots, H, 1), s) ? CKDA_OK : CKDA_ERR_CUDA;
  }
  const bool part_q = a.Hq < a.H, part_k = a.Hk < a.H, part_v = a.Hv < a.H;
  float *rho = reinterpret_cast<float *>(a.ws + l.rho), *kappa = reinterpret_cast<float *>(a.ws + l.kappa);
  Pass &pq = p.pass[0];
  pq.ix = 3; pq.iy = 2; pq.iz = 1; pq.iw = 0;
  pq.hx = a.H; pq.hy = a.Hv; pq.hz = a.Hk; pq.hw = a.Hq; pq.dx = a.dv; pq.dz = a.dk;
  pq.sz = a.dv; pq.sx = 1; pq.seg_in = segS; pq.end_slot = segS;
  pq.part = part_q; pq.out = part_q ? a.ws + l.pq : static_cast<uint8_t *>(b->dq); pq.ho = a.Hq;
  pq.dots = rho;
  Pass &pk = p.pass[1];
  pk = pq;
  pk.ix = 2; pk.iy = 3; pk.iz = 0; pk.iw = 1;
  pk.hx = a.Hv; pk.hy = a.H; pk.hz = a.Hq; pk.hw = a.Hk; pk.rev = 1;
  pk.seg_in = segX; pk.end_slot = nullptr;
  pk.part = part_k; pk.out = part_k ? a.ws + l.pk : static_cast<uint8_t *>(b->dk); pk.ho = a.Hk;
  pk.dots = kappa;
  Pass &pv = p.pass[2];
  pv = pk;
  pv.ix = 1; pv.iy = 0; pv.iz = 3; pv.iw = -1;
  pv.hx = a.Hk; pv.hy = a.Hq; pv.hz = a.H; pv.dx = a.dk; pv.dz = a.dv; pv.sz = 1; pv.sx = a.dv;
  pv.end = b->dS0;
  pv.part = part_v; pv.out = part_v ? a.ws + l.pv : static_cast<uint8_t *>(b->dv); pv.ho = a.Hv;
  pv.dots = nullptr;
  if (!launch<kGrad>(p, dim3(slots, H, 3), s)) return CKDA_ERR_CUDA;
  DecayParams d = {};
  d.S = segS; d.X = segX; d.rho = rho; d.kappa = kappa;
  d.dg = a.g_fixed ? reinterpret_cast<float *>(a.ws + l.dg) : b->dg;
  d.H = a.H; d.elems = p.elems; d.rows = rows; d.slots = p.slots;
  lin_decay_kernel<<<dim3(slots, H), 256, 0, s>>>(d);
  if (part_q) launch_share(pq.out, b->dq, rows, a.H, a.Hq, a.dk, true, a.status, s);
  if (part_k) launch_share(pk.out, b->dk, rows, a.H, a.Hk, a.dk, true, a.status, s);
  if (part_v) launch_share(pv.out, b->dv, rows, a.H, a.Hv, a.dv, true, a.status, s);
  if (a.g_fixed) launch_fixed(d.dg, b->dg, rows, a.H, a.status, s);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // namespace lin
}  // namespace ckda
