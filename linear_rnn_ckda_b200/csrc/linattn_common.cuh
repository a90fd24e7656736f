// linattn_common.cuh -- what the linear attention kernels share: how blocks find their tokens
// and how a chunk's summed log decays are held.
#pragma once

#include "common.cuh"
#include "linattn.h"

namespace ckda {
namespace lin {

constexpr int kC = 64;    // tokens per chunk

// Pieces of L tokens that len tokens take (their sum may pass 32 bits)
__host__ __device__ __forceinline__ int pieces_of(int len, int L) { return (int)(((long)len + L - 1) / L); }

// Pieces of `L` tokens of every sequence (chunks, or segments of several chunks) are numbered in
// one array, `spare` further slots after each sequence's.  Packed: sequence n starts at
// cu[n] / L + n (1 + spare), which leaves room for its ceil(len / L) pieces before the next;
// a table written by plan_kernel gives each slot's sequence (-1: none).
struct Slots {
  const int32_t *cu;
  const int *table;       // packed: [count]
  const int *status;      // non-zero: bad offsets, nothing runs
  int N, T, L, spare;
  __host__ __device__ __forceinline__ long base(int n) const {
    return cu ? (long)cu[n] / L + (long)n * (1 + spare) : (long)n * (pieces_of(T, L) + spare);
  }
};
inline long slot_count(bool packed, int N, int T, int L, int spare) {
  return packed ? (long)T / L + (long)N * (1 + spare) + 1 : (long)N * (pieces_of(T, L) + spare);
}

// One slot's tokens: rows [row0, row0 + len) of the token axis, piece `piece` of `pieces`.
struct Piece {
  int n, piece, pieces, len;
  long row0;
};
__device__ __forceinline__ bool find_piece(const Slots &s, long slot, Piece &p) {
  long first;
  int total;
  if (s.cu) {
    // (only the plan writes this code, so all threads read the same)
    if (*s.status == CKDA_ERR_SEQLENS) return false;
    p.n = s.table[slot];
    if (p.n < 0) return false;
    first = s.cu[p.n];
    total = s.cu[p.n + 1] - (int)first;
  } else {
    p.n = (int)(slot / (pieces_of(s.T, s.L) + s.spare));
    first = (long)p.n * s.T;
    total = s.T;
  }
  p.piece = (int)(slot - s.base(p.n));
  p.pieces = pieces_of(total, s.L);
  if (p.piece >= p.pieces) return false;
  p.row0 = first + (long)p.piece * s.L;
  p.len = min(s.L, total - p.piece * s.L);
  return true;
}

// Checks a packed batch's offsets (status word) and writes the table, of `count` slots, of the slot
// numbering that a call uses (linattn_simt.cu).
struct PlanTable {
  int *table;
  int L, spare;
  long count;
};
int launch_plan(const int32_t *cu, int N, int T, const PlanTable &t, int *status, cudaStream_t s);

// The tensor-core path (linattn_tc.cu): bf16 inputs.
size_t tc_workspace(bool packed, int N, int B, int T, int H, int Hq, int Hk, int Hv, int dk, int dv,
                    bool g_fixed, bool back);
int launch_tc(const LinArgs &a, const LinBwdArgs *b, cudaStream_t s);
// dg from the row dots rho = q . dq and kappa = k . dk, each [slices, H, rows] (slices summed in
// order), and the states around every piece and their gradients (linattn_simt.cu).
struct DecayParams {
  const float *S, *X;       // [slots, H, elems]: incoming states and each sequence's end; the gradients
                            // of the states after the pieces and (with S0) of each sequence's S0
  const float *rho, *kappa, *g;
  int g_fixed, has_S0;
  float *dg;                // [rows, H]
  int H, elems, slices;
  long rows;
  Slots slots;
};
void launch_decay(const DecayParams &p, long slots, cudaStream_t s);
// Sums over the heads that share one head of x [rows, Hx, d], and of a fixed decay's gradient
// over the rows (linattn_simt.cu).
void launch_share(const void *part, void *out, long rows, int H, int Hx, int d, bool bf16,
                  const int *status, cudaStream_t s);
void launch_fixed(const float *part, float *dg, long rows, int H, const int *status, cudaStream_t s);

// Log decays in base 2 as 64-bit fixed point, 32 bits of fraction: each is rounded by 2^-33 at most,
// sums and differences of them are exact, so the weight between two tokens keeps fp32 accuracy however large the sums before them are (an
// fp32 sum of a few thousand would lose 2^-12 of it), and 2^x splits into its integer word and
// its fraction word for nothing.  2^x below -200 is 0 in fp32, so clamping there changes no
// result, keeps -inf (a reset) finite and bounds a chunk's sum by 12,927 (64 x 140 log2 e).
// (A NaN has no fixed-point form: its chunk's factors are set to NaN, chunk_is_nan.)
__device__ __forceinline__ long long fixed_log2(float g) {
  return __double2ll_rn((double)fmaxf(g, -140.f) * 6196328018.8645515);   // log2(e) 2^32
}
// 2^x, 0 below 2^-126 (the fraction's power lies in [1, 2], where the approximation's fast form
// is as good as any)
__device__ __forceinline__ float exp2_fixed(long long x) {
  const int n = (int)(x >> 32);
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint2float_rn((uint32_t)x) * 2.3283064365386963e-10f));
  return n < -126 ? 0.f : r * __int_as_float((min(n, 126) + 127) << 23);
}
// Whether a log decay of the warp's tokens, two per lane, is NaN
__device__ __forceinline__ bool chunk_is_nan(float g0, float g1) {
  return __any_sync(0xffffffffu, isnan(g0) || isnan(g1)) != 0;
}
// Sums over the warp's tokens, two per lane (x0, x1): returns the sum up to and with the second.
__device__ __forceinline__ long long scan_pairs(long long x0, long long x1) {
  const int lane = threadIdx.x & 31;
  long long sum = x0 + x1;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += y;
  }
  return sum;
}

}  // namespace lin
}  // namespace ckda
