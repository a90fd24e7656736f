// linattn_common.cuh -- what the linear attention kernels share: how blocks find their tokens
// and how a chunk's summed log decays are held.
#pragma once

#include "common.cuh"
#include "linattn.h"

namespace ckda {
namespace lin {

constexpr int kC = 64;    // tokens per chunk

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
    return cu ? (long)cu[n] / L + (long)n * (1 + spare) : (long)n * ((T + L - 1) / L + spare);
  }
};
inline long slot_count(bool packed, int N, int T, int L, int spare) {
  return packed ? (long)T / L + (long)N * (1 + spare) + 1 : (long)N * ((T + L - 1) / L + spare);
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
    p.n = (int)(slot / ((s.T + s.L - 1) / s.L + s.spare));
    first = (long)p.n * s.T;
    total = s.T;
  }
  p.piece = (int)(slot - s.base(p.n));
  p.pieces = (total + s.L - 1) / s.L;
  if (p.piece >= p.pieces) return false;
  p.row0 = first + (long)p.piece * s.L;
  p.len = min(s.L, total - p.piece * s.L);
  return true;
}

// Checks a packed batch's offsets (status word) and writes the slot tables of the one or two
// slot numberings a call uses.  Host side in linattn_abi.cu.
struct PlanTable {
  int *table;
  int L, spare;
  long count;
};
int launch_plan(const int32_t *cu, int N, int T, const PlanTable *tables, int n_tables, int *status,
                cudaStream_t s);

// The tensor-core path (linattn_tc.cu): bf16 inputs.
size_t tc_workspace(bool packed, int N, int B, int T, int H, int Hq, int Hk, int Hv, int dk, int dv,
                    bool g_fixed, bool back);
int launch_tc(const LinArgs &a, const LinBwdArgs *b, cudaStream_t s);
// Sums over the heads that share one head of x [rows, Hx, d], and of a fixed decay's gradient
// over the rows (linattn_simt.cu).
void launch_share(const void *part, void *out, long rows, int H, int Hx, int d, bool bf16,
                  const int *status, cudaStream_t s);
void launch_fixed(const float *part, float *dg, long rows, int H, const int *status, cudaStream_t s);

// Log decays in base 2.  exp2 of anything below -200 is 0 in fp32, so clamping there changes no
// result, keeps -inf (a reset) finite, and bounds a chunk's sum by 12,800.
constexpr float kMinLog2 = -200.f;
__device__ __forceinline__ double log2_decay(float g) {
  const double x = (double)g * 1.4426950408889634;
  return x < (double)kMinLog2 ? (double)kMinLog2 : x;     // NaN stays NaN
}
// A sum G is summed in fp64 and held as two floats, hi a multiple of 2^-8 and lo the rest, so
// that the difference of two sums (hi exactly, lo to 2^-33) keeps fp32 accuracy when both are
// large and near each other; a single fp32 sum of a few thousand would lose 2^-12 of the weight.
__device__ __forceinline__ float2 split_sum(double G) {
  const float hi = (float)(rint(G * 256.0) * 0.00390625);
  return make_float2(hi, (float)(G - (double)hi));
}
__device__ __forceinline__ float pair_weight(float2 a, float2 b) {     // 2^(a - b)
  return exp2f((a.x - b.x) + (a.y - b.y));
}

}  // namespace lin
}  // namespace ckda
