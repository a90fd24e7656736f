// linattn_simt.cu -- linear attention with a decay for each head in exact fp32 on CUDA cores:
// forward and gradients, chunks of 64 tokens.
//
//   1. lin_local_kernel: every chunk's own state  sum_j e^{G_C - G_j} k_j v_j^T  (and, backwards,
//      its own state gradient  sum_i e^{G_i} q_i dO_i^T), all chunks side by side;
//   2. lin_scan_kernel: the walk over a sequence's chunks, S <- e^{G_C} S + own, elementwise:
//      one thread per four state entries, the next chunks' loads in flight;
//   3. lin_pass_kernel: outputs or one gradient of every chunk, all chunks side by side.
//
// As on the tensor cores (linattn_tc.cu) the output and the three gradients are one product with
// the roles exchanged, X the queries, Y the keys, Z the values, M the state the chunk starts with
// (o, dq) or the state gradient it ends with (dk, dv):
//   out_i = rowf_i M^T x_i + sum_j e^{+-(G_i - G_j)} (x_i . y_j) z_j
//   o : q, k, v forwards    dq : dO, v, k forwards    dk : v, dO, q    dv : k, q, dO backwards
// and q . dq, k . dk of each token go to lin_decay_kernel for the decays' gradients.  A sequence
// of one chunk (a short prompt) is one launch: the pass reads S0 itself and writes S_T.
//
// Bound: fp32 FMA and shared-memory loads; few chunks are split over columns of the output, which
// repeats the scores, so that a small call occupies more SMs.  Measured: B2 T37 H3 64 x 64 forward
// 22 us (one launch), B2 T515 H4 32 x 64 gradients 52 us (five).
#include "linattn_common.cuh"

namespace ckda {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kLd = 132;     // row stride of a 64 x 128 fp32 tile: 16-byte rows, banks shifted by 4
constexpr int kLdP = 68;     // of a 64 x 64 one
constexpr int kTile = kC * kLd;
constexpr int kTileP = kC * kLdP;

// Loads rows [0, len) x columns [c0, c0 + cols) of head hx of x [rows, Hx, d] into a tile of row
// stride ld, zeros past len, d or where x is NULL.
__device__ void load_tile(float *t, int ld, const float *x, long row0, int len, int Hx, int hx, int d,
                          int c0, int cols) {
  const float *src = x + ((size_t)row0 * Hx + hx) * d + c0;
  const int n4 = cols / 4;
  for (int i = threadIdx.x; i < kC * n4; i += kThreads) {
    const int r = i / n4, c = (i - r * n4) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x && r < len && c0 + c < d) f = *reinterpret_cast<const float4 *>(src + (size_t)r * Hx * d + c);
    *reinterpret_cast<float4 *>(t + r * ld + c) = f;
  }
}

// A sum as two floats, hi a multiple of 2^-8 and lo the rest: the difference of two sums is
// (hi - hi), exact, plus (lo - lo), to 2^-33.
__device__ __forceinline__ float2 split_sum(long long G) {
  return make_float2((float)(int)(G >> 24) * 0.00390625f,
                     (float)(int)(G & 0xffffff) * 2.3283064365386963e-10f);
}
__device__ __forceinline__ float pair_weight(float2 a, float2 b) {     // 2^(a - b)
  return exp2f((a.x - b.x) + (a.y - b.y));
}
// The chunk's sums G_i (hi, lo; base 2) to sG[0 .. 63], rows past len continuing the last;
// e^{G_i} to sE and e^{G_C - G_i} (0 past len) to sW.  One warp; the caller synchronises.
__device__ void chunk_gates(float2 *sG, float *sE, float *sW, const float *g, long row0, int len,
                            int H, int h, int g_fixed) {
  const int lane = threadIdx.x;
  if (lane >= 32) return;
  long long x[2];
  float gl[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * lane + u;
    gl[u] = i < len ? g[g_fixed ? (size_t)h : (size_t)(row0 + i) * H + h] : 0.f;
    x[u] = fixed_log2(gl[u]);
  }
  const bool bad = chunk_is_nan(gl[0], gl[1]);
  const long long sum = scan_pairs(x[0], x[1]);
  const long long all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * lane + u;
    const long long G = u ? sum : sum - x[1];
    sG[i] = bad ? make_float2(nanf(""), 0.f) : split_sum(G);
    sE[i] = bad ? nanf("") : exp2_fixed(G);
    sW[i] = i >= len ? 0.f : bad ? nanf("") : exp2_fixed(all - G);
  }
}

// acc[4][NJ] += A (64 x K) B (K x 16 NJ) for this thread's rows 4 ty .. 4 ty + 3.  A is stored
// [row][k] (AKC: k contiguous) or [k][row]; B [k][column], columns NJ tx .. NJ tx + NJ - 1.
template <int NJ, bool AKC>
__device__ __forceinline__ void mm(float (&acc)[4][NJ], const float *A, int lda, const float *B, int ldb, int K) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float a[4][4], b[4][NJ];       // [k][..]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = AKC ? *reinterpret_cast<const float4 *>(A + (4 * ty + i) * lda + k)
                           : *reinterpret_cast<const float4 *>(A + (k + i) * lda + 4 * ty);
      if (AKC) {
        a[0][i] = f.x; a[1][i] = f.y; a[2][i] = f.z; a[3][i] = f.w;
      } else {
        a[i][0] = f.x; a[i][1] = f.y; a[i][2] = f.z; a[i][3] = f.w;
      }
      const float *bp = B + (k + i) * ldb + NJ * tx;
      if constexpr (NJ == 4) {
        const float4 e = *reinterpret_cast<const float4 *>(bp);
        b[i][0] = e.x; b[i][1] = e.y; b[i][2] = e.z; b[i][3] = e.w;
      } else {
        const float2 e = *reinterpret_cast<const float2 *>(bp);
        b[i][0] = e.x; b[i][1] = e.y;
      }
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(a[kk][i], b[kk][j], acc[i][j]);
  }
}
// the same with B stored [column][k], columns tx + 16 j (free of bank conflicts)
__device__ __forceinline__ void mm_scores(float (&acc)[4][4], const float *A, const float *B, int K) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * kLd + k);
      b[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * kLd + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
        acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
        acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
        acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
      }
  }
}
template <int NJ>
__device__ __forceinline__ void zero(float (&acc)[4][NJ]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
}
template <int NJ>
__device__ __forceinline__ void put_row(float *dst, const float (&v)[NJ]) {
  if constexpr (NJ == 4) *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<float2 *>(dst) = make_float2(v[0], v[1]);
}

// The status word of an unpacked batch (a packed one's plan writes it).
__device__ __forceinline__ void clear_status(const Slots &s, int *status) {
  if (!s.cu && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *status = 0;
}

// ---------------------------------------------------------------- chunks' own states
struct LocalParams {
  const float *y[2], *z[2];  // k, v; q, dO
  int hy[2], hz[2];
  const float *g;
  float *own[2];             // [slots, H, dk, dv]
  float *decay;              // [slots, H]: e^{G_C}
  int *status;
  int H, ndk, ndv, g_fixed, cols;
  Slots slots;
};
// blockIdx: (slot, head, (direction, block of 64 rows, slice of 16 NJ columns)); direction 1: own
// state gradients, with weights e^{G_i}.
template <int NJ>
__global__ void __launch_bounds__(kThreads) lin_local_kernel(const LocalParams p) {
  __shared__ __align__(16) float sY[kTileP], sZ[kTileP];
  __shared__ float2 sG[kC];
  __shared__ float sE[kC], sW[kC];
  clear_status(p.slots, p.status);
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, blocks = (p.ndk + 63) / 64;
  const int slice = blockIdx.z % p.cols, m0 = 64 * (blockIdx.z / p.cols % blocks), back = blockIdx.z / (p.cols * blocks);
  const int c0 = 16 * NJ * slice, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  chunk_gates(sG, sE, sW, p.g, u.row0, u.len, p.H, h, p.g_fixed);
  load_tile(sY, kLdP, p.y[back], u.row0, u.len, p.hy[back], head_of(h, p.H, p.hy[back]), p.ndk, m0, 64);
  load_tile(sZ, kLdP, p.z[back], u.row0, u.len, p.hz[back], head_of(h, p.H, p.hz[back]), p.ndv, c0, 16 * NJ);
  __syncthreads();
  const float *w = back ? sE : sW;
  for (int i = threadIdx.x; i < kC * 4 * NJ; i += kThreads) {
    const int r = i / (4 * NJ);
    float4 *z = reinterpret_cast<float4 *>(sZ + r * kLdP + (i - r * 4 * NJ) * 4);
    *z = make_float4(z->x * w[r], z->y * w[r], z->z * w[r], z->w * w[r]);
  }
  __syncthreads();
  const size_t at = (size_t)blockIdx.x * p.H + h;
  if (threadIdx.x == 0 && blockIdx.z == 0) p.decay[at] = sE[kC - 1];
  float acc[4][NJ];
  zero(acc);
  mm<NJ, false>(acc, sY, kLdP, sZ, kLdP, kC);
  float *out = p.own[back] + at * p.ndk * p.ndv + c0 + NJ * tx;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (m0 + 4 * ty + i < p.ndk && c0 + NJ * tx < p.ndv) put_row<NJ>(out + (size_t)(m0 + 4 * ty + i) * p.ndv, acc[i]);
}

// ---------------------------------------------------------------- walk over the chunks
// blockIdx: (sequence, head, direction x block of 4 x 128 entries); replaces each chunk's own state
// by the state before it (direction 1: after it).  keep: the end states also go to the spare slots.
struct ScanParams {
  float *own[2];
  const float *init[2];
  float *end[2];
  const float *decay;
  int H, elems, blocks, keep;
  Slots slots;
};
__global__ void __launch_bounds__(128) lin_scan_kernel(const ScanParams p) {
  if (p.slots.cu && *p.slots.status) return;
  const int n = blockIdx.x, h = blockIdx.y, back = blockIdx.z >= p.blocks;
  const int e = ((blockIdx.z - (back ? p.blocks : 0)) * 128 + threadIdx.x) * 4;
  if (e >= p.elems) return;
  float *const own = back ? p.own[1] : p.own[0];
  const float *const init = back ? p.init[1] : p.init[0];
  float *const end = back ? p.end[1] : p.end[0];
  const int len = p.slots.cu ? p.slots.cu[n + 1] - p.slots.cu[n] : p.slots.T;
  const int nc = pieces_of(len, kC);
  const long base = p.slots.base(n);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (init) S = *reinterpret_cast<const float4 *>(init + ((size_t)n * p.H + h) * p.elems + e);
  constexpr int kAhead = 4;
  for (int c0 = 0; c0 < nc; c0 += kAhead) {
    float4 d[kAhead];
    float a[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + u >= nc) continue;
      const size_t at = (size_t)(base + (back ? nc - 1 - c0 - u : c0 + u)) * p.H + h;
      d[u] = *reinterpret_cast<const float4 *>(own + at * p.elems + e);
      a[u] = p.decay[at];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + u >= nc) continue;
      const size_t at = (size_t)(base + (back ? nc - 1 - c0 - u : c0 + u)) * p.H + h;
      *reinterpret_cast<float4 *>(own + at * p.elems + e) = S;
      S.x = fmaf(a[u], S.x, d[u].x); S.y = fmaf(a[u], S.y, d[u].y);
      S.z = fmaf(a[u], S.z, d[u].z); S.w = fmaf(a[u], S.w, d[u].w);
    }
  }
  if (p.keep) *reinterpret_cast<float4 *>(own + ((size_t)(base + nc) * p.H + h) * p.elems + e) = S;
  if (end) *reinterpret_cast<float4 *>(end + ((size_t)n * p.H + h) * p.elems + e) = S;
}

// ---------------------------------------------------------------- outputs and gradients
struct SimtPass {
  const float *x, *y, *z, *w;  // w: partner of the row dots, or NULL
  int hx, hy, hz, hw, dx, dz;
  int rev, across;             // across: z channels are the state's rows (dq, dk), else its columns
  const float *state;          // [slots, H, dk, dv], or (one chunk a sequence) [N, H, dk, dv] or NULL
  float *out;                  // [rows, H, dz]
  float *dots;                 // [slices, H, rows]
  float *end;                  // one chunk a sequence: S_T
};
struct PassParams {
  SimtPass pass[3];
  const float *g;
  int *status;
  int H, g_fixed, elems, single, slices;
  long rows;
  Slots slots;
};
constexpr int kPassSmem = (3 * kTile + kTileP + 4 * kC) * 4;
constexpr int kSingleSmem = kPassSmem + kTile * 4;

// blockIdx: (slot, head, pass x slice of 16 NJ output columns)
template <int NJ>
__global__ void __launch_bounds__(kThreads) lin_pass_kernel(const PassParams p) {
  extern __shared__ __align__(16) float sm[];
  float *sX = sm, *sY = sX + kTile, *sZ = sY + kTile, *sP = sZ + kTile;
  float2 *sG = reinterpret_cast<float2 *>(sP + kTileP);
  float *sE = reinterpret_cast<float *>(sG + kC), *sW = sE + kC;
  float *sS = p.single ? sW + kC : sY;           // the state's rows, over Y once the scores are done
  if (p.single) clear_status(p.slots, p.status);
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int pi = blockIdx.z / p.slices;
  const SimtPass &ps = p.pass[pi];
  const int h = blockIdx.y, c0 = 16 * NJ * (blockIdx.z - pi * p.slices), tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (c0 >= ps.dz) return;
  chunk_gates(sG, sE, sW, p.g, u.row0, u.len, p.H, h, p.g_fixed);
  load_tile(sX, kLd, ps.x, u.row0, u.len, ps.hx, head_of(h, p.H, ps.hx), ps.dx, 0, ps.dx);
  load_tile(sY, kLd, ps.y, u.row0, u.len, ps.hy, head_of(h, p.H, ps.hy), ps.dx, 0, ps.dx);
  load_tile(sZ, kLd, ps.z, u.row0, u.len, ps.hz, head_of(h, p.H, ps.hz), ps.dz, c0, 16 * NJ);
  __syncthreads();
  {
    float acc[4][4];
    zero(acc);
    mm_scores(acc, sX, sY, ps.dx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * ty + i, c = tx + 16 * j;
        const float w = ps.rev ? pair_weight(sG[c], sG[r]) : pair_weight(sG[r], sG[c]);
        sP[r * kLdP + c] = (ps.rev ? c >= r && c < u.len : c <= r) ? acc[i][j] * w : 0.f;
      }
  }
  float acc[4][NJ];
  zero(acc);
  const float *S = ps.state;
  if (S) S += ((size_t)(p.single ? u.n : blockIdx.x) * p.H + h) * p.elems;
  for (int m0 = 0; S && m0 < ps.dx; m0 += 64) {    // rowf (x M): the state's x channels 64 at a time
    const int nr = min(64, ps.dx - m0);
    __syncthreads();                               // (sY's scores, or the rows before, are done)
    if (ps.across) {
      // [z][x] rows, transposed on the way: lanes take rows, so the stores are free of conflicts
      for (int i = tid; i < 16 * NJ * (nr / 4); i += kThreads) {
        const int n = i % (16 * NJ), k = i / (16 * NJ) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + n < ps.dz) f = *reinterpret_cast<const float4 *>(S + (size_t)(c0 + n) * ps.dx + m0 + k);
        sS[k * kLd + n] = f.x; sS[(k + 1) * kLd + n] = f.y; sS[(k + 2) * kLd + n] = f.z; sS[(k + 3) * kLd + n] = f.w;
      }
    } else {
      for (int i = tid; i < nr * 4 * NJ; i += kThreads) {
        const int r = i / (4 * NJ), c = (i - r * 4 * NJ) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + c < ps.dz) f = *reinterpret_cast<const float4 *>(S + (size_t)(m0 + r) * ps.dz + c0 + c);
        *reinterpret_cast<float4 *>(sS + r * kLd + c) = f;
      }
    }
    __syncthreads();
    mm<NJ, true>(acc, sX + m0, kLd, sS, kLd, nr);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] *= (ps.rev ? sW : sE)[4 * ty + i];
  __syncthreads();                                 // (sP)
  mm<NJ, true>(acc, sP, kLdP, sZ, kLd, kC);
  const int col = c0 + NJ * tx;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (ps.out && r < u.len && col < ps.dz) put_row<NJ>(ps.out + ((size_t)(u.row0 + r) * p.H + h) * ps.dz + col, acc[i]);
    if (ps.dots) {                                 // over the 16 threads of a row, then the slices
      float d = 0.f;
      if (r < u.len && col < ps.dz) {
        const float *w = ps.w + ((size_t)(u.row0 + r) * ps.hw + head_of(h, p.H, ps.hw)) * ps.dz + col;
#pragma unroll
        for (int j = 0; j < NJ; ++j) d = fmaf(w[j], acc[i][j], d);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      if (tx == 0 && r < u.len)
        ps.dots[((size_t)(blockIdx.z - pi * p.slices) * p.H + h) * p.rows + u.row0 + r] = d;
    }
  }
  if (!p.single || !ps.end) return;
  // S_T = e^{G_C} S0 + sum_j e^{G_C - G_j} k_j v_j^T
  __syncthreads();
  for (int i = tid; i < kC * 4 * NJ; i += kThreads) {
    const int r = i / (4 * NJ);
    float4 *z = reinterpret_cast<float4 *>(sZ + r * kLd + (i - r * 4 * NJ) * 4);
    *z = make_float4(z->x * sW[r], z->y * sW[r], z->z * sW[r], z->w * sW[r]);
  }
  __syncthreads();
  float *end = ps.end + ((size_t)u.n * p.H + h) * p.elems;
  for (int m0 = 0; m0 < ps.dx; m0 += 64) {
    zero(acc);
    mm<NJ, false>(acc, sY + m0, kLd, sZ, kLd, kC);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m0 + 4 * ty + i;
      if (r >= ps.dx || col >= ps.dz) continue;
      if (S) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(sE[kC - 1], S[(size_t)r * ps.dz + col + j], acc[i][j]);
      }
      put_row<NJ>(end + (size_t)r * ps.dz + col, acc[i]);
    }
  }
}

// ---------------------------------------------------------------- decay gradients
// dg_t = e^{g_t} <S_{t-1}, R_t> = <S_out, X> + sum_{s >= t} (q_s . dq_s - k_s . dk_s) over a piece (a
// segment or chunk), S_out the state after it and X its gradient.  At the piece's first token that is
// <S_in, gradient of S_in>, which is known by itself: 0 for a sequence without S0, else the value that
// ends the piece before.  The sums of a long piece miss it by their rounding errors, and the difference
// is spread over the tokens by the size of what was summed (tied at both ends, a random walk keeps
// 1 / sqrt 3 of its error, and a common factor on all terms goes).  A token that keeps nothing of
// the state (e^{g_t} = 0) has no gradient.  One block per (piece, head).
__global__ void __launch_bounds__(256) lin_decay_kernel(const DecayParams p) {
  __shared__ double s_all[4][8], s_sum[8], s_abs[8];
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = (size_t)h * p.rows + u.row0, all_rows = (size_t)p.H * p.rows;
  auto term = [&](int i, double &x, double &size) {
    x = size = 0.0;
    for (int y = 0; i >= 0 && y < p.slices; ++y) {
      const float a = p.rho[y * all_rows + row + i], b = p.kappa[y * all_rows + row + i];
      x += (double)a - (double)b;
      size += (double)(fabsf(a) + fabsf(b));
    }
  };
  double t[4] = {0.0, 0.0, 0.0, 0.0};            // <S_out, X>, the same before the piece; sum, sum of sizes
  {
    const long slot = blockIdx.x;
    const bool first = u.piece == 0, tie = !first || p.has_S0;
    auto state = [&](const float *x, long s) { return reinterpret_cast<const float4 *>(x + ((size_t)s * p.H + h) * p.elems); };
    const float4 *S1 = state(p.S, slot + 1), *X1 = state(p.X, slot);
    const float4 *S0 = state(p.S, slot), *X0 = tie ? state(p.X, first ? slot + u.pieces : slot - 1) : X1;
#pragma unroll 4
    for (int e = tid; e < p.elems / 4; e += 256) {
      const float4 a = S1[e], b = X1[e], c = S0[e], d = X0[e];
      t[0] += (double)fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
      t[1] += (double)fmaf(c.x, d.x, fmaf(c.y, d.y, fmaf(c.z, d.z, c.w * d.w)));
    }
    if (!tie) t[1] = 0.0;
  }
  for (int i = tid; i < u.len; i += 256) {
    double x, size;
    term(i, x, size);
    t[2] += x;
    t[3] += size;
  }
#pragma unroll
  for (int y = 0; y < 4; ++y) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t[y] += __shfl_xor_sync(0xffffffffu, t[y], off);
    if (lane == 0) s_all[y][warp] = t[y];
  }
  __syncthreads();
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    t[y] = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) t[y] += s_all[y][w];
  }
  double run = t[0], runs = 0.0;                 // <S_out, X>; with what has been summed, and its size
  const double start = t[1], share = (start - (run + t[2])) / t[3];
  const bool tied = isfinite(share);             // (not where there is nothing to spread over, or no number)
  // 256 tokens at a time from the end; thread 0 takes the last of them
  for (int top = u.len; top > 0; top -= 256) {
    const int i = top - 1 - tid;
    double x, size;
    term(i, x, size);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, off), z = __shfl_up_sync(0xffffffffu, size, off);
      if (lane >= off) {
        x += y;
        size += z;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_sum[warp] = x;
      s_abs[warp] = size;
    }
    __syncthreads();
    double before = 0.0, befores = 0.0, all = 0.0, alls = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) {
        before += s_sum[w];
        befores += s_abs[w];
      }
      all += s_sum[w];
      alls += s_abs[w];
    }
    if (i >= 0) {
      const size_t at = (size_t)(u.row0 + i) * p.H + h;
      double d = run + before + x;
      if (tied) d = i == 0 ? start : d + share * (runs + befores + size);
      const float g = p.g[p.g_fixed ? (size_t)h : at];
      p.dg[at] = !isnan(g) && exp2_fixed(fixed_log2(g)) == 0.f ? 0.f : (float)d;
    }
    run += all;
    runs += alls;
  }
}

// ---------------------------------------------------------------- sums over shared heads, fixed decays
// out[row, hx, c] = sum over the H / Hx heads that read head hx, in order
template <typename T>
__global__ void lin_share_kernel(const float *__restrict__ part, T *__restrict__ out, long n, int H,
                                 int Hx, int d, const int *__restrict__ status) {
  if (*status) return;
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int r = H / Hx;
  const long c = i % d, rh = i / d;            // rh = row * Hx + hx; its first head is rh * r
  float s = 0.f;
  for (int j = 0; j < r; ++j) s += part[((size_t)rh * r + j) * d + c];
  out[i] = from_f32<T>(s);
}
// dg[h] = sum over rows of part[row, h], one block per head, fp64 sums in a fixed order
__global__ void __launch_bounds__(256) lin_fixed_kernel(const float *__restrict__ part,
                                                        float *__restrict__ dg, long rows, int H,
                                                        const int *__restrict__ status) {
  if (*status) return;
  __shared__ double s[256];
  double x = 0.0;
  for (long r = threadIdx.x; r < rows; r += 256) x += (double)part[r * H + blockIdx.x];
  s[threadIdx.x] = x;
  __syncthreads();
  for (int off = 128; off > 0; off >>= 1) {
    if (threadIdx.x < off) s[threadIdx.x] += s[threadIdx.x + off];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[blockIdx.x] = (float)s[0];
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Columns of an output that one block computes (16 NJ): 64, or 32 where that alone makes up for
// few chunks (two blocks an SM at most).
int slice_columns(long units, int d) { return d > 32 && units * (d / 64 + (d < 64)) >= 148 ? 64 : 32; }

// Workspace past the header: the slot table, decays, the chunks' states, and backwards the state
// gradients and what decay gradients, shared heads and fixed decays are summed from.
struct SimtLayout {
  long slots;
  bool single;              // one chunk a sequence, forward: no states in between
  int cols;                 // output columns of a block
  size_t table, decay, S, X, rho, kappa, pq, pk, pv, dg, total;
};
SimtLayout layout(bool packed, int N, int T, int B, int H, int Hq, int Hk, int Hv, int dk, int dv,
                  bool g_fixed, bool back) {
  SimtLayout L;
  const size_t rows = (size_t)B * T;
  L.slots = slot_count(packed, N, T, kC, 1);
  L.single = !packed && !back && T > 0 && T <= kC;
  const int most = dk > dv ? dk : dv;
  L.cols = slice_columns(((long)T / kC + 1) * (packed ? 1 : B) * H * (back ? 3 : 1), back ? most : dv);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += round256(bytes); return r; };
  const size_t states = L.single ? 0 : (size_t)L.slots * H * dk * dv * 4, slices = (dk + L.cols - 1) / L.cols;
  L.table = take(packed ? (size_t)L.slots * 4 : 0);
  L.decay = take(L.single ? 0 : (size_t)L.slots * H * 4);
  L.S = take(states);
  L.X = take(back ? states : 0);
  L.rho = take(back ? slices * rows * H * 4 : 0);
  L.kappa = take(back ? slices * rows * H * 4 : 0);
  L.pq = take(back && Hq < H ? rows * H * dk * 4 : 0);
  L.pk = take(back && Hk < H ? rows * H * dk * 4 : 0);
  L.pv = take(back && Hv < H ? rows * H * dv * 4 : 0);
  L.dg = take(back && g_fixed ? rows * H * 4 : 0);
  L.total = at;
  return L;
}

template <int NJ>
int run_cols(const LinArgs &a, const LinBwdArgs *b, const SimtLayout &L, cudaStream_t s) {
  const int elems = a.dk * a.dv;
  const unsigned slots = (unsigned)L.slots, H = (unsigned)a.H;
  float *S = reinterpret_cast<float *>(a.ws + L.S), *X = reinterpret_cast<float *>(a.ws + L.X);
  const Slots sl{a.cu, reinterpret_cast<const int *>(a.ws + L.table), a.status, a.N, a.T, kC, 1};
  const long rows = (long)a.B * a.T;
  auto f32 = [](const void *p) { return static_cast<const float *>(p); };
  if (a.cu) {
    const PlanTable t{reinterpret_cast<int *>(a.ws + L.table), kC, 1, L.slots};
    const int rc = launch_plan(a.cu, a.N, a.T, t, a.status, s);
    if (rc != CKDA_OK) return rc;
  }
  if (!L.single) {
    LocalParams l = {};
    l.y[0] = f32(a.k); l.z[0] = f32(a.v); l.hy[0] = a.Hk; l.hz[0] = a.Hv; l.own[0] = S;
    if (b) {
      l.y[1] = f32(a.q); l.z[1] = f32(b->dO); l.hy[1] = a.Hq; l.hz[1] = a.H; l.own[1] = X;
    }
    l.g = a.g; l.decay = reinterpret_cast<float *>(a.ws + L.decay); l.status = a.status;
    l.H = a.H; l.ndk = a.dk; l.ndv = a.dv; l.g_fixed = a.g_fixed; l.cols = (a.dv + 16 * NJ - 1) / (16 * NJ); l.slots = sl;
    const dim3 grid(slots, H, (unsigned)(l.cols * ((a.dk + 63) / 64) * (b ? 2 : 1)));
    if (slots > 0) lin_local_kernel<NJ><<<grid, kThreads, 0, s>>>(l);
    ScanParams c = {};
    c.own[0] = S; c.own[1] = X;
    c.init[0] = a.S0; c.init[1] = b ? b->dS_T : nullptr;
    c.end[0] = a.S_T; c.end[1] = b ? b->dS0 : nullptr;
    c.decay = l.decay; c.H = a.H; c.elems = elems; c.blocks = (elems / 4 + 127) / 128; c.keep = b != nullptr; c.slots = sl;
    lin_scan_kernel<<<dim3((unsigned)a.N, H, (unsigned)(c.blocks * (b ? 2 : 1))), 128, 0, s>>>(c);
  }
  if (rows == 0 || (!b && !a.o && !L.single)) return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
  const int smem = L.single ? kSingleSmem : kPassSmem;
  if (cudaFuncSetAttribute(lin_pass_kernel<NJ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return CKDA_ERR_CUDA;
  PassParams p = {};
  p.g = a.g; p.status = a.status; p.H = a.H; p.g_fixed = a.g_fixed; p.elems = elems; p.single = L.single; p.rows = rows;
  p.slots = sl;
  if (!b) {
    p.pass[0] = SimtPass{f32(a.q), f32(a.k), f32(a.v), nullptr, a.Hq, a.Hk, a.Hv, 0, a.dk, a.dv, 0, 0,
                         L.single ? a.S0 : S, static_cast<float *>(a.o), nullptr, L.single ? a.S_T : nullptr};
    p.slices = (a.dv + 16 * NJ - 1) / (16 * NJ);
    lin_pass_kernel<NJ><<<dim3(slots, H, (unsigned)p.slices), kThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
  }
  const bool part_q = a.Hq < a.H, part_k = a.Hk < a.H, part_v = a.Hv < a.H;
  float *rho = reinterpret_cast<float *>(a.ws + L.rho), *kappa = reinterpret_cast<float *>(a.ws + L.kappa);
  float *pq = part_q ? reinterpret_cast<float *>(a.ws + L.pq) : static_cast<float *>(b->dq);
  float *pk = part_k ? reinterpret_cast<float *>(a.ws + L.pk) : static_cast<float *>(b->dk);
  float *pv = part_v ? reinterpret_cast<float *>(a.ws + L.pv) : static_cast<float *>(b->dv);
  const float *q = f32(a.q), *k = f32(a.k), *v = f32(a.v), *dO = f32(b->dO);
  p.pass[0] = SimtPass{dO, v, k, q, a.H, a.Hv, a.Hk, a.Hq, a.dv, a.dk, 0, 1, S, pq, rho, nullptr};
  p.pass[1] = SimtPass{v, dO, q, k, a.Hv, a.H, a.Hq, a.Hk, a.dv, a.dk, 1, 1, X, pk, kappa, nullptr};
  p.pass[2] = SimtPass{k, q, dO, nullptr, a.Hk, a.Hq, a.H, 0, a.dk, a.dv, 1, 0, X, pv, nullptr, nullptr};
  const int most = a.dk > a.dv ? a.dk : a.dv;
  p.slices = (most + 16 * NJ - 1) / (16 * NJ);
  lin_pass_kernel<NJ><<<dim3(slots, H, (unsigned)(3 * p.slices)), kThreads, smem, s>>>(p);
  DecayParams d = {};
  d.S = S; d.X = X; d.rho = rho; d.kappa = kappa; d.g = a.g; d.g_fixed = a.g_fixed; d.has_S0 = a.S0 != nullptr; d.slices = (a.dk + 16 * NJ - 1) / (16 * NJ);
  d.dg = a.g_fixed ? reinterpret_cast<float *>(a.ws + L.dg) : b->dg;
  d.H = a.H; d.elems = elems; d.rows = rows; d.slots = sl;
  launch_decay(d, L.slots, s);
  if (part_q) launch_share(pq, b->dq, rows, a.H, a.Hq, a.dk, false, a.status, s);
  if (part_k) launch_share(pk, b->dk, rows, a.H, a.Hk, a.dk, false, a.status, s);
  if (part_v) launch_share(pv, b->dv, rows, a.H, a.Hv, a.dv, false, a.status, s);
  if (a.g_fixed) launch_fixed(d.dg, b->dg, rows, a.H, a.status, s);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
int run_simt(const LinArgs &a, const LinBwdArgs *b, cudaStream_t s) {
  const SimtLayout L = layout(a.cu != nullptr, a.N, a.T, a.B, a.H, a.Hq, a.Hk, a.Hv, a.dk, a.dv, a.g_fixed, b != nullptr);
  return L.cols == 64 ? run_cols<4>(a, b, L, s) : run_cols<2>(a, b, L, s);
}

// ---------------------------------------------------------------- packed batches
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t *cu, int N, int T, PlanTable t, int *status) {
  bool bad = false;
  for (int n = threadIdx.x; n < N; n += 1024) {
    const int s = cu[n], e = cu[n + 1];
    bad |= s < 0 || e < s || e > T || (n == 0 && s != 0) || (n == N - 1 && e != T);
  }
  const bool any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = any ? CKDA_ERR_SEQLENS : CKDA_OK;
  if (any) return;
  const Slots s{cu, nullptr, nullptr, N, T, t.L, t.spare};
  for (int n = threadIdx.x; n < N; n += 1024) {
    const long b = s.base(n), next = n + 1 < N ? s.base(n + 1) : t.count;
    const int pieces = pieces_of(cu[n + 1] - cu[n], t.L);
    for (long i = b; i < next; ++i) t.table[i] = i - b < pieces ? n : -1;
  }
}

}  // namespace

void launch_decay(const DecayParams &p, long slots, cudaStream_t s) {
  lin_decay_kernel<<<dim3((unsigned)slots, (unsigned)p.H), 256, 0, s>>>(p);
}
void launch_share(const void *part, void *out, long rows, int H, int Hx, int d, bool bf16,
                  const int *status, cudaStream_t s) {
  const long n = rows * Hx * d;
  if (n == 0) return;
  const unsigned grid = (unsigned)((n + 255) / 256);
  const float *in = static_cast<const float *>(part);
  if (bf16)
    lin_share_kernel<<<grid, 256, 0, s>>>(in, static_cast<__nv_bfloat16 *>(out), n, H, Hx, d, status);
  else
    lin_share_kernel<<<grid, 256, 0, s>>>(in, static_cast<float *>(out), n, H, Hx, d, status);
}
void launch_fixed(const float *part, float *dg, long rows, int H, const int *status, cudaStream_t s) {
  lin_fixed_kernel<<<H, 256, 0, s>>>(part, dg, rows, H, status);
}

int launch_plan(const int32_t *cu, int N, int T, const PlanTable &t, int *status, cudaStream_t s) {
  plan_kernel<<<1, 1024, 0, s>>>(cu, N, T, t, status);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // namespace lin

// fp32 inputs run in exact fp32 on CUDA cores, bf16 ones on the tensor cores.
size_t linattn_fwd_workspace(int B, int T, int H, int dk, int dv, int N, bool packed, int io_dtype) {
  if (io_dtype == CKDA_BF16) return lin::tc_workspace(packed, N, B, T, H, H, H, H, dk, dv, false, false);
  return lin::layout(packed, N, T, B, H, H, H, H, dk, dv, false, false).total;
}
size_t linattn_bwd_workspace(const LinArgs &a, bool packed) {
  if (a.io_dtype == CKDA_BF16)
    return lin::tc_workspace(packed, a.N, a.B, a.T, a.H, a.Hq, a.Hk, a.Hv, a.dk, a.dv, a.g_fixed, true);
  return lin::layout(packed, a.N, a.T, a.B, a.H, a.Hq, a.Hk, a.Hv, a.dk, a.dv, a.g_fixed, true).total;
}
int launch_linattn_fwd(const LinArgs &a, cudaStream_t s) {
  return a.io_dtype == CKDA_BF16 ? lin::launch_tc(a, nullptr, s) : lin::run_simt(a, nullptr, s);
}
int launch_linattn_bwd(const LinBwdArgs &b, cudaStream_t s) {
  return b.f.io_dtype == CKDA_BF16 ? lin::launch_tc(b.f, &b, s) : lin::run_simt(b.f, &b, s);
}

}  // namespace ckda
