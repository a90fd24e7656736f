// linattn_simt.cu -- linear attention with a decay for each head in exact fp32 on CUDA cores:
// forward and gradients, chunks of 64 tokens, three launches each way.
//
//   1. lin_local_kernel: every chunk's own state  sum_j e^{G_C - G_j} k_j v_j^T  (and, backwards,
//      its own state gradient  sum_i e^{G_i} q_i dO_i^T), all chunks side by side;
//   2. lin_scan_kernel: the walk over a sequence's chunks, S <- e^{G_C} S + own, elementwise:
//      one thread per four state entries, the next chunks' loads in flight;
//   3. lin_out_kernel / lin_grad_kernel: outputs or gradients of every chunk from the state it
//      starts with (and the state gradient it ends with), all chunks side by side.
//
// Gradients: with X the gradient with respect to the state after the chunk,
//   dq_i = e^{G_i} S_in dO_i + sum_{j <= i} e^{G_i - G_j} (dO_i . v_j) k_j
//   dk_j = e^{G_C - G_j} X v_j + sum_{i >= j} e^{G_i - G_j} (dO_i . v_j) q_i
//   dv_j = e^{G_C - G_j} X^T k_j + sum_{i >= j} e^{G_i - G_j} (q_i . k_j) dO_i
//   dg_t = <S_out, X> + sum_{s >= t, s in the chunk} (q_s . dq_s - k_s . dk_s)
// The last follows from each G_i's derivative: outputs and gradients are sums of terms
// e^{G_a - G_b}, the q side carrying +G and the k side -G.
//
// Bound: fp32 FMA and shared-memory loads (64 x d x d products per chunk and head); the states
// between chunks add 64 KB written and read three times per 64 tokens at d = 128.
#include "linattn_common.cuh"

namespace ckda {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kLd = 132;     // row stride of a 64 x 128 fp32 tile: 16-byte rows, banks shifted by 4
constexpr int kLdP = 68;     // of a 64 x 64 one
constexpr int kTile = kC * kLd;
constexpr int kTileP = kC * kLdP;

struct ChunkParams {
  const void *q, *k, *v, *dO;
  const float *g;
  float *own_S, *own_X;      // [slots, H, dk, dv]: chunks' own states, then states at the borders
  float *decay;              // [slots, H]: e^{G_C}
  void *o;
  float *dq, *dk, *dv;       // gradients, or per-head shares of them (shared heads)
  float *dg;                 // [rows, H]
  int part_q, part_k, part_v;
  int H, Hq, Hk, Hv, ndk, ndv, g_fixed;
  Slots slots;
};

// Loads rows [0, len) of head `hx` of x [rows, Hx, d] into a 64 x 128 fp32 tile, zeros elsewhere.
__device__ void load_tile(float *t, const void *x, long row0, int len, int Hx, int hx, int d) {
  const float *src = static_cast<const float *>(x) + ((size_t)row0 * Hx + hx) * d;
  for (int i = threadIdx.x; i < kC * 32; i += kThreads) {
    const int r = i >> 5, c = (i & 31) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x && r < len && c < d) {
      f = *reinterpret_cast<const float4 *>(src + (size_t)r * Hx * d + c);
    }
    *reinterpret_cast<float4 *>(t + r * kLd + c) = f;
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
// e^{G_i} to sE and e^{G_C - G_i} to sW.  One warp; the caller synchronises.
__device__ void chunk_gates(float2 *sG, float *sE, float *sW, const float *g, long row0, int len,
                            int H, int h, int g_fixed) {
  const int lane = threadIdx.x;
  if (lane >= 32) return;
  long long x[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * lane + u;
    x[u] = i < len ? fixed_log2(g[g_fixed ? (size_t)h : (size_t)(row0 + i) * H + h]) : 0;
  }
  const long long sum = scan_pairs(x[0], x[1]);
  const long long all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = 2 * lane + u;
    const long long G = u ? sum : sum - x[1];
    sG[i] = split_sum(G);
    sE[i] = exp2_fixed(G);
    sW[i] = i < len ? exp2_fixed(all - G) : 0.f;
  }
}

// acc[4][NJ] += A (64 x K) B (K x 16 NJ) for this thread's rows 4 ty .. 4 ty + 3.  KC: the
// operand is stored [row][k] (k contiguous); else [k][row].  Columns: tx + 16 j with a KC B,
// 4 tx + 64 (j / 4) + j % 4 otherwise (both free of bank conflicts).
template <int NJ, bool AKC, bool BKC>
__device__ __forceinline__ void mm(float (&acc)[4][NJ], const float *A, int lda, const float *B,
                                   int ldb, int K, int jmax) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
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
    }
    if (BKC) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < jmax) f = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * ldb + k);
        b[0][j] = f.x; b[1][j] = f.y; b[2][j] = f.z; b[3][j] = f.w;
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(B + (k + kk) * ldb + 4 * tx + 16 * j);
          b[kk][j] = f.x; b[kk][j + 1] = f.y; b[kk][j + 2] = f.z; b[kk][j + 3] = f.w;
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
template <int NJ>
__device__ __forceinline__ void zero(float (&acc)[4][NJ]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
}
// column of acc[.][j]
template <bool BKC>
__device__ __forceinline__ int col_of(int j) {
  const int tx = threadIdx.x & 15;
  return BKC ? tx + 16 * j : 4 * tx + 64 * (j >> 2) + (j & 3);
}

// ---------------------------------------------------------------- chunks' own states
// blockIdx: (slot, head, direction); direction 1: own_X from q, dO with weights e^{G_i}.
__global__ void __launch_bounds__(kThreads) lin_local_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) float sm[];
  float *sY = sm, *sZ = sm + kTile;
  float2 *sG = reinterpret_cast<float2 *>(sZ + kTile);
  float *sE = reinterpret_cast<float *>(sG + kC), *sW = sE + kC;
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, back = blockIdx.z;
  chunk_gates(sG, sE, sW, p.g, u.row0, u.len, p.H, h, p.g_fixed);
  const int Hy = back ? p.Hq : p.Hk, Hz = back ? p.H : p.Hv;
  load_tile(sY, back ? p.q : p.k, u.row0, u.len, Hy, h * Hy / p.H, p.ndk);
  load_tile(sZ, back ? p.dO : p.v, u.row0, u.len, Hz, h * Hz / p.H, p.ndv);
  __syncthreads();
  const float *w = back ? sE : sW;
  for (int i = threadIdx.x; i < kC * 32; i += kThreads) {
    const int r = i >> 5, c = (i & 31) * 4;
    float4 *z = reinterpret_cast<float4 *>(sZ + r * kLd + c);
    const float s = r < u.len ? w[r] : 0.f;
    *z = make_float4(z->x * s, z->y * s, z->z * s, z->w * s);
  }
  __syncthreads();
  const size_t at = (size_t)blockIdx.x * p.H + h;
  if (threadIdx.x == 0 && !back) p.decay[at] = sE[kC - 1];
  float *out = (back ? p.own_X : p.own_S) + at * p.ndk * p.ndv;
  const int ty = threadIdx.x >> 4;
  for (int m0 = 0; m0 < p.ndk; m0 += 64) {
    float acc[4][8];
    zero(acc);
    mm<8, false, false>(acc, sY + m0, kLd, sZ, kLd, kC, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m0 + 4 * ty + i;
      if (r >= p.ndk) continue;
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const int c = col_of<false>(j);
        if (c < p.ndv)
          *reinterpret_cast<float4 *>(out + (size_t)r * p.ndv + c) =
              make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
      }
    }
  }
}

// ---------------------------------------------------------------- walk over the chunks
// blockIdx: (sequence, head, block of 4 x 128 entries); replaces each chunk's own state by the
// state before it (back: after it).  keep_end: the end state also goes to the spare slot.
struct ScanParams {
  float *own;
  const float *decay, *init;
  float *end;
  int H, elems, back, keep_end;
  Slots slots;
};
__global__ void __launch_bounds__(128) lin_scan_kernel(const ScanParams p) {
  if (p.slots.cu && *p.slots.status) return;
  const int n = blockIdx.x, h = blockIdx.y;
  const int e = (blockIdx.z * 128 + threadIdx.x) * 4;
  if (e >= p.elems) return;
  const int len = p.slots.cu ? p.slots.cu[n + 1] - p.slots.cu[n] : p.slots.T;
  const int nc = (len + kC - 1) / kC;
  const long base = p.slots.base(n);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.init) S = *reinterpret_cast<const float4 *>(p.init + ((size_t)n * p.H + h) * p.elems + e);
  constexpr int kAhead = 4;
  for (int c0 = 0; c0 < nc; c0 += kAhead) {
    float4 d[kAhead];
    float a[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + u >= nc) continue;
      const size_t at = (size_t)(base + (p.back ? nc - 1 - c0 - u : c0 + u)) * p.H + h;
      d[u] = *reinterpret_cast<const float4 *>(p.own + at * p.elems + e);
      a[u] = p.decay[at];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (c0 + u >= nc) continue;
      const size_t at = (size_t)(base + (p.back ? nc - 1 - c0 - u : c0 + u)) * p.H + h;
      *reinterpret_cast<float4 *>(p.own + at * p.elems + e) = S;
      S.x = fmaf(a[u], S.x, d[u].x); S.y = fmaf(a[u], S.y, d[u].y);
      S.z = fmaf(a[u], S.z, d[u].z); S.w = fmaf(a[u], S.w, d[u].w);
    }
  }
  if (p.keep_end) *reinterpret_cast<float4 *>(p.own + ((size_t)(base + nc) * p.H + h) * p.elems + e) = S;
  if (p.end) *reinterpret_cast<float4 *>(p.end + ((size_t)n * p.H + h) * p.elems + e) = S;
}

// Copies rows [r0, r0 + 64) x all columns of a [R][Cc] state into a tile (zeros outside).
__device__ void load_state(float *t, const float *S, int r0, int R, int Cc) {
  for (int i = threadIdx.x; i < 64 * 32; i += kThreads) {
    const int r = i >> 5, c = (i & 31) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < R && c < Cc) f = *reinterpret_cast<const float4 *>(S + (size_t)(r0 + r) * Cc + c);
    *reinterpret_cast<float4 *>(t + r * kLd + c) = f;
  }
}

// P[i][j] = acc o 2^{G_i - G_j} for j <= i (columns of a KC product), 0 above the diagonal.
__device__ __forceinline__ void store_scores(float *P, const float (&acc)[4][4], const float2 *sG) {
  const int ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * ty + i, c = col_of<true>(j);
      P[r * kLdP + c] = c <= r ? acc[i][j] * pair_weight(sG[r], sG[c]) : 0.f;
    }
}

// ---------------------------------------------------------------- outputs
__global__ void __launch_bounds__(kThreads) lin_out_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sK = sQ + kTile, *sV = sK + kTile, *sP = sV + kTile;
  float2 *sG = reinterpret_cast<float2 *>(sP + kTileP);
  float *sE = reinterpret_cast<float *>(sG + kC), *sW = sE + kC;
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, ty = threadIdx.x >> 4;
  chunk_gates(sG, sE, sW, p.g, u.row0, u.len, p.H, h, p.g_fixed);
  load_tile(sQ, p.q, u.row0, u.len, p.Hq, h * p.Hq / p.H, p.ndk);
  load_tile(sK, p.k, u.row0, u.len, p.Hk, h * p.Hk / p.H, p.ndk);
  load_tile(sV, p.v, u.row0, u.len, p.Hv, h * p.Hv / p.H, p.ndv);
  __syncthreads();
  {
    float acc[4][4];
    zero(acc);
    mm<4, true, true>(acc, sQ, kLd, sK, kLd, p.ndk, 4);
    store_scores(sP, acc, sG);
  }
  float acc[4][8];
  zero(acc);
  const float *S = p.own_S + ((size_t)blockIdx.x * p.H + h) * p.ndk * p.ndv;
  for (int m0 = 0; m0 < p.ndk; m0 += 64) {      // e^{G} (q S), the state's rows 64 at a time
    __syncthreads();                            // (sK's scores are done)
    load_state(sK, S, m0, p.ndk, p.ndv);
    __syncthreads();
    mm<8, true, false>(acc, sQ + m0, kLd, sK, kLd, min(64, p.ndk - m0), 8);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] *= sE[4 * ty + i];
  mm<8, true, false>(acc, sP, kLdP, sV, kLd, kC, 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= u.len) continue;
    float *o = static_cast<float *>(p.o) + ((size_t)(u.row0 + r) * p.H + h) * p.ndv;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col_of<false>(j) < p.ndv) o[col_of<false>(j)] = acc[i][j];
  }
}

// ---------------------------------------------------------------- gradients
// Writes one gradient, or this head's share of it (part).  Columns of an NC product.
__device__ __forceinline__ void store_grad(float *out, int part, const float (&acc)[4][8], const Piece &u,
                                           int Hx, int H, int h, int d) {
  const int ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= u.len) continue;
    const size_t off = part ? ((size_t)(u.row0 + r) * H + h) * d
                            : ((size_t)(u.row0 + r) * Hx + h) * d;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = col_of<false>(j);
      if (c >= d) continue;
      out[off + c] = acc[i][j];
    }
  }
}
// rows' dot products x_r . acc_r, summed over the 16 threads of a row, added to s[r] * sign
__device__ __forceinline__ void row_dots(float *s, const float *X, const float (&acc)[4][8], float sign) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) d = fmaf(X[(4 * ty + i) * kLd + col_of<false>(j)], acc[i][j], d);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (tx == 0) s[4 * ty + i] += sign * d;
  }
}

__global__ void __launch_bounds__(kThreads) lin_grad_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sK = sQ + kTile, *sV = sK + kTile, *sD = sV + kTile, *sS = sD + kTile;
  float *sP = sS + kTile;                      // scores' gradients, then scores
  float2 *sG = reinterpret_cast<float2 *>(sP + kTileP);
  float *sE = reinterpret_cast<float *>(sG + kC), *sW = sE + kC, *sR = sW + kC;
  __shared__ float s_red[kThreads / 32];
  Piece u;
  if (!find_piece(p.slots, blockIdx.x, u)) return;
  const int h = blockIdx.y, tid = threadIdx.x, ty = tid >> 4;
  const int dk = p.ndk, dv = p.ndv;
  chunk_gates(sG, sE, sW, p.g, u.row0, u.len, p.H, h, p.g_fixed);
  if (tid < kC) sR[tid] = 0.f;
  load_tile(sQ, p.q, u.row0, u.len, p.Hq, h * p.Hq / p.H, dk);
  load_tile(sK, p.k, u.row0, u.len, p.Hk, h * p.Hk / p.H, dk);
  load_tile(sV, p.v, u.row0, u.len, p.Hv, h * p.Hv / p.H, dv);
  load_tile(sD, p.dO, u.row0, u.len, p.H, h, dv);
  const size_t elems = (size_t)dk * dv;
  const float *S = p.own_S + ((size_t)blockIdx.x * p.H + h) * elems;
  const float *S_out = p.own_S + ((size_t)(blockIdx.x + 1) * p.H + h) * elems;
  const float *X = p.own_X + ((size_t)blockIdx.x * p.H + h) * elems;
  // <S_out, X>, the part of dg that every token of the chunk shares
  float dot = 0.f;
  for (size_t e = tid; e < elems; e += kThreads) dot = fmaf(S_out[e], X[e], dot);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  if ((tid & 31) == 0) s_red[tid >> 5] = dot;
  __syncthreads();
  {
    float acc[4][4];
    zero(acc);
    mm<4, true, true>(acc, sD, kLd, sV, kLd, dv, 4);
    store_scores(sP, acc, sG);
  }
  float acc[4][8];
  // dq: dO S^T (column n = key channel, 64 state rows at a time), then the chunk's own part
  zero(acc);
  for (int m0 = 0; m0 < dk; m0 += 64) {
    __syncthreads();
    load_state(sS, S, m0, dk, dv);
    __syncthreads();
    float part[4][4];
    zero(part);
    mm<4, true, true>(part, sD, kLd, sS, kLd, dv, 4);
    // columns m0 + tx + 16 j go through shared memory to the NC layout of acc
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sS[(4 * ty + i) * kLd + col_of<true>(j)] = part[i][j] * sE[4 * ty + i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m0 == 0) acc[i][j] = sS[(4 * ty + i) * kLd + 4 * (tid & 15) + j];
        else acc[i][4 + j] = sS[(4 * ty + i) * kLd + 4 * (tid & 15) + j];
  }
  mm<8, true, false>(acc, sP, kLdP, sK, kLd, kC, 8);
  row_dots(sR, sQ, acc, 1.f);
  store_grad(p.dq, p.part_q, acc, u, p.Hq, p.H, h, dk);
  // dk: X v_j likewise
  zero(acc);
  for (int m0 = 0; m0 < dk; m0 += 64) {
    __syncthreads();
    load_state(sS, X, m0, dk, dv);
    __syncthreads();
    float part[4][4];
    zero(part);
    mm<4, true, true>(part, sV, kLd, sS, kLd, dv, 4);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sS[(4 * ty + i) * kLd + col_of<true>(j)] = part[i][j] * sW[4 * ty + i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m0 == 0) acc[i][j] = sS[(4 * ty + i) * kLd + 4 * (tid & 15) + j];
        else acc[i][4 + j] = sS[(4 * ty + i) * kLd + 4 * (tid & 15) + j];
  }
  mm<8, false, false>(acc, sP, kLdP, sQ, kLd, kC, 8);
  row_dots(sR, sK, acc, -1.f);
  store_grad(p.dk, p.part_k, acc, u, p.Hk, p.H, h, dk);
  __syncthreads();                            // the scores' gradients and sR are done
  {
    float sc[4][4];
    zero(sc);
    mm<4, true, true>(sc, sQ, kLd, sK, kLd, dk, 4);
    store_scores(sP, sc, sG);
  }
  // dv: X^T k_j, state rows 64 at a time, then the chunk's own part
  zero(acc);
  for (int m0 = 0; m0 < dk; m0 += 64) {
    __syncthreads();
    load_state(sS, X, m0, dk, dv);
    __syncthreads();
    mm<8, true, false>(acc, sK + m0, kLd, sS, kLd, min(64, dk - m0), 8);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] *= sW[4 * ty + i];
  mm<8, false, false>(acc, sP, kLdP, sD, kLd, kC, 8);
  store_grad(p.dv, p.part_v, acc, u, p.Hv, p.H, h, dv);
  // dg: suffix sums within the chunk (two rows per lane, from the end)
  if (tid < 32) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += s_red[w];
    const int i1 = kC - 1 - 2 * tid, i0 = i1 - 1;
    const float r1 = sR[i1], r0 = sR[i0];
    float sum = r0 + r1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, sum, off);
      if (tid >= off) sum += y;
    }
    if (i0 < u.len) p.dg[(size_t)(u.row0 + i0) * p.H + h] = all + sum;
    if (i1 < u.len) p.dg[(size_t)(u.row0 + i1) * p.H + h] = all + (sum - r0);
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

// Workspace past the header: the slot table, decays, the chunks' states, and backwards the state
// gradients and what shared heads and fixed decays sum over.
struct SimtLayout {
  long slots;
  size_t table, decay, S, X, pq, pk, pv, dg, total;
};
SimtLayout layout(bool packed, int N, int T, int B, int H, int Hq, int Hk, int Hv, int dk, int dv,
                  bool g_fixed, bool back) {
  SimtLayout L;
  const size_t rows = (size_t)B * T;
  L.slots = slot_count(packed, N, T, kC, 1);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t r = at; at += round256(bytes); return r; };
  L.table = take(packed ? (size_t)L.slots * 4 : 0);
  L.decay = take((size_t)L.slots * H * 4);
  L.S = take((size_t)L.slots * H * dk * dv * 4);
  L.X = take(back ? (size_t)L.slots * H * dk * dv * 4 : 0);
  L.pq = take(back && Hq < H ? rows * H * dk * 4 : 0);
  L.pk = take(back && Hk < H ? rows * H * dk * 4 : 0);
  L.pv = take(back && Hv < H ? rows * H * dv * 4 : 0);
  L.dg = take(back && g_fixed ? rows * H * 4 : 0);
  L.total = at;
  return L;
}

constexpr int kLocalSmem = (2 * kTile + 4 * kC) * 4;
constexpr int kOutSmem = (3 * kTile + kTileP + 4 * kC) * 4;
constexpr int kGradSmem = (5 * kTile + kTileP + 5 * kC) * 4;

template <typename K>
bool set_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

int run_simt(const LinArgs &a, const LinBwdArgs *b, cudaStream_t s) {
  const SimtLayout L = layout(a.cu != nullptr, a.N, a.T, a.B, a.H, a.Hq, a.Hk, a.Hv, a.dk, a.dv,
                              a.g_fixed, b != nullptr);
  ChunkParams p = {};
  p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.o = a.o;
  p.own_S = reinterpret_cast<float *>(a.ws + L.S);
  p.own_X = reinterpret_cast<float *>(a.ws + L.X);
  p.decay = reinterpret_cast<float *>(a.ws + L.decay);
  p.H = a.H; p.Hq = a.Hq; p.Hk = a.Hk; p.Hv = a.Hv; p.ndk = a.dk; p.ndv = a.dv; p.g_fixed = a.g_fixed;
  p.slots = Slots{a.cu, reinterpret_cast<const int *>(a.ws + L.table), a.status, a.N, a.T, kC, 1};
  if (a.cu) {
    const PlanTable t{reinterpret_cast<int *>(a.ws + L.table), kC, 1, L.slots};
    const int rc = launch_plan(a.cu, a.N, a.T, &t, 1, a.status, s);
    if (rc != CKDA_OK) return rc;
  }
  if (b) {
    p.dO = b->dO;
    p.part_q = a.Hq < a.H; p.part_k = a.Hk < a.H; p.part_v = a.Hv < a.H;
    p.dq = p.part_q ? reinterpret_cast<float *>(a.ws + L.pq) : static_cast<float *>(b->dq);
    p.dk = p.part_k ? reinterpret_cast<float *>(a.ws + L.pk) : static_cast<float *>(b->dk);
    p.dv = p.part_v ? reinterpret_cast<float *>(a.ws + L.pv) : static_cast<float *>(b->dv);
    p.dg = a.g_fixed ? reinterpret_cast<float *>(a.ws + L.dg) : b->dg;
  }
  const dim3 grid((unsigned)L.slots, (unsigned)a.H, b ? 2 : 1);
  const int elems = a.dk * a.dv;
  const dim3 scan((unsigned)a.N, (unsigned)a.H, (unsigned)((elems / 4 + 127) / 128));
  if (!set_smem(lin_local_kernel, kLocalSmem) || !set_smem(lin_out_kernel, kOutSmem) ||
      !set_smem(lin_grad_kernel, kGradSmem))
    return CKDA_ERR_CUDA;
  if (grid.x > 0) lin_local_kernel<<<grid, kThreads, kLocalSmem, s>>>(p);
  ScanParams f{p.own_S, p.decay, a.S0, a.S_T, a.H, elems, 0, b != nullptr, p.slots};
  lin_scan_kernel<<<scan, 128, 0, s>>>(f);
  if (b) {
    ScanParams r{p.own_X, p.decay, b->dS_T, b->dS0, a.H, elems, 1, 0, p.slots};
    lin_scan_kernel<<<scan, 128, 0, s>>>(r);
  }
  const dim3 flat(grid.x, grid.y);
  if (grid.x > 0 && !b && a.o) lin_out_kernel<<<flat, kThreads, kOutSmem, s>>>(p);
  if (b) {
    const long rows = (long)a.B * a.T;
    if (grid.x > 0) lin_grad_kernel<<<flat, kThreads, kGradSmem, s>>>(p);
    if (p.part_q) launch_share(p.dq, b->dq, rows, a.H, a.Hq, a.dk, false, a.status, s);
    if (p.part_k) launch_share(p.dk, b->dk, rows, a.H, a.Hk, a.dk, false, a.status, s);
    if (p.part_v) launch_share(p.dv, b->dv, rows, a.H, a.Hv, a.dv, false, a.status, s);
    if (a.g_fixed) launch_fixed(p.dg, b->dg, rows, a.H, a.status, s);
  }
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

// ---------------------------------------------------------------- packed batches
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t *cu, int N, int T, PlanTable t0,
                                                    PlanTable t1, int *status) {
  bool bad = false;
  for (int n = threadIdx.x; n < N; n += 1024) {
    const int s = cu[n], e = cu[n + 1];
    bad |= s < 0 || e < s || e > T || (n == 0 && s != 0) || (n == N - 1 && e != T);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) *status = CKDA_ERR_SEQLENS;
    return;
  }
  for (int x = 0; x < 2; ++x) {
    const PlanTable t = x ? t1 : t0;
    if (!t.table) continue;
    const Slots s{cu, nullptr, nullptr, N, T, t.L, t.spare};
    for (int n = threadIdx.x; n < N; n += 1024) {
      const long b = s.base(n), next = n + 1 < N ? s.base(n + 1) : t.count;
      const int pieces = (cu[n + 1] - cu[n] + t.L - 1) / t.L;
      for (long i = b; i < next; ++i) t.table[i] = i - b < pieces ? n : -1;
    }
  }
}

}  // namespace

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

int launch_plan(const int32_t *cu, int N, int T, const PlanTable *tables, int n_tables, int *status,
                cudaStream_t s) {
  PlanTable none{nullptr, 1, 0, 0};
  plan_kernel<<<1, 1024, 0, s>>>(cu, N, T, n_tables > 0 ? tables[0] : none,
                                 n_tables > 1 ? tables[1] : none, status);
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
