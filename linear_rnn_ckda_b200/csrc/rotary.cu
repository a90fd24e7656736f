// rotary.cu -- rotary positions: channel pairs of q and k turned by position times frequency.
//
//   (x_a, x_b) -> scale (x_a cos t - x_b sin t, x_b cos t + x_a sin t),  t = pos * f_i
//
// for the first 2 n_freqs channels of every head (pair i: channels i and i + n_freqs, or
// 2 i and 2 i + 1), the others copied; the inverse turns by -t, which with the same scale is
// the gradient.
//
// The angle is needed modulo one turn.  Each frequency is held as a 64-bit fixed-point
// fraction of a turn, F = f / (2 pi) * 2^64 modulo 2^64, to two units (the product is taken in four
// fp64 parts), and pos * F in wrapping 64-bit integer arithmetic is the angle's fraction of a turn, off
// by at most 2^-63 of a turn per position (an fp32 product is a tenth of a radian off at a million
// tokens); no range reduction follows.  One fp32 rounding of the fraction costs 2^-25 of half a turn.
//
// Bound: HBM, q and k read and written once.  A warp takes a token (or some of its heads, when
// tokens are few): its first loads are in flight while it fills a table of the token's cos and
// sin in shared memory; then each lane keeps the entries of its own 16-byte vector in
// registers and turns that vector of one head after another.  Warps share nothing but the
// fixed-point frequencies, formed once a block.  (With a table per block, a block barrier per
// token pair and table entries read for every vector, 268 MB took 66 us.)
#include "common.cuh"
#include "linattn.h"

namespace ckda {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotItems = 4;       // vectors (pairs of them) per lane in flight
// Blocks per SM: the registers of four bf16 items (eight table entries each) leave room for two
// (46.6 us against 52 with three and 59 with four, 268 MB), those of fp32 for four (19.0 us
// against 21.8 with three, 84 MB).
template <typename T>
constexpr int kRotBlocks = sizeof(T) == 2 ? 2 : 4;

struct RotParams {
  const void *q, *k, *pos;
  void *q_out, *k_out;
  const double *freqs;
  long tasks;                      // tokens x groups
  int nf, Hq, Hk, d, pos64, inverse, groups, per_group, turn_items, iph;
  float scale;
};

// A vector as 32-bit words (two bf16 values or one float each), or one element.
template <typename T, int V>
struct Vec {
  using Type = uint4;
};
template <typename T>
struct Vec<T, 1> {
  using Type = T;
};
__device__ __forceinline__ void turn(float &x, float &y, float2 c) {
  // (fused as written, so that every path rounds alike)
  const float u = fmaf(x, c.x, -__fmul_rn(y, c.y));
  y = fmaf(y, c.x, __fmul_rn(x, c.y));
  x = u;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// a word of first channels with the word of their partners
template <typename T>
__device__ __forceinline__ void turn_words(uint32_t &a, uint32_t &b, const float2 *c) {
  if constexpr (sizeof(T) == 2) {
    float x0 = low(a), y0 = low(b), x1 = high(a), y1 = high(b);
    turn(x0, y0, c[0]);
    turn(x1, y1, c[1]);
    a = pack2(x0, x1);
    b = pack2(y0, y1);
  } else {
    float x = __uint_as_float(a), y = __uint_as_float(b);
    turn(x, y, c[0]);
    a = __float_as_uint(x);
    b = __float_as_uint(y);
  }
}

// V: elements per vector (1: any size and alignment).  An item is one vector of first channels
// with the one of their partners (half layout), or one vector of adjacent pairs (INTER, V >= 2;
// V = 1 takes its two channels one by one), or one vector of copied channels.  A head has iph
// items, turn_items of them turned; lane l takes item l % iph (iph <= 32) of every (32 / iph)-th
// head, or items l, l + 32, .. of every head.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRotThreads, kRotBlocks<T>) rotary_kernel(const RotParams p) {
  extern __shared__ uint64_t rot_smem[];
  uint64_t *freq = rot_smem;                                     // [nf]
  float2 *table = reinterpret_cast<float2 *>(rot_smem + p.nf) + (threadIdx.x >> 5) * p.nf;
  const int lane = threadIdx.x & 31;
  using VT = typename Vec<T, V>::Type;
  constexpr bool kTwo = !INTER || V == 1;                        // an item has a second vector
  constexpr int kE = INTER && V > 1 ? V / 2 : V;                 // table entries of an item
  for (int i = threadIdx.x; i < p.nf; i += kRotThreads) {
    // f / (2 pi) with 1 / (2 pi) as a sum of three doubles: products and their rounding errors, whose
    // fractions of a turn, [-1/2, 1/2], become integers (their sum wraps as turns do)
    constexpr double kInv0 = 0x1.45f306dc9c883p-3, kInv1 = -0x1.6b01ec5417056p-57, kInv2 = -0x1.6447e493ad4cep-111;
    const double f = p.freqs[i], x = f * kInv0, y = f * kInv1;
    auto units = [](double t) { return (uint64_t)__double2ll_rn((t - rint(t)) * 18446744073709551616.0); };
    freq[i] = units(x) + units(fma(f, kInv0, -x)) + units(y) + units(fma(f, kInv1, -y) + f * kInv2);
  }
  __syncthreads();
  const int rows = p.iph <= 32 ? 32 / p.iph : 1;                 // heads a warp takes at once
  const int sub = p.iph <= 32 ? lane / p.iph : 0;
  const bool idle = sub >= rows;

  for (long task = (long)blockIdx.x * kRotWarps + (threadIdx.x >> 5); task < p.tasks;
       task += (long)gridDim.x * kRotWarps) {
    const long tok = p.groups == 1 ? task : task / p.groups;
    const int grp = p.groups == 1 ? 0 : (int)(task - tok * p.groups);
    const int h0 = grp * p.per_group, h1 = min(p.Hq + p.Hk, h0 + p.per_group);
    bool filled = false;
    for (int iv = p.iph <= 32 ? lane - sub * p.iph : lane; iv - lane < p.iph || !filled; iv += 32) {
      const bool on = !idle && iv < p.iph, turned = iv < p.turn_items;
      const int ca = turned ? (kTwo && INTER ? 2 * iv : iv * V) : 2 * p.nf + (iv - p.turn_items) * V;
      const int cb = INTER ? ca + 1 : ca + p.nf;
      float2 cs[kE];
      for (int h = h0; h < h1 || !filled; h += rows * kRotItems) {
        VT a[kRotItems], b[kRotItems];
        T *dst[kRotItems];
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
          const int hh = h + sub + u * rows;
          dst[u] = nullptr;
          if (!on || hh >= h1) continue;
          const bool is_q = hh < p.Hq;
          const size_t off = is_q ? ((size_t)tok * p.Hq + hh) * p.d : ((size_t)tok * p.Hk + (hh - p.Hq)) * p.d;
          const T *src = static_cast<const T *>(is_q ? p.q : p.k) + off;
          dst[u] = static_cast<T *>(is_q ? p.q_out : p.k_out) + off;
          a[u] = *reinterpret_cast<const VT *>(src + ca);
          if (kTwo && turned) b[u] = *reinterpret_cast<const VT *>(src + cb);
        }
        if (!filled) {
          filled = true;
          const long long at = p.pos64 ? static_cast<const long long *>(p.pos)[tok]
                                       : (long long)static_cast<const int *>(p.pos)[tok];
          for (int i = lane; i < p.nf; i += 32) {
            float sn, cn;                                        // half turns in [-1, 1)
            sincospif((float)(long long)((uint64_t)at * freq[i]) * 1.0842021724855044e-19f, &sn, &cn);   // 2^-63
            table[i] = make_float2(cn * p.scale, (p.inverse ? -sn : sn) * p.scale);
          }
          __syncwarp();
        }
        if (h == h0 && on && turned) {
#pragma unroll
          for (int e = 0; e < kE; ++e) cs[e] = table[iv * kE + e];
        }
#pragma unroll
        for (int u = 0; u < kRotItems; ++u) {
          if (!dst[u]) continue;
          if (turned) {
            if constexpr (V == 1) {
              float x = to_f32(a[u]), y = to_f32(b[u]);
              turn(x, y, cs[0]);
              a[u] = from_f32<T>(x);
              b[u] = from_f32<T>(y);
            } else if constexpr (INTER) {
              if constexpr (sizeof(T) == 2) {
                uint32_t *w[4] = {&a[u].x, &a[u].y, &a[u].z, &a[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float x = low(*w[e]), y = high(*w[e]);
                  turn(x, y, cs[e]);
                  *w[e] = pack2(x, y);
                }
              } else {
                turn_words<T>(a[u].x, a[u].y, cs);
                turn_words<T>(a[u].z, a[u].w, cs + 1);
              }
            } else {
              constexpr int n = 4 / sizeof(T);
              turn_words<T>(a[u].x, b[u].x, cs);
              turn_words<T>(a[u].y, b[u].y, cs + n);
              turn_words<T>(a[u].z, b[u].z, cs + 2 * n);
              turn_words<T>(a[u].w, b[u].w, cs + 3 * n);
            }
          }
          *reinterpret_cast<VT *>(dst[u] + ca) = a[u];
          if (kTwo && turned) *reinterpret_cast<VT *>(dst[u] + cb) = b[u];
        }
      }
      if (p.iph <= 32) break;
    }
    __syncwarp();                                                // (the table is free)
  }
}

template <typename T, int V, bool INTER>
int launch_typed(const RotaryArgs &a, cudaStream_t s) {
  RotParams p;
  p.q = a.q; p.k = a.k; p.pos = a.pos; p.q_out = a.q_out; p.k_out = a.k_out; p.freqs = a.freqs;
  p.nf = a.n_freqs; p.Hq = a.Hq; p.Hk = a.Hk; p.d = a.d;
  p.pos64 = a.pos64; p.inverse = a.inverse; p.scale = a.scale;
  p.turn_items = INTER && V > 1 ? 2 * a.n_freqs / V : a.n_freqs / V;
  p.iph = p.turn_items + (a.d - 2 * a.n_freqs) / V;
  const int heads = a.Hq + a.Hk;
  // a token's heads go to several warps while there are fewer warps than the GPU holds, down to
  // what one pass of a warp takes
  const int pass = (p.iph <= 32 ? 32 / p.iph : 1) * kRotItems, most = (heads + pass - 1) / pass;
  const long room = 148L * kRotBlocks<T> * kRotWarps;
  long groups = a.n >= room ? 1 : room / a.n;
  if (groups > most) groups = most;
  p.per_group = (int)((heads + groups - 1) / groups);
  p.groups = (heads + p.per_group - 1) / p.per_group;
  p.tasks = a.n * p.groups;
  long blocks = (p.tasks + kRotWarps - 1) / kRotWarps;
  if (blocks > 148 * kRotBlocks<T>) blocks = 148 * kRotBlocks<T>;
  const size_t smem = (size_t)p.nf * 8 * (1 + kRotWarps);
  rotary_kernel<T, V, INTER><<<(unsigned)blocks, kRotThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

template <typename T>
int launch_vec(const RotaryArgs &a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                        (a.Hk ? reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out) : 0);
  // 16-byte vectors where every vector boundary falls on one: head size, the turned part and,
  // in the half layout, its half
  const bool wide = (any & 15) == 0 && a.d % V == 0 &&
                    (a.interleaved ? 2 * a.n_freqs : a.n_freqs) % V == 0;
  if (a.interleaved) return wide ? launch_typed<T, V, true>(a, s) : launch_typed<T, 1, true>(a, s);
  return wide ? launch_typed<T, V, false>(a, s) : launch_typed<T, 1, false>(a, s);
}

}  // namespace

int launch_rotary(const RotaryArgs &a, cudaStream_t s) {
  if (a.n == 0) return CKDA_OK;
  return a.io_dtype == CKDA_BF16 ? launch_vec<__nv_bfloat16>(a, s) : launch_vec<float>(a, s);
}

}  // namespace ckda
