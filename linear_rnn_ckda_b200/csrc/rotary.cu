// rotary.cu -- rotary positions: channel pairs of q and k turned by position times frequency.
//
//   (x_a, x_b) -> scale (x_a cos t - x_b sin t, x_b cos t + x_a sin t),  t = pos * f_i
//
// for the first 2 n_freqs channels of every head (pair i: channels i and i + n_freqs, or
// 2 i and 2 i + 1), the others copied; the inverse turns by -t, which with the same scale is
// the gradient.
//
// The angle is needed modulo one turn.  Each frequency is held as a 64-bit fixed-point
// fraction of a turn, F = f / (2 pi) * 2^64 modulo 2^64, and pos * F in wrapping 64-bit integer
// arithmetic is the angle's fraction of a turn: nothing is lost to the size of the position
// (an fp32 product is a tenth of a radian off at a million tokens), and no range reduction
// follows.  One fp32 rounding of the fraction costs 2^-25 of half a turn.
//
// Bound: HBM, q and k read and written once.  A block takes a few tokens: its threads put
// their loads in flight, fill a table of cos and sin in shared memory (one pair per token and
// frequency, shared by all heads), and turn 16-byte vectors from registers.
#include "common.cuh"
#include "linattn.h"

namespace ckda {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotItems = 2;       // items per thread held in registers at once
constexpr int kRotTable = 2048;    // table entries (tokens of a block x frequencies)

struct FastDiv {                   // n / d for n < 2^31 by one multiplication
  uint32_t d, mul, shift;
};
FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  return (uint32_t)(((uint64_t)__umulhi(n, f.mul) + n) >> f.shift);
}

struct RotParams {
  const void *q, *k, *pos;
  void *q_out, *k_out;
  const double *freqs;
  long n;
  int nf, Hq, Hk, d, interleaved, pos64, inverse, tokens;
  float scale;
  FastDiv by_iph, by_heads, by_nf;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};

// V: elements per vector (1: any size and alignment).  An item is one vector of first channels
// with the one of their partners (half layout), or one vector of adjacent pairs (interleaved,
// V >= 2; V = 1 takes its two channels one by one), or one vector of copied channels.
template <typename T, int V>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const RotParams p) {
  __shared__ float2 table[kRotTable];
  const long t0 = (long)blockIdx.x * p.tokens;
  const int nt = (int)(p.n - t0 < p.tokens ? p.n - t0 : p.tokens);
  const int heads = p.Hq + p.Hk;
  const bool inter = p.interleaved != 0;
  const int turn_items = inter ? (V == 1 ? p.nf : 2 * p.nf / V) : p.nf / V;
  const int iph = (int)p.by_iph.d;
  const uint32_t items = (uint32_t)nt * heads * iph;
  using VT = Vec<T, V>;

  for (uint32_t base = 0; base < items || base == 0; base += kRotThreads * kRotItems) {
    VT a[kRotItems], b[kRotItems];
    T *dst[kRotItems];
    int at[kRotItems], tok[kRotItems];   // first frequency (-1: copied, -2: none), token
    int ca[kRotItems], cb[kRotItems];
#pragma unroll
    for (int u = 0; u < kRotItems; ++u) {
      const uint32_t it = base + u * kRotThreads + threadIdx.x;
      at[u] = -2;
      tok[u] = 0; ca[u] = cb[u] = 0; dst[u] = nullptr;
      if (it >= items) continue;
      const uint32_t row = div_by(it, p.by_iph), iv = it - row * iph;
      const uint32_t tk = div_by(row, p.by_heads), h = row - tk * heads;
      tok[u] = (int)tk;
      const bool is_q = (int)h < p.Hq;
      const size_t off = is_q ? ((size_t)(t0 + tk) * p.Hq + h) * p.d
                              : ((size_t)(t0 + tk) * p.Hk + (h - p.Hq)) * p.d;
      const T *src = static_cast<const T *>(is_q ? p.q : p.k) + off;
      dst[u] = static_cast<T *>(is_q ? p.q_out : p.k_out) + off;
      if ((int)iv < turn_items) {
        at[u] = inter ? (V == 1 ? (int)iv : (int)iv * (V / 2)) : (int)iv * V;
        ca[u] = inter ? (V == 1 ? 2 * (int)iv : (int)iv * V) : (int)iv * V;
        cb[u] = inter ? (V == 1 ? ca[u] + 1 : -1) : ca[u] + p.nf;
      } else {
        at[u] = -1;
        ca[u] = 2 * p.nf + ((int)iv - turn_items) * V;
        cb[u] = -1;
      }
      a[u] = *reinterpret_cast<const VT *>(src + ca[u]);
      if (cb[u] >= 0) b[u] = *reinterpret_cast<const VT *>(src + cb[u]);
    }
    if (base == 0) {
      for (uint32_t i = threadIdx.x; i < (uint32_t)nt * p.nf; i += kRotThreads) {
        const uint32_t tk = div_by(i, p.by_nf), fi = i - tk * p.nf;
        const double turns = p.freqs[fi] * 0.15915494309189533577;   // 1 / (2 pi)
        const double frac = (turns - floor(turns)) * 4294967296.0;
        const double hi = floor(frac);
        const uint64_t F = ((uint64_t)hi << 32) + (uint64_t)((frac - hi) * 4294967296.0);
        const long long at_pos = p.pos64 ? static_cast<const long long *>(p.pos)[t0 + tk]
                                         : (long long)static_cast<const int *>(p.pos)[t0 + tk];
        const uint64_t u = (uint64_t)at_pos * F;
        // half turns in [-1, 1)
        float sn, cs;
        sincospif((float)(long long)u * 1.0842021724855044e-19f, &sn, &cs);   // 2^-63
        table[i] = make_float2(cs * p.scale, (p.inverse ? -sn : sn) * p.scale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kRotItems; ++u) {
      if (at[u] == -2) continue;
      if (at[u] >= 0) {
        const float2 *cs = table + tok[u] * p.nf + at[u];
        if (inter && V > 1) {
#pragma unroll
          for (int e = 0; e + 1 < V; e += 2) {
            const float2 c = cs[e / 2];
            const float x = to_f32(a[u].x[e]), y = to_f32(a[u].x[e + 1]);
            a[u].x[e] = from_f32<T>(x * c.x - y * c.y);
            a[u].x[e + 1] = from_f32<T>(y * c.x + x * c.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 c = cs[e];
            const float x = to_f32(a[u].x[e]), y = to_f32(b[u].x[e]);
            a[u].x[e] = from_f32<T>(x * c.x - y * c.y);
            b[u].x[e] = from_f32<T>(y * c.x + x * c.y);
          }
        }
      }
      *reinterpret_cast<VT *>(dst[u] + ca[u]) = a[u];
      if (cb[u] >= 0) *reinterpret_cast<VT *>(dst[u] + cb[u]) = b[u];
    }
  }
}

template <typename T, int V>
int launch_typed(const RotaryArgs &a, cudaStream_t s) {
  RotParams p;
  p.q = a.q; p.k = a.k; p.pos = a.pos; p.q_out = a.q_out; p.k_out = a.k_out; p.freqs = a.freqs;
  p.n = a.n; p.nf = a.n_freqs; p.Hq = a.Hq; p.Hk = a.Hk; p.d = a.d;
  p.interleaved = a.interleaved; p.pos64 = a.pos64; p.inverse = a.inverse; p.scale = a.scale;
  const int turn_items = a.interleaved ? (V == 1 ? a.n_freqs : 2 * a.n_freqs / V) : a.n_freqs / V;
  const int iph = turn_items + (a.d - 2 * a.n_freqs) / V;
  const int heads = p.Hq + p.Hk;
  // tokens per block: enough items to fill the block's registers once, while the table holds
  // them and every SM still has a few blocks
  long tokens = (long)kRotThreads * kRotItems / ((long)heads * iph);
  if (a.n_freqs > 0 && tokens > kRotTable / a.n_freqs) tokens = kRotTable / a.n_freqs;
  if (tokens > a.n / 592) tokens = a.n / 592;
  if (tokens < 1) tokens = 1;
  p.tokens = (int)tokens;
  p.by_iph = fast_div((uint32_t)iph);
  p.by_heads = fast_div((uint32_t)heads);
  p.by_nf = fast_div((uint32_t)(a.n_freqs > 0 ? a.n_freqs : 1));
  const long blocks = (a.n + tokens - 1) / tokens;
  rotary_kernel<T, V><<<(unsigned)blocks, kRotThreads, 0, s>>>(p);
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
  return wide ? launch_typed<T, V>(a, s) : launch_typed<T, 1>(a, s);
}

}  // namespace

int launch_rotary(const RotaryArgs &a, cudaStream_t s) {
  if (a.n == 0) return CKDA_OK;
  return a.io_dtype == CKDA_BF16 ? launch_vec<__nv_bfloat16>(a, s) : launch_vec<float>(a, s);
}

}  // namespace ckda
