// linattn.h -- launch interface of linear attention with a decay for each head (linattn_*.cu)
// and of rotary positions (rotary.cu).
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t     (per sequence and head)
//
// Over a chunk of C tokens with G_i = g_1 + .. + g_i (from the chunk's first token):
//   o_i   = e^{G_i} S_in^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j
//   S_out = e^{G_C} S_in + sum_j e^{G_C - G_j} k_j v_j^T
// Every factor is the exponential of a sum of log decays over a range of tokens, so none
// exceeds 1 and nothing is divided.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ckda {
// The head of a tensor with Hx heads that head h of H reads, h Hx / H without the product, which
// passes 32 bits from 46,342 heads on (Hx divides H).
__host__ __device__ inline int head_of(int h, int H, int Hx) { return h / (H / Hx); }

// CKDA_OK when the current device is sm_100, else the CKDA_ERR_* code a call returns.
int check_device();
// ckda_debug_wait_injection's settings: the chunk (-1: off) and the bound of its wait (0: the usual one).
int wait_injection(uint64_t *wait_ns);

struct LinArgs {
  const void *q, *k, *v;      // [rows, Hq, dk], [rows, Hk, dk], [rows, Hv, dv]
  const float *g;             // [rows, H], or [H] (g_fixed)
  const float *S0;            // [N, H, dk, dv] or NULL
  const int32_t *cu;          // device offsets [N + 1], or NULL
  void *o;                    // [rows, H, dv] or NULL
  float *S_T;                 // [N, H, dk, dv] or NULL
  int N, B, T, H, Hq, Hk, Hv, dk, dv, g_fixed, io_dtype;
  int *status;                // workspace header
  uint8_t *ws;                // workspace past the header
};

struct LinBwdArgs {
  LinArgs f;                  // the forward's inputs (o, S_T unused)
  const void *dO;             // [rows, H, dv] in the io dtype, or NULL (zero)
  const float *dS_T;          // [N, H, dk, dv] or NULL (zero)
  void *dq, *dk, *dv;         // shaped as q, k, v, in the io dtype
  float *dg;                  // shaped as g
  float *dS0;                 // [N, H, dk, dv] or NULL
};

struct LinDecodeArgs {
  const void *q, *k, *v;      // [B, Hq, dk], [B, Hk, dk], [B, Hv, dv]
  const float *g;             // [B, H] or [H]
  float *S;                   // [B, H, dk, dv], updated in place
  void *o;                    // [B, H, dv] or NULL
  int B, H, Hq, Hk, Hv, dk, dv, g_fixed, io_dtype;
};

struct RotaryArgs {
  const void *q, *k;          // [n, Hq, d], [n, Hk, d] (Hk may be 0)
  const void *pos;            // [n] int32 or int64
  const double *freqs;        // [n_freqs] radians per position
  void *q_out, *k_out;
  long n;
  int n_freqs, Hq, Hk, d, interleaved, pos64, inverse, io_dtype;
  float scale;
};

size_t linattn_fwd_workspace(int B, int T, int H, int dk, int dv, int N, bool packed, int io_dtype);
size_t linattn_bwd_workspace(const LinArgs &a, bool packed);
int launch_linattn_fwd(const LinArgs &a, cudaStream_t s);
int launch_linattn_bwd(const LinBwdArgs &a, cudaStream_t s);
int launch_linattn_decode(const LinDecodeArgs &a, cudaStream_t s);
int launch_rotary(const RotaryArgs &a, cudaStream_t s);

}  // namespace ckda
