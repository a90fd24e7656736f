// linattn_abi.cu -- host side of the C ABI of linear attention with a decay for each head and of
// rotary positions (include/ckda.h): argument checks, workspace, dispatch.  As in ckda_abi.cu
// nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/ckda.h"
#include "internal.h"
#include "linattn.h"

namespace {

bool valid_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_io(int t) { return t == CKDA_F32 || t == CKDA_BF16; }
bool shares(int H, int Hx) { return Hx > 0 && Hx <= H && H % Hx == 0; }

// (an empty call's tensors have no storage to point at)
bool any_tokens(int B, int T) { return B != 0 && T != 0; }
bool has_decays(const float *g, int B, int T, int decay) {
  return g != nullptr || (decay == CKDA_DECAY_PER_TOKEN && !any_tokens(B, T));
}

// Sizes and types common to the three calls.
int check_sizes(long long B, long long T, int H, int Hq, int Hk, int Hv, int dk, int dv, int decay,
                int io_dtype) {
  if (!valid_dim(dk) || !valid_dim(dv) || B < 0 || T < 0 || H <= 0 || H > 65535 || !shares(H, Hq) ||
      !shares(H, Hk) || !shares(H, Hv))
    return CKDA_ERR_DIM;
  if (!valid_io(io_dtype) || (decay != CKDA_DECAY_PER_TOKEN && decay != CKDA_DECAY_PER_HEAD))
    return CKDA_ERR_DTYPE;
  // token rows are 32-bit coordinates, whole chunks of 64 too; row x head counts stay far below 2^63
  if (B * T > INT32_MAX - 63 || B * T * H > (1LL << 41)) return CKDA_ERR_DIM;
  return CKDA_OK;
}
int check_seqs(const void *cu, int n_seqs, int B, int T) {
  if (!cu) return B > INT32_MAX / 2 ? CKDA_ERR_DIM : CKDA_OK;
  return (B != 1 || n_seqs < 0 || (n_seqs == 0 && T > 0)) ? CKDA_ERR_DIM : CKDA_OK;
}

}  // namespace

extern "C" {

size_t ckda_linattn_fwd_workspace_size(int B, int T, int H, int dk, int dv, int io_dtype, int n_seqs) {
  if (B < 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0 || n_seqs < 0) return ckda::kWorkspaceHeader;
  return ckda::kWorkspaceHeader +
         ckda::linattn_fwd_workspace(B, T, H, dk, dv, n_seqs > 0 ? n_seqs : B, n_seqs > 0, io_dtype);
}

size_t ckda_linattn_bwd_workspace_size(int B, int T, int H, int Hq, int Hk, int Hv, int dk, int dv,
                                       int decay, int io_dtype, int n_seqs) {
  if (B < 0 || T < 0 || H <= 0 || dk <= 0 || dv <= 0 || n_seqs < 0) return ckda::kWorkspaceHeader;
  ckda::LinArgs a = {};
  a.N = n_seqs > 0 ? n_seqs : B;
  a.B = B; a.T = T; a.H = H; a.Hq = Hq; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv;
  a.g_fixed = decay == CKDA_DECAY_PER_HEAD;
  a.io_dtype = io_dtype;
  return ckda::kWorkspaceHeader + ckda::linattn_bwd_workspace(a, n_seqs > 0);
}

int ckda_linattn_fwd(const void *q, const void *k, const void *v, const float *g, const float *S0,
                     const int32_t *cu_seqlens, int n_seqs, int B, int T, int H, int Hq, int Hk,
                     int Hv, int dk, int dv, int decay, int io_dtype, void *o, float *S_T,
                     void *workspace, size_t workspace_bytes, void *stream) {
  if ((any_tokens(B, T) && (!q || !k || !v)) || !has_decays(g, B, T, decay)) return CKDA_ERR_NULL;
  int rc = check_sizes(B, T, H, Hq, Hk, Hv, dk, dv, decay, io_dtype);
  if (rc == CKDA_OK) rc = check_seqs(cu_seqlens, n_seqs, B, T);
  if (rc != CKDA_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(S0, 16) ||
      !aligned(o, 16) || !aligned(S_T, 16) || !aligned(cu_seqlens, 4))
    return CKDA_ERR_ALIGN;
  const size_t need = ckda_linattn_fwd_workspace_size(B, T, H, dk, dv, io_dtype, cu_seqlens ? n_seqs : 0);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return CKDA_ERR_WORKSPACE;
  rc = ckda::check_device();
  if (rc != CKDA_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the status word: a packed batch's plan and an fp32 batch's first kernel write it themselves
  if ((!cu_seqlens && io_dtype == CKDA_BF16) || (cu_seqlens && n_seqs == 0) || (long long)B * T == 0)
    if (cudaMemsetAsync(workspace, 0, ckda::kWorkspaceHeader, s) != cudaSuccess) return CKDA_ERR_CUDA;
  ckda::LinArgs a = {};
  a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.cu = cu_seqlens; a.o = o; a.S_T = S_T;
  a.N = cu_seqlens ? n_seqs : B;
  a.B = B; a.T = T; a.H = H; a.Hq = Hq; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv;
  a.g_fixed = decay == CKDA_DECAY_PER_HEAD;
  a.io_dtype = io_dtype;
  a.status = static_cast<int *>(workspace);
  a.ws = static_cast<uint8_t *>(workspace) + ckda::kWorkspaceHeader;
  if (a.N == 0) return CKDA_OK;
  return ckda::launch_linattn_fwd(a, s);
}

int ckda_linattn_bwd(const void *q, const void *k, const void *v, const float *g, const float *S0,
                     const int32_t *cu_seqlens, int n_seqs, int B, int T, int H, int Hq, int Hk,
                     int Hv, int dk, int dv, int decay, int io_dtype, const void *dO,
                     const float *dS_T, void *dq, void *dk_out, void *dv_out, float *dg, float *dS0,
                     void *workspace, size_t workspace_bytes, void *stream) {
  if ((any_tokens(B, T) && (!q || !k || !v || !dq || !dk_out || !dv_out)) ||
      !has_decays(g, B, T, decay) || !has_decays(dg, B, T, decay))
    return CKDA_ERR_NULL;
  int rc = check_sizes(B, T, H, Hq, Hk, Hv, dk, dv, decay, io_dtype);
  if (rc == CKDA_OK) rc = check_seqs(cu_seqlens, n_seqs, B, T);
  if (rc != CKDA_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) || !aligned(S0, 16) ||
      !aligned(dO, 16) || !aligned(dS_T, 16) || !aligned(dq, 16) || !aligned(dk_out, 16) ||
      !aligned(dv_out, 16) || !aligned(dg, 4) || !aligned(dS0, 16) || !aligned(cu_seqlens, 4))
    return CKDA_ERR_ALIGN;
  const size_t need = ckda_linattn_bwd_workspace_size(B, T, H, Hq, Hk, Hv, dk, dv, decay, io_dtype,
                                                      cu_seqlens ? n_seqs : 0);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return CKDA_ERR_WORKSPACE;
  rc = ckda::check_device();
  if (rc != CKDA_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the status word: a packed batch's plan and an fp32 batch's first kernel write it themselves
  if ((!cu_seqlens && io_dtype == CKDA_BF16) || (cu_seqlens && n_seqs == 0) || (long long)B * T == 0)
    if (cudaMemsetAsync(workspace, 0, ckda::kWorkspaceHeader, s) != cudaSuccess) return CKDA_ERR_CUDA;
  ckda::LinBwdArgs b = {};
  ckda::LinArgs &a = b.f;
  a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.cu = cu_seqlens;
  a.N = cu_seqlens ? n_seqs : B;
  a.B = B; a.T = T; a.H = H; a.Hq = Hq; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv;
  a.g_fixed = decay == CKDA_DECAY_PER_HEAD;
  a.io_dtype = io_dtype;
  a.status = static_cast<int *>(workspace);
  a.ws = static_cast<uint8_t *>(workspace) + ckda::kWorkspaceHeader;
  b.dO = dO; b.dS_T = dS_T; b.dq = dq; b.dk = dk_out; b.dv = dv_out; b.dg = dg; b.dS0 = dS0;
  if (a.N == 0 || (long)B * T == 0) {
    // no token: a fixed decay's gradient is an empty sum
    if (a.g_fixed && cudaMemsetAsync(dg, 0, (size_t)H * 4, s) != cudaSuccess) return CKDA_ERR_CUDA;
    if (a.N == 0) return CKDA_OK;
  }
  return ckda::launch_linattn_bwd(b, s);
}

int ckda_linattn_decode_step(const void *q, const void *k, const void *v, const float *g, float *S,
                             int B, int H, int Hq, int Hk, int Hv, int dk, int dv, int decay,
                             int io_dtype, void *o, void *stream) {
  if ((B != 0 && (!q || !k || !v || !S)) || !has_decays(g, B, 1, decay)) return CKDA_ERR_NULL;
  int rc = check_sizes(B, 1, H, Hq, Hk, Hv, dk, dv, decay, io_dtype);
  if (rc != CKDA_OK) return rc;
  if ((long long)B * H * (dv / 16) > INT32_MAX) return CKDA_ERR_DIM;   // (a warp takes 16 state columns)
  const uintptr_t es = io_dtype == CKDA_BF16 ? 2 : 4;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(g, 4) || !aligned(S, 16) ||
      !aligned(o, es))
    return CKDA_ERR_ALIGN;
  rc = ckda::check_device();
  if (rc != CKDA_OK) return rc;
  ckda::LinDecodeArgs a = {};
  a.q = q; a.k = k; a.v = v; a.g = g; a.S = S; a.o = o;
  a.B = B; a.H = H; a.Hq = Hq; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv;
  a.g_fixed = decay == CKDA_DECAY_PER_HEAD;
  a.io_dtype = io_dtype;
  return ckda::launch_linattn_decode(a, static_cast<cudaStream_t>(stream));
}

int ckda_rotary(const void *q, const void *k, const void *pos, const double *freqs, long long n_tokens,
                int Hq, int Hk, int d, int n_freqs, int layout, int pos_int64, float scale, int inverse,
                int io_dtype, void *q_out, void *k_out, void *stream) {
  if (n_tokens > 0 && (!q || !pos || !q_out || (Hk > 0 && (!k || !k_out)))) return CKDA_ERR_NULL;
  if (n_freqs > 0 && !freqs) return CKDA_ERR_NULL;
  if (n_tokens < 0 || n_tokens > INT32_MAX || Hq <= 0 || Hk < 0 || d <= 0 || d > 1024 ||
      n_freqs < 0 || 2 * n_freqs > d || (long long)Hq + Hk > 65535)
    return CKDA_ERR_DIM;
  if (!valid_io(io_dtype) || (layout != CKDA_ROTARY_HALF && layout != CKDA_ROTARY_INTERLEAVED))
    return CKDA_ERR_DTYPE;
  const uintptr_t es = io_dtype == CKDA_BF16 ? 2 : 4;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(q_out, es) || !aligned(k_out, es) ||
      !aligned(pos, pos_int64 ? 8 : 4) || !aligned(freqs, 8))
    return CKDA_ERR_ALIGN;
  const int rc = ckda::check_device();
  if (rc != CKDA_OK) return rc;
  ckda::RotaryArgs a = {};
  a.q = q; a.k = k; a.pos = pos; a.freqs = freqs; a.q_out = q_out; a.k_out = k_out;
  a.n = (long)n_tokens; a.n_freqs = n_freqs; a.Hq = Hq; a.Hk = Hk; a.d = d;
  a.interleaved = layout == CKDA_ROTARY_INTERLEAVED;
  a.pos64 = pos_int64 != 0; a.inverse = inverse != 0; a.io_dtype = io_dtype; a.scale = scale;
  return ckda::launch_rotary(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
