// linattn_decode.cu -- one token of linear attention with a decay for each head, state in place:
//   S <- exp(g) S + k v^T,   o = S^T q
//
// Bound: HBM, each fp32 state read and written once (131,072 bytes a head of 128 x 128).  A warp
// owns 16 state columns over every key channel: lane l holds columns 4 (l % 4) .. + 3 of rows
// l / 4 + 8 m, so a load covers 8 rows x 64 contiguous bytes and o's sum over rows is in-thread
// sums and three shuffles.  Warps share nothing, so the block's warp count is free: few heads
// are spread one warp per block over the SMs, many take eight.  Measured: B256 H32 128 x 128, 1,082
// MB, 177 to 188 us (88 to 93 % of the copy rate); B1 H16 13 us, of which the host's call is most.
#include "common.cuh"
#include "linattn.h"

namespace ckda {
namespace {

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(256, 2) linattn_decode_kernel(const LinDecodeArgs p, uint32_t tasks) {
  constexpr int slices = DV / 16;
  __shared__ float2 s_kq[8][DK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * (blockDim.x >> 5) + warp;   // below 2^31: B H dv / 16 is checked
  if (task >= tasks) return;
  const uint32_t head = task / slices, slice = task % slices;    // head = b * H + h
  const int col = slice * 16 + (lane & 3) * 4, r0 = lane >> 2;
  float *S = p.S + (size_t)head * DK * DV + col;
  constexpr int kRows = DK / 8;
  float4 st[kRows];
#pragma unroll
  for (int m = 0; m < kRows; ++m)
    st[m] = __ldcs(reinterpret_cast<const float4 *>(S + (r0 + 8 * m) * DV));
  const uint32_t b = head / (uint32_t)p.H;
  const int h = (int)(head - b * p.H);
  const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.Hq + head_of(h, p.H, p.Hq)) * DK;
  const T *k = static_cast<const T *>(p.k) + ((size_t)b * p.Hk + head_of(h, p.H, p.Hk)) * DK;
  const T *v = static_cast<const T *>(p.v) + ((size_t)b * p.Hv + head_of(h, p.H, p.Hv)) * DV + col;
  for (int i = lane; i < DK; i += 32) s_kq[warp][i] = make_float2(to_f32(k[i]), to_f32(q[i]));
  const float al = expf(p.g[p.g_fixed ? (uint32_t)h : head]);
  const float v0 = to_f32(v[0]), v1 = to_f32(v[1]), v2 = to_f32(v[2]), v3 = to_f32(v[3]);
  __syncwarp();
  float o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    const float2 kq = s_kq[warp][r0 + 8 * m];
    st[m].x = fmaf(al, st[m].x, kq.x * v0); st[m].y = fmaf(al, st[m].y, kq.x * v1);
    st[m].z = fmaf(al, st[m].z, kq.x * v2); st[m].w = fmaf(al, st[m].w, kq.x * v3);
    __stcs(reinterpret_cast<float4 *>(S + (r0 + 8 * m) * DV), st[m]);
    o0 = fmaf(kq.y, st[m].x, o0); o1 = fmaf(kq.y, st[m].y, o1);
    o2 = fmaf(kq.y, st[m].z, o2); o3 = fmaf(kq.y, st[m].w, o3);
  }
  if (p.o == nullptr) return;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    o0 += __shfl_xor_sync(0xffffffffu, o0, off);
    o1 += __shfl_xor_sync(0xffffffffu, o1, off);
    o2 += __shfl_xor_sync(0xffffffffu, o2, off);
    o3 += __shfl_xor_sync(0xffffffffu, o3, off);
  }
  if (r0 == 0) {
    T *o = static_cast<T *>(p.o) + (size_t)head * DV + col;
    o[0] = from_f32<T>(o0); o[1] = from_f32<T>(o1);
    o[2] = from_f32<T>(o2); o[3] = from_f32<T>(o3);
  }
}

template <int DK, int DV, typename T>
int launch_typed(const LinDecodeArgs &a, cudaStream_t s) {
  const long tasks = (long)a.B * a.H * (DV / 16);
  long warps = tasks / (148 * 4);
  warps = warps < 1 ? 1 : warps > 8 ? 8 : warps;
  linattn_decode_kernel<DK, DV, T><<<(unsigned)((tasks + warps - 1) / warps), (unsigned)(32 * warps), 0, s>>>(
      a, (uint32_t)tasks);
  return cudaGetLastError() == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}
template <int DK, typename T>
int launch_dv(const LinDecodeArgs &a, cudaStream_t s) {
  switch (a.dv) {
    case 16: return launch_typed<DK, 16, T>(a, s);
    case 32: return launch_typed<DK, 32, T>(a, s);
    case 64: return launch_typed<DK, 64, T>(a, s);
    case 128: return launch_typed<DK, 128, T>(a, s);
  }
  return CKDA_ERR_DIM;
}
template <typename T>
int launch_dk(const LinDecodeArgs &a, cudaStream_t s) {
  switch (a.dk) {
    case 16: return launch_dv<16, T>(a, s);
    case 32: return launch_dv<32, T>(a, s);
    case 64: return launch_dv<64, T>(a, s);
    case 128: return launch_dv<128, T>(a, s);
  }
  return CKDA_ERR_DIM;
}

}  // namespace

int launch_linattn_decode(const LinDecodeArgs &a, cudaStream_t s) {
  if ((long)a.B * a.H == 0) return CKDA_OK;
  return a.io_dtype == CKDA_BF16 ? launch_dk<__nv_bfloat16>(a, s) : launch_dk<float>(a, s);
}

}  // namespace ckda
