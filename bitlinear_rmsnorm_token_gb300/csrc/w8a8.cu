// w8a8.cu -- projections with 8-bit weights: per-channel weight quantisation
// and the int8 x int8 contraction.
#include "common.cuh"
#include "internal.h"
#include "rowquant.cuh"

namespace bitnet {
namespace {

constexpr int kWarps = 8;

// One warp per output channel: absmax over its K weights, then the codes.
__global__ void __launch_bounds__(kWarps * 32) k_quant_w8(const float* __restrict__ w, int64_t N, int K,
                                                          int8_t* __restrict__ codes, float* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (n >= N) return;
  const float4* row = reinterpret_cast<const float4*>(w + n * K);
  float m = 0.0f;
  for (int i = lane; i < K / 4; i += 32) {
    const float4 v = __ldg(row + i);
    m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  m = warp_max(m);
  const float sc = __fdiv_rn(127.0f, fmaxf(m, 1e-30f));
  uint32_t* out = reinterpret_cast<uint32_t*>(codes + n * K);
  for (int i = lane; i < K / 4; i += 32) {
    const float4 v = __ldg(row + i);
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t p = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float r = fminf(fmaxf(rintf(__fmul_rn(f[j], sc)), -127.0f), 127.0f);
      p |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xffu) << (8 * j);
    }
    out[i] = p;
  }
  if (lane == 0) scale[n] = sc;
}

// A warp per output: 16-byte chunks of the two rows, dp4a.
template <typename YT>
__global__ void __launch_bounds__(kWarps * 32) k_w8a8_dot(const int8_t* __restrict__ a,
                                                          const float* __restrict__ a_scale,
                                                          const int8_t* __restrict__ w,
                                                          const float* __restrict__ w_scale, int M, int N, int K,
                                                          YT* __restrict__ y, int32_t* __restrict__ acc_out) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= N) return;
  const uint4* wr = reinterpret_cast<const uint4*>(w + static_cast<int64_t>(n) * K);
  const float inv_w = __frcp_rn(w_scale[n]);
  for (int m = blockIdx.y; m < M; m += gridDim.y) {
    const uint4* ar = reinterpret_cast<const uint4*>(a + static_cast<int64_t>(m) * K);
    int acc = 0;
    for (int i = lane; i < K / 16; i += 32) {
      const uint4 x = __ldg(wr + i), v = __ldg(ar + i);
      acc = __dp4a(static_cast<int>(x.x), static_cast<int>(v.x), acc);
      acc = __dp4a(static_cast<int>(x.y), static_cast<int>(v.y), acc);
      acc = __dp4a(static_cast<int>(x.z), static_cast<int>(v.z), acc);
      acc = __dp4a(static_cast<int>(x.w), static_cast<int>(v.w), acc);
    }
    acc = warp_sum_int(acc);
    if (lane == 0) {
      const int64_t at = static_cast<int64_t>(m) * N + n;
      y[at] = round_out<YT>(rescale_elem(static_cast<float>(acc), __frcp_rn(a_scale[m]), inv_w));
      if (acc_out) acc_out[at] = acc;
    }
  }
}

}  // namespace

cudaError_t launch_quant_w8(const float* w, int64_t N, int64_t K, int8_t* codes, float* scale, cudaStream_t s) {
  k_quant_w8<<<static_cast<unsigned>((N + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(w, N, static_cast<int>(K), codes,
                                                                                     scale);
  return cudaGetLastError();
}

cudaError_t launch_w8a8(DeviceContext* ctx, const int8_t* a, const float* a_scale, const int8_t* w,
                        const float* w_scale, int64_t M, int64_t K, int64_t N, void* y, int y_dtype, int32_t* acc_out,
                        cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((N + kWarps - 1) / kWarps), static_cast<unsigned>(M < 1024 ? M : 1024));
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  switch (y_dtype) {
    case BITNET_DTYPE_F32:
      k_w8a8_dot<<<grid, kWarps * 32, 0, s>>>(a, a_scale, w, w_scale, m, n, k, static_cast<float*>(y), acc_out);
      break;
    case BITNET_DTYPE_F16:
      k_w8a8_dot<<<grid, kWarps * 32, 0, s>>>(a, a_scale, w, w_scale, m, n, k, static_cast<__half*>(y), acc_out);
      break;
    case BITNET_DTYPE_BF16:
      k_w8a8_dot<<<grid, kWarps * 32, 0, s>>>(a, a_scale, w, w_scale, m, n, k, static_cast<__nv_bfloat16*>(y),
                                              acc_out);
      break;
    default:
      return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace bitnet
