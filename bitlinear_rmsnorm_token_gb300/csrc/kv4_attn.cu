// kv4_attn.cu -- softmax attention over the paged 4-bit key/value cache.
//
// o[t, h] = sum_j p_j v_j, p = softmax_j(scale q[t, h] . k_j) over the keys the
// masks leave, with the running maximum and sum of a one-pass softmax in fp32.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "rowquant.cuh"

namespace bitnet {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One CTA per (query row, head); warp w takes keys w, w + 4, ...; a lane holds
// D / 32 consecutive dimensions.
template <int D, typename QT, typename OT>
__global__ void __launch_bounds__(kWarps * 32) k_kv4_attn_row(KvView c, const QT* __restrict__ q, int Hq, int max_q,
                                                              float scale, int causal, int window,
                                                              OT* __restrict__ out, unsigned* err) {
  using B = KvBlock<D>;
  constexpr int kPer = D / 32;
  __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, h = blockIdx.y;
  const int b = kv_seq_of_row(c.q_start, c.num_seqs, t, lane);
  if (b < 0) return;
  bool bad = false;
  const int len = kv_len_of(c, b, &bad);
  const int n = c.q_start[b + 1] - c.q_start[b];
  if (n > max_q) bad = true;
  const int64_t pos = static_cast<int64_t>(len) - n + (t - c.q_start[b]);
  const int64_t j1 = causal ? min(static_cast<int64_t>(len), pos + 1) : len;
  const int64_t j0 = causal && window > 0 ? max(static_cast<int64_t>(0), pos - window + 1) : 0;
  const int kvh = h / (Hq / c.heads);
  const QT* qr = q + (static_cast<int64_t>(t) * Hq + h) * D + kPer * lane;
  float qv[kPer], o[kPer], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    qv[i] = static_cast<float>(qr[i]) * scale;
    o[i] = 0.0f;
  }
  for (int64_t j = j0 + warp; j < j1; j += kWarps) {
    const int page = c.page_table[static_cast<int64_t>(b) * c.max_pages + (j >> 6)];
    if (page < 0 || page >= c.num_pages) {
      bad = true;
      continue;
    }
    const uint8_t* blk = c.cache + (static_cast<int64_t>(page) * c.heads + kvh) * B::kBytes;
    const int slot = static_cast<int>(j & (kKvPage - 1));
    const float2 km = *reinterpret_cast<const float2*>(blk + B::offKMeta + slot * 8);
    const float2 vm = *reinterpret_cast<const float2*>(blk + B::offVMeta + slot * 8);
    float dot = 0.0f;
    const uint8_t* kc = blk + B::offK + slot * B::kRow + kPer / 2 * lane;
    const uint8_t* vc = blk + B::offV + slot * B::kRow + kPer / 2 * lane;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      dot += qv[i] * (static_cast<float>((kc[i / 2] >> (4 * (i & 1))) & 15) * km.x + km.y);
    dot = warp_sum_f(dot);
    const float m2 = fmaxf(m, dot);
    const float f = __expf(m - m2), p = __expf(dot - m2);
    m = m2;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      o[i] = o[i] * f + p * (static_cast<float>((vc[i / 2] >> (4 * (i & 1))) & 15) * vm.x + vm.y);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
    if (bad) atomicOr(err, kErrBadIndex);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_o[warp][kPer * lane + i] = o[i];
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
  float f[kWarps], ll = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.0f : __expf(s_m[w] - mm);
    ll += s_l[w] * f[w];
  }
  const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float r = 0.0f;
    for (int w = 0; w < kWarps; ++w) r += s_o[w][d] * f[w];
    out[(static_cast<int64_t>(t) * Hq + h) * D + d] = round_out<OT>(r * inv);
  }
}

template <int D, typename QT, typename OT>
cudaError_t launch_row(const DeviceContext* ctx, const KvView& c, const void* q, int64_t T, int Hq, int max_q,
                       float scale, int causal, int window, void* out, cudaStream_t s) {
  k_kv4_attn_row<D, QT, OT><<<dim3(static_cast<unsigned>(T), static_cast<unsigned>(Hq)), kWarps * 32, 0, s>>>(
      c, static_cast<const QT*>(q), Hq, max_q, scale, causal, window, static_cast<OT*>(out), ctx->err_word);
  return cudaGetLastError();
}

template <typename QT, typename OT>
cudaError_t launch_d(const DeviceContext* ctx, const KvView& c, int head_dim, const void* q, int64_t T, int Hq,
                     int max_q, float scale, int causal, int window, void* out, cudaStream_t s) {
  return head_dim == 128 ? launch_row<128, QT, OT>(ctx, c, q, T, Hq, max_q, scale, causal, window, out, s)
                         : launch_row<256, QT, OT>(ctx, c, q, T, Hq, max_q, scale, causal, window, out, s);
}

}  // namespace

cudaError_t launch_kv4_attention(DeviceContext* ctx, const KvView& c, int head_dim, const void* q, int q_dtype,
                                 int64_t T, int Hq, int max_q_len, float scale, int causal, int window, void* out,
                                 int out_dtype, cudaStream_t s, int* status) {
  *status = BITNET_OK;
  const int64_t rows = static_cast<int64_t>(Hq / c.heads) * max_q_len;
  if (kv4_decode_supported(head_dim, q_dtype, rows))
    return launch_kv4_decode(ctx, c, head_dim, q, q_dtype, T, Hq, rows, scale, causal, window, out, out_dtype, s,
                             status);
  auto with_out = [&](auto* qt) {
    using QT = std::remove_pointer_t<decltype(qt)>;
    if (out_dtype == BITNET_DTYPE_F32)
      return launch_d<QT, float>(ctx, c, head_dim, q, T, Hq, max_q_len, scale, causal, window, out, s);
    return launch_d<QT, QT>(ctx, c, head_dim, q, T, Hq, max_q_len, scale, causal, window, out, s);
  };
  switch (q_dtype) {
    case BITNET_DTYPE_F32: return with_out(static_cast<float*>(nullptr));
    case BITNET_DTYPE_F16: return with_out(static_cast<__half*>(nullptr));
    case BITNET_DTYPE_BF16: return with_out(static_cast<__nv_bfloat16*>(nullptr));
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace bitnet
