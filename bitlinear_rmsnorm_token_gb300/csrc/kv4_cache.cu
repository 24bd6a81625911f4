// kv4_cache.cu -- writing rows into the paged 4-bit key/value cache and reading
// them back.
//
// Row quantisation: min and max over the D values (exact), scale = (max - min)
// / 15, code = round(15 (x - min) / (max - min)), ties to even, of the exact
// quotient.  The quotient is formed in fp32 as (x - min) * (15 / (max - min)),
// whose error is below 4 * 2^-24 * 15 < 4e-6 (one rounding each of the
// difference, the range, its reciprocal and the product); where it lies within
// 1e-5 of the border between two codes the code is decided in double instead
// (about one value in 50 000), so that it never depends on that rounding.
// A row with max - min < 1e-30 (a constant row) has scale 0 and codes 0.
//
// D / 16 lanes share a row, 16 values each: two or four 16-byte loads per lane,
// a min/max exchange over the row's lanes, one 8-byte store of codes.  Bound by
// memory for many rows, by one row's latency for few.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "rowquant.cuh"

namespace bitnet {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ int quant_code(float x, float lo, float hi, float inv) {
  const float t = __fmul_rn(__fsub_rn(x, lo), inv);
  float r = rintf(t);
  if (fabsf(fabsf(t - r) - 0.5f) < 1e-5f)
    r = static_cast<float>(rint((static_cast<double>(x) - lo) * 15.0 / (static_cast<double>(hi) - lo)));
  return static_cast<int>(fminf(fmaxf(r, 0.0f), 15.0f));
}

// Where row `row` of the plan (token * heads + head) lives in the cache, or
// null: a token outside every sequence, a position before the sequence's
// first, or a page outside the cache (recorded).
template <int D>
__device__ __forceinline__ uint8_t* locate(const KvView& c, int t, int head, int lane, int* slot, unsigned* err) {
  const int b = kv_seq_of_row(c.q_start, c.num_seqs, t, lane);
  if (b < 0) return nullptr;
  bool bad = false;
  const int len = kv_len_of(c, b, &bad);
  const int64_t pos = static_cast<int64_t>(len) - (static_cast<int64_t>(c.q_start[b + 1]) - t);
  uint8_t* p = nullptr;
  if (pos >= 0 && pos < len) {
    const int page = c.page_table[static_cast<int64_t>(b) * c.max_pages + (pos >> 6)];
    if (page < 0 || page >= c.num_pages) bad = true;
    else p = c.cache + (static_cast<int64_t>(page) * c.heads + head) * KvBlock<D>::kBytes;
    *slot = static_cast<int>(pos & (kKvPage - 1));
  }
  if (bad && lane == 0) atomicOr(err, kErrBadIndex);
  return p;
}

// A warp takes 512 / D heads of one token's keys or values (blockIdx.y: keys,
// values).
template <int D, typename T, bool kRead>
__global__ void __launch_bounds__(kWarps * 32) k_kv4_rows(KvView c, T* __restrict__ k, T* __restrict__ v, int T_rows,
                                                          unsigned* err) {
  constexpr int kLanes = D / 16;       // lanes per row
  constexpr int kRows = 32 / kLanes;   // rows per warp
  using B = KvBlock<D>;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int groups = (c.heads + kRows - 1) / kRows;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / groups);
  if (t >= T_rows) return;
  const int head = static_cast<int>(w % groups) * kRows + lane / kLanes;
  const bool on = head < c.heads;
  const int l = lane % kLanes;
  int slot = 0;
  uint8_t* blk = locate<D>(c, t, on ? head : 0, lane, &slot, err);
  if (!blk) return;  // the same for all lanes
  const bool is_v = blockIdx.y != 0;
  T* x = (is_v ? v : k) + (static_cast<int64_t>(t) * c.heads + (on ? head : 0)) * D + 16 * l;
  uint2* codes = reinterpret_cast<uint2*>(blk + (is_v ? B::offV : B::offK) + slot * B::kRow + 8 * l);
  float2* meta = reinterpret_cast<float2*>(blk + (is_v ? B::offVMeta : B::offKMeta) + slot * 8);
  if constexpr (kRead) {
    if (!on) return;
    const uint2 w2 = *codes;
    const float2 sm = *meta;
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t word = i < 8 ? w2.x : w2.y;
      f[i] = __fadd_rn(__fmul_rn(static_cast<float>((word >> (4 * (i & 7))) & 15u), sm.x), sm.y);
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(x)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
      union { T h[16]; uint4 u[2]; } o;
#pragma unroll
      for (int i = 0; i < 16; ++i) o.h[i] = round_out<T>(f[i]);
      reinterpret_cast<uint4*>(x)[0] = o.u[0];
      reinterpret_cast<uint4*>(x)[1] = o.u[1];
    }
  } else {
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = load4(x + 4 * i);
      f[4 * i] = q.x;
      f[4 * i + 1] = q.y;
      f[4 * i + 2] = q.z;
      f[4 * i + 3] = q.w;
    }
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      lo = fminf(lo, f[i]);
      hi = fmaxf(hi, f[i]);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (!on) return;
    const float span = __fsub_rn(hi, lo);
    const bool flat = span < 1e-30f;
    const float scale = flat ? 0.0f : __fdiv_rn(span, 15.0f);
    const float inv = flat ? 0.0f : __fdiv_rn(15.0f, span);
    uint2 w2 = make_uint2(0u, 0u);
    if (!flat) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w2.x |= static_cast<uint32_t>(quant_code(f[i], lo, hi, inv)) << (4 * i);
        w2.y |= static_cast<uint32_t>(quant_code(f[8 + i], lo, hi, inv)) << (4 * i);
      }
    }
    *codes = w2;
    if (l == 0) *meta = make_float2(scale, lo);
  }
}

template <int D, typename T, bool kRead>
cudaError_t launch_rows(const DeviceContext* ctx, const KvView& c, void* k, void* v, int64_t T_rows, cudaStream_t s) {
  const int64_t groups = (c.heads + 512 / D - 1) / (512 / D);
  const int64_t ctas = (T_rows * groups + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  k_kv4_rows<D, T, kRead><<<dim3(static_cast<unsigned>(ctas), 2), kWarps * 32, 0, s>>>(
      c, static_cast<T*>(k), static_cast<T*>(v), static_cast<int>(T_rows), ctx->err_word);
  return cudaGetLastError();
}

template <bool kRead>
cudaError_t launch_rows_any(const DeviceContext* ctx, const KvView& c, int head_dim, void* k, void* v, int dtype,
                            int64_t T_rows, cudaStream_t s) {
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return head_dim == 128 ? launch_rows<128, T, kRead>(ctx, c, k, v, T_rows, s)
                           : launch_rows<256, T, kRead>(ctx, c, k, v, T_rows, s);
  };
  switch (dtype) {
    case BITNET_DTYPE_F32: return go(static_cast<float*>(nullptr));
    case BITNET_DTYPE_F16: return go(static_cast<__half*>(nullptr));
    case BITNET_DTYPE_BF16: return go(static_cast<__nv_bfloat16*>(nullptr));
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_kv4_append(const DeviceContext* ctx, const KvView& c, int head_dim, const void* k, const void* v,
                              int dtype, int64_t T, cudaStream_t s) {
  return launch_rows_any<false>(ctx, c, head_dim, const_cast<void*>(k), const_cast<void*>(v), dtype, T, s);
}

cudaError_t launch_kv4_read(const DeviceContext* ctx, const KvView& c, int head_dim, void* k, void* v, int dtype,
                            int64_t T, cudaStream_t s) {
  return launch_rows_any<true>(ctx, c, head_dim, k, v, dtype, T, s);
}

}  // namespace bitnet
