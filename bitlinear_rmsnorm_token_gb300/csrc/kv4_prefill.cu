// kv4_prefill.cu -- attention of many query rows per sequence over the paged
// 4-bit cache (prompts, chunks of prompts, whole texts) on the 5th-generation
// tensor cores.
//
// A tile is 128 query rows of a (sequence, kv head): row r is query head
// h G + r % G of token r / G, so the heads that share keys share the tile.  A CTA
// takes two tiles (head_dim 128) or one (256) and walks the pages that their rows
// see, 64 keys at a time, with the running maximum and sum of a one-pass softmax:
//   S[128, 64]  = Q K^T   (tcgen05, fp16 operands, both in shared memory)
//   p = 2^(c S - ref)
//   O[128, D] += W V      (W from tensor memory)
// O, S and W live in tensor memory; W takes S's place.  A row's reference only
// moves when its maximum has grown by 2^8 (O is then rescaled), so most pages are
// taken without a maximum, scores to W in one pass.
//
// What stands for K and V depends on the query type:
//   bf16: the stored values rounded to fp16 (11 bits: 1/8 of the rounding that the
//     queries and the output have), times a power of two of the page's largest
//     key and of the largest value met; W = p as fp16.  c S is one fma, and the
//     softmax, which sets the pace, has 5 instructions a pair of scores instead of
//     11 (chunk of 4096 over 12288 tokens: see the last line).
//   fp16, fp32: the codes as c - 8, exact, with the scales outside the products
//     (kv4.cuh): x = s_j S + (m_j + 8 s_j) sum(q), W = p s_j times a power of two,
//     and sum p_j (m_j + 8 s_j) beside O.  fp32 queries and their W are two fp16
//     parts each (22 bits), two products where 16-bit ones take one.
//
// Warps: 4 per tile for the softmax (a thread a row), 8 or 12 that decode pages
// into the operands' swizzled layout (values transposed: rows are dimensions, in
// the order that keeps the stores of a warp on different banks), a producer of
// raw pages, and an MMA issuer per tile.  S is double buffered, so that the next
// page's scores are computed while a page's softmax runs.
// Few tiles on a long cache: the pages are split over gridDim.z and the parts
// joined by a second launch, in order.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "rowquant.cuh"

namespace bitnet {
namespace {

constexpr int kRows = 128;          // rows of a tile
constexpr float kLazy = 8.0f;       // a row's maximum may pass its reference by this many powers of two
constexpr int kWExp = 6;            // value scales are below 2^(kWExp + 1) after their power of two: times 2^kLazy < 2^15

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
// e of 2^e <= v < 2^(e+1), kept in [-100, 100].
__device__ __forceinline__ int pow2_exp(float v) { return min(max((__float_as_int(v) >> 23) - 127, -100), 100); }

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs of floats in one 64-bit register: two operations an instruction.
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_pack(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Codes in bits 0-3 (4-7) of both halves of w, other bits ignored, to fp16 c - 8.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x64006400u;  // 1024 + c
  const uint32_t k = 0x64086408u;                      // 1032
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  const uint32_t x = (w & 0x00f000f0u) | 0x64006400u;    // 1024 + 16 c
  const uint32_t k = 0x2c002c00u, m = 0xd480d480u;       // 1/16, -72
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k),
                            *reinterpret_cast<const __half2*>(&m));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands: A's column c holds K elements 2c, 2c + 1.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// c s + mid of two codes, s in two parts: one rounding of the sum (and of mid).
__device__ __forceinline__ uint32_t decode_h2(uint32_t c, uint32_t hi, uint32_t lo, uint32_t mid) {
  const __half2 x = *reinterpret_cast<const __half2*>(&c);
  const __half2 t = __hfma2(x, *reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&mid));
  const __half2 r = __hfma2(x, *reinterpret_cast<const __half2*>(&hi), t);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A page's per-key factors, and what the softmax has to know of the page.
struct __align__(16) PageMeta {
  float ks[kKvPage], kmid[kKvPage];  // s, m + 8 s of the keys
  float vs[kKvPage], vmid[kKvPage];  // s 2^(kWExp - e), m + 8 s of the values
  int key0;           // position of the page's first token
  int ok;             // 0: no such page, its keys are masked
  int e;              // the power of two that the value scales (bf16: values) lie below
  float gk;           // bf16: what a unit of S counts (the keys' power of two)
};

// bf16: s (two parts) and m + 8 s of a page's rows as fp16, times the operands' powers of two; zeros for tokens that do
// not exist and for rows that are not finite (they stand for unspecified values, and must not reach other queries).
struct __align__(16) PageTab {
  uint4 k[kKvPage];  // each twice, for both halves of a word: s high, s low, m + 8 s
  __half v_hi[kKvPage], v_lo[kKvPage], v_mid[kKvPage];
};

template <int D, bool kSplit, bool kDeq>
struct Layout {
  static constexpr int kT = D == 128 ? 2 : 1;                // tiles per CTA
  static constexpr int kParts = kSplit ? 2 : 1;
  // Decode warps: heads of 128, groups of 4 that take every kGroups-th page each; heads of 256, 8 that decode the keys
  // of every page and 4 the values.  Raw page slots (whole turns of the groups) and operand stages (at least a turn):
  // no group can then be a phase ahead of what a barrier's parity tells.
  static constexpr bool kByRole = D == 256;
  static constexpr int kGroups = D == 128 && !kSplit ? 2 : 1;
  static constexpr int kKeyWarps = kByRole ? 8 : 4, kValWarps = 4;
  static constexpr int kDecodeWarps = kByRole ? kKeyWarps + kValWarps : 4 * kGroups;
  static constexpr int kPageWarps = kByRole ? kDecodeWarps : 4;  // warps that take part in a page
  static constexpr int kRaw = D == 128 ? (kSplit ? 2 : 4) : (kSplit ? 1 : 2);
  static constexpr int kK = D == 128 ? (kSplit ? 2 : 3) : 1;
  static constexpr int kV = D == 128 ? (kSplit ? 2 : 3) : (kSplit ? 1 : 2);
  static_assert(kRaw % kGroups == 0 && kK >= kGroups && kV >= kGroups, "see above");
  static constexpr int kMeta = 4;
  static constexpr int kSoftWarps = 4 * kT;
  static constexpr int kProducer = kSoftWarps + kDecodeWarps;  // then an MMA warp per tile
  static constexpr int kMma0 = kProducer + 1;
  static constexpr int kThreads = 32 * (kMma0 + kT);
  static constexpr int kQPart = kRows * D * 2;               // bytes of one part of a tile's queries
  static constexpr int kOp = kKvPage * D * 2;                // bytes of a page's keys (values) as fp16
  static constexpr int offQ = 0;
  static constexpr int offK = offQ + kT * kParts * kQPart;
  static constexpr int offV = offK + kK * kOp;
  static constexpr int offRaw = offV + kV * kOp;
  static constexpr int offMeta = offRaw + kRaw * KvBlock<D>::kBytes;
  static constexpr int kNumBars = 2 * kRaw + 2 * kK + 2 * kV + 2 * kMeta + 7 * kT + 4;
  static constexpr int offBar = offMeta + kMeta * static_cast<int>(sizeof(PageMeta));
  static constexpr int offRow = offBar + kNumBars * 8;       // float2 per row: sum(q), its factor
  static constexpr int offTab = (offRow + kT * kRows * 8 + 15) / 16 * 16;  // two pages' factors of each group
  static constexpr int offMisc = offTab + (kDeq ? 2 * kGroups * static_cast<int>(sizeof(PageTab)) : 0);  // 48 ints
  static constexpr int kBytes = offMisc + 192;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "over the 227 KB of shared memory a CTA may use");
  // tensor memory: scores (two buffers) and output of each tile
  static constexpr int kCols = 512;
  __host__ __device__ static constexpr int s_col(int t, int buf) { return D == 128 ? 256 * t + 64 * buf : 256 + 64 * buf; }
  __host__ __device__ static constexpr int o_col(int t) { return D == 128 ? 256 * t + 128 : 0; }
};

struct Problem {
  KvView c;
  int Hq, G, T, max_q;
  float scale;  // |softmax scale| * log2(e)
  float sign;   // its sign, given to the queries
  int causal, window;
  unsigned* err;
  float* part;  // [splits][T * Hq][D + 4], or null
};

template <int D, typename QT, typename OT>
__global__ void __launch_bounds__(
    Layout<D, std::is_same<QT, float>::value, std::is_same<QT, __nv_bfloat16>::value>::kThreads, 1)
    k_kv4_prefill(const Problem p, const QT* __restrict__ q, OT* __restrict__ out) {
  constexpr bool kSplit = std::is_same<QT, float>::value, kDeq = std::is_same<QT, __nv_bfloat16>::value;
  using L = Layout<D, kSplit, kDeq>;
  using B = KvBlock<D>;
  constexpr int kT = L::kT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  PageMeta* metas = reinterpret_cast<PageMeta*>(smem + L::offMeta);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::offBar);
  uint64_t* raw_empty = raw_full + L::kRaw;
  uint64_t* k_full = raw_empty + L::kRaw;
  uint64_t* k_empty = k_full + L::kK;
  uint64_t* v_full = k_empty + L::kK;
  uint64_t* v_empty = v_full + L::kV;
  uint64_t* meta_full = v_empty + L::kV;
  uint64_t* meta_empty = meta_full + L::kMeta;
  uint64_t* s_full = meta_empty + L::kMeta;  // [tile][buffer]
  // [tile][buffer]: a warp may be done with page j + 1 before another is with page j, but not with page j + 2
  uint64_t* p_full = s_full + 2 * kT;
  uint64_t* pv_done = p_full + 2 * kT;       // [tile]
  uint64_t* drained = pv_done + kT;          // [tile]: only on giving up
  uint64_t* tab_full = drained + kT;         // [group or role][2]: the table of factors is written (bf16)
  uint64_t* o_done = tab_full + 4;            // [tile]: the last product is done
  int* misc = reinterpret_cast<int*>(smem + L::offMisc);
  volatile int* abort_flag = misc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
  // misc[2 .. 6]: sequence, pair of tiles, first row, rows and length; misc[8..]: running sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  // ---- which rows: unit `want` of kv head `head`, the last units (longest rows of a causal prompt) first
  const int head = blockIdx.x % p.c.heads;
  const int want = gridDim.x / p.c.heads - 1 - blockIdx.x / p.c.heads;
  if (threadIdx.x == 0) misc[2] = -1;
  if (threadIdx.x == 32) {
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], L::kPageWarps);
    }
    for (int i = 0; i < L::kK; ++i) {
      mbar_init(&k_full[i], L::kKeyWarps);
      mbar_init(&k_empty[i], kT);
    }
    for (int i = 0; i < L::kV; ++i) {
      mbar_init(&v_full[i], L::kValWarps);
      mbar_init(&v_empty[i], kT);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&tab_full[i], i < 2 ? L::kKeyWarps : L::kValWarps);
    for (int i = 0; i < L::kMeta; ++i) {
      mbar_init(&meta_full[i], L::kPageWarps);
      mbar_init(&meta_empty[i], L::kSoftWarps);
    }
    for (int i = 0; i < kT; ++i) {
      mbar_init(&s_full[2 * i], 1);
      mbar_init(&s_full[2 * i + 1], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&drained[i], 1);
      mbar_init(&o_done[i], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  {
    int base = 0;
    for (int c0 = 0; c0 < p.c.num_seqs; c0 += L::kThreads) {
      const int i = c0 + threadIdx.x;
      int units = 0, n_i = 0, q_i = 0, len_i = 0;
      if (i < p.c.num_seqs) {
        bool bad = false;
        q_i = p.c.q_start[i];
        const int64_t n64 = static_cast<int64_t>(p.c.q_start[i + 1]) - q_i;
        len_i = kv_len_of(p.c, i, &bad);
        if (n64 < 0 || n64 > p.max_q || q_i < 0 || q_i + n64 > p.T) bad = true;
        else n_i = static_cast<int>(n64);
        if (bad) atomicOr(p.err, kErrBadIndex);
        units = (n_i * p.G + kT * kRows - 1) / (kT * kRows);
      }
      int x = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) misc[8 + warp] = x;
      __syncthreads();
      // running sums over the warps, a lane each
      int ws = lane < L::kThreads / 32 ? misc[8 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o) ws += y;
      }
      const int total = __shfl_sync(0xffffffffu, ws, 31);
      const int before = warp ? __shfl_sync(0xffffffffu, ws, warp - 1) : 0;
      const int lo = base + before + x - units;
      if (want >= lo && want < lo + units) {
        misc[2] = i;
        misc[3] = want - lo;
        misc[4] = q_i;
        misc[5] = n_i;
        misc[6] = len_i;
      }
      base += total;
    }
  }
  __syncthreads();
  const int b = misc[2];
  if (b < 0) return;  // the grid is sized for any division of the rows
  if (warp == L::kMma0) {
    tmem_alloc(tmem_slot, L::kCols);
    tmem_relinquish();
  }
  const int row0 = misc[3] * kT * kRows;              // first row of the CTA
  const int q0 = misc[4], n = misc[5], len = misc[6];
  const int rows = n * p.G;
  const int pos0 = len - n;                           // position of the sequence's first query token
  // pages that any of the CTA's rows sees
  int page0 = 0, pages = (len + kKvPage - 1) / kKvPage;
  if (p.causal) {
    const int last = pos0 + (min(row0 + kT * kRows, rows) - 1) / p.G;  // position of the last row
    pages = last < 0 ? 0 : min(pages, last / kKvPage + 1);
    if (p.window > 0) page0 = max(0, pos0 + row0 / p.G - p.window + 1) / kKvPage;
  }
  pages = max(0, pages - page0);
  if (gridDim.z > 1) {  // this part's pages (at most 2^25 pages and 64 parts: 32 bits)
    const unsigned all = pages, a = all * blockIdx.z / gridDim.z;
    pages = static_cast<int>(all * (blockIdx.z + 1) / gridDim.z - a);
    page0 += static_cast<int>(a);
  }
  // ---- the first pages, under way while the queries are read
  auto load_page = [&](int j) {
    const int rs = j % L::kRaw;
    const int page = p.c.page_table[static_cast<int64_t>(b) * p.c.max_pages + page0 + j];
    if (page < 0 || page >= p.c.num_pages) {
      atomicOr(p.err, kErrBadIndex);
      mbar_arrive(&raw_full[rs]);
    } else {
      mbar_arrive_expect_tx(&raw_full[rs], B::kBytes);
      bulk_load(smem + L::offRaw + rs * B::kBytes,
                p.c.cache + (static_cast<int64_t>(page) * p.c.heads + head) * B::kBytes, B::kBytes, &raw_full[rs]);
    }
  };
  if (warp == L::kProducer && lane == 0)
    for (int j = 0; j < min(pages, L::kRaw); ++j) load_page(j);
  // ---- queries, scaled by a power of two per row, as fp16 (one part or two): D / 8 lanes to a row, 8 dimensions
  // each, all warps, the loads of a lane's rows in flight
  float2* row_q = reinterpret_cast<float2*>(smem + L::offRow);
  {
    constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes of a row, rows of a warp at a time
    constexpr int kStep = L::kThreads / 32 * kAt, kBatch = (kT * kRows + kStep - 1) / kStep;
    constexpr int kVecs = sizeof(QT) / 2;             // 16-byte loads of 8 dimensions
    const int c = lane % kLanes;
    const int t0 = warp * kAt + lane / kLanes;
    {
      uint4 raw[kBatch][kVecs];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int row = row0 + t0 + k * kStep;
        const int i = row / p.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            q + (static_cast<int64_t>(q0 + i) * p.Hq + head * p.G + (row - i * p.G)) * D + 8 * c);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) raw[k][u] = row < rows && t0 + k * kStep < kT * kRows ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int rr = t0 + k * kStep, tl = rr / kRows, rt = rr % kRows;
          if (rr >= kT * kRows) break;  // the same for the whole warp
        const QT* x = reinterpret_cast<const QT*>(raw[k]);
        float v[8], top = 0.0f;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          v[d] = static_cast<float>(x[d]);
          top = fmaxf(top, fabsf(v[d]));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = pow2_exp(top);
        const float f = p.sign * pow2(14 - e);
        // chunk c of the row: dimensions 8c + 0, 4, 1, 5, 2, 6, 3, 7, the order in which a word of codes decodes
        uint8_t* dst = smem + L::offQ + tl * L::kParts * L::kQPart + (c >> 3) * (kRows * 128) + (rt >> 3) * 1024 +
                       (rt & 7) * 128 + (((c & 7) ^ (rt & 7)) << 4);
        float h[8], sum = 0.0f;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          v[d] *= f;
          h[d] = __half2float(__float2half_rn(v[d]));
          sum += h[d];
        }
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(pack_h2(h[0], h[4]), pack_h2(h[1], h[5]), pack_h2(h[2], h[6]), pack_h2(h[3], h[7]));
        if constexpr (kSplit) {
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            h[d] = __half2float(__float2half_rn(v[d] - h[d]));
            sum += h[d];
          }
          *reinterpret_cast<uint4*>(dst + L::kQPart) =
              make_uint4(pack_h2(h[0], h[4]), pack_h2(h[1], h[5]), pack_h2(h[2], h[6]), pack_h2(h[3], h[7]));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (c == 0) row_q[rr] = make_float2(sum, p.scale * pow2(e - 14));
      }
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < L::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;  // this warp's quarter of the TMEM lanes
    const int tile = warp >> 2;
    const int tile_r0 = row0 + tile * kRows;
    const int r = tile_r0 + (threadIdx.x & 127);  // row of the item
    const bool row_on = r < rows;
    const int i_tok = row_on ? r / p.G : 0;
    const int64_t q_at = static_cast<int64_t>(q0 + i_tok) * p.Hq + head * p.G + (row_on ? r - i_tok * p.G : 0);
    const float2 row = row_q[threadIdx.x];
    const float qc = row.y;
    const f2 qsum2 = f2_pack(row.x, row.x);
    const int pos = row_on ? pos0 + i_tok : len - 1;
    const int key_hi = p.causal ? min(pos, len - 1) : len - 1;
    const int key_lo = p.causal && p.window > 0 ? pos - p.window + 1 : 0;
    // pages between these need no mask for any row of the tile
    const int free_hi = p.causal ? min(pos0 + tile_r0 / p.G, len - 1) : len - 1;
    const int free_lo = p.causal && p.window > 0 ? pos0 + (min(tile_r0 + kRows, rows) - 1) / p.G - p.window + 1 : 0;
    float m_ref = -INFINITY;
    f2 l2 = 0, z2 = 0;  // sums of the even and of the odd keys
    int e_run = 0;      // values count up to 2^e_run in O
    // O by f, once the product before page j is done with it.
    auto rescale = [&](int j, float f) -> bool {
      if (!mbar_wait(&pv_done[tile], (j - 1) & 1, p.err, abort_flag)) return false;
      tc_fence_after();
      __syncwarp();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tmem_read_x16(tmem + lanes + static_cast<uint32_t>(L::o_col(tile) + c), o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st_32x32b_x16(tmem + lanes + static_cast<uint32_t>(L::o_col(tile) + c), o);
      }
      tmem_st_wait();
      return true;
    };
    // Half hf (32 keys) of a page's scores, as x of p = 2^(c x - ref).
    auto load_x = [&](uint32_t s_addr, const PageMeta& meta, int hf, f2 (&x)[16]) {
      uint32_t sv[32];
      tmem_read_x32(s_addr + 32 * hf, sv);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = f2_pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
      if constexpr (!kDeq) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const ulonglong2 ks = *reinterpret_cast<const ulonglong2*>(&meta.ks[32 * hf + 2 * i]);
          const ulonglong2 km = *reinterpret_cast<const ulonglong2*>(&meta.kmid[32 * hf + 2 * i]);
          x[i] = f2_fma(x[i], ks.x, f2_mul(km.x, qsum2));
          x[i + 1] = f2_fma(x[i + 1], ks.y, f2_mul(km.y, qsum2));
        }
      }
    };
    // The half's probabilities to W (w0 and, two parts, w1), added to lp and zp.  kMasked: x is -inf where a key is
    // hidden, whose value row must not matter whatever it holds.
    auto weigh = [&](const PageMeta& meta, int hf, const f2 (&x)[16], f2 qg2, f2 ref2, float live, f2& lp, f2& zp,
                     uint32_t* w0, uint32_t* w1, auto masked_tag) {
      constexpr bool kMasked = decltype(masked_tag)::value;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        [[maybe_unused]] ulonglong2 vs, vm;
        if constexpr (!kDeq) {
          vs = *reinterpret_cast<const ulonglong2*>(&meta.vs[32 * hf + 2 * i]);
          vm = *reinterpret_cast<const ulonglong2*>(&meta.vmid[32 * hf + 2 * i]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float wa, wb, xa, xb;
          f2_unpack(x[i + k], xa, xb);
          f2_unpack(f2_fma(x[i + k], qg2, ref2), wa, wb);
          wa = ex2(wa);
          wb = ex2(wb);
          if constexpr (kMasked) {
            if (xa == -INFINITY) wa = 0.0f;
            if (xb == -INFINITY) wb = 0.0f;
          }
          const f2 pr = f2_pack(wa, wb);
          lp = f2_add(lp, pr);
          if constexpr (!kDeq) {
            f2 vmk = k ? vm.y : vm.x;
            f2_unpack(f2_mul(pr, k ? vs.y : vs.x), wa, wb);
            if constexpr (kMasked) {
              float ma, mb;
              f2_unpack(vmk, ma, mb);
              if (xa == -INFINITY) wa = ma = 0.0f;
              if (xb == -INFINITY) wb = mb = 0.0f;
              vmk = f2_pack(ma, mb);
            }
            zp = f2_fma(pr, vmk, zp);
          }
          if constexpr (kMasked) {
            wa *= live;
            wb *= live;
          }
          w0[i + k] = pack_h2(wa, wb);
          if constexpr (kSplit) {
            const __half2 h = *reinterpret_cast<const __half2*>(&w0[i + k]);
            w1[i + k] = pack_h2(wa - __low2float(h), wb - __high2float(h));
          }
        }
      }
    };
    // A page that every row of the warp sees whole, against the references as they are: no maximum is taken. A row's
    // sum above 2^kLazy (as every probability above it makes) gives the page back to the other path, which moves the
    // reference; otherwise each probability is within what W holds.
    auto page_fast = [&](uint32_t s_addr, const PageMeta& meta, int de) -> bool {
      const float qg = kDeq ? qc * meta.gk : qc, ref = static_cast<float>(de) - m_ref;
      const f2 qg2 = f2_pack(qg, qg), ref2 = f2_pack(ref, ref);
      f2 lp = 0, zp = 0;
      uint32_t w0[32];
      [[maybe_unused]] uint32_t w1[32];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        f2 x[16];
        load_x(s_addr, meta, hf, x);
        weigh(meta, hf, x, qg2, ref2, 1.0f, lp, zp, w0 + 16 * hf, w1 + 16 * hf, std::false_type{});
      }
      float a, b;
      f2_unpack(lp, a, b);
      const float un = pow2(-de);
      if (__any_sync(0xffffffffu, (a + b) * un > 256.0f)) return false;  // 2^kLazy
      const f2 un2 = f2_pack(un, un);
      l2 = f2_fma(lp, un2, l2);
      z2 = f2_fma(zp, un2, z2);
      tmem_st_32x32b_x32(s_addr, w0);
      if constexpr (kSplit) tmem_st_32x32b_x32(s_addr + 32, w1);
      return true;
    };
    // Any page: the maximum first, then the same sums in the same order (a row's bits do not depend on the rows beside
    // it).  live: 0 where the page's values are too small to count beside those met.
    auto page = [&](int j, uint32_t s_addr, const PageMeta& meta, int de, float live) -> bool {
      const float qg = kDeq ? qc * meta.gk : qc;
      const int hi = meta.ok ? key_hi - meta.key0 : -1, lo = key_lo - meta.key0;
      auto load_masked = [&](int hf, f2 (&x)[16]) {
        load_x(s_addr, meta, hf, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = 32 * hf + 2 * i;
          float a, b;
          f2_unpack(x[i], a, b);
          if (key > hi || key < lo) a = -INFINITY;
          if (key + 1 > hi || key + 1 < lo) b = -INFINITY;
          x[i] = f2_pack(a, b);
        }
      };
      float top = -INFINITY;
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        f2 x[16];
        load_masked(hf, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a, b;
          f2_unpack(x[i], a, b);
          top = fmaxf(top, fmaxf(a, b));
        }
      }
      float f = 1.0f;
      if (top != -INFINITY) {
        const float m = top * qg;
        if (m_ref == -INFINITY) {
          m_ref = m;  // nothing summed yet
        } else if (m > m_ref + kLazy) {
          f = ex2(m_ref - m);
          m_ref = m;
          const f2 ff = f2_pack(f, f);
          l2 = f2_mul(l2, ff);
          z2 = f2_mul(z2, ff);
        }
      }
      if (j > 0 && __any_sync(0xffffffffu, f != 1.0f) && !rescale(j, f)) return false;
      const float ref = static_cast<float>(de) - (m_ref == -INFINITY ? 0.0f : m_ref);
      const f2 qg2 = f2_pack(qg, qg), ref2 = f2_pack(ref, ref);
      f2 lp = 0, zp = 0;
      // (both halves' W are held back until the scores have been read)
      uint32_t w0[32];
      [[maybe_unused]] uint32_t w1[32];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        f2 x[16];
        load_masked(hf, x);
        weigh(meta, hf, x, qg2, ref2, live, lp, zp, w0 + 16 * hf, w1 + 16 * hf, std::true_type{});
      }
      const float un = pow2(-de);
      const f2 un2 = f2_pack(un, un);
      l2 = f2_fma(lp, un2, l2);
      z2 = f2_fma(zp, un2, z2);
      tmem_st_32x32b_x32(s_addr, w0);
      if constexpr (kSplit) tmem_st_32x32b_x32(s_addr + 32, w1);
      return true;
    };
    bool ok = true;
    for (int j = 0; j < pages; ++j) {
      const int buf = j & 1, ms = j % L::kMeta;
      const uint32_t s_addr = tmem + lanes + static_cast<uint32_t>(L::s_col(tile, buf));
      if (!mbar_wait(&meta_full[ms], (j / L::kMeta) & 1, p.err, abort_flag) ||
          !mbar_wait(&s_full[2 * tile + buf], (j >> 1) & 1, p.err, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      __syncwarp();
      const PageMeta& meta = metas[ms];
      // ---- the values' power of two: O moves with it (seldom: it has some room); a page of smaller values is weighed
      // by 2^de, and not at all beyond 2^-40 (its probabilities still count)
      const int e = meta.e;
      if (j == 0) {
        e_run = e + 1;
      } else if (e > e_run) {
        if (!rescale(j, pow2(max(e_run - e - 1, -120)))) {
          ok = false;
          break;
        }
        e_run = e + 1;
      }
      const bool small = e - e_run < -40;
      const int de = small ? 0 : e - e_run;
      const bool masked = !meta.ok || meta.key0 < free_lo || meta.key0 + kKvPage - 1 > free_hi;
      const bool fast = !masked && !small && __all_sync(0xffffffffu, m_ref != -INFINITY);
      if (!fast || !page_fast(s_addr, meta, de)) ok = page(j, s_addr, meta, de, small ? 0.0f : 1.0f);
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&p_full[2 * tile + buf]);
        mbar_arrive(&meta_empty[ms]);
      }
    }
    float l, z;
    {
      float a, b;
      f2_unpack(l2, a, b);
      l = a + b;
      f2_unpack(z2, a, b);
      z = a + b;
    }
    // ---- the row's result
    // (a barrier of its own: this warp may be up to two products ahead of pv_done, whose parity says nothing then)
    if (ok && (pages == 0 || mbar_wait(&o_done[tile], 0, p.err, abort_flag))) {
      tc_fence_after();
      __syncwarp();
      const float un_w = pow2(e_run - kWExp);
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // no key seen: zeros; NaN stays
      const bool any_on = tile_r0 + 32 * (warp & 3) < rows;
      if (any_on) {
#pragma unroll 1
        for (int a = 0; a < D / 32; ++a) {
          // dimensions 32 a ..: columns d (D / 8) + 4 a .. + 3 hold dimension d of the groups of 8
          uint32_t o[32];
          if (pages > 0) tmem_read_8x4(tmem + lanes + static_cast<uint32_t>(L::o_col(tile) + 4 * a), D / 8, o);
          if (row_on) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int d = 0; d < 8; ++d) v[8 * k + d] = pages > 0 ? fmaf(__uint_as_float(o[4 * d + k]), un_w, z) : 0.0f;
            if (p.part) {
              float* dst = p.part + (static_cast<int64_t>(blockIdx.z) * p.T * p.Hq + q_at) * (D + 4) + 32 * a;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
              OT* dst = out + q_at * D + 32 * a;
              constexpr int kPer = 16 / static_cast<int>(sizeof(OT));
#pragma unroll
              for (int i = 0; i < 32 / kPer; ++i) {
                union { OT v[kPer]; uint4 u; } pk;
#pragma unroll
                for (int k = 0; k < kPer; ++k) pk.v[k] = round_out<OT>(v[i * kPer + k] * inv);
                reinterpret_cast<uint4*>(dst)[i] = pk.u;
              }
            }
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (p.part && row_on)
          *reinterpret_cast<float2*>(p.part + (static_cast<int64_t>(blockIdx.z) * p.T * p.Hq + q_at) * (D + 4) + D) =
              make_float2(m_ref, l);
      }
    }
  } else if (warp < L::kProducer) {
    // ------------------------------------------------------------ decode
    // Pages first, first + step, .. : their keys and / or values, by kU threads.
    auto decode_pages = [&](auto threads, auto keys_tag, auto vals_tag, int ut, int first, int step, uint64_t* tab_bar,
                            PageTab* tabs) {
      constexpr int kU = decltype(threads)::value;
      constexpr bool kKeys = decltype(keys_tag)::value, kVals = decltype(vals_tag)::value;
      constexpr int kWords = D / 8;  // words of a row
      for (int j = first, it = 0; j < pages; j += step, ++it) {
        const int rs = j % L::kRaw, ks = j % L::kK, vs = j % L::kV, ms = j % L::kMeta;
        const int page = p.c.page_table[static_cast<int64_t>(b) * p.c.max_pages + page0 + j];
        const bool ok = page >= 0 && page < p.c.num_pages;
        const int key0 = (page0 + j) * kKvPage;
        if (!mbar_wait(&raw_full[rs], (j / L::kRaw) & 1, p.err, abort_flag)) return;
        const uint8_t* raw = smem + L::offRaw + rs * B::kBytes;
        const float2* kmeta = reinterpret_cast<const float2*>(raw + B::offKMeta);
        const float2* vmeta = reinterpret_cast<const float2*>(raw + B::offVMeta);
        // ---- factors: every warp finds the page's largest value (value scale), and key where it decodes keys
        if (!mbar_wait(&meta_empty[ms], ((j / L::kMeta) & 1) ^ 1, p.err, abort_flag)) return;
        PageMeta& meta = metas[ms];
        auto largest = [&](const float2* m) {
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = m[lane + 32 * i];
            // bf16: what the row's values lie below, of finite rows
            const float most = kDeq ? fmaf(8.0f, fabsf(v.x), fabsf(fmaf(8.0f, v.x, v.y))) : v.x;
            if (ok && key0 + lane + 32 * i < len && (!kDeq || most < INFINITY)) top = fmaxf(top, most);
          }
          return pow2_exp(warp_max(top));
        };
        // thread ut's row of the page: a key, or a value from thread kKvPage on (where both are decoded)
        auto factor = [&](const float2* m, bool is_v, int key, int e) {
          const float2 sm = m[key];
          const float mid = fmaf(8.0f, sm.x, sm.y);
          if constexpr (kDeq) {
            const bool use = ok && key0 + key < len && fmaf(8.0f, fabsf(sm.x), fabsf(mid)) < INFINITY;
            const float f = pow2(kWExp - e), sc = use ? sm.x * f : 0.0f;
            const __half hi = __float2half_rn(sc), lo = __float2half_rn(sc - __half2float(hi));
            const __half md = __float2half_rn(use ? mid * f : 0.0f);
            PageTab& tab = tabs[it & 1];
            if (is_v) {
              tab.v_hi[key] = hi;
              tab.v_lo[key] = lo;
              tab.v_mid[key] = md;
            } else {
              const uint32_t h2 = __half_as_ushort(hi), l2 = __half_as_ushort(lo), m2 = __half_as_ushort(md);
              tab.k[key] = make_uint4(h2 | (h2 << 16), l2 | (l2 << 16), m2 | (m2 << 16), 0u);
            }
          } else {
            (is_v ? meta.vs : meta.ks)[key] = is_v ? sm.x * pow2(kWExp - e) : sm.x;
            (is_v ? meta.vmid : meta.kmid)[key] = mid;
          }
        };
        if constexpr (kKeys) {
          const int e = kDeq ? largest(kmeta) : 0;
          if (ut < kKvPage) factor(kmeta, false, ut, e);
          if (ut == 0) {
            meta.key0 = key0;
            meta.ok = ok ? 1 : 0;
            meta.gk = pow2(e - kWExp);
          }
        }
        if constexpr (kVals) {
          const int e = largest(vmeta);
          const int key = kKeys ? ut - kKvPage : ut;
          if (key >= 0 && key < kKvPage) factor(vmeta, true, key, e);
          if (key == 0) meta.e = e;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&meta_full[ms]);
        if constexpr (kDeq) {  // written by several warps; the other table may still be in use for the page before
          if (lane == 0) mbar_arrive(&tab_bar[it & 1]);
          if (!mbar_wait(&tab_bar[it & 1], (it >> 1) & 1, p.err, abort_flag)) return;
        }
        // ---- keys: a word (8 dimensions) to a 16-byte chunk of the key's operand row, a thread its word column
        if constexpr (kKeys) {
          if (!mbar_wait(&k_empty[ks], ((j / L::kK) & 1) ^ 1, p.err, abort_flag)) return;
          constexpr int kStep = kU / kWords;
          const int w = ut % kWords, key = ut / kWords;
          const uint8_t* src = raw + B::offK + key * B::kRow + 4 * w;
          uint8_t* dst = smem + L::offK + ks * L::kOp + (w >> 3) * (kKvPage * 128);
          uint32_t a[kKvPage / kStep];
#pragma unroll
          for (int i = 0; i < kKvPage / kStep; ++i)
            a[i] = ok ? *reinterpret_cast<const uint32_t*>(src + i * kStep * B::kRow) : 0x88888888u;
#pragma unroll
          for (int i = 0; i < kKvPage / kStep; ++i) {
            const int at = key + i * kStep;
            const uint32_t a8 = a[i] >> 8;
            uint4 o = make_uint4(codes_lo(a[i]), codes_hi(a[i]), codes_lo(a8), codes_hi(a8));
            if constexpr (kDeq) {
              const uint4 f = tabs[it & 1].k[at];
              o = make_uint4(decode_h2(o.x, f.x, f.y, f.z), decode_h2(o.y, f.x, f.y, f.z), decode_h2(o.z, f.x, f.y, f.z),
                             decode_h2(o.w, f.x, f.y, f.z));
            }
            *reinterpret_cast<uint4*>(dst + at * 128 + (((w & 7) ^ (at & 7)) << 4)) = o;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[ks]);
        }
        // ---- values, transposed: a word of 8 consecutive keys to 8 chunks, one per dimension; dimension 8 w + d is
        // operand row d (D / 8) + w, so that a warp's chunks of one d lie in consecutive rows (different banks)
        if constexpr (kVals) {
          if (!mbar_wait(&v_empty[vs], ((j / L::kV) & 1) ^ 1, p.err, abort_flag)) return;
          static_assert(8 * kWords % kU == 0, "whole turns of the group");
#pragma unroll 1
          for (int id = ut; id < 8 * kWords; id += kU) {
            const int w = id % kWords, kg = id / kWords;
            const uint8_t* src = raw + B::offV + 8 * kg * B::kRow + 4 * w;
            uint8_t* dst = smem + L::offV + vs * L::kOp + (w >> 3) * 1024 + (w & 7) * 128 + ((kg ^ (w & 7)) << 4);
            uint32_t a[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] = ok ? *reinterpret_cast<const uint32_t*>(src + k * B::kRow) : 0x88888888u;
            [[maybe_unused]] uint4 fh, fl, fm;
            if constexpr (kDeq) {  // of the 8 keys, neighbours in the halves of a word
              fh = reinterpret_cast<const uint4*>(tabs[it & 1].v_hi)[kg];
              fl = reinterpret_cast<const uint4*>(tabs[it & 1].v_lo)[kg];
              fm = reinterpret_cast<const uint4*>(tabs[it & 1].v_mid)[kg];
            }
            auto put = [&](uint8_t* at, uint4 o) {
              if constexpr (kDeq)
                o = make_uint4(decode_h2(o.x, fh.x, fl.x, fm.x), decode_h2(o.y, fh.y, fl.y, fm.y),
                               decode_h2(o.z, fh.z, fl.z, fm.z), decode_h2(o.w, fh.w, fl.w, fm.w));
              *reinterpret_cast<uint4*>(at) = o;
            };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t sel = c | ((4 + c) << 8);
              uint32_t pr[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) pr[k] = prmt_b32(a[2 * k], a[2 * k + 1], sel);
              put(dst + 2 * c * kWords * 128,
                  make_uint4(codes_lo(pr[0]), codes_lo(pr[1]), codes_lo(pr[2]), codes_lo(pr[3])));
              put(dst + (2 * c + 1) * kWords * 128,
                  make_uint4(codes_hi(pr[0]), codes_hi(pr[1]), codes_hi(pr[2]), codes_hi(pr[3])));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[vs]);
        }
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    const int uw = warp - L::kSoftWarps, ut = threadIdx.x - 32 * L::kSoftWarps;
    PageTab* tabs = reinterpret_cast<PageTab*>(smem + L::offTab);
    if constexpr (L::kByRole) {
      if (uw < L::kKeyWarps)
        decode_pages(std::integral_constant<int, 32 * L::kKeyWarps>{}, Yes{}, No{}, ut, 0, 1, tab_full, tabs);
      else
        decode_pages(std::integral_constant<int, 32 * L::kValWarps>{}, No{}, Yes{}, ut - 32 * L::kKeyWarps, 0, 1,
                     tab_full + 2, tabs);
    } else {
      const int group = uw >> 2;
      decode_pages(std::integral_constant<int, 128>{}, Yes{}, Yes{}, ut - 128 * group, group, L::kGroups,
                   tab_full + 2 * group, tabs + 2 * group);
    }
  } else if (warp == L::kProducer) {
    // ------------------------------------------------------------ raw pages
    if (lane == 0) {
      int j = min(pages, L::kRaw);
      for (; j < pages; ++j) {
        if (!mbar_wait(&raw_empty[j % L::kRaw], ((j / L::kRaw) & 1) ^ 1, p.err, abort_flag)) break;
        load_page(j);
      }
      if (*abort_flag)  // given up: copies still in flight must land before the CTA's shared memory goes
        for (int i = max(0, j - L::kRaw); i < j; ++i) mbar_wait(&raw_full[i % L::kRaw], (i / L::kRaw) & 1, p.err);
    }
  } else {
    // ------------------------------------------------------------ MMA issue, a warp per tile
    if (warp < L::kMma0 + kT && lane == 0) {
      const int t = warp - L::kMma0;
      constexpr uint32_t id_s = idesc_f16_f32(kRows, kKvPage), id_o = idesc_f16_f32(kRows, D);
      const uint32_t q_addr = smem_u32(smem + L::offQ + t * L::kParts * L::kQPart);
      auto scores = [&](int j) {
        const int ks = j % L::kK;
        if (!mbar_wait(&k_full[ks], (j / L::kK) & 1, p.err, abort_flag)) return false;
        tc_fence_after();
        const uint32_t k_addr = smem_u32(smem + L::offK + ks * L::kOp);
        const uint32_t d = tmem + static_cast<uint32_t>(L::s_col(t, j & 1));
#pragma unroll
        for (int part = 0; part < L::kParts; ++part)
#pragma unroll
          for (int s = 0; s < D / 64; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f16(d, sw128_kmajor_desc(q_addr + part * L::kQPart + s * (kRows * 128)) + 2 * k,
                         sw128_kmajor_desc(k_addr + s * (kKvPage * 128)) + 2 * k, id_s, (part | s | k) != 0 ? 1u : 0u);
        tc_commit(&s_full[2 * t + (j & 1)]);
        tc_commit(&k_empty[ks]);
        return true;
      };
      bool ok = pages == 0 || scores(0);
      for (int j = 0; ok && j < pages; ++j) {
        if (j + 1 < pages) {
          // the other score buffer holds W of the page before: its product must be done with it
          if (j > 0 && !mbar_wait(&pv_done[t], (j - 1) & 1, p.err, abort_flag)) break;
          if (!scores(j + 1)) break;
        }
        const int vs = j % L::kV;
        if (!mbar_wait(&v_full[vs], (j / L::kV) & 1, p.err, abort_flag)) break;
        if (!mbar_wait(&p_full[2 * t + (j & 1)], (j >> 1) & 1, p.err, abort_flag)) break;
        tc_fence_after();
        const uint32_t v_addr = smem_u32(smem + L::offV + vs * L::kOp);
#pragma unroll
        for (int part = 0; part < L::kParts; ++part)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f16_ta(tmem + static_cast<uint32_t>(L::o_col(t)),
                          tmem + static_cast<uint32_t>(L::s_col(t, j & 1) + 32 * part + 8 * k),
                          sw128_kmajor_desc(v_addr) + 2 * k, id_o, (j | part | k) != 0 ? 1u : 0u);
        tc_commit(j + 1 < pages ? &pv_done[t] : &o_done[t]);
        tc_commit(&v_empty[vs]);
      }
      if (*abort_flag) {  // given up: the products in flight must end before shared and tensor memory go
        tc_commit(&drained[t]);
        mbar_wait(&drained[t], 0, p.err);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == L::kMma0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// Joins the page ranges of a row, in order: a warp per (row, query head).
template <int D, typename OT>
__global__ void __launch_bounds__(128) k_kv4_join_rows(const Problem p, int splits, OT* __restrict__ out) {
  constexpr int kPer = D / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t all = static_cast<int64_t>(p.T) * p.Hq;
  if (row >= all) return;
  const int b = kv_seq_of_row(p.c.q_start, p.c.num_seqs, static_cast<int>(row / p.Hq), lane);
  if (b < 0) return;
  const int q0 = p.c.q_start[b];
  const int64_t n = static_cast<int64_t>(p.c.q_start[b + 1]) - q0;
  if (n < 0 || n > p.max_q || q0 < 0 || q0 + n > p.T) return;  // left out, as its scores were
  const float* src = p.part + row * (D + 4);
  const int64_t stride = all * (D + 4);
  float m = -INFINITY, l = 0.0f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, src[s * stride + D]);
  if (m == -INFINITY) m = 0.0f;
  for (int s = 0; s < splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(src + s * stride + D);
    const float f = ex2(ml.x - m);
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(src + s * stride)[32 * i + lane];
      o[4 * i] = fmaf(f, v.x, o[4 * i]);
      o[4 * i + 1] = fmaf(f, v.y, o[4 * i + 1]);
      o[4 * i + 2] = fmaf(f, v.z, o[4 * i + 2]);
      o[4 * i + 3] = fmaf(f, v.w, o[4 * i + 3]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) {
    union { OT v[4]; uint2 u2; uint4 u4; } pk;
#pragma unroll
    for (int c = 0; c < 4; ++c) pk.v[c] = round_out<OT>(o[4 * i + c] * inv);
    OT* dst = out + row * D + 128 * i + 4 * lane;
    if constexpr (sizeof(OT) == 4) *reinterpret_cast<uint4*>(dst) = pk.u4;
    else *reinterpret_cast<uint2*>(dst) = pk.u2;
  }
}

template <int D, typename QT, typename OT>
cudaError_t launch_t(DeviceContext* ctx, Problem p, const void* q, void* out, cudaStream_t s, int* status) {
  using L = Layout<D, std::is_same<QT, float>::value, std::is_same<QT, __nv_bfloat16>::value>;
  // units of kT * 128 rows: any division of T rows into sequences of at most max_q has at most this many
  const int64_t per = L::kT * kRows;
  const int64_t units = static_cast<int64_t>(p.T) * p.G / per + (p.c.num_seqs < p.T ? p.c.num_seqs : p.T);
  if (units * p.c.heads > 0x7fffffff) {
    *status = BITNET_ERR_UNSUPPORTED_SHAPE;
    return cudaSuccess;
  }
  // Too few units for the SMs: split the pages, at least 8 to a part.
  int64_t splits = 1;
  if (units * p.c.heads < ctx->num_sms) splits = ctx->num_sms / (units * p.c.heads);
  const int64_t most = (p.c.max_pages + 7) / 8;
  if (splits > most) splits = most;
  if (splits > 64) splits = 64;
  uint8_t* ws = nullptr;
  if (splits > 1) {
    const size_t bytes = static_cast<size_t>(splits) * p.T * p.Hq * (D + 4) * 4;
    if ((*status = pool_alloc(ctx, reinterpret_cast<void**>(&ws), bytes, s))) return cudaSuccess;
    p.part = reinterpret_cast<float*>(ws);
  }
  auto kern = k_kv4_prefill<D, QT, OT>;
  cudaError_t e = allow_smem(ctx, reinterpret_cast<const void*>(kern), L::kAlloc);
  if (e == cudaSuccess) {
    kern<<<dim3(static_cast<unsigned>(units * p.c.heads), 1, static_cast<unsigned>(splits)), L::kThreads, L::kAlloc, s>>>(
        p, static_cast<const QT*>(q), static_cast<OT*>(out));
    e = cudaGetLastError();
  }
  if (splits > 1) {
    if (e == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.T) * p.Hq + 3) / 4));
      cfg.blockDim = dim3(128);
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, k_kv4_join_rows<D, OT>, static_cast<const Problem>(p), static_cast<int>(splits),
                             static_cast<OT*>(out));
    }
    pool_free(ws, s);
  }
  return e;
}

}  // namespace

cudaError_t launch_kv4_prefill(DeviceContext* ctx, const KvView& c, int head_dim, const void* q, int q_dtype, int64_t T,
                               int Hq, int max_q_len, float scale, int causal, int window, void* out, int out_dtype,
                               cudaStream_t s, int* status) {
  Problem p = {};
  p.c = c;
  p.Hq = Hq;
  p.G = Hq / c.heads;
  p.T = static_cast<int>(T);
  p.max_q = max_q_len;
  p.scale = fabsf(scale) * 1.4426950408889634f;
  p.sign = scale < 0.0f ? -1.0f : 1.0f;
  p.causal = causal;
  p.window = window < (1 << 30) ? window : 1 << 30;  // keeps position - window within 32 bits
  p.err = ctx->err_word;
  if (T * p.G > 0x3fffffff) {  // rows of an item are counted in 32 bits
    *status = BITNET_ERR_UNSUPPORTED_SHAPE;
    return cudaSuccess;
  }
  auto go = [&](auto* qt, auto* ot) {
    using QT = std::remove_pointer_t<decltype(qt)>;
    using OT = std::remove_pointer_t<decltype(ot)>;
    return head_dim == 128 ? launch_t<128, QT, OT>(ctx, p, q, out, s, status)
                           : launch_t<256, QT, OT>(ctx, p, q, out, s, status);
  };
  float* f = nullptr;
  __half* h = nullptr;
  __nv_bfloat16* bf = nullptr;
  const bool f32_out = out_dtype == BITNET_DTYPE_F32;
  switch (q_dtype) {
    case BITNET_DTYPE_F32: return go(f, f);
    case BITNET_DTYPE_F16: return f32_out ? go(h, f) : go(h, h);
    case BITNET_DTYPE_BF16: return f32_out ? go(bf, f) : go(bf, bf);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace bitnet
