// kv4.cuh -- layout and addressing of the paged 4-bit key/value cache.
//
// The cache is [num_pages][num_kv_heads] blocks; a block holds the keys and the
// values of kKvPage consecutive tokens of one kv head, D = head_dim:
//   [64][D/2]  key codes   (byte j of a token: dimension 2j in the low four
//   [64][D/2]  value codes  bits, 2j + 1 in the high four)
//   [64][2]    float (scale, minimum) of each key row
//   [64][2]    float (scale, minimum) of each value row
// so a block is one contiguous, 1024-byte sized copy and everything a pass over
// 64 tokens of a head needs.  A stored value is code * scale + minimum.
//
// One scale and minimum per row make both products of attention run on the
// integer codes:  q . k_j = s_j (q . c_j) + m_j sum(q)  and
// sum_j p_j v_j = sum_j (p_j s_j) c_j + sum_j p_j m_j.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bitnet.h"

namespace bitnet {

constexpr int kKvPage = BITNET_KV4_PAGE;

template <int D>
struct KvBlock {
  static constexpr int kRow = D / 2;                 // bytes of a row's codes
  static constexpr int offK = 0;
  static constexpr int offV = kKvPage * kRow;
  static constexpr int offKMeta = 2 * kKvPage * kRow;
  static constexpr int offVMeta = offKMeta + kKvPage * 8;
  static constexpr int kBytes = offVMeta + kKvPage * 8;
  static_assert(kBytes % 1024 == 0, "blocks stay 1 KB aligned");
};

// What a kernel sees of a bitnet_kv4 descriptor.
struct KvView {
  uint8_t* cache;
  const int32_t* q_start;
  const int32_t* kv_lens;
  const int32_t* page_table;
  int64_t num_pages;
  int num_seqs;
  int max_pages;
  int heads;  // kv heads
};

// The sequence that owns row t: the last b with q_start[b] <= t (q_start is
// non-decreasing), or -1 before the first and behind the last row.  All 32
// lanes call it with the same t: a 33-ary search, one load per lane and round
// (two rounds for up to 1024 sequences).
__device__ __forceinline__ int kv_seq_of_row(const int32_t* __restrict__ q_start, int num_seqs, int t, int lane) {
  int lo = 0, hi = num_seqs + 1;  // the count of entries <= t is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;  // probes, ascending
    const bool le = i < hi && q_start[i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) {
      hi = lo;
    } else {
      const int last = lo + (c - 1) * step;  // entry `last` is <= t, entry last + step is not
      hi = min(hi, last + step);
      lo = last + 1;
    }
  }
  return lo == 0 || lo == num_seqs + 1 ? -1 : lo - 1;
}

// Keys of sequence b, as the page table can hold them; *bad is set where the
// plan says otherwise.
__device__ __forceinline__ int kv_len_of(const KvView& c, int b, bool* bad) {
  const int n = c.kv_lens[b];
  const int64_t most = static_cast<int64_t>(c.max_pages) * kKvPage;
  if (n < 0 || n > most) *bad = true;
  return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}

}  // namespace bitnet
