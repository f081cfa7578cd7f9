// Where rows of packed tensors belong in a paged cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kPage = 16;

// Where row t of the packed tensors belongs: the sequence s with cu[s] <= t <
// cu[s + 1], its token seq_lens[s] - n_s + (t - cu[s]), and that token's slot
// (page * 16 + place).  -1: t is no sequence's row (left alone), or its offsets,
// length or page id are unusable (recorded in the status word).
__device__ __forceinline__ long long token_slot(int t, const int* __restrict__ cu,
                                                const int* __restrict__ seq_lens,
                                                const int* __restrict__ block_table, int num_seqs,
                                                int total, int max_blocks, int num_pages,
                                                int* status, int lane) {
  int lo = 0, hi = num_seqs;   // cu[lo] <= t < cu[hi] is narrowed by 32 probes a round
  if (t < __ldg(cu) || t >= __ldg(cu + num_seqs)) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && __ldg(cu + at) <= t;
    // the first probe above t bounds the range (offsets are non-decreasing)
    const int n = __ffs(~__ballot_sync(0xffffffffu, le)) - 1;
    const int below = n < 0 ? 32 : n;
    lo += below * step;
    hi = min(hi, lo + step);
  }
  const int first = __ldg(cu + lo), n = __ldg(cu + lo + 1) - first;
  const int L = __ldg(seq_lens + lo);
  if (first < 0 || n < 0 || first + (long long)n > total || t < first || t >= first + n || L < n ||
      (long long)L > (long long)max_blocks * kPage) {
    if (lane == 0) atomicExch(status, kDevInvalidArg);
    return -1;
  }
  const int pos = L - n + (t - first);
  const int id = __ldg(block_table + (size_t)lo * max_blocks + pos / kPage);
  if (id < 0 || id >= num_pages) {
    if (lane == 0) atomicExch(status, kDevBadBlockTable);
    return -1;
  }
  return (long long)id * kPage + pos % kPage;
}

}  // namespace
}  // namespace fa
