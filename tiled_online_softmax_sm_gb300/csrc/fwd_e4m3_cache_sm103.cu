// Instances of the tcgen05 forward that read the e4m3 paged cache: chunks of new
// tokens, under a window or not.
//
// The recurrence and the two 128-row query tiles are the forward's.  A tile's
// pages are staged as codes (half the bytes of bf16 in flight) and a fourth
// warpgroup widens them into the K/V ring: code * 2^e is exact in bf16, so the
// MMAs multiply the cached values themselves.  The heads of a group are rows of
// one tile, so K and V are staged and widened once for all of them.  With few
// units their tile lists are cut into parts for all SMs, merged by a second
// launch: 64 tokens of one sequence over 8192 keys 139 -> 31 us.
//
// Bound by the two tiles' chain of MMAs and by issue slots.  16 x 512-token
// chunks over [512, 8192] tokens (H = 32, Hkv = 8, d = 128): 527 us, 1061
// TFLOP/s, 0.54 of the bf16 GEMM rate (the bf16 cache's 447 us have no widening
// warps beside the softmax); a copy without softmax and widening takes 376 us,
// DRAM would need 41.  Below 128 rows a unit has one tile and its time does not
// depend on the rows (64 sequences, 229 us, 2.3 TB/s).
#include "fwd_bf16_sm103.cuh"

namespace fa {

cudaError_t launch_fwd_e4m3_cache(const FwdParams& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? launch<128, true, false, true, true>(p, stream, why)
                    : launch<64, true, false, true, true>(p, stream, why);
}

}  // namespace fa
