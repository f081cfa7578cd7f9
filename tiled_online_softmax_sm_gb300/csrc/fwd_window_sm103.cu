// Sliding-window instances of the tcgen05 forward: dense and packed bf16.
//
// Only tiles that hold a visible key are loaded and multiplied: the window's,
// from an entry that differs from unit to unit (neighbours then read different
// tiles at a time), and last the sinks'.  The next units are worked out by an
// idle warp, since units are short: n = m = 8192, window 1024, 4 sinks, H = 32,
// d = 128 is 1024 units of 11 tiles, 149 us, 866 TFLOP/s of visible pairs (0.44 of
// the GEMM rate).  80 to 89 % of a unit's tiles is visible; of the rest, in
// copies that leave it out, O's rounded row sum costs 6 %, the sinks' tile 5 %,
// the stores of O 3 %, and each unit's first tile and epilogue about 12 %.
// 16 ragged sequences at d = 64 under a window of 256 (units of three tiles, 67 %
// visible): 114 us, 297 TFLOP/s.
#include "fwd_bf16_sm103.cuh"

namespace fa {

cudaError_t launch_fwd_window(const FwdParams& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? launch<128, false, false, true>(p, stream, why)
                    : launch<64, false, false, true>(p, stream, why);
}

}  // namespace fa
