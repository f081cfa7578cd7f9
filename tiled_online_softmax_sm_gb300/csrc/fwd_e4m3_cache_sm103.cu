// Instances of the tcgen05 forward that read the e4m3 paged cache.
#include "fwd_bf16_sm103.cuh"

namespace fa {

cudaError_t launch_fwd_e4m3_cache(const FwdParams& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? launch<128, true, false, true, true>(p, stream, why)
                    : launch<64, true, false, true, true>(p, stream, why);
}

}  // namespace fa
