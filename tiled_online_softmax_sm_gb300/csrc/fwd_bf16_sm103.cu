// Dense, packed and paged forward instances of the tcgen05 kernel.
#include "fwd_bf16_sm103.cuh"

namespace fa {

cudaError_t launch_fwd_bf16(const FwdParams& p, cudaStream_t stream, const char** why) {
  const bool paged = p.block_table != nullptr;
  if (p.fp8) {
    if (p.d == 128 && p.dv == 128 && !paged) return launch<128, false, true>(p, stream, why);
    *why = "fwd e4m3: supported d == dv == 128, dense";
    return cudaErrorInvalidValue;
  }
  if (p.d == 128 && p.dv == 128)
    return paged ? launch<128, true, false>(p, stream, why) : launch<128, false, false>(p, stream, why);
  if (p.d == 64 && p.dv == 64)
    return paged ? launch<64, true, false>(p, stream, why) : launch<64, false, false>(p, stream, why);
  *why = "fwd_bf16: unsupported head dim";
  return cudaErrorInvalidValue;
}

}  // namespace fa
