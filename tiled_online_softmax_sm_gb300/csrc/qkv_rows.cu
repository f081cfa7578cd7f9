// Norms of queries and keys for each head, the position rotation in the same
// pass, and (paged form) K and V into the bf16 paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w    over the d values of a head
//   (a, b) -> (a c - b s, b c + a s)     for the pairs of the first rot_dim values
//
// A row is 2 d bytes read and 2 d written, and the d values need two reductions'
// worth of nothing else, so the pass is bound by memory traffic.  D / 8 lanes
// share a row; a lane holds four rotary pairs of it as two pieces of four values:
// the halves' pairs (p, p + rot_dim/2) for p = 4 l .. 4 l + 3, or eight values in
// a row when pairs are neighbours, so both values of a pair are in one lane and
// only the sum of squares crosses lanes.  The table's entries of a lane's pairs
// serve every row of the token that the warp handles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint2 ld_row(const void* p) {
  uint2 v;   // (not .nc: q may be its own output)
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void widen(const uint2& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xffff0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xffff0000u);
}

// A warp's share: kSteps times 32 / (D / 8) rows of one token, of its q heads,
// then its k heads, then (paged) its v heads.
template <int D, bool PAGED, int kSteps>
__global__ void __launch_bounds__(kWarps * 32)
qkv_rows_kernel(const QkvRowsParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLanes, l = lane % kLanes;
  const int heads = p.H + (PAGED ? 2 : 1) * p.Hkv;
  const int shares = (heads + kSteps * kRows - 1) / (kSteps * kRows);
  const uint32_t item = blockIdx.x * (uint32_t)kWarps + (threadIdx.x >> 5);   // below 2^32
  const uint32_t tok = item / (uint32_t)shares;
  if (tok >= (uint32_t)p.total) return;
  const int t = (int)tok;
  const int r0 = (int)(item - tok * (uint32_t)shares) * (kSteps * kRows) + sub;
  // this lane's two pieces of a row
  const int rl = p.rot_dim / 8;                    // lanes whose values are rotated
  const int off_a = l < rl && !p.interleaved ? 4 * l : 8 * l;
  const int off_b = l < rl && !p.interleaved ? 4 * l + p.rot_dim / 2 : 8 * l + 4;

  uint2 a[kSteps], b[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = r0 + i * kRows;
    const __nv_bfloat16* src;
    if (row < p.H) src = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + row * D;
    else if (row < p.H + p.Hkv) src = static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + (row - p.H) * D;
    else src = static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride + (row - p.H - p.Hkv) * D;
    a[i] = b[i] = make_uint2(0u, 0u);
    if (row < heads) {
      a[i] = ld_row(src + off_a);
      b[i] = ld_row(src + off_b);
    }
  }
  // cos and sin of the lane's pairs 4 l .. 4 l + 3
  float c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  bool bad = false;
  if (p.rot_dim > 0) {
    int x[kMaxAxes];
#pragma unroll
    for (int k = 0; k < kMaxAxes; ++k) {
      x[k] = k < p.num_axes ? __ldg(p.positions + (size_t)k * p.total + t) : 0;
      bad = bad || x[k] < 0 || x[k] >= p.max_positions;
    }
    if (!bad && l < rl) {
      const int half = p.rot_dim / 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pair = 4 * l + e;
        int at = x[kMaxAxes - 1];
#pragma unroll
        for (int k = kMaxAxes - 2; k >= 0; --k) at = pair < p.section_end[k] ? x[k] : at;
        const float2 cs = __ldg(reinterpret_cast<const float2*>(p.cos_sin) + (size_t)at * half + pair);
        c[e] = cs.x;
        s[e] = cs.y;
      }
    }
  }
  if (bad) {   // (the same in every lane)
    if (lane == 0) atomicExch(p.status, kDevInvalidArg);
    return;
  }
  long long slot = 0;
  if constexpr (PAGED) {
    slot = token_slot(t, p.cu, p.seq_lens, p.block_table, p.num_seqs, p.total, p.max_blocks, p.num_pages,
                      p.status, lane);
    if (slot < 0) return;
  }
  uint2 wqa = make_uint2(0u, 0u), wqb = wqa, wka = wqa, wkb = wqa;
  if (p.q_weight != nullptr) {
    wqa = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q_weight) + off_a));
    wqb = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q_weight) + off_b));
  }
  if (p.k_weight != nullptr) {
    wka = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.k_weight) + off_a));
    wkb = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.k_weight) + off_b));
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = r0 + i * kRows;
    const bool is_q = row < p.H, is_v = row >= p.H + p.Hkv;
    float xa[4], xb[4];
    widen(a[i], xa);
    widen(b[i], xb);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], sum));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const bool norm = is_q ? p.q_weight != nullptr : p.k_weight != nullptr;
    if (norm) {
      const float r = rsqrtf(sum * (1.f / D) + p.eps);
      float wa[4], wb[4];
      widen(is_q ? wqa : wka, wa);
      widen(is_q ? wqb : wkb, wb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xa[e] = xa[e] * r * wa[e];
        xb[e] = xb[e] * r * wb[e];
      }
    }
    float ya[4], yb[4];
    if (l >= rl) {   // not rotated (times 0 would turn an inf into a NaN)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ya[e] = xa[e];
        yb[e] = xb[e];
      }
    } else if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ya[2 * e] = xa[2 * e] * c[e] - xa[2 * e + 1] * s[e];
        ya[2 * e + 1] = xa[2 * e + 1] * c[e] + xa[2 * e] * s[e];
        yb[2 * e] = xb[2 * e] * c[e + 2] - xb[2 * e + 1] * s[e + 2];
        yb[2 * e + 1] = xb[2 * e + 1] * c[e + 2] + xb[2 * e] * s[e + 2];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ya[e] = xa[e] * c[e] - xb[e] * s[e];
        yb[e] = xb[e] * c[e] + xa[e] * s[e];
      }
    }
    uint2 oa = make_uint2(ptx::pack_bf16x2(ya[0], ya[1]), ptx::pack_bf16x2(ya[2], ya[3]));
    uint2 ob = make_uint2(ptx::pack_bf16x2(yb[0], yb[1]), ptx::pack_bf16x2(yb[2], yb[3]));
    if ((PAGED && is_v) || (!norm && l >= rl)) {   // as they are
      oa = a[i];
      ob = b[i];
    }
    if (row >= heads) continue;
    __nv_bfloat16* dst;
    bool in = true;
    if (is_q) {
      const size_t at = (size_t)t * p.H + row;
      in = FA_IN_BOUNDS(at, (size_t)p.total * p.H, p.status);
      dst = static_cast<__nv_bfloat16*>(p.q_out) + at * D;
    } else if constexpr (PAGED) {
      const int h = row - p.H - (is_v ? p.Hkv : 0);
      const size_t at = (size_t)((slot / kPage * p.Hkv + h) * kPage + slot % kPage);
      in = FA_IN_BOUNDS(at, (size_t)p.num_pages * p.Hkv * kPage, p.status);
      dst = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + at * D;
    } else {
      const size_t at = (size_t)t * p.Hkv + (row - p.H);
      in = FA_IN_BOUNDS(at, (size_t)p.total * p.Hkv, p.status);
      dst = static_cast<__nv_bfloat16*>(p.k_out) + at * D;
    }
    if (in) {
      *reinterpret_cast<uint2*>(dst + off_a) = oa;
      *reinterpret_cast<uint2*>(dst + off_b) = ob;
    }
  }
}

template <int D, bool PAGED>
void launch(const QkvRowsParams& p, cudaStream_t stream) {
  constexpr int kSteps = 4;
  const int heads = p.H + (PAGED ? 2 : 1) * p.Hkv;
  constexpr int kEach = kSteps * 256 / D;
  const long long items = (long long)p.total * ((heads + kEach - 1) / kEach);
  qkv_rows_kernel<D, PAGED, kSteps>
      <<<(unsigned)((items + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_qkv_rows(const QkvRowsParams& p, cudaStream_t stream) {
  if (p.k_cache != nullptr) p.d == 128 ? launch<128, true>(p, stream) : launch<64, true>(p, stream);
  else p.d == 128 ? launch<128, false>(p, stream) : launch<64, false>(p, stream);
  return cudaGetLastError();
}

}  // namespace fa
