// Norms of queries and keys for each head, the position rotation in the same
// pass, and (paged form) K and V into the bf16 paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w    over the d values of a head
//   (a, b) -> (a c - b s, b c + a s)     for the pairs of the first rot_dim values
//
// A row is 2 d bytes read and 2 d written.  D / 8 lanes share a row; a lane holds
// four rotary pairs of it: values 4 l .. 4 l + 3 and as many rot_dim / 2 further on,
// or eight values in a row when pairs are neighbours, so both values of a pair are
// in one lane and only the sum of squares crosses lanes.  Norm weight, cos and sin
// of a value are the same in every row of the token: their products are formed once
// (y_i = (x_i C_i + x_partner S_i) / rms), which leaves 3 packed fp32 instructions for
// two values.  That matters: with the weights, cos and sin applied one after the
// other, row by row, the pass was bound by instructions (126 us for 21 300 tokens of
// 32 + 8 + 8 heads, d = 128).
//
// Where a token's rows go (a search of cu_seqlens, then the block table: four
// dependent loads) is looked up behind its first rows' loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kSteps = 4;     // rows that a lane works on
// Blocks an SM: at 5 nothing is spilled.  us for 21 300 tokens (see above): 5 87, and when
// that took 89 (the norms formed one row after the other) 4 96, 6 99; 2 steps at 8 blocks 115,
// 3 steps at 6 97.
constexpr int kBlocks = 5;

__device__ __forceinline__ uint2 ld_row(const void* p) {
  uint2 v;   // (not .nc: q may be its own output)
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// The two bf16 values of a word as packed fp32.
__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return ptx::f2_bits(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint64_t swapped(uint64_t v) {
  float lo, hi;
  ptx::f2_split(v, lo, hi);
  return ptx::f2_bits(hi, lo);
}

__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  ptx::f2_split(v, lo, hi);
  return ptx::pack_bf16x2(lo, hi);
}

// Squares leave fp32 where values reach 2^60 or (with an eps that does not hide it) fall
// to 2^-75: a row's 1 / sqrt(mean square + eps) is taken as it is only within 2^-50 .. 2^50.
__device__ __forceinline__ bool out_of_range(float r) {
  return __float_as_uint(r) - 0x26800000u > 0x58800000u - 0x26800000u;   // (a NaN, too)
}

// The sum of the squares of a lane's values, and of its row's (in all of the row's lanes).
__device__ __forceinline__ float lane_squares(const uint64_t (&x)[4]) {
  float lo, hi;
  ptx::f2_split(ptx::ffma2(x[0], x[0], ptx::ffma2(x[1], x[1], ptx::ffma2(x[2], x[2], ptx::fmul2(x[3], x[3])))), lo, hi);
  return lo + hi;
}
template <int LANES>
__device__ __forceinline__ float row_squares(const uint64_t (&x)[4]) {
  float sum = lane_squares(x);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The power of two that brings a row's largest magnitude to about 1 (to within 2^33, so that
// the factor is a normal number).
template <int LANES>
__device__ __forceinline__ float unit_scale(const uint64_t (&x)[4]) {
  float most = 0.f, lo, hi;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ptx::f2_split(x[k], lo, hi);
    most = fmaxf(most, fmaxf(fabsf(lo), fabsf(hi)));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100);
  return __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
}

// A group is up to kSteps * 32 / (D / 8) heads of q, of k or of v of one token; a
// token's groups are shared out over `parts` warps.  A warp's next group is on its
// way while it works on one.
template <int D, bool PAGED, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kBlocks)
qkv_rows_kernel(const QkvRowsParams p, int parts) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  constexpr int kEach = kSteps * kRows;
  const int lane = threadIdx.x & 31;
  const int sub = lane / kLanes, l = lane % kLanes;
  const uint32_t wid = blockIdx.x * (uint32_t)kWarps + (threadIdx.x >> 5);   // below 2^32
  const uint32_t tok = wid / (uint32_t)parts;
  if (tok >= (uint32_t)p.total) return;
  const int t = (int)tok, part = (int)(wid - tok * (uint32_t)parts);
  const int q_groups = (p.H + kEach - 1) / kEach, k_groups = (p.Hkv + kEach - 1) / kEach;
  const int groups = q_groups + (PAGED ? 2 : 1) * k_groups;
  const int g0 = (int)((long long)part * groups / parts), g1 = (int)((long long)(part + 1) * groups / parts);
  const int rl = p.rot_dim / 8;                    // lanes whose values are rotated
  const int off_a = l < rl && !INTER ? 4 * l : 8 * l;
  const int off_b = l < rl && !INTER ? 4 * l + p.rot_dim / 2 : 8 * l + 4;
  const bool all = rl == kLanes;                   // every lane's are
  auto kind_of = [&](int g) { return g < q_groups ? 0 : g < q_groups + k_groups ? 1 : 2; };   // q, k, v
  auto head_of = [&](int g) { return (g - (g < q_groups ? 0 : g < q_groups + k_groups ? q_groups : q_groups + k_groups)) * kEach + sub; };
  uint2 a[kSteps], b[kSteps], na[kSteps], nb[kSteps];
  auto source = [&](int g) __attribute__((always_inline)) {   // the lane's first row of the group
    const int kind = kind_of(g);
    return (kind == 0 ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride
            : kind == 1 ? static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride
                        : static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride) + head_of(g) * D;
  };
  auto fetch = [&](int g) __attribute__((always_inline)) {
    const int heads = kind_of(g) == 0 ? p.H : p.Hkv, h0 = head_of(g);
    const __nv_bfloat16* src = source(g);
#pragma unroll
    for (int e = 0; e < kSteps; ++e) {
      na[e] = nb[e] = make_uint2(0x3f803f80u, 0x3f803f80u);   // (ones: rows past the last head are in range)
      if (h0 + e * kRows < heads) {
        na[e] = ld_row(src + e * kRows * D + off_a);
        nb[e] = ld_row(src + e * kRows * D + off_b);
      }
    }
  };
  fetch(g0);
  // positions, cos and sin of the lane's pairs, the token's slot
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
  long long slot = 0;
  if constexpr (PAGED)
    slot = token_slot(t, p.cu, p.seq_lens, p.block_table, p.num_seqs, p.total, p.max_blocks, p.num_pages,
                      p.status, lane);
  if (bad || slot < 0) {   // (the same in every lane)
    if (slot >= 0 && lane == 0) atomicExch(p.status, kDevInvalidArg);
    return;
  }
  uint64_t C[4], S[4];
  int made = -1;           // the kind that C and S are of
  bool norm = false;
  for (int g = g0; g < g1; ++g) {
    const int kind = kind_of(g), heads = kind == 0 ? p.H : p.Hkv, h0 = head_of(g);
#pragma unroll
    for (int e = 0; e < kSteps; ++e) {
      a[e] = na[e];
      b[e] = nb[e];
    }
    if (g + 1 < g1) fetch(g + 1);
    // output row of head h: first + h * step
    __nv_bfloat16* dst;
    size_t first, limit;
    int step = 1;
    if (kind == 0 || !PAGED) {
      dst = static_cast<__nv_bfloat16*>(kind == 0 ? p.q_out : p.k_out);
      first = (size_t)t * heads;
      limit = (size_t)p.total * heads;
    } else {
      dst = static_cast<__nv_bfloat16*>(kind == 1 ? p.k_cache : p.v_cache);
      first = (size_t)(slot / kPage * p.Hkv * kPage + slot % kPage);
      limit = (size_t)p.num_pages * p.Hkv * kPage;
      step = kPage;
    }
    if (kind < 2 && kind != made) {
      made = kind;
      const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(kind == 0 ? p.q_weight : p.k_weight);
      norm = weight != nullptr;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (norm) {
        const uint2 wa = __ldg(reinterpret_cast<const uint2*>(weight + off_a));
        const uint2 wb = __ldg(reinterpret_cast<const uint2*>(weight + off_b));
        ptx::f2_split(widen(wa.x), w[0], w[1]);
        ptx::f2_split(widen(wa.y), w[2], w[3]);
        ptx::f2_split(widen(wb.x), w[4], w[5]);
        ptx::f2_split(widen(wb.y), w[6], w[7]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (INTER) {   // values 2 e and 2 e + 1 are a pair
          C[e] = ptx::f2_bits(w[2 * e] * c[e], w[2 * e + 1] * c[e]);
          S[e] = ptx::f2_bits(-w[2 * e + 1] * s[e], w[2 * e] * s[e]);
        } else {                 // values e and 4 + e are
          const int x = 2 * (e & 1);
          C[e] = ptx::f2_bits(w[2 * e] * c[x], w[2 * e + 1] * c[x + 1]);
          S[e] = e < 2 ? ptx::f2_bits(-w[4 + x] * s[x], -w[5 + x] * s[x + 1])
                       : ptx::f2_bits(w[x] * s[x], w[x + 1] * s[x + 1]);
        }
      }
    }
    // a row (its bits, its values and 1 / its norm) rotated and stored
    auto finish = [&](int h, uint32_t (&y)[4], const uint64_t (&x)[4], float r) __attribute__((always_inline)) {
      if (!PAGED || kind < 2) {
        const uint64_t r2 = ptx::f2_bits(r, r);
        uint64_t z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = ptx::fmul2(x[k], r2);
        if (norm || l < rl) {          // (the rest as they are)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint64_t v = ptx::fmul2(z[k], C[k]);
            if (all || l < rl)         // (elsewhere an inf times S = 0 would be a NaN)
              v = ptx::ffma2(INTER ? swapped(z[k]) : z[k ^ 2], S[k], v);
            y[k] = narrow(v);
          }
        }
      }
      const size_t row = first + (size_t)h * step;
      if (h < heads && FA_IN_BOUNDS(row, limit, p.status)) {
        *reinterpret_cast<uint2*>(dst + row * D + off_a) = make_uint2(y[0], y[1]);
        *reinterpret_cast<uint2*>(dst + row * D + off_b) = make_uint2(y[2], y[3]);
      }
    };
    // (all rows' norms before the first is used: the sums' shuffles go side by side, and the
    // check of their range is one branch a group; 87.4 us, with a branch for each row 90.2)
    float r[kSteps];
#pragma unroll
    for (int e = 0; e < kSteps; ++e) r[e] = 1.f;
    if (norm && (!PAGED || kind < 2)) {
#pragma unroll
      for (int e = 0; e < kSteps; ++e) {
        const uint64_t x[4] = {widen(a[e].x), widen(a[e].y), widen(b[e].x), widen(b[e].y)};
        r[e] = lane_squares(x);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int e = 0; e < kSteps; ++e) r[e] += __shfl_xor_sync(0xffffffffu, r[e], o);
      bool out = false;
#pragma unroll
      for (int e = 0; e < kSteps; ++e) {
        r[e] = rsqrtf(r[e] * (1.f / D) + p.eps);
        out = out || out_of_range(r[e]);
      }
      if (__any_sync(0xffffffffu, out)) {   // rows read again, one at a time: registers are short
        const __nv_bfloat16* src = source(g);
#pragma unroll 1
        for (int e = 0; e < kSteps; ++e) {
          uint32_t y[4] = {0u, 0u, 0u, 0u};
          if (h0 + e * kRows < heads) {
            const uint2 lo = ld_row(src + e * kRows * D + off_a), hi = ld_row(src + e * kRows * D + off_b);
            y[0] = lo.x;
            y[1] = lo.y;
            y[2] = hi.x;
            y[3] = hi.y;
          }
          uint64_t x[4] = {widen(y[0]), widen(y[1]), widen(y[2]), widen(y[3])};
          const float scale = unit_scale<kLanes>(x), mean = row_squares<kLanes>(x) * (1.f / D);
          // (not for the sake of a large eps, which times the factor's square could leave fp32)
          const float f = mean > 0x1p100f || mean + p.eps < 0x1p-100f ? scale : 1.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = ptx::fmul2(x[k], ptx::f2_bits(f, f));
          finish(h0 + e * kRows, y, x, rsqrtf(row_squares<kLanes>(x) * (1.f / D) + p.eps * f * f));
        }
        continue;
      }
    }
#pragma unroll
    for (int e = 0; e < kSteps; ++e) {
      uint32_t y[4] = {a[e].x, a[e].y, b[e].x, b[e].y};
      const uint64_t x[4] = {widen(y[0]), widen(y[1]), widen(y[2]), widen(y[3])};
      finish(h0 + e * kRows, y, x, r[e]);
    }
  }
}

template <int D, bool PAGED>
void launch(const QkvRowsParams& p, cudaStream_t stream) {
  constexpr int kEach = kSteps * 256 / D;
  const int groups = (p.H + kEach - 1) / kEach + (PAGED ? 2 : 1) * ((p.Hkv + kEach - 1) / kEach);
  // As many warps a token as one wave has room for, up to one a group: latency counts
  // there; beyond, a warp that keeps a token's C, S and slot is the cheapest.  us with
  // one, two and six warps a token (32 + 8 + 8 heads, d = 128): 64 tokens 7.7, 5.5, 3.7;
  // 1024 8.7, 7.1, 8.9; 4096 19, 20, 27; 16384 69, 74, 113.
  const int wave = 152 * kWarps * kBlocks / (p.total < 1 ? 1 : p.total);
  const int parts = wave < 1 ? 1 : wave < groups ? wave : groups;
  const long long warps = (long long)p.total * parts;
  const unsigned blocks = (unsigned)((warps + kWarps - 1) / kWarps);
  if (p.interleaved) qkv_rows_kernel<D, PAGED, true><<<blocks, kWarps * 32, 0, stream>>>(p, parts);
  else qkv_rows_kernel<D, PAGED, false><<<blocks, kWarps * 32, 0, stream>>>(p, parts);
}

}  // namespace

cudaError_t launch_qkv_rows(const QkvRowsParams& p, cudaStream_t stream) {
  if (p.k_cache != nullptr) p.d == 128 ? launch<128, true>(p, stream) : launch<64, true>(p, stream);
  else p.d == 128 ? launch<128, false>(p, stream) : launch<64, false>(p, stream);
  return cudaGetLastError();
}

}  // namespace fa
