// The paged KV cache in e4m3: quantising new K/V rows as they are written, and
// reading cached rows back as bf16.
//
// Format.  A row (one token of one kv head, d values) is stored as d e4m3
// codes and one scale byte b: value = code * 2^(b - 127).  The exponent
// e = b - 127 is the smallest integer >= -127 with
//     max |x| over the row's finite values <= 448 * 2^e
// (448 is e4m3's largest value).  A power of two costs e4m3 no precision: it
// moves the exponent, the codes keep their 4 significant bits, and
// x * 2^-e is exact in fp32, so each code is one round-to-nearest-even of the
// input and nothing depends on a division's rounding.  From the bf16 bits of
// the maximum (exponent field E, 7-bit fraction f), 448 = 1.75 * 2^8 gives
//     b = max(0, E - 8 + (f > 0x60)).
// inf and NaN do not enter the maximum; e4m3 has no inf, so both become its NaN.
//
// Both kernels: one warp per (token, up to 8 heads).  A row is d/8
// lanes of 16 bytes of bf16 (write) or d/16 lanes of 16 codes (read), so a
// warp's loads and stores are whole 32-byte sectors.  The token's sequence is
// found by a 32-way search of cu_seqlens (two rounds for up to 1024
// sequences); in the write kernel the row loads are in flight behind it.
// Bound by memory traffic: 3 bytes a value plus one byte a row; 6.5 TB/s
// written and 6.7 read back (64 sequences, 8 heads, d = 128: 0.95 and 0.98 of a
// plain copy).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

// A warp's share: HEADS rows of K and of V.
template <int D, int HEADS, bool WRITE>
struct Share {
  static constexpr int kLanes = WRITE ? D / 8 : D / 16;     // lanes per row
  static constexpr int kRows = 32 / kLanes;                 // rows per warp step
  static constexpr int kSteps = HEADS / kRows;              // of K, and then as many of V
  static constexpr int kAll = 2 * kSteps;
  static_assert(HEADS % kRows == 0, "whole steps");
};

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Lanes of row `sub` hold 8 values each (4 words of bf16 pairs).
template <int D, int HEADS>
__global__ void __launch_bounds__(kWarps * 32)
kv_write_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                long long k_stride, long long v_stride, uint8_t* __restrict__ k_cache,
                uint8_t* __restrict__ v_cache, uint8_t* __restrict__ k_scale,
                uint8_t* __restrict__ v_scale, const int* __restrict__ block_table,
                const int* __restrict__ seq_lens, const int* __restrict__ cu, int num_seqs,
                int total, int Hkv, int num_pages, int max_blocks, int* status) {
  using P = Share<D, HEADS, true>;
  constexpr int kLanes = P::kLanes, kRows = P::kRows, kSteps = P::kSteps, kAll = P::kAll;
  const int lane = threadIdx.x & 31;
  const int blocks_h = (Hkv + HEADS - 1) / HEADS;
  const uint32_t item = blockIdx.x * (uint32_t)kWarps + (threadIdx.x >> 5);   // below 2^32
  const uint32_t row_t = item / (uint32_t)blocks_h;
  if (row_t >= (uint32_t)total) return;
  const int t = (int)row_t;
  const int h0 = (int)(item - row_t * (uint32_t)blocks_h) * HEADS;
  const int sub = lane / kLanes, col = (lane % kLanes) * 8;
  uint4 x[kAll];
#pragma unroll
  for (int i = 0; i < kAll; ++i) {
    const __nv_bfloat16* src = (i >= kSteps ? v + t * v_stride : k + t * k_stride) + col;
    const int h = h0 + i % kSteps * kRows + sub;
    x[i] = h < Hkv ? ld_stream(src + h * D) : make_uint4(0u, 0u, 0u, 0u);
  }
  const long long slot = token_slot(t, cu, seq_lens, block_table, num_seqs, total, max_blocks,
                                    num_pages, status, lane);
  if (slot < 0) return;
  const long long row0 = (slot / kPage) * Hkv * kPage + slot % kPage;
  const size_t first = (size_t)(row0 + (long long)(h0 + sub) * kPage);   // step 0's cache row
#pragma unroll
  for (int i = 0; i < kAll; i += 2) {
    uint32_t w[2][4] = {{x[i].x, x[i].y, x[i].z, x[i].w},
                        {x[i + 1].x, x[i + 1].y, x[i + 1].z, x[i + 1].w}};
    // Magnitudes as 15-bit integers order like the values.  The maxima of the
    // two steps' rows share a register on their way through the warp.
    auto row_maxima = [&]() __attribute__((always_inline)) -> uint32_t {
      uint32_t m[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        m[r] = __vmaxu2(__vmaxu2(w[r][0] & 0x7fff7fffu, w[r][1] & 0x7fff7fffu),
                        __vmaxu2(w[r][2] & 0x7fff7fffu, w[r][3] & 0x7fff7fffu));
      uint32_t mx = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1)
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      return mx;
    };
    uint32_t mx = row_maxima();
    // (adding 0x80 carries into bit 15 exactly for magnitudes of inf and NaN)
    if (__any_sync(0xffffffffu, ((mx + 0x00800080u) & 0x80008000u) != 0u)) {
      // rare: inf and NaN become NaN and stay out of the maximum
      uint32_t nan[2][4] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[r][e] & 0x7fffu) >= 0x7f80u) { w[r][e] &= 0xffff0000u; nan[r][e] |= 0x7fffu; }
          if (((w[r][e] >> 16) & 0x7fffu) >= 0x7f80u) { w[r][e] &= 0xffffu; nan[r][e] |= 0x7fff0000u; }
        }
      mx = row_maxima();
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[r][e] |= nan[r][e];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int amax = (int)(r == 0 ? mx & 0xffffu : mx >> 16);
      const int b = max(0, (amax >> 7) - 8 + ((amax & 0x7f) > 0x60 ? 1 : 0));
      const float inv = __uint_as_float((uint32_t)(254 - b) << 23);   // 2^-(b - 127), exact
      uint32_t code[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        code[e] = ptx::pack_e4m3x2(__uint_as_float(w[r][e] << 16) * inv,
                                   __uint_as_float(w[r][e] & 0xffff0000u) * inv);
      uint8_t* cache = i + r >= kSteps ? v_cache : k_cache;
      uint8_t* scales = i + r >= kSteps ? v_scale : k_scale;
      const int step = (i + r) % kSteps;
      const int h = h0 + step * kRows + sub;
      const size_t row = first + (size_t)(step * kRows * kPage);
      if (h < Hkv && FA_IN_BOUNDS(row, (size_t)num_pages * Hkv * kPage, status)) {
        *reinterpret_cast<uint2*>(cache + row * D + col) =
            make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
        if (col == 0) scales[row] = (uint8_t)b;
      }
    }
  }
}

template <int D, int HEADS>
__global__ void __launch_bounds__(kWarps * 32)
kv_read_kernel(const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
               const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
               const int* __restrict__ block_table, const int* __restrict__ seq_lens,
               const int* __restrict__ cu, __nv_bfloat16* __restrict__ k,
               __nv_bfloat16* __restrict__ v, int num_seqs, int total, int Hkv, int num_pages,
               int max_blocks, int* status) {
  using P = Share<D, HEADS, false>;
  constexpr int kLanes = P::kLanes, kRows = P::kRows, kSteps = P::kSteps, kAll = P::kAll;
  const int lane = threadIdx.x & 31;
  const int blocks_h = (Hkv + HEADS - 1) / HEADS;
  const uint32_t item = blockIdx.x * (uint32_t)kWarps + (threadIdx.x >> 5);   // below 2^32
  const uint32_t row_t = item / (uint32_t)blocks_h;
  if (row_t >= (uint32_t)total) return;
  const int t = (int)row_t;
  const int h0 = (int)(item - row_t * (uint32_t)blocks_h) * HEADS;
  const int sub = lane / kLanes, col = (lane % kLanes) * 16;
  const long long slot = token_slot(t, cu, seq_lens, block_table, num_seqs, total, max_blocks,
                                    num_pages, status, lane);
  if (slot < 0) return;
  const long long row0 = (slot / kPage) * Hkv * kPage + slot % kPage;
  // Whole 32-byte sectors a store where the outputs allow it: 232 against 250 us
  // for 64 prefixes (518 MB of codes and scales, d = 128).
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  uint4 x[kAll];
  uint32_t b[kAll];
#pragma unroll
  for (int i = 0; i < kAll; ++i) {
    const uint8_t* cache = i >= kSteps ? v_cache : k_cache;
    const uint8_t* scales = i >= kSteps ? v_scale : k_scale;
    const int h = h0 + i % kSteps * kRows + sub;
    const size_t row = (size_t)(row0 + (long long)(h < Hkv ? h : 0) * kPage);
    x[i] = ld_stream(cache + row * D + col);
    b[i] = __ldg(scales + row);
  }
#pragma unroll
  for (int i = 0; i < kAll; ++i) {
    __nv_bfloat16* out = i >= kSteps ? v : k;
    const int h = h0 + i % kSteps * kRows + sub;
    const float s = ptx::exp2_byte(b[i]);
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float lo, hi;
      ptx::unpack_e4m3x2(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu, lo, hi);
      r[e] = ptx::pack_bf16x2(lo * s, hi * s);   // exact: 4 significant bits
    }
    const size_t row = (size_t)t * Hkv + h;
    if (h < Hkv && FA_IN_BOUNDS(row, (size_t)total * Hkv, status)) {
      uint4* dst = reinterpret_cast<uint4*>(out + row * D + col);
      const uint4 lo = make_uint4(r[0], r[1], r[2], r[3]), hi = make_uint4(r[4], r[5], r[6], r[7]);
      if (wide) {
        ptx::st_global_v8(dst, lo, hi);
      } else {
        dst[0] = lo;
        dst[1] = hi;
      }
    }
  }
}

template <int HEADS>
unsigned blocks(const KvRowsParams& p) {
  const long long items = (long long)p.total * ((p.Hkv + HEADS - 1) / HEADS);
  return (unsigned)((items + kWarps - 1) / kWarps);
}

template <int D, int HEADS>
void write(const KvRowsParams& p, cudaStream_t stream) {
  kv_write_kernel<D, HEADS><<<blocks<HEADS>(p), kWarps * 32, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(p.k), static_cast<const __nv_bfloat16*>(p.v), p.k_stride,
      p.v_stride, static_cast<uint8_t*>(p.k_cache), static_cast<uint8_t*>(p.v_cache),
      static_cast<uint8_t*>(p.k_scale), static_cast<uint8_t*>(p.v_scale), p.block_table,
      p.seq_lens, p.cu, p.num_seqs, p.total, p.Hkv, p.num_pages, p.max_blocks, p.status);
}

template <int D, int HEADS>
void read(const KvRowsParams& p, cudaStream_t stream) {
  kv_read_kernel<D, HEADS><<<blocks<HEADS>(p), kWarps * 32, 0, stream>>>(
      static_cast<const uint8_t*>(p.k_cache), static_cast<const uint8_t*>(p.v_cache),
      static_cast<const uint8_t*>(p.k_scale), static_cast<const uint8_t*>(p.v_scale),
      p.block_table, p.seq_lens, p.cu, static_cast<__nv_bfloat16*>(const_cast<void*>(p.k)),
      static_cast<__nv_bfloat16*>(const_cast<void*>(p.v)), p.num_seqs, p.total, p.Hkv,
      p.num_pages, p.max_blocks, p.status);
}

}  // namespace

// Heads per warp: 512 values of K and of V (four heads at d = 128, eight at
// d = 64), or half as many where the other half of the lanes would have no row.
// us for 64 x [512, 8192] tokens, with one or both of K and V a warp and eight
// heads, and with this: d = 128, 8 heads, write 264, 261, read 270, 252; 2
// heads, write 210, 87, read 176, 90; d = 64, 8 heads, write 174, 133, read 166,
// 130; 2 heads, write 169, 86, read 141, 87.
cudaError_t launch_kv_write_e4m3(const KvRowsParams& p, cudaStream_t stream) {
  if (p.d == 128) p.Hkv <= 2 ? write<128, 2>(p, stream) : write<128, 4>(p, stream);
  else (p.Hkv - 1) % 8 < 4 ? write<64, 4>(p, stream) : write<64, 8>(p, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_e4m3(const KvRowsParams& p, cudaStream_t stream) {
  p.d == 128 ? read<128, 4>(p, stream) : read<64, 8>(p, stream);
  return cudaGetLastError();
}

}  // namespace fa
