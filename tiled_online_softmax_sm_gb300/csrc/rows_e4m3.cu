// Attention of a few query rows over the e4m3 paged cache: one token per
// sequence (decode), or a chunk of new tokens in units of at most 32 rows
// (tokens x grouped heads of one kv head).
//
// The keys of one (sequence, kv head) are split over the warps of a
// thread-block cluster (flash-decoding, "S12 FlashAttention", 它还解锁了什么 and
// 练习 1); each warp runs the online-softmax recurrence over its pages, and the
// splits' states are merged inside the cluster through distributed shared
// memory: one launch, no workspace, and a fixed order of additions.
//
// Mask.  The n query tokens of a sequence are the last n of its L keys; the
// one at position p sees key j when j <= p and (window == 0, or j > p - window,
// or j < sinks).  Only pages that hold a visible key are looked up and read:
// the sinks' pages, then the pages from the first windowed key to the end.
//
// Per page and warp (16 tokens; S and O are formed transposed, so the rows of
// the mma tiles are tokens and value dims, all 16 of them in use, and the
// query rows are the 8-wide column side):
//   S^T = K Q^T   m16n8k16 f16: A = K codes widened to f16 (exact), B = Q in f16
//                 scaled per row by a power of two (exact: bf16 has 8 bits,
//                 f16 11; elements 2^-29 below their row's largest lose bits)
//   x = S * 2^(k exponent) * (scale log2 e, Q's power of two), masked
//   p = 2^(x - m) for the sum l, w = 2^(x + v exponent - r) for the values
//   O^T += V^T w  A = V codes widened to f16 (exact), B = w in f16
// The V scales ride on the weights, so m and r are separate references: w is
// at most 2^8 and a weight only underflows when its token's contribution is
// 2^-32 of the largest one's.  Both are raised lazily, when a score passes
// them by more than 8 (log2 units): a vote per page instead of reductions.
// O = 2^(r - m) acc / l, in fp32, rounded once to bf16.
//
// The lanes' shares of a row are chosen so that no shuffle or ldmatrix is
// needed: lane (r = lane / 4, c = lane % 4) reads tokens r, r + 8 of K at dims
// [c D/4, (c + 1) D/4) and tokens 2c, 2c + 1, 2c + 8, 2c + 9 of V at dims
// [r D/8, (r + 1) D/8), whole 16-byte units, conflict free under the tensor
// copies' swizzle; any order of the reduced dims serves as long as Q's
// fragments use the same one.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include "fa_internal.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kPage = 16;
constexpr int kWarps = 4;             // splits per CTA
constexpr int kStages = 3;            // pages in flight per warp
constexpr int kMaxRankedSeqs = 256;   // launches with more sequences keep index order
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;         // log2 units a score may pass its reference by

template <int D, int NT>
struct Geo {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kPage * D;                        // K or V page, bytes
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kMerge = kWarps * kRows * D * 4;
  static constexpr int kBody = kRing > kMerge ? kRing : kMerge;  // the merge reuses the ring
  static constexpr int kSmem = kBody + 1024;                     // + alignment slack
};

struct Args {
  const __nv_bfloat16* q;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int* block_table;
  const int* seq_lens;
  const int* cu_q;
  __nv_bfloat16* o;
  float* lse;
  long long lse_row, lse_head;   // strides of the LSE
  int num_seqs, total_q, max_q, H, Hkv, num_pages, max_blocks, C, ranked;
  int block_q, num_blocks;       // query tokens per unit, units per (sequence, kv head)
  float scale_log2;
  int causal, window, sinks;
  int skip_first_copy;
  int* status;
};

// 16-byte unit u of row t in a tile whose rows are D bytes, as the tensor
// copies lay it out (128-byte swizzle for D = 128, 64-byte for D = 64).
template <int D>
__device__ __forceinline__ uint32_t unit_at(int t, int u) {
  return D == 128 ? (uint32_t)(t * 128 + ((u ^ (t & 7)) << 4))
                  : (uint32_t)(t * 64 + ((u ^ ((t >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 2)
rows_e4m3_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const Args a) {
  using G_ = Geo<D, NT>;
  constexpr int kRows = G_::kRows;
  constexpr int kTile = G_::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ int s_len[kMaxRankedSeqs];
  __shared__ int s_order[kMaxRankedSeqs];
  __shared__ __align__(16) uint8_t s_scales[kWarps][kStages][2][16];
  __shared__ uint64_t s_bar[kWarps][kStages];
  __shared__ float s_m[kWarps][kRows], s_r[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_cm[kRows], s_cr[kRows], s_cl[kRows];   // the CTA's merged state

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int C = a.C;
  const int cta = C > 1 ? (int)ptx::cluster_rank() : 0;
  const int unit = blockIdx.x / C;
  // longest sequences first (CTAs start in block order): each CTA ranks the
  // lengths, ties by index; skipped when every cluster fits at once
  if (a.ranked) {
    for (int t = threadIdx.x; t < a.num_seqs; t += blockDim.x) s_len[t] = __ldg(a.seq_lens + t);
    __syncthreads();
    for (int t = threadIdx.x; t < a.num_seqs; t += blockDim.x) {
      const int Lt = s_len[t];
      int rank = 0;
      for (int u = 0; u < a.num_seqs; ++u) rank += (s_len[u] > Lt) || (s_len[u] == Lt && u < t);
      s_order[rank] = t;
    }
    __syncthreads();
  }
  const int g = unit % a.Hkv;
  const int qb = unit / a.Hkv % a.num_blocks;
  const int seq = unit / a.Hkv / a.num_blocks;
  const int s = a.ranked ? s_order[seq] : seq;
  const int G = a.H / a.Hkv;
  int L = __ldg(a.seq_lens + s);   // keys, the new tokens' among them
  int q0 = s, n = 1;
  bool bad_seq = L < 0 || (long long)L > (long long)a.max_blocks * kPage;
  if (a.cu_q != nullptr) {
    q0 = __ldg(a.cu_q + s);
    n = __ldg(a.cu_q + s + 1) - q0;
    bad_seq = bad_seq || q0 < 0 || n < 0 || n > a.max_q || (long long)q0 + n > a.total_q;
  }
  if (bad_seq) {
    if (threadIdx.x == 0) atomicExch(a.status, kDevInvalidArg);
    L = 0;
    if (a.cu_q != nullptr) return;   // every CTA of the cluster: its rows are left alone
  }
  // this unit's tokens of the sequence's n, and the first one's position
  int p0 = L - n + qb * a.block_q;
  q0 += qb * a.block_q;
  n = min(n - qb * a.block_q, a.block_q);
  if (n <= 0) return;
  const int rows = n * G;            // row i * G + h: token i, head h of the group

  // keys some row sees: [0, sink_end) and [first, last)
  int first = 0, last = L, sink_end = 0;
  if (a.causal) {
    last = max(0, p0 + n);
    if (a.window > 0) {
      first = (int)max(0ll, (long long)p0 + 1 - a.window);
      sink_end = min(a.sinks, first);
    }
  }
  const int w0 = first / kPage;                                  // first windowed page
  const int w1 = (last + kPage - 1) / kPage;
  const int ns = min((sink_end + kPage - 1) / kPage, w0);        // sink pages before it
  const int np = ns + max(0, w1 - w0);
  const int splits = C * kWarps;
  const int x = cta * kWarps + warp;
  const int tb = (int)((long long)x * np / splits);
  const int te = (int)((long long)(x + 1) * np / splits);
  auto page_of = [&](int t) { return t < ns ? t : w0 + (t - ns); };
  const int* bt_row = a.block_table + (size_t)s * a.max_blocks;

  uint8_t* ring = smem + warp * kStages * 2 * kTile;
  const uint32_t ring_a = ptx::smem_u32(ring);
  const uint32_t scales_a = ptx::smem_u32(&s_scales[warp][0][0][0]);
  const uint32_t bars = ptx::smem_u32(&s_bar[warp][0]);
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) ptx::mbar_init(bars + 8 * st, 1);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __syncwarp();

  // page ids of the next 32 list entries, one per lane; the next 32 are loaded
  // while these are used, so a refill never waits for the table
  int ids = tb + lane < te ? __ldg(bt_row + page_of(tb + lane)) : 0;
  int ids_next = tb + 32 + lane < te ? __ldg(bt_row + page_of(tb + 32 + lane)) : 0;
  int issued = tb;
  uint32_t bad_mask = 0;   // stages whose page id was out of range (page 0 was read instead)
  auto issue = [&](int st) {
    const int k = issued - tb;
    if (k > 0 && (k & 31) == 0) {
      ids = ids_next;
      const int nx = issued + 32 + lane;
      ids_next = nx < te ? __ldg(bt_row + page_of(nx)) : 0;
    }
    int id = __shfl_sync(0xffffffffu, ids, k & 31);
    ++issued;
    const bool bad = id < 0 || id >= a.num_pages;
    bad_mask = (bad_mask & ~(1u << st)) | ((bad ? 1u : 0u) << st);
    if (bad) id = 0;
    if (lane == 0) {
      if (bad) atomicExch(a.status, kDevBadBlockTable);
      const uint32_t bar = bars + 8 * st;
      const int row = (id * a.Hkv + g) * kPage;
      const uint32_t dst = ring_a + st * 2 * kTile;
      ptx::mbar_arrive_expect_tx(bar, 2 * kTile + 32);
      ptx::tma_load_2d(dst, &tmK, 0, row, bar);
      ptx::tma_load_2d(dst + kTile, &tmV, 0, row, bar);
      ptx::bulk_load(scales_a + st * 32, a.k_scale + row, 16, bar);
      ptx::bulk_load(scales_a + st * 32 + 16, a.v_scale + row, 16, bar);
    }
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st) {
    if (issued >= te) break;
    // test hook: the first page is never requested, so its wait runs out
    if (a.skip_first_copy && st == 0) { ++issued; continue; }
    issue(st);
  }

  // Q fragments (B operand): column = query row r of the tile, lane c's dims
  const int r = lane >> 2, c = lane & 3;
  uint32_t qf[NT][D / 16][2];
  float qfac[NT][2];    // scale log2 e and Q's power of two, for columns 2c, 2c + 1
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = 8 * t + r;
    uint32_t w[D / 8];
    if (row < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((size_t)(q0 + row / G) * a.H + g * G + row % G) * D + c * (D / 4));
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        const uint4 v = __ldg(src + u);
        w[4 * u] = v.x;
        w[4 * u + 1] = v.y;
        w[4 * u + 2] = v.z;
        w[4 * u + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int u = 0; u < D / 8; ++u) w[u] = 0u;
    }
    uint32_t mx = 0u;
#pragma unroll
    for (int u = 0; u < D / 8; ++u) mx = __vmaxu2(mx, w[u] & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // multiply by 2^e with the largest element landing in [2^14, 2^15)
    const int e = min(127, 141 - (int)(mx >> 7));
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
#pragma unroll
      for (int hlf = 0; hlf < 2; ++hlf)
        qf[t][u][hlf] = ptx::pack_f16x2(__uint_as_float(w[2 * u + hlf] << 16) * up,
                                        __uint_as_float(w[2 * u + hlf] & 0xffff0000u) * up);
    const float f = a.scale_log2 * ptx::exp2_byte((uint32_t)(127 - e));
    qfac[t][0] = __shfl_sync(0xffffffffu, f, 8 * c);       // lane of row 2c
    qfac[t][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);   // lane of row 2c + 1
  }

  float acc[NT][D / 16][4];
  float m[NT][2], rr[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[t][e] = rr[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
  }
  bool timed_out = false;
  int st = 0;
  uint32_t parity = 0;
  int t_page = tb;
  for (; t_page < te; ++t_page) {
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(bars + 8 * st, parity, a.status))) {
      timed_out = true;
      break;
    }
    const uint32_t kb = ring_a + st * 2 * kTile, vb = kb + kTile;
    const int j0 = page_of(t_page) * kPage;
    const bool bad = (bad_mask >> st) & 1u;
    // every row sees all 16 keys, and all of them are keys of the sequence
    const bool whole = !bad && j0 + kPage <= (a.causal ? p0 + 1 : L) &&
                       (a.window == 0 || j0 > p0 + n - 1 - a.window || j0 + kPage <= a.sinks);

    // S^T for the page: rows = tokens, columns = query rows
    float sa[NT][4], sb[NT][4];   // even and odd k-steps: two chains
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[t][e] = sb[t][e] = 0.f;
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      const int un = D == 128 ? 2 * c + u : c;
      const uint4 x0 = lds128(kb + unit_at<D>(r, un));
      const uint4 x1 = lds128(kb + unit_at<D>(r + 8, un));
      const uint32_t k0[4] = {x0.x, x0.y, x0.z, x0.w}, k1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t fa[4];
        ptx::e4m3x4_to_f16x2(k0[y], fa[0], fa[2]);
        ptx::e4m3x4_to_f16x2(k1[y], fa[1], fa[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          ptx::mma_f16_16816(y & 1 ? sb[t] : sa[t], fa, qf[t][4 * u + y][0], qf[t][4 * u + y][1]);
      }
    }
    // scale bytes of this lane's tokens r and r + 8
    uint32_t kx[2], vx[2];
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf) {
      kx[hlf] = s_scales[warp][st][0][r + 8 * hlf];
      vx[hlf] = s_scales[warp][st][1][r + 8 * hlf];
    }
    const float kf[2] = {ptx::exp2_byte(kx[0]), ptx::exp2_byte(kx[1])};
    const float vf[2] = {(float)((int)vx[0] - 127), (float)((int)vx[1] - 127)};

    float xs[NT][4];
    bool raise = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = (sa[t][e] + sb[t][e]) * kf[e >> 1] * qfac[t][e & 1];
        if (!whole) {
          const int j = j0 + r + 8 * (e >> 1);
          const int row = 8 * t + 2 * c + (e & 1);
          const int p = p0 + row / G;
          bool see = !bad && j < L;
          if (a.causal) {
            see = see && j <= p;
            if (a.window > 0) see = see && (j > p - a.window || j < a.sinks);
          }
          if (!see) v = -INFINITY;
        }
        xs[t][e] = v;
        raise = raise || v > m[t][e & 1] + kRaise || v + vf[e >> 1] > rr[t][e & 1] + kRaise;
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(xs[t][e], xs[t][e + 2]);
          float mo = fmaxf(xs[t][e] + vf[0], xs[t][e + 2] + vf[1]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, off));
          }
          const float mn = fmaxf(m[t][e], mx), ro = fmaxf(rr[t][e], mo);
          // from no reference, or to none, there is nothing to rescale
          l[t][e] *= m[t][e] == -INFINITY ? 1.f : ptx::ex2(m[t][e] - mn);
          const float al = rr[t][e] == -INFINITY ? 1.f : ptx::ex2(rr[t][e] - ro);
          m[t][e] = mn;
          rr[t][e] = ro;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[t][i][e] *= al;
            acc[t][i][e + 2] *= al;
          }
        }
    }
    uint32_t wb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float rm = m[t][e & 1] == -INFINITY ? 0.f : m[t][e & 1];
        const float ro = rr[t][e & 1] == -INFINITY ? 0.f : rr[t][e & 1];
        l[t][e & 1] += ptx::ex2(xs[t][e] - rm);
        w[e] = ptx::ex2(xs[t][e] + vf[e >> 1] - ro);
      }
      wb[t][0] = ptx::movmatrix_trans(ptx::pack_f16x2(w[0], w[1]));
      wb[t][1] = ptx::movmatrix_trans(ptx::pack_f16x2(w[2], w[3]));
    }

    // O^T += V^T w: tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims [r D/8, (r + 1) D/8)
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int tok = 2 * c + (y & 1) + 8 * (y >> 1);
      if constexpr (D == 128) {
        const uint4 v = lds128(vb + unit_at<D>(tok, r));
        vw[y][0] = v.x;
        vw[y][1] = v.y;
        vw[y][2] = v.z;
        vw[y][3] = v.w;
      } else {
        const uint2 v = lds64(vb + unit_at<D>(tok, r >> 1) + (r & 1) * 8);
        vw[y][0] = v.x;
        vw[y][1] = v.y;
      }
      if (!whole) {
        // keys no row sees may hold anything: 0 * NaN would be NaN
        const int j = j0 + tok;
        if (bad || j >= last || (j < first && j >= sink_end)) {
#pragma unroll
          for (int u = 0; u < D / 32; ++u) vw[y][u] = 0u;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
#pragma unroll
      for (int hlf = 0; hlf < 2; ++hlf) {
        // bytes (token 2c, token 2c + 1) of two dims, then of tokens + 8
        const uint32_t sel = hlf ? 0x7362u : 0x5140u;
        uint32_t fa[4];
        ptx::e4m3x4_to_f16x2(__byte_perm(vw[0][u], vw[1][u], sel), fa[0], fa[1]);
        ptx::e4m3x4_to_f16x2(__byte_perm(vw[2][u], vw[3][u], sel), fa[2], fa[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) ptx::mma_f16_16816(acc[t][2 * u + hlf], fa, wb[t][0], wb[t][1]);
      }
    __syncwarp();
    if (issued < te) {
      if (lane == 0) ptx::fence_proxy_async_smem();
      issue(st);
    }
    if (++st == kStages) {
      st = 0;
      parity ^= 1u;
    }
  }
  if (timed_out) {
    // let the copies in flight land (each wait is bounded) before the ring is
    // reused below
    if (lane == 0) {
      for (int t = t_page + 1; t < issued; ++t) {
        if (++st == kStages) {
          st = 0;
          parity ^= 1u;
        }
        ptx::mbar_wait(bars + 8 * st, parity, nullptr);
      }
    }
    __syncwarp();
  }

  // ---- merge the CTA's warps, then the cluster's CTAs
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], off);
      if (r == 0) {
        const int row = 8 * t + 2 * c + e;
        s_m[warp][row] = m[t][e];
        s_r[warp][row] = rr[t][e];
        s_l[warp][row] = l[t][e];
      }
    }
  __syncthreads();   // every warp is done with its ring, too
  float* buf = reinterpret_cast<float*>(smem);   // [kWarps][kRows][D]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * t + 2 * c + e;
      float ro = s_r[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) ro = fmaxf(ro, s_r[w][row]);
      const float f = rr[t][e] == -INFINITY ? 0.f : ptx::ex2(rr[t][e] - ro);
      float4* dst = reinterpret_cast<float4*>(buf + ((size_t)warp * kRows + row) * D + r * (D / 8));
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        dst[i] = make_float4(acc[t][2 * i][e] * f, acc[t][2 * i][e + 2] * f,
                             acc[t][2 * i + 1][e] * f, acc[t][2 * i + 1][e + 2] * f);
    }
  if (threadIdx.x < kRows) {
    const int row = threadIdx.x;
    float M = -INFINITY, R = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, s_m[w][row]);
      R = fmaxf(R, s_r[w][row]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (s_m[w][row] != -INFINITY) sum += s_l[w][row] * ptx::ex2(s_m[w][row] - M);
    s_cm[row] = M;
    s_cr[row] = R;
    s_cl[row] = sum;
  }
  __syncthreads();
  constexpr int kVecs = kRows * D / 4;
  if (C > 1) {
    for (int v = threadIdx.x; v < kVecs; v += kWarps * 32) {
      float4 sum = reinterpret_cast<float4*>(buf)[v];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 y = reinterpret_cast<float4*>(buf)[w * kVecs + v];
        sum.x += y.x;
        sum.y += y.y;
        sum.z += y.z;
        sum.w += y.w;
      }
      reinterpret_cast<float4*>(buf)[v] = sum;
    }
    __syncwarp();
    ptx::cluster_sync();
  }
  // CTA `cta` finishes every C-th 4-value piece of the rows
  for (int v = threadIdx.x * C + cta; v < kVecs; v += kWarps * 32 * C) {
    const int row = v / (D / 4);
    if (row >= rows) break;
    float M = -INFINITY, R = -INFINITY;
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (C == 1) {
      M = s_cm[row];
      R = s_cr[row];
      sum = s_cl[row];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = reinterpret_cast<float4*>(buf)[w * kVecs + v];
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
      }
    } else {
      const uint32_t am = ptx::smem_u32(&s_cm[row]), ar = ptx::smem_u32(&s_cr[row]),
                     al = ptx::smem_u32(&s_cl[row]), ab = ptx::smem_u32(buf + 4 * v);
      for (int k = 0; k < C; ++k) {
        M = fmaxf(M, ptx::ld_cluster_f32(ptx::cluster_map(am, k)));
        R = fmaxf(R, ptx::ld_cluster_f32(ptx::cluster_map(ar, k)));
      }
      for (int k = 0; k < C; ++k) {
        const float mk = ptx::ld_cluster_f32(ptx::cluster_map(am, k));
        const float rk = ptx::ld_cluster_f32(ptx::cluster_map(ar, k));
        const float lk = ptx::ld_cluster_f32(ptx::cluster_map(al, k));
        const float4 z = ptx::ld_cluster_f32x4(ptx::cluster_map(ab, k));
        if (mk == -INFINITY) continue;   // this CTA's keys were all masked
        sum += lk * ptx::ex2(mk - M);
        const float f = ptx::ex2(rk - R);
        y.x += z.x * f;
        y.y += z.y * f;
        y.z += z.z * f;
        y.w += z.w * f;
      }
    }
    const float f = sum > 0.f ? ptx::ex2(R - M) / sum : (sum == 0.f ? 0.f : sum);
    const size_t tok = (size_t)(q0 + row / G);
    const size_t orow = tok * a.H + g * G + row % G;
    if (FA_IN_BOUNDS(orow, (size_t)a.total_q * a.H, a.status)) {
      *reinterpret_cast<uint2*>(a.o + orow * D + (v % (D / 4)) * 4) =
          make_uint2(ptx::pack_bf16x2(y.x * f, y.y * f), ptx::pack_bf16x2(y.z * f, y.w * f));
      if (v % (D / 4) == 0 && a.lse != nullptr)
        a.lse[tok * a.lse_row + (g * G + row % G) * a.lse_head] =
            sum == 0.f ? -INFINITY : (M + __log2f(sum)) * kLn2;
    }
  }
  __syncwarp();
  if (C > 1) ptx::cluster_sync();   // no CTA leaves while another reads its shared memory
}

// Failure-detection test hook, as the bf16 decode's: with
// FA_TEST_FORCE_WAIT_TIMEOUT=1 every warp skips its first page copy, its
// bounded wait expires and FA_ERR_TIMEOUT is recorded.  Unset in normal use.
int skip_first_copy_for_tests() {
  const char* v = getenv("FA_TEST_FORCE_WAIT_TIMEOUT");
  return (v != nullptr && v[0] == '1') ? 1 : 0;
}

template <int D, int NT>
cudaError_t launch(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  using G_ = Geo<D, NT>;
  CUtensorMap tmK, tmV;
  const uint64_t dims[2] = {(uint64_t)D, (uint64_t)p.num_pages * p.Hkv * kPage};
  const uint64_t strides[1] = {(uint64_t)D};
  const uint32_t box[2] = {(uint32_t)D, (uint32_t)kPage};
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_tmap_bf16(&tmK, p.k_cache, 2, dims, strides, box, sw, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
      !make_tmap_bf16(&tmV, p.v_cache, 2, dims, strides, box, sw, CU_TENSOR_MAP_DATA_TYPE_UINT8)) {
    *why = "tensor map for the e4m3 caches";
    return cudaErrorInvalidValue;
  }
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) {
    *why = "query SM count";
    return e;
  }
  // Cluster size: doubled while the machine has room for more CTAs and a warp
  // still keeps at least two pages (the longest sequence the table or the
  // window allows).
  const int G = p.H / p.Hkv;
  const int block_q = 8 * NT / G < p.max_q ? 8 * NT / G : p.max_q;
  const int num_blocks = (p.max_q + block_q - 1) / block_q;
  const long long units = (long long)p.num_seqs * num_blocks * p.Hkv;
  long long pages = p.max_blocks;
  if (p.causal && p.window > 0) {
    const long long w = ((long long)p.window + block_q + 30) / 16 + (p.sinks + 15ll) / 16;
    if (w < pages) pages = w;
  }
  const int room = (NT == 1 ? 4 : 2) * sms;
  int C = 1;
  while (C < 8 && units * C < room && pages >= 4ll * C * kWarps) C *= 2;
  Args a{static_cast<const __nv_bfloat16*>(p.q), static_cast<const uint8_t*>(p.k_scale),
         static_cast<const uint8_t*>(p.v_scale), p.block_table, p.seq_lens, p.cu_q,
         static_cast<__nv_bfloat16*>(p.o), p.lse, p.cu_q ? 1 : p.H, p.cu_q ? p.total_q : 1,
         p.num_seqs, p.total_q, p.max_q, p.H, p.Hkv, p.num_pages, p.max_blocks, C,
         p.num_seqs > 1 && p.num_seqs <= kMaxRankedSeqs && units * C > room ? 1 : 0,
         block_q, num_blocks, p.scale * kLog2e, p.causal, p.window, p.sinks, skip_first_copy_for_tests(), p.status};
  auto kernel = rows_e4m3_kernel<D, NT>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G_::kSmem);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute(rows_e4m3)";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = G_::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, tmK, tmV, a);
  if (e != cudaSuccess) *why = "rows_e4m3 launch";
  return e;
}

template <int D>
cudaError_t by_rows(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  const long long rows = (long long)p.max_q * (p.H / p.Hkv);
  if (rows <= 8) return launch<D, 1>(p, stream, why);
  if (rows <= 16) return launch<D, 2>(p, stream, why);
  return launch<D, 4>(p, stream, why);
}

}  // namespace

cudaError_t launch_rows_e4m3(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? by_rows<128>(p, stream, why) : by_rows<64>(p, stream, why);
}

}  // namespace fa
