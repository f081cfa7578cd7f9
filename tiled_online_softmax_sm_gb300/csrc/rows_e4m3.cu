// Attention of a few query rows over the e4m3 paged cache: one token per
// sequence (decode), or a short chunk whose tokens times grouped heads make at
// most 32 rows per kv head (rows_e4m3_form).
//
// The keys of a unit (sequence, kv head) are split over warps (flash-decoding,
// "S12 FlashAttention", 它还解锁了什么 and 练习 1), each of which runs the
// online-softmax recurrence over its pages.  Two forms:
//
//   rows_cluster_kernel  The warps of a thread-block cluster of 1 to 8 CTAs
//       share a unit and merge their states through distributed shared memory,
//       in one launch.
//   rows_stream_kernel   For few long units, which clusters of 8 would leave
//       most SMs idle on, and with a workspace: the units' pages form one long
//       list, of which every warp of a one-wave grid takes an equal piece,
//       whatever the lengths.  A warp leaves one (m, r, l, O) partial per unit
//       it touches in the workspace, and rows_merge_kernel, launched behind it
//       as a programmatic dependent, merges each unit's partials in a fixed
//       order.
//
// Up to 8 rows it is bound by HBM once there is work for all warps: 64 sequences
// of [512, 8192] tokens (d = 128, 8 kv heads of 4; 517 MB) take 84 us (6.1 TB/s,
// 0.90 of a plain copy), and no less in a copy that skips all the arithmetic.
// With more rows the chain of each page bounds it (loads, MMAs, exponentials,
// transpose, MMAs) at 12 warps an SM: 4 new tokens of the same sequences take 147
// us (0.52), of 16 such sequences 47 (134 MB, 0.42; the copies alone 35).
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
//   p = 2^(x - m) for the sum l, w = 2^(x - m + v exponent - r) for the values
//   O^T += V^T w  A = V codes widened to f16 (exact), B = w in f16
// The V scales ride on the weights, so the weights have a reference of their own,
// r, kept relative to m (small numbers: at scores of 2^20 a sum of score and
// exponent would be off by 2^-4).  Both are raised lazily, when an exponent of p
// or w passes 15: a vote per page instead of reductions.  m is raised to the
// largest score, r to 7 below the largest weighted one, so w uses f16's upper
// range: it is at most 2^15, exact to 11 bits down to 2^-21 of the largest weight
// times 2^(v exponent), and zero below 2^-32 of it.  O = 2^r acc / l, in fp32,
// rounded once to bf16.
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

#include "fa_internal.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kPage = 16;
constexpr int kWarps = 4;             // warps per CTA
constexpr int kMaxRanked = 256;       // cluster launches with more sequences keep index order
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 15.f;          // largest exponent of p and w (f16 holds up to 2^16)
constexpr float kUnder = 7.f;         // how far r lies below the largest weighted score when raised
// The reference of a row that has seen no key (its r is 0): finite, so that
// 2^(x - m) is 0 for a masked x = -inf without a guard, and below every score of
// finite rows.
constexpr float kNone = -3.4e38f;

template <int D, int NT, bool STREAM>
struct Geo {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kPage * D;                        // K or V page, bytes
  // pages in flight per warp and CTAs per SM
  static constexpr int kStages = NT == 4 ? 6 : NT == 2 || STREAM ? 4 : 3;
  static constexpr int kCtasPerSm = NT == 4 ? 2 : NT == 2 || STREAM ? 3 : 4;
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kMerge = kWarps * kRows * D * 4;
  static constexpr int kBody = STREAM || kRing > kMerge ? kRing : kMerge;  // the merge reuses the ring
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
  float scale_log2;
  int causal, window, sinks;
  int skip_first_copy;
  int* status;
  // stream form: the list's offsets, left for the merge (num_seqs + 1), and the
  // partials [warps + units][kRows], of m, r, l and then O
  int* pre;
  float* part_s;
  float* part_o;
  size_t part_rows;
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

// One sequence's query rows and the keys they see.
struct Seq {
  int q0, n;       // first query row of the packed q, query tokens
  int L;           // keys, the new tokens' among them
  int first, last, sink_end;  // keys some row sees: [0, sink_end) and [first, last)
  int ns, w0, np;  // pages: 0 .. ns - 1, then w0, w0 + 1, ...; np of them
  bool bad;        // offsets or length out of range
};

__device__ __forceinline__ Seq load_seq(const Args& a, int s) {
  Seq Q;
  Q.L = __ldg(a.seq_lens + s);
  Q.q0 = s;
  Q.n = 1;
  Q.bad = Q.L < 0 || (long long)Q.L > (long long)a.max_blocks * kPage;
  if (a.cu_q != nullptr) {
    Q.q0 = __ldg(a.cu_q + s);
    Q.n = __ldg(a.cu_q + s + 1) - Q.q0;
    Q.bad = Q.bad || Q.q0 < 0 || Q.n < 0 || Q.n > a.max_q || (long long)Q.q0 + Q.n > a.total_q;
    if (Q.bad) Q.n = 0;   // its rows are left alone
  }
  if (Q.bad) Q.L = 0;
  Q.first = 0;
  Q.last = Q.L;
  Q.sink_end = 0;
  if (a.causal && a.window > 0) {
    Q.first = (int)max(0ll, (long long)Q.L - Q.n + 1 - a.window);
    Q.sink_end = min(a.sinks, Q.first);
  }
  Q.w0 = Q.first / kPage;
  Q.ns = min((Q.sink_end + kPage - 1) / kPage, Q.w0);
  Q.np = Q.n > 0 ? Q.ns + max(0, (Q.last + kPage - 1) / kPage - Q.w0) : 0;
  return Q;
}

__device__ __forceinline__ int page_of(const Seq& Q, int t) {
  return t < Q.ns ? t : Q.w0 + (t - Q.ns);
}

// The recurrence's state of a warp, in fragment layout: columns 2c, 2c + 1 of
// row tile t; l holds this lane's tokens only until it is summed up.
template <int D, int NT>
struct State {
  float acc[NT][D / 16][4];
  float m[NT][2], r[NT][2], l[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = kNone;
        r[t][e] = l[t][e] = 0.f;
      }
    }
  }

  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], off);
  }
};

// Q fragments (B operand): column = query row r of the tile, lane c's dims;
// fac: scale log2 e and Q's power of two, for columns 2c, 2c + 1.
template <int D, int NT>
struct Query {
  uint32_t f[NT][D / 16][2];
  float fac[NT][2];

  __device__ __forceinline__ void load(const Args& a, const Seq& Q, int g, int G, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int rows = Q.n * G;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = 8 * t + r;
      uint32_t w[D / 8];
      if (row < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((size_t)(Q.q0 + row / G) * a.H + g * G + row % G) * D + c * (D / 4));
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
      // multiply by 2^e with the largest element landing in [2^14, 2^15) (below it
      // for rows under 2^-106, where a larger e would make fac a subnormal)
      const int e = min(120, 141 - (int)(mx >> 7));
      const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf)
          f[t][u][hlf] = ptx::pack_f16x2(__uint_as_float(w[2 * u + hlf] << 16) * up,
                                         __uint_as_float(w[2 * u + hlf] & 0xffff0000u) * up);
      const float k = a.scale_log2 * ptx::exp2_byte((uint32_t)(127 - e));
      fac[t][0] = __shfl_sync(0xffffffffu, k, 8 * c);       // lane of row 2c
      fac[t][1] = __shfl_sync(0xffffffffu, k, 8 * c + 4);   // lane of row 2c + 1
    }
  }
};

// S^T of a page: rows = tokens r, r + 8, columns = query rows 2c, 2c + 1.
template <int D, int NT>
__device__ __forceinline__ void scores(uint32_t kb, const Query<D, NT>& q, int lane,
                                       float (&s)[NT][4]) {
  const int r = lane >> 2, c = lane & 3;
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
        ptx::mma_f16_16816(y & 1 ? sb[t] : sa[t], fa, q.f[t][4 * u + y][0], q.f[t][4 * u + y][1]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = sa[t][e] + sb[t][e];
}

// The recurrence's step over one page whose raw scores are s: keys j0 ..
// j0 + 15, V tile at vb, scale bytes (K's 16, then V's 16) at sc.
template <int D, int NT>
__device__ __forceinline__ void absorb(const Args& a, const Seq& Q, int G, const Query<D, NT>& q,
                                       const float (&s)[NT][4], uint32_t vb, const uint8_t* sc,
                                       int j0, bool bad, int lane, State<D, NT>& S) {
  const int r = lane >> 2, c = lane & 3;
  const int p0 = Q.L - Q.n;   // position of the first query token
  // every row sees all 16 keys, and all of them are keys of the sequence
  const bool whole = !bad && j0 + kPage <= (a.causal ? p0 + 1 : Q.L) &&
                     (a.window == 0 || j0 > Q.L - 1 - a.window || j0 + kPage <= a.sinks);
  // V: tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims [r D/8, (r + 1) D/8)
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
  }
  // scale bytes of this lane's tokens r and r + 8
  const float kf[2] = {ptx::exp2_byte(sc[r]), ptx::exp2_byte(sc[r + 8])};
  const float vf[2] = {ptx::log2_byte(sc[16 + r]), ptx::log2_byte(sc[24 + r])};
  float xs[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      // the powers of two first: s times K's alone may overflow where Q's takes it
      // back.  (Bounded, so that a row of zeros has score 0 whatever its scale.)
      xs[t][e] = s[t][e] * fminf(kf[e >> 1] * q.fac[t][e & 1], 3.4028234e38f);
  if (!whole) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + r + 8 * (e >> 1);
        const int row = 8 * t + 2 * c + (e & 1);
        const int p = p0 + row / G;
        bool see = !bad && j < Q.L;
        if (a.causal) {
          see = see && j <= p;
          if (a.window > 0) see = see && (j > p - a.window || j < a.sinks);
        }
        if (!see) xs[t][e] = -INFINITY;
      }
    // keys no row sees may hold anything: 0 * NaN would be NaN
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int j = j0 + 2 * c + (y & 1) + 8 * (y >> 1);
      if (bad || j >= Q.last || (j < Q.first && j >= Q.sink_end)) {
#pragma unroll
        for (int u = 0; u < D / 32; ++u) vw[y][u] = 0u;
      }
    }
  }
  float xp[NT][4], xw[NT][4];   // the exponents of p and w
  auto exponents = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xp[t][e] = xs[t][e] - S.m[t][e & 1];
        xw[t][e] = xp[t][e] + (vf[e >> 1] - S.r[t][e & 1]);
      }
  };
  exponents();
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e & 1] = ptx::fmax3(top[e & 1], xp[t][e], xw[t][e]);
  if (__any_sync(0xffffffffu, fmaxf(top[0], top[1]) > kTop)) {
    float mn[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(xs[t][e], xs[t][e + 2]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mn[t][e] = fmaxf(S.m[t][e], mx);
      }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float up = S.m[t][e] - mn[t][e];
        float mo = fmaxf(xs[t][e] - mn[t][e] + vf[0], xs[t][e + 2] - mn[t][e] + vf[1]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, off));
        const float ro = fmaxf(S.r[t][e] + up, mo - kUnder);
        S.l[t][e] *= ptx::ex2(up);   // (from none: 0 * 0)
        const float al = ptx::ex2(S.r[t][e] + up - ro);
        S.m[t][e] = mn[t][e];
        S.r[t][e] = ro;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          S.acc[t][i][e] *= al;
          S.acc[t][i][e + 2] *= al;
        }
      }
    exponents();
  }
  uint32_t wb[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      S.l[t][e & 1] += ptx::ex2(xp[t][e]);
      w[e] = ptx::ex2(xw[t][e]);
    }
    wb[t][0] = ptx::movmatrix_trans(ptx::pack_f16x2(w[0], w[1]));
    wb[t][1] = ptx::movmatrix_trans(ptx::pack_f16x2(w[2], w[3]));
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
      for (int t = 0; t < NT; ++t) ptx::mma_f16_16816(S.acc[t][2 * u + hlf], fa, wb[t][0], wb[t][1]);
    }
}

__device__ __forceinline__ float max4(float a, float b, float c, float d) {
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// A warp's ring of pages in flight.
template <int D, int kStages>
struct Ring {
  static constexpr int kTile = kPage * D;
  uint32_t data, scales, bars;
  const uint8_t* sc;
  int wst;          // stage waited for next, and its phase
  uint32_t wph;
  int ist;          // stage issued next
  int pending;      // stages issued and not waited for
  uint32_t bad;     // stages whose page id was out of range (page 0 was read instead)

  __device__ __forceinline__ void init(uint8_t* ring, uint8_t* scale_area, uint64_t* bar, int lane) {
    data = ptx::smem_u32(ring);
    sc = scale_area;
    scales = ptx::smem_u32(scale_area);
    bars = ptx::smem_u32(bar);
    wst = ist = pending = 0;
    wph = bad = 0u;
    if (lane == 0) {
      for (int st = 0; st < kStages; ++st) ptx::mbar_init(bars + 8 * st, 1);
      ptx::fence_mbar_init();
      ptx::fence_proxy_async_smem();
    }
    __syncwarp();
  }

  // Copies page `id` of kv head g into the next stage.
  __device__ __forceinline__ void issue(const Args& a, const CUtensorMap* tmK,
                                        const CUtensorMap* tmV, int id, int g, int lane,
                                        bool skip = false) {
    const bool out = id < 0 || id >= a.num_pages;
    bad = (bad & ~(1u << ist)) | ((out ? 1u : 0u) << ist);
    if (out) id = 0;
    if (lane == 0 && !skip) {
      if (out) atomicExch(a.status, kDevBadBlockTable);
      const uint32_t bar = bars + 8 * ist;
      const int row = (id * a.Hkv + g) * kPage;
      const uint32_t dst = data + ist * 2 * kTile;
      ptx::mbar_arrive_expect_tx(bar, 2 * kTile + 32);
      ptx::tma_load_2d(dst, tmK, 0, row, bar);
      ptx::tma_load_2d(dst + kTile, tmV, 0, row, bar);
      ptx::bulk_load(scales + ist * 32, a.k_scale + row, 16, bar);
      ptx::bulk_load(scales + ist * 32 + 16, a.v_scale + row, 16, bar);
    }
    ist = ist + 1 == kStages ? 0 : ist + 1;
    ++pending;
  }

  // Waits for the next stage; its index, or -1 when the wait ran out.
  __device__ __forceinline__ int wait(int* status) {
    const int st = wst;
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(bars + 8 * st, wph, status))) return -1;
    step();
    return st;
  }

  __device__ __forceinline__ void step() {
    --pending;
    if (++wst == kStages) {
      wst = 0;
      wph ^= 1u;
    }
  }

  // After a wait ran out: gives the copies in flight time to land (each wait
  // is bounded) before their shared memory is given up or reused.
  __device__ __forceinline__ void drain(int lane) {
    while (pending > 0) {
      if (lane == 0) ptx::mbar_wait(bars + 8 * wst, wph, nullptr);
      step();
    }
    __syncwarp();
  }
};

// Pages t0 .. t1 - 1 of a unit's list, whose copies come out of the ring in
// order; refill() issues the next copy, if there is one, into the stage just
// freed.  False when a wait ran out.
template <int D, int NT, int kStages, typename Refill>
__device__ __forceinline__ bool run_pages(const Args& a, const Seq& Q, int G,
                                          const Query<D, NT>& q, Ring<D, kStages>& ring, int t0, int t1,
                                          int lane, State<D, NT>& S, Refill refill) {
  constexpr int kTile = kPage * D;
  for (int t = t0; t < t1; ++t) {
    const int st = ring.wait(a.status);
    if (st < 0) return false;
    float sx[NT][4];
    scores<D, NT>(ring.data + st * 2 * kTile, q, lane, sx);
    absorb<D, NT>(a, Q, G, q, sx, ring.data + st * 2 * kTile + kTile, ring.sc + st * 32,
                  page_of(Q, t) * kPage, (ring.bad >> st) & 1u, lane, S);
    __syncwarp();
    refill();
  }
  return true;
}

// ------------------------------------------------------------- cluster form
// Longest sequences first, since CTAs start in block order: the sequence of rank
// s when they are counted into classes of length (four an octave, by index within
// one).  Every CTA counts for itself; skipped when all clusters fit at once.  64
// x [512, 8192] tokens, 8 kv heads: 112 us in index order, 85 so; 256 x [100,
// 1000]: 62 and 61 (and 84 when every pair of sequences was compared).
constexpr int kClasses = 128;
struct Order {
  uint32_t count[kMaxRanked / 32][kClasses / 4];   // bytes: of 32 sequences, then of those before them
  uint16_t first[kClasses];
  int pick;
};

__device__ __forceinline__ int by_length(const Args& a, int s, Order& o) {
  constexpr int kEach = kMaxRanked / (kWarps * 32);
  static_assert(kMaxRanked / 32 * kClasses / 4 == kEach * kWarps * 32, "one word a thread and turn");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int cls[kEach], before[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = threadIdx.x + i * kWarps * 32;
    // (exponent and two bits of the length: 0 for none, at most 126)
    const int L = t < a.num_seqs ? max(0, __ldg(a.seq_lens + t)) : 0;
    cls[i] = kClasses - 1 - (L > 0 ? (int)(__float_as_uint((float)L) >> 21) - 127 * 4 + 1 : 0);
    (&o.count[0][0])[t] = 0u;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool mine = (int)threadIdx.x + i * kWarps * 32 < a.num_seqs;
    const uint32_t same = __match_any_sync(0xffffffffu, mine ? cls[i] : -1);
    before[i] = __popc(same & ((1u << lane) - 1u));
    if (mine && before[i] == 0)
      reinterpret_cast<uint8_t*>(o.count[warp + i * kWarps])[cls[i]] = (uint8_t)__popc(same);
  }
  __syncthreads();
  if (warp == 0) {   // lane: four classes
    uint32_t sum = 0u, last = 0u;
#pragma unroll
    for (int k = 0; k < kMaxRanked / 32; ++k) {
      sum += last;   // at most 224 a byte
      last = o.count[k][lane];
      o.count[k][lane] = sum;
    }
    int n[4], run = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[e] = run;
      run += (int)((sum >> 8 * e) & 0xffu) + (int)((last >> 8 * e) & 0xffu);
    }
    int scan = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += v;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o.first[4 * lane + e] = (uint16_t)(scan - run + n[e]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = threadIdx.x + i * kWarps * 32;
    if (t < a.num_seqs && s == o.first[cls[i]] + before[i] +
                                   reinterpret_cast<uint8_t*>(o.count[warp + i * kWarps])[cls[i]])
      o.pick = t;
  }
  __syncthreads();
  return o.pick;
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, Geo<D, NT, false>::kCtasPerSm)
rows_cluster_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const Args a) {
  using G_ = Geo<D, NT, false>;
  constexpr int kRows = G_::kRows;
  constexpr int kTile = G_::kTile;
  constexpr int kStages = G_::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(16) uint8_t s_scales[kWarps][kStages][32];
  __shared__ uint64_t s_bar[kWarps][kStages];
  __shared__ float s_m[kWarps][kRows], s_r[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_cm[kRows], s_cr[kRows], s_cl[kRows];   // the CTA's merged state
  __shared__ Order s_order;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int C = a.C;
  const int cta = C > 1 ? (int)ptx::cluster_rank() : 0;
  const int unit = blockIdx.x / C;
  const int g = unit % a.Hkv;
  const int G = a.H / a.Hkv;
  int s = unit / a.Hkv;
  if (a.ranked) s = by_length(a, s, s_order);
  const Seq Q = load_seq(a, s);
  if (Q.bad && threadIdx.x == 0) atomicExch(a.status, kDevInvalidArg);
  if (Q.n == 0) return;              // every CTA of the cluster
  const int rows = Q.n * G;          // row i * G + h: token i, head h of the group
  const int splits = C * kWarps;
  const int x = cta * kWarps + warp;
  const int tb = (int)((long long)x * Q.np / splits);
  const int te = (int)((long long)(x + 1) * Q.np / splits);
  const int* bt_row = a.block_table + (size_t)s * a.max_blocks;

  Ring<D, kStages> ring;
  ring.init(smem + warp * kStages * 2 * kTile, &s_scales[warp][0][0], &s_bar[warp][0], lane);
  // page ids of the next 32 list entries, one per lane; the 32 behind them are
  // loaded while these are used, so a refill never waits for the table
  int ids = tb + lane < te ? __ldg(bt_row + page_of(Q, tb + lane)) : 0;
  int ids_next = tb + 32 + lane < te ? __ldg(bt_row + page_of(Q, tb + 32 + lane)) : 0;
  int issued = tb;
  auto issue = [&](bool skip) {
    const int k = issued - tb;
    if (k > 0 && (k & 31) == 0) {
      ids = ids_next;
      const int nx = issued + 32 + lane;
      ids_next = nx < te ? __ldg(bt_row + page_of(Q, nx)) : 0;
    }
    ring.issue(a, &tmK, &tmV, __shfl_sync(0xffffffffu, ids, k & 31), g, lane, skip);
    ++issued;
  };
  // (test hook: the first page is never requested, so its wait runs out)
  for (int k = 0; k < kStages && issued < te; ++k) issue(a.skip_first_copy && k == 0);

  Query<D, NT> q;
  q.load(a, Q, g, G, lane);
  State<D, NT> S;
  S.clear();
  if (tb < te && !run_pages<D, NT, kStages>(a, Q, G, q, ring, tb, te, lane, S, [&]() {
        if (issued < te) {
          if (lane == 0) ptx::fence_proxy_async_smem();
          issue(false);
        }
      }))
    ring.drain(lane);

  // ---- merge the CTA's warps, then the cluster's CTAs
  S.sum_l();
  if (r == 0) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e;
        s_m[warp][row] = S.m[t][e];
        s_r[warp][row] = S.r[t][e];
        s_l[warp][row] = S.l[t][e];
      }
  }
  __syncthreads();   // every warp is done with its ring, too
  float* buf = reinterpret_cast<float*>(smem);   // [kWarps][kRows][D]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * t + 2 * c + e;
      const float M = max4(s_m[0][row], s_m[1][row], s_m[2][row], s_m[3][row]);
      const float ro = max4(s_r[0][row] + s_m[0][row], s_r[1][row] + s_m[1][row],
                            s_r[2][row] + s_m[2][row], s_r[3][row] + s_m[3][row]) - M;
      const float f = ptx::ex2(S.r[t][e] + (S.m[t][e] - M) - ro);
      float4* dst = reinterpret_cast<float4*>(buf + ((size_t)warp * kRows + row) * D + r * (D / 8));
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        dst[i] = make_float4(S.acc[t][2 * i][e] * f, S.acc[t][2 * i][e + 2] * f,
                             S.acc[t][2 * i + 1][e] * f, S.acc[t][2 * i + 1][e + 2] * f);
    }
  if (threadIdx.x < kRows) {
    const int row = threadIdx.x;
    float M = -INFINITY, R = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, s_m[w][row]);
      R = fmaxf(R, s_r[w][row] + s_m[w][row]);
    }
    R -= M;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum += s_l[w][row] * ptx::ex2(s_m[w][row] - M);
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
        const float mk = ptx::ld_cluster_f32(ptx::cluster_map(am, k));
        M = fmaxf(M, mk);
        R = fmaxf(R, ptx::ld_cluster_f32(ptx::cluster_map(ar, k)) + mk);
      }
      R -= M;
      for (int k = 0; k < C; ++k) {
        const float mk = ptx::ld_cluster_f32(ptx::cluster_map(am, k));
        const float rk = ptx::ld_cluster_f32(ptx::cluster_map(ar, k));
        const float lk = ptx::ld_cluster_f32(ptx::cluster_map(al, k));
        const float4 z = ptx::ld_cluster_f32x4(ptx::cluster_map(ab, k));
        sum += lk * ptx::ex2(mk - M);
        const float f = ptx::ex2(rk + (mk - M) - R);
        y.x += z.x * f;
        y.y += z.y * f;
        y.z += z.z * f;
        y.w += z.w * f;
      }
    }
    const float f = sum > 0.f ? ptx::ex2(R) / sum : (sum == 0.f ? 0.f : sum);
    const size_t tok = (size_t)(Q.q0 + row / G);
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

// -------------------------------------------------------------- stream form
constexpr int kMaxSeqs = 1024;   // sequences whose page counts a CTA sums up

template <int D, int NT>
constexpr int kStreamWarps = 152 * Geo<D, NT, true>::kCtasPerSm * kWarps;   // one wave

// pre[s]: list pages of sequences 0 .. s - 1 (s = 0 .. num_seqs).
__device__ __forceinline__ void sum_pages(const Args& a, int* pre, int* warp_sum, bool report) {
  const int per = (a.num_seqs + kWarps * 32 - 1) / (kWarps * 32);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = min(a.num_seqs, (int)threadIdx.x * per), s1 = min(a.num_seqs, s0 + per);
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const Seq Q = load_seq(a, s);
    if (Q.bad && report) atomicExch(a.status, kDevInvalidArg);
    mine += Q.np * a.Hkv;
    pre[s + 1] = mine;
  }
  int run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  int base = run - mine;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  for (int s = s0; s < s1; ++s) pre[s + 1] += base;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}

// Warps that share `total` pages: at least two each, so no share is empty.
__device__ __forceinline__ int sharers(int warps, int total) {
  return total == 0 ? 0 : max(1, min(warps, total / 2));
}

// The sequence whose pages hold list position x.
__device__ __forceinline__ int seq_of(const int* pre, int num_seqs, int x) {
  int lo = 0, hi = num_seqs;   // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, Geo<D, NT, true>::kCtasPerSm)
rows_stream_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const Args a) {
  using G_ = Geo<D, NT, true>;
  constexpr int kRows = G_::kRows;
  constexpr int kTile = G_::kTile;
  constexpr int kStages = G_::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(16) uint8_t s_scales[kWarps][kStages][32];
  __shared__ uint64_t s_bar[kWarps][kStages];
  __shared__ int s_pre[kMaxSeqs + 1];
  __shared__ int s_sum[kWarps];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int G = a.H / a.Hkv;
  // the merge behind this kernel may start its own set-up (it waits for this
  // kernel's completion before it reads the partials)
  asm volatile("griddepcontrol.launch_dependents;");
  Ring<D, kStages> ring;
  ring.init(smem + warp * kStages * 2 * kTile, &s_scales[warp][0][0], &s_bar[warp][0], lane);
  sum_pages(a, s_pre, s_sum, blockIdx.x == 0);
  const int total = s_pre[a.num_seqs];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.num_seqs; i += kWarps * 32)
      if (FA_IN_BOUNDS(i, kMaxSeqs + 1, a.status)) a.pre[i] = s_pre[i];
  const int W = sharers(gridDim.x * kWarps, total);
  const int wid = blockIdx.x * kWarps + warp;
  if (wid >= W) return;
  const int xb = (int)((long long)wid * total / W);
  const int xe = (int)((long long)(wid + 1) * total / W);

  // the copies' cursor: position ix, in unit (is, ig), whose list starts at i0
  int ix = xb, is = seq_of(s_pre, a.num_seqs, xb), i0 = 0, i1 = 0, ig = 0;
  int ins = 0, iw0 = 0;
  int ids = 0;
  auto enter = [&]() {       // the unit of position ix
    while (s_pre[is + 1] <= ix) ++is;
    const int np = (s_pre[is + 1] - s_pre[is]) / a.Hkv;
    ig = (ix - s_pre[is]) / np;
    i0 = s_pre[is] + ig * np;
    i1 = i0 + np;
    const Seq Q = load_seq(a, is);
    ins = Q.ns;
    iw0 = Q.w0;
  };
  auto fetch_ids = [&]() {   // the ids of the next 32 pages of the unit, one per lane
    const int t = ix - i0 + lane;
    ids = ix + lane < min(i1, xe)
              ? __ldg(a.block_table + (size_t)is * a.max_blocks + (t < ins ? t : iw0 + (t - ins)))
              : 0;
  };
  int k_ids = 0;
  auto issue = [&](bool skip) {
    if (ix >= i1) {
      enter();
      k_ids = 32;
    }
    if (k_ids == 32) {
      fetch_ids();
      k_ids = 0;
    }
    ring.issue(a, &tmK, &tmV, __shfl_sync(0xffffffffu, ids, k_ids), ig, lane, skip);
    ++k_ids;
    ++ix;
  };
  for (int k = 0; k < kStages && ix < xe; ++k) issue(a.skip_first_copy && k == 0);

  int s = seq_of(s_pre, a.num_seqs, xb);
  Query<D, NT> q;
  State<D, NT> S;
  for (int x = xb; x < xe;) {
    while (s_pre[s + 1] <= x) ++s;
    const Seq Q = load_seq(a, s);
    const int g = (x - s_pre[s]) / Q.np;
    const int u0 = s_pre[s] + g * Q.np;
    const int x1 = min(xe, u0 + Q.np);
    q.load(a, Q, g, G, lane);
    S.clear();
    if (!run_pages<D, NT, kStages>(a, Q, G, q, ring, x - u0, x1 - u0, lane, S, [&]() {
          if (ix < xe) {
            if (lane == 0) ptx::fence_proxy_async_smem();
            issue(false);
          }
        })) {
      ring.drain(lane);
      return;
    }
    // this unit's partial: along the list the (warp, unit) pairs are numbered
    // by the sum of the two
    S.sum_l();
    const size_t slot = (size_t)(wid + s * a.Hkv + g) * kRows;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + 2 * c + e;
        if (row >= Q.n * G || !FA_IN_BOUNDS(slot + row, a.part_rows, a.status)) continue;
        if (r == 0)
          *reinterpret_cast<float4*>(a.part_s + (slot + row) * 4) =
              make_float4(S.m[t][e], S.r[t][e], S.l[t][e], 0.f);
        float4* dst = reinterpret_cast<float4*>(a.part_o + (slot + row) * D + r * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          dst[i] = make_float4(S.acc[t][2 * i][e], S.acc[t][2 * i][e + 2], S.acc[t][2 * i + 1][e],
                               S.acc[t][2 * i + 1][e + 2]);
      }
    x = x1;
  }
}

// Merge of the stream form: a block per (unit, row), or a warp where few
// sharers meet.  M = max m_k, R = max (r_k + m_k) - M, l = sum 2^(m_k - M) l_k,
// O = 2^R / l * sum 2^(r_k + (m_k - M) - R) O_k (a rounding of R cancels); warp w
// of a block takes partials w, w + 8, ..., and the warps' sums are added in
// order.  Latency counts here: the list's offsets come from the stream kernel,
// and partials are loaded eight at a time.
constexpr int kMergeWarps = 8;
template <int D, int NT, int WPP>
__global__ void __launch_bounds__(kMergeWarps * 32)
rows_merge_kernel(const Args a, int warps) {
  constexpr int kRows = 8 * NT;
  constexpr int kPairs = kMergeWarps / WPP;
  constexpr int kVec = D / 32;   // values per lane
  __shared__ float s_mr[kMergeWarps][2];
  __shared__ float s_red[kMergeWarps][D + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv;
  const int max_rows = a.max_q * G;
  const unsigned pair = blockIdx.x * kPairs + warp / WPP;
  const int unit = (int)(pair / (unsigned)max_rows), row = (int)(pair % (unsigned)max_rows);
  const int s = unit / a.Hkv, g = unit % a.Hkv;
  const int part = warp % WPP;
  const bool in = s < a.num_seqs;
  Seq Q{};
  if (in) Q = load_seq(a, s);
  const bool live = in && row < Q.n * G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = __ldcg(a.pre + a.num_seqs);
  int w0 = 0, w1 = -1;     // the warps that share the unit
  if (live && Q.np > 0) {
    const int W = sharers(warps, total);
    const long long x0 = __ldcg(a.pre + s) + (long long)g * Q.np, x1 = x0 + Q.np - 1;
    w0 = (int)(((x0 + 1) * W - 1) / total);
    w1 = (int)(((x1 + 1) * W - 1) / total);
  }
  const size_t slot0 = (size_t)unit * kRows + row;
  const float4* ps = reinterpret_cast<const float4*>(a.part_s);
  // the first eight of this warp's partials are on their way before the
  // references are known
  float v[8][kVec];
  float4 st[8];
  auto fetch = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int w = k0 + u * WPP;
      st[u] = make_float4(kNone, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[u][i] = 0.f;
      if (w <= w1) {
        const size_t at = slot0 + (size_t)w * kRows;
        st[u] = __ldcg(ps + at);
        const float* po = a.part_o + at * D + lane * kVec;
        if constexpr (kVec == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(po));
          v[u][0] = x.x;
          v[u][1] = x.y;
          v[u][2] = x.z;
          v[u][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(po));
          v[u][0] = x.x;
          v[u][1] = x.y;
        }
      }
    }
  };
  fetch(w0 + part);
  float M = kNone, R = kNone;
  for (int w = w0 + (WPP == 1 ? lane : (int)threadIdx.x); w <= w1; w += WPP * 32) {
    const float4 x = __ldcg(ps + slot0 + (size_t)w * kRows);
    M = fmaxf(M, x.x);
    R = fmaxf(R, x.y + x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, o));
  }
  if constexpr (WPP > 1) {
    if (lane == 0) {
      s_mr[warp][0] = M;
      s_mr[warp][1] = R;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPP; ++w) {
      M = fmaxf(M, s_mr[w][0]);
      R = fmaxf(R, s_mr[w][1]);
    }
  }
  R -= M;
  float l = 0.f, y[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) y[i] = 0.f;
  for (int k = w0 + part; k <= w1; k += 8 * WPP) {
    if (k > w0 + part) fetch(k);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = ptx::ex2(st[u].y + (st[u].x - M) - R);
      l += st[u].z * ptx::ex2(st[u].x - M);
#pragma unroll
      for (int i = 0; i < kVec; ++i) y[i] = fmaf(v[u][i], f, y[i]);
    }
  }
  if constexpr (WPP > 1) {
    if (lane == 0) s_red[warp][D] = l;
#pragma unroll
    for (int i = 0; i < kVec; ++i) s_red[warp][lane * kVec + i] = y[i];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < WPP; ++w) {
      l += s_red[warp + w][D];
#pragma unroll
      for (int i = 0; i < kVec; ++i) y[i] += s_red[warp + w][lane * kVec + i];
    }
  }
  if (!live) return;
  const float f = l > 0.f ? ptx::ex2(R) / l : (l == 0.f ? 0.f : l);
  const size_t tok = (size_t)(Q.q0 + row / G);
  const int head = g * G + row % G;
  const size_t orow = tok * a.H + head;
  if (FA_IN_BOUNDS(orow, (size_t)a.total_q * a.H, a.status)) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + orow * D + lane * kVec);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) dst[i] = ptx::pack_bf16x2(y[2 * i] * f, y[2 * i + 1] * f);
    if (lane == 0 && a.lse != nullptr)
      a.lse[tok * a.lse_row + head * a.lse_head] = l == 0.f ? -INFINITY : (M + __log2f(l)) * kLn2;
  }
}

// The most pages a unit can have: the table's, or the window's.
long long unit_pages(int max_blocks, int max_q, int causal, int window, int sinks) {
  if (!causal || window <= 0) return max_blocks;
  const long long w = ((long long)window + max_q + 30) / 16 + (sinks + 15ll) / 16;
  return w < max_blocks ? w : max_blocks;
}

// The stream form, for few long units that clusters of 8 leave most of the
// machine idle on: 1 x 131072 tokens 191 (C = 8) against 55 us, 1 x 8192 17.4
// against 13.4, 4 x [512, 8192] 16.4 against 14.5; but 1 x 1000 7.5 against 8.5.
template <int D, int NT>
bool few_units(long long units) {
  return 2 * 8 * units <= Geo<D, NT, false>::kCtasPerSm * 152;
}
template <int D, int NT>
bool takes_shares(int num_seqs, int Hkv, int max_blocks, long long pages) {
  const long long units = (long long)num_seqs * Hkv;
  return num_seqs <= kMaxSeqs && units * max_blocks <= 0x7fffffffLL && pages >= 128 &&
         few_units<D, NT>(units);
}

template <int D, int NT>
cudaError_t launch(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  using GC = Geo<D, NT, false>;
  using GS = Geo<D, NT, true>;
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
  const long long units = (long long)p.num_seqs * p.Hkv;
  const long long pages = unit_pages(p.max_blocks, p.max_q, p.causal, p.window, p.sinks);
  Args a{static_cast<const __nv_bfloat16*>(p.q), static_cast<const uint8_t*>(p.k_scale),
         static_cast<const uint8_t*>(p.v_scale), p.block_table, p.seq_lens, p.cu_q,
         static_cast<__nv_bfloat16*>(p.o), p.lse, p.cu_q ? 1 : p.H, p.cu_q ? p.total_q : 1,
         p.num_seqs, p.total_q, p.max_q, p.H, p.Hkv, p.num_pages, p.max_blocks, 1, 0,
         p.scale * kLog2e, p.causal, p.window, p.sinks, skip_first_copy_for_tests(), p.status,
         nullptr, nullptr, nullptr, 0};
  constexpr int W = kStreamWarps<D, NT>;
  constexpr int kRows = GS::kRows;
  cudaError_t e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = GC::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Cluster size: while a warp keeps two pages and the clusters, longest first,
  // make about two waves of CTAs, or one where a window makes all units alike
  // (its pages are then the least of the table's).  us for C = 1, 2, 4, 8 at
  // d = 128, 4 rows, 8 kv heads: 16 x [512, 8192] tokens 94, 55, 38, 35;
  // 64 x [512, 8192] 127, 93, 107, 130; 128 x [512, 8192] 178, 192, 212, 269;
  // under a window of 2048, 64 sequences 52, 59, 68, 95.
  const int room = GC::kCtasPerSm * 152;
  const bool alike = p.causal && p.window > 0 && 2 * pages <= p.max_blocks;
  int C = 1;
  while (C < 8 && 4 * units * 2 * C <= (alike ? 4 : 7) * room && pages >= 4ll * C * kWarps) C *= 2;
  if (p.workspace != nullptr && takes_shares<D, NT>(p.num_seqs, p.Hkv, p.max_blocks, pages)) {
    const size_t slots = (size_t)(W + units) * kRows;
    a.part_rows = slots;
    a.part_s = static_cast<float*>(p.workspace);
    a.part_o = a.part_s + slots * 4;
    a.pre = reinterpret_cast<int*>(a.part_o + slots * D);
    auto kernel = rows_stream_kernel<D, NT>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GS::kSmem);
    if (e == cudaSuccess) {
      kernel<<<W / kWarps, kWarps * 32, GS::kSmem, stream>>>(tmK, tmV, a);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
      *why = "rows_stream launch";
      return e;
    }
    // one warp per (unit, row), or eight where units are shared by many warps
    const long long pairs = units * p.max_q * (p.H / p.Hkv);
    const bool wide = W > 12 * units;
    cfg.gridDim = dim3((unsigned)(wide ? pairs : (pairs + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    e = wide ? cudaLaunchKernelEx(&cfg, rows_merge_kernel<D, NT, kMergeWarps>, a, W)
             : cudaLaunchKernelEx(&cfg, rows_merge_kernel<D, NT, 1>, a, W);
    if (e != cudaSuccess) *why = "rows_merge launch";
    return e;
  }
  a.C = C;
  a.ranked = p.num_seqs > 1 && p.num_seqs <= kMaxRanked && units * C > room;
  auto kernel = rows_cluster_kernel<D, NT>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GC::kSmem);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute(rows_cluster)";
    return e;
  }
  cfg.gridDim = dim3((unsigned)(units * C));
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, tmK, tmV, a);
  if (e != cudaSuccess) *why = "rows_cluster launch";
  return e;
}

template <int D>
cudaError_t by_rows(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  const long long rows = (long long)p.max_q * (p.H / p.Hkv);
  if (rows <= 8) return launch<D, 1>(p, stream, why);
  if (rows <= 16) return launch<D, 2>(p, stream, why);
  return launch<D, 4>(p, stream, why);
}

// Workspace of the stream form for sequences of max_q tokens.
template <int D, int NT>
size_t stream_bytes(long long units) {
  return (size_t)(kStreamWarps<D, NT> + units) * Geo<D, NT, true>::kRows * (D + 4) * sizeof(float) +
         (kMaxSeqs + 1) * sizeof(int);
}

}  // namespace

size_t rows_e4m3_workspace(int num_seqs, int max_q, int H, int Hkv, int d) {
  const long long rows = (long long)max_q * (H / Hkv), units = (long long)num_seqs * Hkv;
  if (!rows_e4m3_form(max_q, H, Hkv, d)) return cache_parts_bytes(num_seqs, max_q, H, Hkv, d);
  if (num_seqs > kMaxSeqs || rows > kRowsE4m3Max) return 0;
  if (d == 128)
    return rows <= 8 ? stream_bytes<128, 1>(units)
                     : rows <= 16 ? stream_bytes<128, 2>(units) : stream_bytes<128, 4>(units);
  return rows <= 8 ? stream_bytes<64, 1>(units)
                   : rows <= 16 ? stream_bytes<64, 2>(units) : stream_bytes<64, 4>(units);
}

bool rows_e4m3_few_units(int num_seqs, int Hkv) {   // (the 8-row form's limit is the largest)
  return few_units<128, 1>((long long)num_seqs * Hkv) || few_units<64, 1>((long long)num_seqs * Hkv);
}

namespace {
template <int D>
bool uses_workspace(int num_seqs, int max_q, int H, int Hkv, int max_blocks, long long pages) {
  const long long rows = (long long)max_q * (H / Hkv);
  if (rows <= 8) return takes_shares<D, 1>(num_seqs, Hkv, max_blocks, pages);
  if (rows <= 16) return takes_shares<D, 2>(num_seqs, Hkv, max_blocks, pages);
  return rows <= kRowsE4m3Max && takes_shares<D, 4>(num_seqs, Hkv, max_blocks, pages);
}
}  // namespace

bool rows_e4m3_uses_workspace(int num_seqs, int max_q, int H, int Hkv, int d, int max_blocks,
                              int causal, int window, int sinks) {
  const long long pages = unit_pages(max_blocks, max_q, causal, window, sinks);
  return d == 128 ? uses_workspace<128>(num_seqs, max_q, H, Hkv, max_blocks, pages)
                  : uses_workspace<64>(num_seqs, max_q, H, Hkv, max_blocks, pages);
}

cudaError_t launch_rows_e4m3(const PagedE4m3Params& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? by_rows<128>(p, stream, why) : by_rows<64>(p, stream, why);
}

}  // namespace fa
