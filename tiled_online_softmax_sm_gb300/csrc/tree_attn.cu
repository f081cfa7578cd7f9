// Attention of drafted nodes over a paged cache, bf16 or e4m3, on the tcgen05 tensor
// cores: node i of a sequence sees every key of the context (the first p0 = L - n
// tokens) and the nodes whose bit is set in its row of the mask.
//
// The query rows of a kv head, n nodes times G = H / Hkv heads, are packed into
// tiles of as many whole nodes as 128 rows hold (row r = node r / G, head r % G).
// A unit is one or two such tiles of one (sequence, kv head), so K and V are read
// once for up to 256 rows.  A few dozen nodes are far too few rows to keep the
// tensor cores busy (4 d flops per key and row against 4 d bytes per key): the pass
// is bound by HBM, and what matters is that every SM reads all the time.  So the
// units' K/V tiles (128 keys) form one long list, of which every CTA of a one-wave
// grid takes an equal piece by cost, whatever the lengths.  A unit that lies within
// one piece is finished there; of a unit cut between pieces each CTA leaves its
// rows' (m, l, O) in the workspace, and tree_merge_kernel, launched behind as a
// programmatic dependent, merges them in order (the triples' merge of "S12
// FlashAttention", 练习 1).
//
//   warp 0       copies: query tiles, then K and V tiles a page at a time (TMA,
//                128-byte swizzle)
//   warps 1, 2   tensor memory; lane 0 of warp 1 + w issues the tcgen05.mma of
//                softmax warpgroup w (one thread for both left the tensor pipe idle
//                behind its waits and commits)
//   warp 3       V rows that no node sees are zeroed before the MMA reads them
//   warps 4-11   softmax, thread = query row = tensor-memory lane
//   warps 12-19  e4m3 cache: K and V are widened to bf16 (warp 3 then has no work)
//
// The two softmax warpgroups w have a score tile S_w and an accumulator O_w each.
// A unit of two query tiles gives one to each (every K/V tile is used by both); a
// unit of one query tile gives warpgroup w the K/V tiles j = w mod 2, so that one's
// exponentials run beside the other's MMAs, and the two states merge at the end
// of the segment inside the CTA.
//
// Softmax as in the forward: p = 2^(s scale log2 e - ref), the reference set somewhat
// above the maximum and again only when a tile's maximum passes it by far; two sums are
// kept, of p for the LSE and of the bf16-rounded p that the P V MMA multiplies for O
// (which forms that sum itself at d = 64).
//
// Measured (d = 128, 32 heads of 8, contexts uniform on the range): 64 x 16 nodes over
// [512, 8192] tokens, one query tile a unit, 175 us for 1.04 GB (6.0 TB/s, 0.89 of a
// plain copy; a unit's beginning and end cost as much as three K/V tiles of 350). 4 x
// [48, 64] nodes over [16384, 65536], two query tiles, 128 us for 0.56 GB (4.4 TB/s):
// a K/V tile's MMAs for 256 rows take 2050 clocks at d = 128 (3070 in halves) and its
// exponentials 2050, of the 2500 that HBM takes to bring it.  An MMA of 64 rows or 64
// columns takes as long as one of 128 x 128.  Two CTAs, one query tile each and K and V
// shared through L2, took longer (157 us): L2 delivers every K/V tile twice.  What the
// roles' loops have in common is the instruction cache: with the softmax loops
// unrolled over a whole tile the issuers' code was pushed out of it (64 x 16 198 us).
// A small call (1 x 8 nodes over 1000 tokens, 12 us) is start-up: code that is read for
// the first time, the list, one chain of copy, scores, softmax, values and the merge.
// From the e4m3 cache, half the bytes, the same two take 237 and 153 us: a tile of 128 x
// 128 codes takes the widening warps 1500 clocks beside the softmax, two of them a step,
// the conversions' own rate (the scale as a bf16 product instead of an fp32 one changed
// nothing; codes assembled by integer instructions, all of them or half, 290 and 270 us).
// One warpgroup for it took 246 and 160 us, four rows at once instead of two 283 and 162
// (the instruction cache again); deeper rings gained nothing.
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
constexpr int kTile = 128;        // keys of a K/V tile, rows of a query tile
constexpr int kCtas = 152;        // one per SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's reference is set kRoom above the maximum (log2 units) and set again when the
// maximum passes it by more than kRaise, so p lies within 2^-kRoom .. 2^kRaise of what it
// would be against the maximum itself.  O's fp32 sum of p V grows with p: values of V times
// the row's keys have to stay below 2^119 (with a reference that may lag by 24, and no room,
// below 2^103).  Each raise multiplies O in tensor memory: with scores 4 times as hot as
// random ones 16 x 64 nodes at d = 64 take 58 us, 64 without room, 58 with 16.
constexpr float kRaise = 8.f, kRoom = 8.f;

// E4M3: K and V come from the e4m3 cache.  Warp 0 then stages their codes and scale
// bytes, and two more warpgroups widen them to bf16 (exactly: a code has 4 significant
// bits and its scale is a power of two) into the ring that the MMAs read.
template <int D, bool PAIRS, bool E4M3>
struct Cfg {
  static constexpr int kThreads = E4M3 ? 640 : 384;
  static constexpr int kChunks = D / 64;             // 128-byte pieces of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 64 ? (E4M3 ? 6 : 8) : E4M3 ? 3 : 4;   // K/V ring slots
  static constexpr int kQ = E4M3 && !PAIRS ? 1 : 2;        // query tiles
  static constexpr int kRawTile = kTile * D + kTile;       // staged codes and scale bytes
  static constexpr int kRawStages = !E4M3 ? 0 : D == 64 ? 6 : PAIRS ? 2 : 4;   // tiles staged
  // K/V tiles are laid out in groups of eight keys, a group's 1 KB pieces (64
  // values of each key) side by side, so that one copy brings a whole page
  static constexpr int kGroup = 1024 * kChunks;
  // The sum of the rounded weights, O's divisor: at d = 64 the P V MMA forms it as 16
  // more columns of O, with a block of ones for V (an MMA of 80 columns takes as long as
  // one of 64; 16 x [20, 64] nodes, 24 heads of 8: 62 us where the softmax warps add, 59 so).
  // At d = 128 tensor memory is full.
  static constexpr bool kOnes = D == 64;
  static constexpr int kOnesBytes = kOnes ? kTile * 128 : 0;
  static constexpr int kSmem =
      (kQ + kStages) * kTileBytes + kOnesBytes + kRawStages * kRawTile + 1024;   // + alignment slack
  static constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(128, kOnes ? D + 16 : D, false, true);
};

// Registers of the E4M3 instances: 640 threads at 96, split again among copies and
// issuers, softmax, and widening.
constexpr int kRegsIssue = 64, kRegsSoftmax = 152, kRegsWiden = 56;
static_assert(kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsWiden <= 5 * 96, "register split");

// The unit whose first tile lies in a CTA's piece and whose last one in a later one's.
struct Cut {
  int q0, rows, head0, nt;   // first row of the packed q; rows (0: no such unit); first head; tiles
  int first, weight;         // position of tile 0 in the list, cost of a tile
  int total, sharers;        // the list
};

struct Args {
  const __nv_bfloat16* q;
  const uint8_t* codes[2];   // E4M3: of K and V, and their scale bytes
  const uint8_t* scales[2];
  const int* block_table;
  const int* seq_lens;
  const int* cu_q;
  const int* mask;
  __nv_bfloat16* o;
  float* lse;
  int num_seqs, total_q, max_q, words, H, Hkv, G, tile_nodes, num_pages, max_blocks;
  unsigned long long per_unit;     // 2^40 / (2 * tile_nodes), rounded up
  float scale_log2;
  int skip_first_copy;
  int* status;
  // workspace: per CTA the cut unit that begins in its piece, and two partials per
  // CTA, (m, l, l_p) [2 kCtas][row_cap] and O in float4s [2 kCtas][D / 4][row_cap]
  Cut* cuts;
  float4* part_s;
  float4* part_o;
  int row_cap;
};

// One sequence: its query rows and keys.
struct Seq {
  int q0, n, L;
  bool bad;
};

__device__ __forceinline__ Seq load_seq(const Args& a, int s) {
  Seq Q;
  Q.q0 = __ldg(a.cu_q + s);
  Q.n = __ldg(a.cu_q + s + 1) - Q.q0;
  Q.L = __ldg(a.seq_lens + s);
  Q.bad = Q.q0 < 0 || Q.n < 0 || (long long)Q.q0 + Q.n > a.total_q || Q.n > a.max_q ||
          Q.n > 32ll * a.words || Q.L < Q.n || (long long)Q.L > (long long)a.max_blocks * kPage;
  if (Q.bad) Q.n = 0;
  return Q;
}

// Units of a sequence along its nodes, K/V tiles of each, and the cost of one: with
// two query tiles it takes about a third longer (16 x [20, 64] nodes at d = 64, where both
// occur: 2 : 3 59 us, 3 : 4 57, 4 : 5 58; 2 : 4 cost 12 us more than 2 : 3).  Measured on the
// bf16 cache; the e4m3 one, whose widening takes the same for both, has the same weights.
// (a division by 2 * tile_nodes <= 256 as a product with its reciprocal in 2^-40, which is
// exact below 2^32: the divisions of five roles' segments were a good part of the
// code, and of a small call's time)
__device__ __forceinline__ int node_units(const Args& a, const Seq& Q) {
  return (int)(((unsigned long long)(Q.n + 2 * a.tile_nodes - 1) * a.per_unit) >> 40);
}
__device__ __forceinline__ int ceil_div(int x, int cost) {   // cost 1, 3 or 4; 0 for x < 0
  const uint32_t y = (uint32_t)(max(x, 0) + cost - 1);
  return (int)(cost == 3 ? __umulhi(y, 0xaaaaaaabu) >> 1 : y >> (cost >> 1));
}
__device__ __forceinline__ int key_tiles(const Seq& Q) { return (Q.L + kTile - 1) / kTile; }
__device__ __forceinline__ int tile_cost(const Args& a, const Seq& Q, bool weighed) {
  return !weighed ? 1 : Q.n > a.tile_nodes ? 4 : 3;
}
// Cost of beginning and ending a unit, about three tiles (64 x 16 nodes: 9 174 us, 6 178,
// 4 185).
constexpr int kUnitCost = 9;
// Tiles a CTA from which on costs are weighed.  (Below, a tile costs 1 and a unit
// nothing, so that every piece has a tile; above, a piece is longer than any cost, so
// that of a cut unit every piece between its first and its last tile has one, too.)
constexpr int kWeighedTiles = 8;

// Cost of all units of a sequence.
__device__ __forceinline__ int seq_cost(const Args& a, const Seq& Q, bool weighed) {
  return node_units(a, Q) * a.Hkv * ((weighed ? kUnitCost : 0) + key_tiles(Q) * tile_cost(a, Q, weighed));
}

struct Shared {
  int pre[kMaxTreeSeqs + 1];   // cost of sequences 0 .. s - 1
  int warp_sum[2][32];
  uint64_t raw_full[8], raw_empty[8];   // E4M3: staged tiles
  uint64_t q_full[2], q_empty[2];   // Q tile i
  uint64_t kv_full[8], kv_empty[8]; // ring slots
  uint64_t fix_full[8];             // ring slots: a V tile landed that is to be cleaned
  uint64_t s_full[2][2], p_full[2][2];      // warpgroup, part of the K/V tile
  uint64_t pv_done[2], o_done[2], o_empty[2];
  uint64_t stat_full, stat_empty;   // warpgroup 1's row states are in stat / were read
  uint64_t drain[2];
  float stat[kTile][3];
  uint32_t tmem_base;
  int abort;
};

// The list: sequence s begins at pre[s]; each of its units takes `begin` and then
// its tiles' cost.  The CTA of [xb, xe) has the tiles whose position lies in it.
struct List {
  const int* pre;
  bool weighed;
  int begin, xb, xe;
};

// The part of a unit that lies in this CTA's piece: tiles [j0, j1) of nt.
struct Seg {
  int s, g, node0, nodes;   // nodes of the unit, of one or two query tiles
  Seq Q;
  int first, cost;          // position of tile 0, cost of a tile
  int j0, j1, nt;
  bool pair;                // two query tiles
};

// The copies of a segment go out in the order in which the MMAs use them, so that the
// ring's slots are freed in order: K 0, V 0, K 1, V 1, ... for two query tiles
// (S(j + 1) follows P V(j)); K 0, K 1, V 0, K 2, V 1, K 3, ... for one, whose scores
// are formed two tiles ahead.  Number of the copy of V(j) of nt tiles; behind it comes
// K(j + 1) or K(j + 2), if there is one.
__device__ __forceinline__ int copy_v(bool pair, int j, int nt) {
  return pair ? 2 * j + 1 : min(2, nt) + j + min(j, max(nt - 2, 0));
}

// Steps through the segments of a piece: x is a position in the unit to look at (it
// begins at list.xb) and s its sequence.  False when there are no more.
template <bool PAIRS>
__device__ __forceinline__ bool next_segment(const Args& a, const List& list, int& x, int& s, Seg& S) {
  while (x < list.xe) {
    while (list.pre[s + 1] <= x) ++s;
    S.s = s;
    S.Q = load_seq(a, s);
    S.nt = key_tiles(S.Q);
    S.cost = tile_cost(a, S.Q, list.weighed);
    const int along = node_units(a, S.Q);
    const int unit = list.begin + S.nt * S.cost;
    const unsigned u = (unsigned)(x - list.pre[s]) / (unsigned)unit;
    S.first = list.pre[s] + (int)u * unit + list.begin;
    x = S.first + S.nt * S.cost;
    S.g = along == 1 ? (int)u : (int)(u / (unsigned)along);
    S.node0 = ((int)u - S.g * along) * 2 * a.tile_nodes;
    S.nodes = min(2 * a.tile_nodes, S.Q.n - S.node0);
    S.pair = PAIRS && S.nodes > a.tile_nodes;
    S.j0 = ceil_div(list.xb - S.first, S.cost);
    S.j1 = min(S.nt, ceil_div(list.xe - S.first, S.cost));
    if (S.j0 < S.j1) return true;
  }
  return false;
}

// Which of the keys k0 + 32 c .. + 31 node i sees, as bits.
__device__ __forceinline__ uint32_t sees(const Args& a, const Seq& Q, int i, int key) {
  const int t = key - (Q.L - Q.n);   // the first one's node number; negative: context
  if (t <= -32) return 0xffffffffu;
  const int* row = a.mask + (size_t)(Q.q0 + i) * a.words;
  uint32_t bits;
  if (t < 0) {
    bits = ((uint32_t)__ldg(row) << -t) | ((1u << -t) - 1u);
  } else {
    const int w = t >> 5;
    const uint32_t lo = w < a.words ? (uint32_t)__ldg(row + w) : 0u;
    const uint32_t hi = w + 1 < a.words ? (uint32_t)__ldg(row + w + 1) : 0u;
    bits = __funnelshift_r(lo, hi, t & 31);
  }
  const int left = Q.n - t;          // keys of the sequence from `key` on
  return left >= 32 ? bits : left <= 0 ? 0u : bits & ((1u << left) - 1u);
}

__device__ __forceinline__ float sum_packed(const uint32_t (&p)[16]) {
  float x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    ptx::add_bf16x2_to_f32(x0, x1, p[e]);
    ptx::add_bf16x2_to_f32(x2, x3, p[e + 1]);
  }
  return (x0 + x1) + (x2 + x3);
}

template <int D, bool PAIRS, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, PAIRS, E4M3>::kThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = Cfg<D, PAIRS, E4M3>;
  constexpr int kStages = C::kStages, kThreads = C::kThreads, kRawStages = E4M3 ? C::kRawStages : 1;
  // Scores are formed and used in parts of a K/V tile: halves where units have two query
  // tiles, so that a softmax warpgroup works on one half while the other is multiplied (an
  // MMA of 64 columns takes as long as one of 128, but waiting costs more: 4 x 64 nodes
  // over [16384, 65536] tokens 138 us whole, 129 in halves); whole tiles otherwise, where
  // HBM is the bound (64 x 16 nodes 175 us whole, 182 in halves).
  constexpr int kParts = PAIRS ? 2 : 1, kCols = kTile / kParts;
  constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, kCols, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* sKV = sQ + C::kQ * C::kTileBytes;
  uint8_t* sOnes = sKV + kStages * C::kTileBytes;
  uint8_t* sRaw = sOnes + C::kOnesBytes;
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const status = a.status;
  volatile int* const abort_flag = &sh.abort;
  const uint32_t bar_q = ptx::smem_u32(sh.q_full), bar_qe = ptx::smem_u32(sh.q_empty);
  const uint32_t bar_kvf = ptx::smem_u32(sh.kv_full), bar_kve = ptx::smem_u32(sh.kv_empty);
  const uint32_t bar_fix = ptx::smem_u32(sh.fix_full);
  const uint32_t bar_rf = ptx::smem_u32(sh.raw_full), bar_re = ptx::smem_u32(sh.raw_empty);
  const uint32_t bar_s = ptx::smem_u32(sh.s_full), bar_p = ptx::smem_u32(sh.p_full);
  const uint32_t bar_pv = ptx::smem_u32(sh.pv_done), bar_o = ptx::smem_u32(sh.o_done), bar_oe = ptx::smem_u32(sh.o_empty);
  const uint32_t bar_sf = ptx::smem_u32(&sh.stat_full), bar_se = ptx::smem_u32(&sh.stat_empty);
  const uint32_t bar_drain = ptx::smem_u32(sh.drain);

  // the merge behind this kernel may start its own set-up (it waits for this
  // kernel's completion before it reads the partials)
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 32) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar_q + 8 * i, 1);
      ptx::mbar_init(bar_qe + 8 * i, 2);    // an arrival of each issuer, here and below
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(bar_s + 16 * i + 8 * b, 1);
        ptx::mbar_init(bar_p + 16 * i + 8 * b, kTile);
      }
      ptx::mbar_init(bar_pv + 8 * i, 1);
      ptx::mbar_init(bar_o + 8 * i, 1);
      ptx::mbar_init(bar_oe + 8 * i, kTile);
      ptx::mbar_init(bar_drain + 8 * i, 1);
    }
    for (int i = 0; i < (E4M3 ? kRawStages : 0); ++i) {
      ptx::mbar_init(bar_rf + 8 * i, 33);   // the codes' bytes and each lane's scale bytes
      ptx::mbar_init(bar_re + 8 * i, 8);
    }
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar_kvf + 8 * i, E4M3 ? 8 : 1);   // (an arrival of each widening warp)
      ptx::mbar_init(bar_kve + 8 * i, 2);
      ptx::mbar_init(bar_fix + 8 * i, 1);
    }
    ptx::mbar_init(bar_sf, kTile);
    ptx::mbar_init(bar_se, kTile);
    sh.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if constexpr (C::kOnes) {
    for (int i = threadIdx.x; i < C::kOnesBytes / 16; i += kThreads)
      reinterpret_cast<uint4*>(sOnes)[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&sh.tmem_base), 512);
    ptx::tmem_relinquish();
  }
  // the list: how many tiles there are, whether costs are weighed, the offsets
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(a.num_seqs, (int)threadIdx.x * per), s1 = min(a.num_seqs, s0 + per);
  int tiles = 0;
  List list{sh.pre, false, 0, 0, 0};
  {
    int own[2] = {0, 0};   // of this thread's sequences: tiles, weighed cost
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const Seq Q = load_seq(a, s);
      if (Q.bad && blockIdx.x == 0) atomicExch(status, kDevInvalidArg);
      own[0] += seq_cost(a, Q, false);
      own[1] += seq_cost(a, Q, true);
    }
    int run[2] = {own[0], own[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int v = __shfl_up_sync(0xffffffffu, run[k], o);
        if (lane >= o) run[k] += v;
      }
    if (lane == 31) {
      sh.warp_sum[0][warp] = run[0];
      sh.warp_sum[1][warp] = run[1];
    }
    __syncthreads();
    tiles = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? sh.warp_sum[0][lane] : 0);
    list.weighed = tiles >= kWeighedTiles * (int)gridDim.x;
    list.begin = list.weighed ? kUnitCost : 0;
    const int k = list.weighed ? 1 : 0;
    int at = (k ? run[1] - own[1] : run[0] - own[0]);
    at += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[k][lane] : 0);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      at += per == 1 ? (k ? own[1] : own[0]) : seq_cost(a, load_seq(a, s), list.weighed);
      sh.pre[s + 1] = at;
    }
    if (threadIdx.x == 0) sh.pre[0] = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = sh.tmem_base;
  const int total = sh.pre[a.num_seqs];
  const int W = min((int)gridDim.x, tiles);
  const int cta = blockIdx.x;
  int s_first = 0;   // the sequence that holds position xb
  if (cta < W) {
    list.xb = (int)((long long)cta * total / W);
    list.xe = (int)((long long)(cta + 1) * total / W);
    int hi = a.num_seqs;   // pre[s_first] <= xb < pre[hi]
    while (hi - s_first > 1) {
      const int mid = (s_first + hi) >> 1;
      if (sh.pre[mid] <= list.xb) s_first = mid;
      else hi = mid;
    }
  }

  int x = list.xb, s = s_first;
  Seg S{};
  if constexpr (E4M3) {
    if (warp < 4) ptx::setmaxnreg_dec<kRegsIssue>();
    else if (warp < 12) ptx::setmaxnreg_inc<kRegsSoftmax>();
    else ptx::setmaxnreg_dec<kRegsWiden>();
  }
  // Which nodes' V rows any node of the segment's unit sees, of keys k0 .. k0 + 127 (lane c:
  // 32 of them, c mod 4); the others may hold anything, and 0 * NaN is NaN.
  auto seen_of = [&](int k0) __attribute__((always_inline)) -> uint32_t {
    uint32_t seen = 0u;
#pragma unroll 1
    for (int i = S.node0 + (lane >> 2); i < S.node0 + S.nodes; i += 8) seen |= sees(a, S.Q, i, k0 + 32 * (lane & 3));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, o);
    return seen;
  };
  if (warp == 0) {
    // -------------------------------------------------------------- copies
    int li = 0;                 // tiles issued
    int nq[2] = {0, 0}, half = 0;
    uint32_t to_fix = 0u;       // slots whose last copy went to the fix barrier,
    uint32_t fixes = 0u;        // and the parity of the slots' copies that did
    bool ok = true, skip = a.skip_first_copy != 0;
    while (ok && next_segment<PAIRS>(a, list, x, s, S)) {
      for (int i = 0; i < (S.pair ? 2 : 1) && ok; ++i) {
        // (rows past the sequence's last node are its neighbour's, or zeros behind the
        // last row of all: they only reach their own rows of S and O, which nobody reads)
        const int qb = S.pair ? i : half;
        const int phase = qb == 0 ? nq[0] : nq[1];
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_qe + 8 * qb, (phase & 1) ^ 1, status, abort_flag));
        if (!ok) break;
        if (qb == 0) ++nq[0];
        else ++nq[1];
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(bar_q + 8 * qb, a.tile_nodes * a.G * D * 2);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            ptx::tma_load_3d(ptx::smem_u32(sQ) + qb * C::kTileBytes + c * 16384, &tmQ, 64 * c, S.g * a.G,
                             S.Q.q0 + S.node0 + i * a.tile_nodes, bar_q + 8 * qb);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (!S.pair && C::kQ == 2) half ^= 1;
      const int* ids = a.block_table + (size_t)S.s * a.max_blocks;
      // (lane pg: page pg of tile j)
      auto look_up = [&](int j) {
        return lane < 8 && j < S.j1 && j * kTile + lane * kPage < S.Q.L ? __ldg(ids + j * 8 + lane) : 0;
      };
      auto copy = [&](int which, int j, int id) {
        const int npages = (min(kTile, S.Q.L - j * kTile) + kPage - 1) / kPage;
        if (lane < npages && (id < 0 || id >= a.num_pages)) {
          atomicExch(status, kDevBadBlockTable);
          id = 0;
        }
        if constexpr (E4M3) {
          const int rslot = li % kRawStages;
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_re + 8 * rslot, ((li / kRawStages) & 1) ^ 1, status,
                                                      abort_flag));
          if (!ok) return;
          const uint32_t bar = bar_rf + 8 * rslot, dst = ptx::smem_u32(sRaw) + rslot * C::kRawTile;
          if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, npages * kPage * D);
          __syncwarp();
          if (lane < npages && !skip) {
            const size_t row = (size_t)(id * a.Hkv + S.g) * kPage;
            ptx::bulk_load(dst + lane * kPage * D, (which ? a.codes[1] : a.codes[0]) + row * D, kPage * D, bar);
            ptx::cp_async16(dst + kTile * D + lane * kPage, (which ? a.scales[1] : a.scales[0]) + row);
          }
          if (!skip) ptx::cp_async_arrive(bar);
          skip = false;
          ++li;
          return;
        }
        const int slot = li % kStages;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_kve + 8 * slot, ((li / kStages) & 1) ^ 1, status,
                                                    abort_flag));
        if (!ok) return;
        // (tiles that hold nodes: warp 3 cleans their V rows first)
        const bool cleaned = which == 1 && (j + 1) * kTile > S.Q.L - S.Q.n;
        const uint32_t bar = (cleaned ? bar_fix : bar_kvf) + 8 * slot;
        const uint32_t dst = ptx::smem_u32(sKV) + slot * C::kTileBytes;
        if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, npages * kPage * D * 2);
        __syncwarp();
        if (lane < npages && !skip)
          ptx::tma_load_4d(dst + lane * 2 * C::kGroup, which ? &tmV : &tmK, 0, 0, 0, (id * a.Hkv + S.g) * 2, bar);
        skip = false;
        to_fix = (to_fix & ~(1u << slot)) | ((cleaned ? 1u : 0u) << slot);
        if (cleaned) fixes ^= 1u << slot;
        ++li;
      };
      // page ids of tiles j to j + 3, the last looked up long before its copy
      int i0 = look_up(S.j0), i1 = look_up(S.j0 + 1), i2 = look_up(S.j0 + 2), i3;
      copy(0, S.j0, i0);
      if (!S.pair && ok && S.j0 + 1 < S.j1) copy(0, S.j0 + 1, i1);
      for (int j = S.j0; j < S.j1 && ok; ++j) {
        i3 = look_up(j + 3);
        copy(1, j, i0);
        const int jk = j + (S.pair ? 1 : 2);
        if (ok && jk < S.j1) copy(0, jk, S.pair ? i1 : i2);
        i0 = i1;
        i1 = i2;
        i2 = i3;
      }
    }
    if (!ok && lane == 0) {   // let the copies in flight land before shared memory is released
      for (int l = max(0, li - kRawStages); E4M3 && l < li; ++l)
        ptx::mbar_wait(bar_rf + 8 * (l % kRawStages), (l / kRawStages) & 1, nullptr);
      for (int l = max(0, li - kStages); !E4M3 && l < li; ++l) {
        const int slot = l % kStages;
        if (to_fix >> slot & 1u) ptx::mbar_wait(bar_fix + 8 * slot, (fixes >> slot & 1u) ^ 1u, nullptr);
        else ptx::mbar_wait(bar_kvf + 8 * slot, (l / kStages) & 1, nullptr);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (nq[i] > 0) ptx::mbar_wait(bar_q + 8 * i, (nq[i] - 1) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp <= 2) {
    if (lane == 0) {
      // ------------------------------------------------------ MMA issuers
      const int w = warp - 1;
      const uint64_t qdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sQ), 16, 1024);
      const uint64_t kdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, C::kGroup);
      // (V's second 64 columns lie 1 KB behind the first, or are the ones)
      const uint64_t vdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sKV), C::kOnes ? 0 : 1024, C::kGroup);
      const uint32_t s_tm = tbase + w * kTile, o_tm = tbase + 256 + w * 128;
      int lc = 0;                    // copies of the segments so far
      int nq[2] = {0, 0}, half = 0;  // query tiles used, the buffer of the next single one
      int np = 0, no = 0;            // P tiles, units
      bool ok = true;
      // Every copy is waited for, and its slot released, by both issuers, so that a
      // barrier's phase is never ahead of a wait by two; one that the other issuer
      // alone uses is passed.
      auto landed = [&](int l) {
        return ptx::mbar_wait(bar_kvf + 8 * (l % kStages), (l / kStages) & 1, status, abort_flag);
      };
      auto pass = [&](int l) {
        if (!landed(l)) return false;
        ptx::mbar_arrive(bar_kve + 8 * (l % kStages));
        return true;
      };
      // S = Q K^T over a part of copy l.
      auto score = [&](int l, int part, int qb) {
        const int slot = l % kStages;
        const uint64_t qd = qdesc0 + (uint64_t)(qb * (C::kTileBytes >> 4));
        const uint64_t kd = kdesc0 + (uint64_t)(slot * (C::kTileBytes >> 4) + part * (C::kGroup >> 1));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ptx::mma_ss(s_tm + kCols * part, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                      kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), kIdescS, k > 0);
        ptx::tc_commit(bar_s + 16 * w + 8 * part);
      };
      // O (+)= P V over a part of copy l; false when the wait for P ran out.
      auto values = [&](int l, int part, bool first) {
        if (!ptx::mbar_wait(bar_p + 16 * w + 8 * part, np & 1, status, abort_flag)) return false;
        ptx::tc_fence_after();
        const int slot = l % kStages;
        uint64_t vd = vdesc0 + (uint64_t)(slot * (C::kTileBytes >> 4) + part * (C::kGroup >> 1));
        if constexpr (C::kOnes) vd += (uint64_t)((kStages - slot) * (C::kTileBytes >> 4)) << 16;
#pragma unroll
        for (int k = 0; k < kCols / 16; ++k)
          ptx::mma_ts(o_tm, s_tm + kCols * part + k * 8, vd + (uint64_t)(k * (C::kGroup >> 3)), C::kIdescO,
                      (!first || part > 0 || k > 0) ? 1u : 0u);
        ptx::tc_commit(bar_pv + 8 * w);
        return true;
      };
      while (ok && next_segment<PAIRS>(a, list, x, s, S)) {
        const int nt = S.j1 - S.j0;
        const int step = S.pair ? 1 : 2, j0 = S.pair ? 0 : w;   // this issuer's tiles
        const int qb = S.pair ? w : half;
#pragma unroll
        for (int i = 0; i < 2; ++i) {                           // the query tiles
          if (!S.pair && i != half) continue;
          ok = ok && ptx::mbar_wait(bar_q + 8 * i, nq[i] & 1, status, abort_flag);
          ++nq[i];
          if (ok && (i != qb || j0 >= nt)) ptx::mbar_arrive(bar_qe + 8 * i);
        }
        if (!S.pair && C::kQ == 2) half ^= 1;
        auto k_done = [&](int l, bool last) {      // all of K's scores are on their way
          ptx::tc_commit(bar_kve + 8 * (l % kStages));
          if (last) ptx::tc_commit(bar_qe + 8 * qb);
        };
        for (int j = 0; j < min(step, nt) && ok; ++j) {
          if (!S.pair && j != w) {
            ok = pass(lc + j);
            continue;
          }
          if (!(ok = landed(lc + j))) break;
          ptx::tc_fence_after();
          score(lc + j, 0, qb);
          if constexpr (kParts == 2) score(lc + j, 1, qb);
          k_done(lc + j, j + step >= nt);
        }
        for (int j = 0; j < nt && ok; ++j) {
          const bool mine = S.pair || (j & 1) == w, next = j + step < nt;
          const int lv = lc + copy_v(S.pair, j, nt);            // K(j + step) is the copy behind it
          if (mine) {
            // (the previous unit's O is read out of tensor memory)
            if (j == j0 && !(ok = ptx::mbar_wait(bar_oe + 8 * w, (no++ & 1) ^ 1, status, abort_flag))) break;
            ok = landed(lv) && values(lv, 0, j == j0) && (!next || landed(lv + 1));
            if (!ok) break;
            if constexpr (kParts == 2) {
              if (next) score(lv + 1, 0, qb);
              if (!(ok = values(lv, 1, j == j0))) break;
            }
            ++np;
            ptx::tc_commit(bar_kve + 8 * (lv % kStages));
            if (next) {
              score(lv + 1, kParts - 1, qb);
              k_done(lv + 1, j + 2 * step >= nt);
            } else {
              ptx::tc_commit(bar_o + 8 * w);
            }
          } else {
            ok = pass(lv) && (!next || pass(lv + 1));
          }
        }
        lc += 2 * nt;
      }
      // no tcgen05.mma may still run when the tensor memory is released
      ptx::tc_commit(bar_drain + 8 * w);
      ptx::mbar_wait(bar_drain + 8 * w, 0, nullptr);
    }
    __syncwarp();
  } else if (!E4M3 && warp == 3) {
    // ------------------------------------------------- V rows nobody sees
    int lc = 0;
    uint32_t fixes = 0u;   // parity of each slot's copies to the fix barrier
    bool ok = true;
    while (ok && next_segment<PAIRS>(a, list, x, s, S)) {
      const int fix0 = (S.Q.L - S.Q.n) / kTile;   // first tile with nodes
      for (int j = max(S.j0, fix0); j < S.j1; ++j) {
        const uint32_t seen = seen_of(j * kTile);
        const int slot = (lc + copy_v(S.pair, j - S.j0, S.j1 - S.j0)) % kStages;
        ok = __all_sync(0xffffffffu,
                        ptx::mbar_wait(bar_fix + 8 * slot, fixes >> slot & 1u, status, abort_flag));
        if (!ok) break;
        fixes ^= 1u << slot;
        uint8_t* tile = sKV + slot * C::kTileBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hidden = ~__shfl_sync(0xffffffffu, seen, c);
          while (hidden != 0u) {        // four rows at a time, eight lanes each
            int row = -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int b = __ffs(hidden) - 1;
              if (k == lane >> 3) row = b;
              hidden &= hidden - 1u;    // (0 stays 0)
            }
            if (row >= 0)
#pragma unroll
              for (int h = 0; h < C::kChunks; ++h)
                *reinterpret_cast<uint4*>(tile + (4 * c + (row >> 3)) * C::kGroup + h * 1024 + (row & 7) * 128 +
                                          (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_kvf + 8 * slot);
      }
      lc += 2 * (S.j1 - S.j0);
    }
  } else if (E4M3 && warp >= 12) {
    if constexpr (E4M3) {
      // ---------------------------------------------------------- widening
      // 16 codes of a row (a 16-byte unit) become two units of its bf16 row, where the
      // MMAs' swizzle puts them; rows of V that no node sees become zeros.
      constexpr int kStep = 256 / (D / 16), kB = 2;   // rows a step, steps at once
      const int tid = threadIdx.x - 12 * 32;
      // (d = 128: eight lanes take a half of a row and the other half of the next one, which
      // lie in different banks here and there)
      const int un = D == 128 ? (lane & 3) | ((lane >> 2 ^ lane >> 3) & 1) << 2 : lane & 3;
      const int row0 = D == 128 ? (tid >> 5) * 4 + (lane >> 2 & 1) + (lane >> 4) * 2 : tid >> 2;
      int lc = 0;
      bool ok = true;
      while (ok && next_segment<PAIRS>(a, list, x, s, S)) {
        const int ahead = S.pair ? 1 : 2;
        int kj = S.j0, vj = S.j0;
        while (vj < S.j1 && ok) {                            // in the copies' order
          const bool is_v = !(kj < S.j1 && kj < vj + ahead);
          const int j = is_v ? vj++ : kj++;
          const int slot = lc % kStages, rslot = lc % kRawStages;
          const bool cleaned = is_v && (j + 1) * kTile > S.Q.L - S.Q.n;
          const uint32_t seen = cleaned ? seen_of(j * kTile) : 0u;
          ok = __all_sync(0xffffffffu,
                          ptx::mbar_wait(bar_rf + 8 * rslot, (lc / kRawStages) & 1, status, abort_flag) &&
                              ptx::mbar_wait(bar_kve + 8 * slot, ((lc / kStages) & 1) ^ 1, status, abort_flag));
          if (!ok) break;
          const uint8_t* raw = sRaw + rslot * C::kRawTile;
          uint8_t* tile = sKV + slot * C::kTileBytes;
          auto put = [&](int r, const uint4& lo, const uint4& hi) {
            uint8_t* at = tile + (r >> 3) * C::kGroup + (un >> 2) * 1024 + (r & 7) * 128;
            *reinterpret_cast<uint4*>(at + (((2 * un) & 7) ^ (r & 7)) * 16) = lo;
            *reinterpret_cast<uint4*>(at + (((2 * un + 1) & 7) ^ (r & 7)) * 16) = hi;
          };
#pragma unroll 1
          for (int r0 = row0; r0 < kTile; r0 += kB * kStep) {
            uint4 c[kB];
            uint32_t b[kB];
#pragma unroll
            for (int i = 0; i < kB; ++i) {
              c[i] = *reinterpret_cast<const uint4*>(raw + (r0 + i * kStep) * D + un * 16);
              b[i] = raw[kTile * D + r0 + i * kStep];
            }
            if (cleaned) {
#pragma unroll
              for (int i = 0; i < kB; ++i) {
                const int r = r0 + i * kStep;
                if (!(__shfl_sync(0xffffffffu, seen, r >> 5) >> (r & 31) & 1u)) {
                  c[i] = make_uint4(0u, 0u, 0u, 0u);
                  b[i] = 0u;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < kB; ++i) {
              uint4 lo, hi;
              ptx::widen16(c[i], b[i], lo, hi);
              put(r0 + i * kStep, lo, hi);
            }
          }
          ptx::fence_proxy_async_smem();   // the MMA (and the next copy) come behind these accesses
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(bar_kvf + 8 * slot);
            ptx::mbar_arrive(bar_re + 8 * rslot);
          }
          ++lc;
        }
      }
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ softmax
    const int w = (warp - 4) >> 2;          // warpgroup
    const int quarter = warp & 3;           // tensor-memory lane quarter
    const int r = quarter * 32 + lane;      // row of the query tile
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = lane_base + w * kTile;
    const uint32_t o_col = lane_base + 256 + w * 128;
    const uint64_t sc2 = ptx::f2_bits(a.scale_log2, a.scale_log2);
    int ns = 0, nod[2] = {0, 0}, nstat = 0;
    bool ok = true;
    // for the merge: no unit cut behind this piece, until one is met
    if (threadIdx.x == 128 && FA_IN_BOUNDS(cta, kCtas, status)) a.cuts[cta] = Cut{0, 0, 0, 0, 0, 0, 0, 0};
    while (ok && next_segment<PAIRS>(a, list, x, s, S)) {
      const int nt = S.j1 - S.j0;
      const int tile_rows = a.tile_nodes * a.G;
      const int rows = min(tile_rows, S.nodes * a.G - (S.pair && w == 1 ? tile_rows : 0));   // of this tile
      const bool valid = r < rows;
      const int node = S.node0 + (S.pair && w == 1 ? a.tile_nodes : 0) + r / a.G;
      const int row = (S.pair && w == 1 ? tile_rows : 0) + r;                // of the unit
      // a warp without a valid row leaves P as it is: it reaches only its own rows
      const bool any = quarter * 32 < rows;
      if (threadIdx.x == 128 && S.j0 == 0 && S.j1 < S.nt && FA_IN_BOUNDS(cta, kCtas, status))
        a.cuts[cta] = Cut{S.Q.q0 + S.node0, S.nodes * a.G, S.g * a.G, S.nt, S.first, S.cost, total, W};
      float m_ref = -INFINITY, l_run = 0.f, l_p = 0.f;
      const int step = S.pair ? 1 : 2, jw = S.pair ? 0 : w;
      for (int jl = jw; jl < nt; jl += step) {
        const int k0 = (S.j0 + jl) * kTile;
        const bool masked = k0 + kTile > S.Q.L - S.Q.n;    // the tile holds nodes
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c) vis[c] = valid ? sees(a, S.Q, node, k0 + 32 * c) : 0u;
        }
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          ok = __all_sync(0xffffffffu,
                          ptx::mbar_wait(bar_s + 16 * w + 8 * part, ns & 1, status, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
          if (any) {
            const uint32_t col = s_col + kCols * part;
            uint32_t x0[32], x1[32];
            // 64 scores, those of hidden keys -inf; returns the maximum.  (The loads of a
            // tile without nodes reduce it themselves.)
            auto load = [&](int g) __attribute__((always_inline)) -> float {
              float m0, m1;
              ptx::tmem_ld32_max(col + 64 * g, x0, m0);
              ptx::tmem_ld32_max(col + 64 * g + 32, x1, m1);
              ptx::tmem_wait_ld();
              float top = fmaxf(m0, m1);
              if (masked) {
                const bool low = kParts == 2 ? part == 0 : g == 0;
                const uint32_t v0 = low ? vis[0] : vis[2], v1 = low ? vis[1] : vis[3];
                top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  x0[e] = v0 >> e & 1u ? x0[e] : 0xff800000u;
                  x1[e] = v1 >> e & 1u ? x1[e] : 0xff800000u;
                  top = ptx::fmax3(top, __uint_as_float(x0[e]), __uint_as_float(x1[e]));
                }
              }
              return top;
            };
            float mx = -INFINITY;
            uint64_t nref2 = 0, sum2[2] = {ptx::f2_bits(0.f, 0.f), ptx::f2_bits(0.f, 0.f)};
            // P (bf16 pairs) of 32 scores goes to 16 columns of S whose scores are in
            // registers or done with
            auto form = [&](const uint32_t (&x)[32], int c) __attribute__((always_inline)) {
              uint32_t pp[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float y0, y1;
                ptx::f2_split(
                    ptx::ffma2(ptx::f2_bits(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc2, nref2), y0, y1);
                const float p0 = ptx::ex2(y0), p1 = ptx::ex2(y1);
                sum2[(e / 2) & 1] = ptx::fadd2(sum2[(e / 2) & 1], ptx::f2_bits(p0, p1));
                pp[e / 2] = ptx::pack_bf16x2(p0, p1);
              }
              ptx::tmem_st16(col + c * 16, pp);
              if constexpr (!C::kOnes) l_p += sum_packed(pp);
            };
            // Half a tile: one look.  A whole one: both halves for the maximum, then both
            // again for P.  (Rolled: unrolled over the tile, the code of the softmax warps
            // pushes that of the issuers out of the instruction cache.)
            constexpr int kLooks = kParts == 2 ? 1 : 4;
#pragma unroll 1
            for (int look = 0; look < kLooks; ++look) {
              const float top = load(look & 1);
              if (kParts == 2 || look < 2) {
#pragma unroll
                for (int e = 0; e < 32; ++e)   // (the registers stay theirs until the loads are done)
                  asm volatile("" ::"r"(x0[e]), "r"(x1[e]));
                mx = fmaxf(mx, top);
              }
              if (kParts == 2 || look == 1) {
                const float m_tile = mx * a.scale_log2;   // scale > 0: the maximum commutes with it
                float alpha = 1.f;
                if (valid && (m_tile > m_ref + kRaise || (m_ref == -INFINITY && m_tile > -INFINITY))) {
                  const float raised = m_tile + kRoom;
                  alpha = m_ref == -INFINITY ? 1.f : ptx::ex2(m_ref - raised);
                  m_ref = raised;
                  l_run *= alpha;
                  l_p *= alpha;
                }
                // O is rescaled behind the P V of the part before this one
                if (__any_sync(0xffffffffu, (jl > jw || part > 0) && alpha != 1.f)) {
                  const uint32_t done = kParts == 2 ? part ^ 1 : (ns & 1) ^ 1;   // (the phase before this part's)
                  ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_pv + 8 * w, done, status, abort_flag));
                  if (!ok) break;
                  ptx::tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D / 32 + (C::kOnes ? 1 : 0); ++c) {   // (O, and its sum)
                    uint32_t ov[32];
                    ptx::tmem_ld32(o_col + c * 32, ov);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    ptx::tmem_st32(o_col + c * 32, ov);
                  }
                }
                const float ref = m_ref == -INFINITY ? 0.f : m_ref;
                nref2 = ptx::f2_bits(-ref, -ref);
              }
              if (kParts == 2 || look >= 2) {
                form(x0, 2 * (look & 1));
                form(x1, 2 * (look & 1) + 1);
              }
            }
            if (!ok) break;
            float a0, a1;
            ptx::f2_split(ptx::fadd2(sum2[0], sum2[1]), a0, a1);
            l_run += a0 + a1;
            ptx::tmem_wait_st();
          }
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar_p + 16 * w + 8 * part);
        }
        if (!ok) break;
        ++ns;
      }
      if (!ok) break;
      // ---- the rows of the segment: finished, or left as a partial
      const bool used[2] = {true, S.pair || nt > 1};
      const int ph0 = nod[0] & 1, ph1 = nod[1] & 1;
      ++nod[0];
      if (used[1]) ++nod[1];
      const bool two = !S.pair && nt > 1;     // the two warpgroups' states are to be merged
      const int phs = nstat & 1;
      if (two) ++nstat;
      float c0 = 1.f, c1 = 0.f, m = m_ref;
      if (w == 1 && !S.pair) {
        if (!two) continue;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_se, phs ^ 1, status, abort_flag));
        if (!ok) break;
        sh.stat[r][0] = m_ref;
        sh.stat[r][1] = l_run;
        sh.stat[r][2] = l_p;
        ptx::mbar_arrive(bar_sf);
        continue;
      }
      bool there = w == 0 ? ptx::mbar_wait(bar_o, ph0, status, abort_flag)
                          : ptx::mbar_wait(bar_o + 8, ph1, status, abort_flag);
      if (two)   // (warpgroup 1's states first: behind them its accumulator's phase is this unit's)
        there = there && ptx::mbar_wait(bar_sf, phs, status, abort_flag) &&
                ptx::mbar_wait(bar_o + 8, ph1, status, abort_flag);
      ok = __all_sync(0xffffffffu, there);
      if (!ok) break;
      ptx::tc_fence_after();
      float lp1 = 0.f;
      if constexpr (C::kOnes) {
        uint32_t own, other = 0u;
        ptx::tmem_ld1(o_col + D, own);
        if (two) ptx::tmem_ld1(o_col + 128 + D, other);
        ptx::tmem_wait_ld();
        l_p = __uint_as_float(own);
        lp1 = __uint_as_float(other);
      }
      if (two) {
        const float m1 = sh.stat[r][0], l1 = sh.stat[r][1];
        if constexpr (!C::kOnes) lp1 = sh.stat[r][2];
        ptx::mbar_arrive(bar_se);
        m = fmaxf(m_ref, m1);
        c0 = m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - m);
        c1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - m);
        l_run = c0 * l_run + c1 * l1;
        l_p = c0 * l_p + c1 * lp1;
      }
      const bool whole = S.j0 == 0 && S.j1 == S.nt;
      const size_t tok = (size_t)(S.Q.q0 + node);
      const int head = S.g * a.G + r % a.G;
      const size_t orow = tok * a.H + head;
      const size_t slot = 2 * (size_t)cta + (S.j0 == 0 ? 1 : 0);
      if (whole) {
        // (a NaN sum makes the row NaN; without a visible key it is 0)
        const float inv = l_p > 0.f ? 1.f / l_p : (l_p == 0.f ? 0.f : l_p);
        c0 *= inv;
        c1 *= inv;
      }
      const bool none = l_p == 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x0[32];
        ptx::tmem_ld32(o_col + c * 32, x0);
        if (two) {
          uint32_t x1[32];
          ptx::tmem_ld32(o_col + 128 + c * 32, x1);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x0[e] = __float_as_uint(__uint_as_float(x0[e]) * c0 + __uint_as_float(x1[e]) * c1);
        } else {
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x0[e] = __float_as_uint(__uint_as_float(x0[e]) * c0);
        }
        if (none) {   // (0 * NaN of a V row that others see)
#pragma unroll
          for (int e = 0; e < 32; ++e) x0[e] = 0u;
        }
        if (whole) {
          if (valid && FA_IN_BOUNDS(orow, (size_t)a.total_q * a.H, status)) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + orow * D + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = ptx::pack_bf16x2(__uint_as_float(x0[8 * v + 2 * e]), __uint_as_float(x0[8 * v + 2 * e + 1]));
              dst[v] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        } else if (valid && FA_IN_BOUNDS(row, a.row_cap, status)) {
          // float4s of one column lie side by side over the rows: whole lines a store
          float4* dst = a.part_o + (slot * (D / 4) + c * 8) * a.row_cap + row;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[(size_t)v * a.row_cap] =
                make_float4(__uint_as_float(x0[4 * v]), __uint_as_float(x0[4 * v + 1]),
                            __uint_as_float(x0[4 * v + 2]), __uint_as_float(x0[4 * v + 3]));
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar_oe + 8 * w);
      if (two) ptx::mbar_arrive(bar_oe + 8);
      if (valid && !whole) {
        if (FA_IN_BOUNDS(row, a.row_cap, status))
          a.part_s[slot * a.row_cap + row] = make_float4(m, l_run, l_p, 0.f);
      } else if (valid && a.lse != nullptr) {
        const size_t at = (size_t)head * a.total_q + tok;
        if (FA_IN_BOUNDS(at, (size_t)a.total_q * a.H, status))
          a.lse[at] = l_run > 0.f ? (m + __log2f(l_run)) * kLn2 : (l_run == 0.f ? -INFINITY : l_run);
      }
      __syncwarp();
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tbase, 512);
  }
}

// Merge of the cut units: with M = max m_x, O = sum 2^(m_x - M) O_x / sum 2^(m_x -
// M) l_p_x, the LSE from the exact sums.  Block (cta, 32 rows, 8 float4s of O): the
// unit whose first tile lies in CTA `cta`'s piece; lane = row, warp = float4.  Latency
// counts: eight partials are on their way at a time, in one pass with a running
// maximum.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
tree_merge_kernel(const Args a) {
  const int lane = threadIdx.x & 31, warp = blockIdx.z * kMergeWarps + (threadIdx.x >> 5);
  const int row = blockIdx.y * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 c0 = __ldcg(reinterpret_cast<const int4*>(a.cuts + blockIdx.x));
  const int4 c1 = __ldcg(reinterpret_cast<const int4*>(a.cuts + blockIdx.x) + 1);
  const int q0 = c0.x, rows = c0.y, head0 = c0.z, nt = c0.w, at0 = c1.x, cost = c1.y, total = c1.z, W = c1.w;
  if (row >= rows) return;
  const int first = blockIdx.x;
  // the last tile's CTA: the one whose piece holds its position
  const int last = (int)(((long long)(at0 + (nt - 1) * cost + 1) * W - 1) / total);
  float M = -INFINITY, l = 0.f, lp = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x0 = first; x0 <= last; x0 += 8) {
    float4 st[8], v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int x = x0 + u;
      st[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x <= last) {
        const size_t slot = 2 * (size_t)x + (x == first ? 1 : 0);
        st[u] = __ldcg(a.part_s + slot * a.row_cap + row);
        v[u] = __ldcg(a.part_o + (slot * (D / 4) + warp) * a.row_cap + row);
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, st[u].x);
    const float f = M == -INFINITY ? 1.f : ptx::ex2(M - top);   // (what came before is 0 or NaN, or has an M)
    M = top;
    l *= f;
    lp *= f;
    y.x *= f;
    y.y *= f;
    y.z *= f;
    y.w *= f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float g = st[u].x == -INFINITY ? 0.f : ptx::ex2(st[u].x - top);
      l += g * st[u].y;
      lp += g * st[u].z;
      y.x = fmaf(g, v[u].x, y.x);
      y.y = fmaf(g, v[u].y, y.y);
      y.z = fmaf(g, v[u].z, y.z);
      y.w = fmaf(g, v[u].w, y.w);
    }
  }
  const float inv = lp > 0.f ? 1.f / lp : (lp == 0.f ? 0.f : lp);
  const int head = head0 + row % a.G;
  const size_t tok = (size_t)(q0 + row / a.G), orow = tok * a.H + head;
  if (!FA_IN_BOUNDS(orow, (size_t)a.total_q * a.H, a.status)) return;
  reinterpret_cast<uint2*>(a.o + orow * D)[warp] =
      make_uint2(ptx::pack_bf16x2(y.x * inv, y.y * inv), ptx::pack_bf16x2(y.z * inv, y.w * inv));
  if (warp == 0 && a.lse != nullptr)
    a.lse[(size_t)head * a.total_q + tok] =
        l > 0.f ? (M + __log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
}

// Rows a partial has room for.
int row_cap(int max_q, int G) {
  const long long rows = ((long long)max_q * G + 31) / 32 * 32;
  return (int)(rows < 2 * kTile ? rows : 2 * kTile);
}
constexpr size_t kCutBytes = (kCtas * sizeof(Cut) + 255) / 256 * 256;

template <int D, bool E4M3>
cudaError_t launch(const TreeAttnParams& p, cudaStream_t stream, const char** why) {
  using C = Cfg<D, true, E4M3>;
  using C1 = Cfg<D, false, E4M3>;
  CUtensorMap tmQ, tmK, tmV;
  // (value of 64, key of 8, piece of 64 values, group of 8 keys): one box = a page of
  // one kv head, in the order of the tile
  const uint64_t dims[4] = {64, 8, (uint64_t)C::kChunks, (uint64_t)p.num_pages * p.Hkv * 2};
  const uint64_t strides[3] = {(uint64_t)D * 2, 128, (uint64_t)D * 16};
  const uint32_t box[4] = {64, 8, (uint32_t)C::kChunks, 2};
  const int G = p.H / p.Hkv, tile_nodes = kTile / G;
  // (value of 64, head, node): one box = 64 values of a query tile
  const uint64_t q_dims[3] = {(uint64_t)D, (uint64_t)p.H, (uint64_t)p.total_q};
  const uint64_t q_strides[2] = {(uint64_t)D * 2, (uint64_t)p.H * D * 2};
  const uint32_t q_box[3] = {64, (uint32_t)G, (uint32_t)tile_nodes};
  bool made = make_tmap_bf16(&tmQ, p.q, 3, q_dims, q_strides, q_box);
  if constexpr (E4M3) tmK = tmV = tmQ;   // unused: pages are copied untiled
  else made = made && make_tmap_bf16(&tmK, p.k_cache, 4, dims, strides, box) &&
              make_tmap_bf16(&tmV, p.v_cache, 4, dims, strides, box);
  if (!made) {
    *why = "tensor map for the queries and caches";
    return cudaErrorInvalidValue;
  }
  const auto bytes = [](const void* x) { return static_cast<const uint8_t*>(x); };
  Args a{static_cast<const __nv_bfloat16*>(p.q), {bytes(p.k_cache), bytes(p.v_cache)},
         {bytes(p.k_scale), bytes(p.v_scale)}, p.block_table, p.seq_lens, p.cu_q, p.mask,
         static_cast<__nv_bfloat16*>(p.o), p.lse, p.num_seqs, p.total_q, p.max_q, p.words, p.H, p.Hkv, G,
         tile_nodes, p.num_pages, p.max_blocks, ((1ull << 40) + 2 * tile_nodes - 1) / (2 * tile_nodes), p.scale * kLog2e,
         skip_first_copy_for_tests(), p.status,
         nullptr, nullptr, nullptr, row_cap(p.max_q, G)};
  char* ws = static_cast<char*>(p.workspace);
  a.cuts = reinterpret_cast<Cut*>(ws);
  a.part_s = reinterpret_cast<float4*>(ws + kCutBytes);
  a.part_o = a.part_s + (size_t)2 * kCtas * a.row_cap;
  // (without units of two query tiles the kernel is the smaller one)
  const bool pairs = p.max_q > tile_nodes;
  auto kernel = pairs ? tree_attn_kernel<D, true, E4M3> : tree_attn_kernel<D, false, E4M3>;
  const int smem = pairs ? C::kSmem : C1::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    kernel<<<kCtas, C::kThreads, smem, stream>>>(tmQ, tmK, tmV, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *why = "tree_attn launch";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(kCtas, (unsigned)(a.row_cap / 32), D / 4 / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a);
  if (e != cudaSuccess) *why = "tree_merge launch";
  return e;
}

}  // namespace

size_t tree_attn_workspace(int max_q, int H, int Hkv, int d) {
  return kCutBytes + (size_t)2 * kCtas * row_cap(max_q, H / Hkv) * (d + 4) * sizeof(float);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, cudaStream_t stream, const char** why) {
  if (p.k_scale != nullptr) return p.d == 128 ? launch<128, true>(p, stream, why) : launch<64, true>(p, stream, why);
  return p.d == 128 ? launch<128, false>(p, stream, why) : launch<64, false>(p, stream, why);
}

}  // namespace fa
