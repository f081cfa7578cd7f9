// Attention of drafted nodes over the bf16 paged cache, on the tcgen05 tensor
// cores: node i of a sequence sees every key of the context (the first p0 = L - n
// tokens) and the nodes whose bit is set in its row of the mask.
//
// The query rows of a kv head, n nodes times G = H / Hkv heads, are packed into
// 128-row tiles (row r = node r / G, head r % G).  A unit is one or two such tiles
// of one (sequence, kv head), so K and V are read once for 256 rows.  A few dozen
// nodes are far too few rows to keep the tensor cores busy (4 d flops per key and
// row against 4 d bytes per key): the pass is bound by HBM, and what matters is
// that every SM reads all the time.  So the units' K/V tiles (128 keys) form one
// long list, of which every CTA of a one-wave grid takes an equal piece, whatever
// the lengths.  A unit that lies within one piece is finished there; of a unit cut
// between pieces each CTA leaves its rows' (m, l, O) in the workspace, and
// tree_merge_kernel, launched behind as a programmatic dependent, merges them in
// order (the triples' merge of "S12 FlashAttention", 练习 1).
//
//   warp 0       K and V tiles, a page at a time (TMA, 128-byte swizzle)
//   warp 1       tensor memory; its lane 0 issues every tcgen05.mma
//   warp 2       query rows into shared memory
//   warp 3       V rows that no node sees are zeroed before the MMA reads them
//   warps 4-11   softmax, thread = query row = tensor-memory lane
//
// The two softmax warpgroups w have a score tile S_w and an accumulator O_w each.
// A unit of two row tiles gives one to each (every K/V tile is used by both); a
// unit of one row tile gives warpgroup w the K/V tiles j = w mod 2, so that one's
// exponentials run beside the other's MMAs, and the two states merge at the end
// of the unit inside the CTA.
//
// Softmax as in the forward: p = 2^(s scale log2 e - ref), the reference raised
// only when a tile's maximum passes it by more than 8; two sums are kept, of p for
// the LSE and of the bf16-rounded p that the P V MMA multiplies for O.  A row's 128
// scores are read from tensor memory twice, for the maximum (reduced by the load
// itself) and for p, 32 columns at a time: that keeps a thread within the 168
// registers that 384 threads leave it.
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
constexpr int kThreads = 384;
constexpr int kCtas = 152;        // one per SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;     // log2 units

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;             // 128-byte pieces of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;   // K/V ring slots
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;   // + alignment slack
  static constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, kTile, false, false);
  static constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(128, D, false, true);
};

// The unit that begins in a CTA's piece and ends in a later one's.
struct Cut {
  int seq, row0, rows;   // sequence, first of its rows n * G, rows of the unit
  int head;              // kv head
  int last;              // CTA of the last piece; -1: no such unit
  int late;              // the unit is not the first of this CTA's piece
  int pad[2];
};

struct Args {
  const __nv_bfloat16* q;
  const int* block_table;
  const int* seq_lens;
  const int* cu_q;
  const int* mask;
  __nv_bfloat16* o;
  float* lse;
  int num_seqs, total_q, max_q, words, H, Hkv, G, num_pages, max_blocks;
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

// Units of a sequence along its rows, and K/V tiles of each.
__device__ __forceinline__ int row_units(const Args& a, const Seq& Q) {
  return (Q.n * a.G + 2 * kTile - 1) / (2 * kTile);
}
__device__ __forceinline__ int key_tiles(const Seq& Q) { return (Q.L + kTile - 1) / kTile; }

struct Shared {
  int pre[kMaxTreeSeqs + 1];   // list tiles of sequences 0 .. s - 1
  int warp_sum[kThreads / 32];
  uint64_t q_full[2], q_empty[2];   // Q tile i
  uint64_t kv_full[8], kv_empty[8]; // ring slots
  uint64_t fix_full[8];             // ring slots: a V tile landed that is to be cleaned
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t stat_full, stat_empty;   // warpgroup 1's row states are in stat / were read
  uint64_t drain;
  float stat[kTile][3];
  uint32_t tmem_base;
  int abort;
};

// The part of a unit that lies in this CTA's piece: tiles [j0, j1) of nt.
struct Seg {
  int s, g, row0, rows;   // rows: of the unit, at most 256
  Seq Q;
  int j0, j1, nt;
  bool pair;              // two query tiles
};

// The segment at list position x, and the position behind it.
__device__ __forceinline__ int segment(const Args& a, const int* pre, int x, int xe, int& s, Seg& S) {
  while (pre[s + 1] <= x) ++s;
  S.s = s;
  S.Q = load_seq(a, s);
  S.nt = key_tiles(S.Q);
  const int ru = row_units(a, S.Q);
  const int u = (x - pre[s]) / S.nt;
  const int u0 = pre[s] + u * S.nt;
  S.g = u / ru;
  S.row0 = (u - S.g * ru) * 2 * kTile;
  S.rows = min(2 * kTile, S.Q.n * a.G - S.row0);
  S.pair = S.rows > kTile;
  S.j0 = x - u0;
  S.j1 = min(xe - u0, S.nt);
  return u0 + S.j1;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const Args a) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* sKV = sQ + 2 * C::kTileBytes;
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const status = a.status;
  volatile int* const abort_flag = &sh.abort;
  const uint32_t bar_q = ptx::smem_u32(sh.q_full), bar_qe = ptx::smem_u32(sh.q_empty);
  const uint32_t bar_kvf = ptx::smem_u32(sh.kv_full), bar_kve = ptx::smem_u32(sh.kv_empty);
  const uint32_t bar_fix = ptx::smem_u32(sh.fix_full);
  const uint32_t bar_s = ptx::smem_u32(sh.s_full), bar_p = ptx::smem_u32(sh.p_full);
  const uint32_t bar_o = ptx::smem_u32(sh.o_done), bar_oe = ptx::smem_u32(sh.o_empty);
  const uint32_t bar_sf = ptx::smem_u32(&sh.stat_full), bar_se = ptx::smem_u32(&sh.stat_empty);
  const uint32_t bar_drain = ptx::smem_u32(&sh.drain);

  // the merge behind this kernel may start its own set-up (it waits for this
  // kernel's completion before it reads the partials)
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar_q + 8 * i, 32);
      ptx::mbar_init(bar_qe + 8 * i, 1);
      ptx::mbar_init(bar_s + 8 * i, 1);
      ptx::mbar_init(bar_p + 8 * i, kTile);
      ptx::mbar_init(bar_o + 8 * i, 1);
      ptx::mbar_init(bar_oe + 8 * i, kTile);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar_kvf + 8 * i, 1);
      ptx::mbar_init(bar_kve + 8 * i, 1);
      ptx::mbar_init(bar_fix + 8 * i, 1);
    }
    ptx::mbar_init(bar_sf, kTile);
    ptx::mbar_init(bar_se, kTile);
    ptx::mbar_init(bar_drain, 1);
    sh.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&sh.tmem_base), 512);
    ptx::tmem_relinquish();
  }
  {  // the list's offsets
    const int per = (a.num_seqs + kThreads - 1) / kThreads;
    const int s0 = min(a.num_seqs, (int)threadIdx.x * per), s1 = min(a.num_seqs, s0 + per);
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
      const Seq Q = load_seq(a, s);
      if (Q.bad && blockIdx.x == 0) atomicExch(status, kDevInvalidArg);
      if (Q.n > 0) mine += row_units(a, Q) * a.Hkv * key_tiles(Q);
      sh.pre[s + 1] = mine;
    }
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) sh.warp_sum[warp] = run;
    __syncthreads();
    int base = run - mine;
    for (int w = 0; w < warp; ++w) base += sh.warp_sum[w];
    for (int s = s0; s < s1; ++s) sh.pre[s + 1] += base;
    if (threadIdx.x == 0) sh.pre[0] = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = sh.tmem_base;
  const int total = sh.pre[a.num_seqs];
  const int W = min((int)gridDim.x, total);
  const int cta = blockIdx.x;
  const int xb = cta < W ? (int)((long long)cta * total / W) : 0;
  const int xe = cta < W ? (int)((long long)(cta + 1) * total / W) : 0;
  int s_first = 0;   // the sequence that holds position xb
  if (xb < xe) {
    int hi = a.num_seqs;   // pre[s_first] <= xb < pre[hi]
    while (hi - s_first > 1) {
      const int mid = (s_first + hi) >> 1;
      if (sh.pre[mid] <= xb) s_first = mid;
      else hi = mid;
    }
  }

  if (warp == 0) {
    // ------------------------------------------------------ K and V tiles
    int li = 0;                 // tiles issued
    uint32_t to_fix = 0u;       // slots whose last copy went to the fix barrier,
    uint32_t fixes = 0u;        // and the parity of the slots' copies that did
    bool ok = true, skip = a.skip_first_copy != 0;
    int s = s_first;
    for (int x = xb; x < xe && ok;) {
      Seg S;
      x = segment(a, sh.pre, x, xe, s, S);
      const int* ids = a.block_table + (size_t)S.s * a.max_blocks;
      // (lane pg: page pg of the tile, looked up a tile ahead)
      auto look_up = [&](int j) { return lane < 8 && j * kTile + lane * kPage < S.Q.L ? __ldg(ids + j * 8 + lane) : 0; };
      int id_next = look_up(S.j0);
      for (int j = S.j0; j < S.j1 && ok; ++j) {
        int id = id_next;
        if (j + 1 < S.j1) id_next = look_up(j + 1);
        const int npages = (min(kTile, S.Q.L - j * kTile) + kPage - 1) / kPage;
        if (lane < npages && (id < 0 || id >= a.num_pages)) {
          atomicExch(status, kDevBadBlockTable);
          id = 0;
        }
        const bool fix = (j + 1) * kTile > S.Q.L - S.Q.n;   // the tile holds nodes
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const int slot = li % kStages;
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_kve + 8 * slot, ((li / kStages) & 1) ^ 1, status,
                                                      abort_flag));
          if (!ok) break;
          const bool cleaned = fix && which == 1;
          const uint32_t bar = (cleaned ? bar_fix : bar_kvf) + 8 * slot;
          const uint32_t dst = ptx::smem_u32(sKV) + slot * C::kTileBytes;
          if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, npages * kPage * D * 2);
          __syncwarp();
          if (lane < npages && !skip) {
            const int row = (id * a.Hkv + S.g) * kPage;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              ptx::tma_load_2d(dst + c * 16384 + lane * 2048, which ? &tmV : &tmK, 64 * c, row, bar);
          }
          skip = false;
          to_fix = (to_fix & ~(1u << slot)) | ((cleaned ? 1u : 0u) << slot);
          if (cleaned) fixes ^= 1u << slot;
          ++li;
        }
      }
    }
    if (!ok && lane == 0)   // let the copies in flight land before shared memory is released
      for (int l = max(0, li - kStages); l < li; ++l) {
        const int slot = l % kStages;
        if (to_fix >> slot & 1u) ptx::mbar_wait(bar_fix + 8 * slot, (fixes >> slot & 1u) ^ 1u, nullptr);
        else ptx::mbar_wait(bar_kvf + 8 * slot, (l / kStages) & 1, nullptr);
      }
    __syncwarp();
  } else if (warp == 1 && lane == 0) {
    // -------------------------------------------------------- MMA issuer
    const uint64_t qdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sQ), 16, 1024);
    const uint64_t kdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16, 1024);
    const uint64_t vdesc0 = ptx::smem_desc_sw128(ptx::smem_u32(sKV), 16384, 1024);
    int lc = 0;                    // tiles consumed
    int nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};
    int half = 0;                  // Q buffer of the next one-tile unit
    bool ok = true;
    auto issue_s = [&](int w, int qb, int l) {   // S_w = Q K(l)^T
      const int slot = l % kStages;
      const uint64_t qd = qdesc0 + (uint64_t)(qb * (C::kTileBytes >> 4));
      const uint64_t kd = kdesc0 + (uint64_t)(slot * (C::kTileBytes >> 4));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
        ptx::mma_ss(tbase + w * kTile, qd + off, kd + off, C::kIdescS, k > 0);
      }
      ptx::tc_commit(bar_s + 8 * w);
    };
    auto wait_kv = [&](int l) {
      return ptx::mbar_wait(bar_kvf + 8 * (l % kStages), (l / kStages) & 1, status, abort_flag);
    };
    auto free_kv = [&](int l) { ptx::tc_commit(bar_kve + 8 * (l % kStages)); };
    auto issue_pv = [&](int w, int l, bool first) {   // O_w (+)= P_w V(l)
      if (first && !ptx::mbar_wait(bar_oe + 8 * w, (no[w] & 1) ^ 1, status, abort_flag)) return false;
      if (!ptx::mbar_wait(bar_p + 8 * w, np[w] & 1, status, abort_flag)) return false;
      ++np[w];
      ptx::tc_fence_after();
      const uint64_t vd = vdesc0 + (uint64_t)((l % kStages) * (C::kTileBytes >> 4));
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        ptx::mma_ts(tbase + 256 + w * 128, tbase + w * kTile + k * 8, vd + (uint64_t)(k * 128), C::kIdescO,
                    (!first || k > 0) ? 1u : 0u);
      return true;
    };
    int s = s_first;
    for (int x = xb; x < xe && ok;) {
      Seg S;
      x = segment(a, sh.pre, x, xe, s, S);
      const int nt = S.j1 - S.j0;
      if (S.pair) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ok = ok && ptx::mbar_wait(bar_q + 8 * i, nq[i] & 1, status, abort_flag);
          ++nq[i];
        }
        ok = ok && wait_kv(lc);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          issue_s(i, i, lc);
          if (nt == 1) ptx::tc_commit(bar_qe + 8 * i);
        }
        free_kv(lc);
        for (int j = 0; j < nt; ++j) {
          const bool next = j + 1 < nt;
          ok = wait_kv(lc + 2 * j + 1) && (!next || wait_kv(lc + 2 * j + 2));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ok = ok && issue_pv(i, lc + 2 * j + 1, j == 0);
            if (!ok) break;
            if (!next) ptx::tc_commit(bar_o + 8 * i);
            if (next) {
              issue_s(i, i, lc + 2 * j + 2);
              if (j + 2 == nt) ptx::tc_commit(bar_qe + 8 * i);
            }
          }
          if (!ok) break;
          free_kv(lc + 2 * j + 1);
          if (next) free_kv(lc + 2 * j + 2);
        }
        ++no[0];
        ++no[1];
      } else {
        const int qb = half;
        half ^= 1;
        ok = qb == 0 ? ptx::mbar_wait(bar_q, nq[0] & 1, status, abort_flag)
                     : ptx::mbar_wait(bar_q + 8, nq[1] & 1, status, abort_flag);
        if (qb == 0) ++nq[0];
        else ++nq[1];
        // S of tile j goes to warpgroup j mod 2
        auto score = [&](int w, int j) {
          issue_s(w, qb, lc + 2 * j);
          if (j == nt - 1) ptx::tc_commit(bar_qe + 8 * qb);
          free_kv(lc + 2 * j);
        };
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (ok && w < nt) {
            ok = wait_kv(lc + 2 * w);
            if (!ok) break;
            ptx::tc_fence_after();
            score(w, w);
          }
        for (int j0 = 0; j0 < nt && ok; j0 += 2)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int j = j0 + w;
            if (j >= nt || !ok) break;
            const bool next = j + 2 < nt;
            ok = wait_kv(lc + 2 * j + 1) && (!next || wait_kv(lc + 2 * j + 4));
            if (!ok) break;
            ptx::tc_fence_after();
            ok = issue_pv(w, lc + 2 * j + 1, j == w);
            if (!ok) break;
            if (!next) ptx::tc_commit(bar_o + 8 * w);
            free_kv(lc + 2 * j + 1);
            if (next) score(w, j + 2);
          }
        ++no[0];
        if (nt > 1) ++no[1];
      }
      lc += 2 * nt;
    }
    // no tcgen05.mma may still run when the tensor memory is released
    ptx::tc_commit(bar_drain);
    ptx::mbar_wait(bar_drain, 0, nullptr);
  } else if (warp == 2) {
    // --------------------------------------------------------- query rows
    int nq[2] = {0, 0}, half = 0;
    bool ok = true;
    int s = s_first;
    for (int x = xb; x < xe && ok;) {
      Seg S;
      x = segment(a, sh.pre, x, xe, s, S);
      const int tiles = S.pair ? 2 : 1;
      for (int i = 0; i < tiles; ++i) {
        const int qb = S.pair ? i : half;
        const int phase = qb == 0 ? nq[0] : nq[1];
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_qe + 8 * qb, (phase & 1) ^ 1, status, abort_flag));
        if (!ok) break;
        const int r0 = S.row0 + i * kTile;
        const int rows = min(kTile, S.rows - i * kTile);
        const uint32_t dst = ptx::smem_u32(sQ) + qb * C::kTileBytes;
        // (rows past the last one keep what was there: they only reach their own
        // rows of S and O, which nobody reads)
        for (int e = lane; e < rows * (D / 8); e += 32) {
          const int r = e / (D / 8), u = e % (D / 8);
          const int node = (r0 + r) / a.G, h = (r0 + r) - node * a.G;
          const __nv_bfloat16* src =
              a.q + ((size_t)(S.Q.q0 + node) * a.H + S.g * a.G + h) * D + u * 8;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           dst + (u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4)),
                       "l"(src)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(bar_q + 8 * qb);
        if (qb == 0) ++nq[0];
        else ++nq[1];
      }
      if (!S.pair) half ^= 1;
    }
  } else if (warp == 3) {
    // ------------------------------------------------- V rows nobody sees
    // Their weights are exactly 0, but they may hold anything and 0 * NaN is NaN.
    int lc = 0;
    uint32_t fixes = 0u;   // parity of each slot's copies to the fix barrier
    bool ok = true;
    int s = s_first;
    for (int x = xb; x < xe && ok;) {
      Seg S;
      x = segment(a, sh.pre, x, xe, s, S);
      const int i0 = S.row0 / a.G, i1 = (S.row0 + S.rows - 1) / a.G + 1;   // the unit's nodes
      const int fix0 = (S.Q.L - S.Q.n) / kTile;                            // first tile with nodes
      for (int j = max(S.j0, fix0); j < S.j1; ++j) {
        // lane: the union over every eighth node of 32 keys' bits
        uint32_t seen = 0u;
        for (int i = i0 + (lane >> 2); i < i1; i += 8) seen |= sees(a, S.Q, i, j * kTile + 32 * (lane & 3));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, o);
        const int slot = (lc + 2 * (j - S.j0) + 1) % kStages;
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
                *reinterpret_cast<uint4*>(tile + h * 16384 + (32 * c + row) * 128 + (lane & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_kvf + 8 * slot);
      }
      lc += 2 * (S.j1 - S.j0);
    }
  } else if (warp >= 4) {
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
    int s = s_first;
    if (threadIdx.x == 128 && cta < (int)gridDim.x) {
      // what the merge finds of this CTA: the unit that begins here and is cut
      Cut cut{0, 0, 0, 0, -1, 0, {0, 0}};
      if (xb < xe) {
        int se = s_first;
        Seg S;
        while (sh.pre[se + 1] <= xe - 1) ++se;
        segment(a, sh.pre, xe - 1, xe, se, S);
        const int u0 = xe - 1 - S.j0, u1 = u0 + S.nt;   // the unit of the piece's last tile
        if (u0 >= xb && u1 > xe)
          cut = Cut{S.s, S.row0, S.rows, S.g, (int)(((long long)u1 * W - 1) / total), u0 > xb, {0, 0}};
      }
      a.cuts[cta] = cut;
    }
    for (int x = xb; x < xe && ok;) {
      Seg S;
      const int seg_x = x;
      x = segment(a, sh.pre, x, xe, s, S);
      const int nt = S.j1 - S.j0;
      const int row = S.pair ? w * kTile + r : r;          // of the unit
      const bool valid = row < S.rows;
      const int node = (S.row0 + row) / a.G;
      // a warp without a valid row leaves P as it is: it reaches only its own rows
      const bool any = (S.pair ? w * kTile : 0) + quarter * 32 < S.rows;
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
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar_s + 8 * w, ns & 1, status, abort_flag));
        if (!ok) break;
        ++ns;
        ptx::tc_fence_after();
        if (any) {
          float mx = -INFINITY;
          if (!masked) {
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              uint32_t x0[32], x1[32];
              float m0, m1;
              ptx::tmem_ld32_max(s_col + c * 32, x0, m0);
              ptx::tmem_ld32_max(s_col + c * 32 + 32, x1, m1);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)   // (the registers stay theirs until the loads are done)
                asm volatile("" ::"r"(x0[e]), "r"(x1[e]));
              mx = ptx::fmax3(mx, m0, m1);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x32[32];
              ptx::tmem_ld32(s_col + c * 32, x32);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                mx = fmaxf(mx, vis[c] >> e & 1u ? __uint_as_float(x32[e]) : -INFINITY);
            }
          }
          const float m_tile = mx * a.scale_log2;   // scale > 0: the maximum commutes with it
          const bool raise = valid && (m_tile > m_ref + kRaise || (m_ref == -INFINITY && m_tile > -INFINITY));
          float alpha = 1.f;
          if (raise) {
            alpha = m_ref == -INFINITY ? 1.f : ptx::ex2(m_ref - m_tile);
            m_ref = m_tile;
            l_run *= alpha;
            l_p *= alpha;
          }
          // (S of this tile is complete, so every earlier P V is: they were issued
          // before it)
          if (__any_sync(0xffffffffu, raise && jl > jw && alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              ptx::tmem_ld32(o_col + c * 32, ov);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              ptx::tmem_st32(o_col + c * 32, ov);
            }
          }
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t nref2 = ptx::f2_bits(-ref, -ref);
          // P (bf16 pairs) overwrites S from its first column on: chunk c goes to
          // columns 16 c .. 16 c + 15, which belong to scores read before
          uint32_t sr[2][32];
          ptx::tmem_ld32(s_col, sr[0]);
          uint64_t sum2 = ptx::f2_bits(0.f, 0.f), sum2b = sum2;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ptx::tmem_wait_ld();
            if (c < 3) ptx::tmem_ld32(s_col + (c + 1) * 32, sr[(c + 1) & 1]);
            uint32_t pr[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float s0 = __uint_as_float(sr[c & 1][e]), s1 = __uint_as_float(sr[c & 1][e + 1]);
              if (masked) {
                s0 = vis[c] >> e & 1u ? s0 : -INFINITY;
                s1 = vis[c] >> (e + 1) & 1u ? s1 : -INFINITY;
              }
              float x0, x1;
              ptx::f2_split(ptx::ffma2(ptx::f2_bits(s0, s1), sc2, nref2), x0, x1);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              if (e & 2) sum2b = ptx::fadd2(sum2b, ptx::f2_bits(p0, p1));
              else sum2 = ptx::fadd2(sum2, ptx::f2_bits(p0, p1));
              pr[e / 2] = ptx::pack_bf16x2(p0, p1);
            }
            ptx::tmem_st16(s_col + c * 16, pr);
            l_p += sum_packed(pr);
          }
          float a0, a1;
          ptx::f2_split(ptx::fadd2(sum2, sum2b), a0, a1);
          l_run += a0 + a1;
          ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar_p + 8 * w);
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
      if (two)
        there = there && ptx::mbar_wait(bar_o + 8, ph1, status, abort_flag) &&
                ptx::mbar_wait(bar_sf, phs, status, abort_flag);
      ok = __all_sync(0xffffffffu, there);
      if (!ok) break;
      ptx::tc_fence_after();
      if (two) {
        const float m1 = sh.stat[r][0], l1 = sh.stat[r][1], lp1 = sh.stat[r][2];
        ptx::mbar_arrive(bar_se);
        m = fmaxf(m_ref, m1);
        c0 = m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - m);
        c1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - m);
        l_run = c0 * l_run + c1 * l1;
        l_p = c0 * l_p + c1 * lp1;
      }
      const bool whole = S.j0 == 0 && S.j1 == S.nt;
      const size_t tok = (size_t)(S.Q.q0 + node);
      const int head = S.g * a.G + (S.row0 + row) - node * a.G;
      const size_t orow = tok * a.H + head;
      const size_t slot = 2 * (size_t)cta + (seg_x > xb ? 1 : 0);
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
// M) l_p_x, the LSE from the exact sums.  Block (cta, 32 rows): the unit that
// begins in CTA `cta`'s piece; lane = row, warp = every eighth float4 of O.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
tree_merge_kernel(const Args a) {
  constexpr int kEach = D / 4 / kMergeWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.y * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 c0 = __ldcg(reinterpret_cast<const int4*>(a.cuts + blockIdx.x));
  const int2 c1 = __ldcg(reinterpret_cast<const int2*>(a.cuts + blockIdx.x) + 2);
  const int seq = c0.x, row0 = c0.y, rows = c0.z, g = c0.w, last = c1.x, late = c1.y;
  if (last < 0 || row >= rows) return;
  const int first = blockIdx.x;
  const int q0 = __ldg(a.cu_q + seq);
  auto slot_of = [&](int x) { return (size_t)(2 * x + (x == first ? late : 0)); };
  float M = -INFINITY;
#pragma unroll 4
  for (int x = first; x <= last; ++x) M = fmaxf(M, __ldcg(a.part_s + slot_of(x) * a.row_cap + row).x);
  float l = 0.f, lp = 0.f;
  float4 y[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int x = first; x <= last; ++x) {
    const float4 st = __ldcg(a.part_s + slot_of(x) * a.row_cap + row);
    const float f = st.x == -INFINITY ? 0.f : ptx::ex2(st.x - M);
    l += f * st.y;
    lp += f * st.z;
    const float4* po = a.part_o + (slot_of(x) * (D / 4) + warp * kEach) * a.row_cap + row;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float4 v = __ldcg(po + (size_t)i * a.row_cap);
      y[i].x = fmaf(f, v.x, y[i].x);
      y[i].y = fmaf(f, v.y, y[i].y);
      y[i].z = fmaf(f, v.z, y[i].z);
      y[i].w = fmaf(f, v.w, y[i].w);
    }
  }
  const float inv = lp > 0.f ? 1.f / lp : (lp == 0.f ? 0.f : lp);
  const int node = (row0 + row) / a.G;
  const int head = g * a.G + row0 + row - node * a.G;
  const size_t tok = (size_t)(q0 + node), orow = tok * a.H + head;
  if (!FA_IN_BOUNDS(orow, (size_t)a.total_q * a.H, a.status)) return;
  uint2* dst = reinterpret_cast<uint2*>(a.o + orow * D) + warp * kEach;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    dst[i] = make_uint2(ptx::pack_bf16x2(y[i].x * inv, y[i].y * inv),
                        ptx::pack_bf16x2(y[i].z * inv, y[i].w * inv));
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

template <int D>
cudaError_t launch(const TreeAttnParams& p, cudaStream_t stream, const char** why) {
  using C = Cfg<D>;
  CUtensorMap tmK, tmV;
  // (dim, cache row); one box = 64 values of one page of one kv head
  const uint64_t dims[2] = {(uint64_t)D, (uint64_t)p.num_pages * p.Hkv * kPage};
  const uint64_t strides[1] = {(uint64_t)D * 2};
  const uint32_t box[2] = {64, (uint32_t)kPage};
  if (!make_tmap_bf16(&tmK, p.k_cache, 2, dims, strides, box) ||
      !make_tmap_bf16(&tmV, p.v_cache, 2, dims, strides, box)) {
    *why = "tensor map for the caches";
    return cudaErrorInvalidValue;
  }
  const int G = p.H / p.Hkv;
  Args a{static_cast<const __nv_bfloat16*>(p.q), p.block_table, p.seq_lens, p.cu_q, p.mask,
         static_cast<__nv_bfloat16*>(p.o), p.lse, p.num_seqs, p.total_q, p.max_q, p.words, p.H, p.Hkv, G,
         p.num_pages, p.max_blocks, p.scale * kLog2e, skip_first_copy_for_tests(), p.status,
         nullptr, nullptr, nullptr, row_cap(p.max_q, G)};
  char* ws = static_cast<char*>(p.workspace);
  a.cuts = reinterpret_cast<Cut*>(ws);
  a.part_s = reinterpret_cast<float4*>(ws + kCutBytes);
  a.part_o = a.part_s + (size_t)2 * kCtas * a.row_cap;
  auto kernel = tree_attn_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e == cudaSuccess) {
    kernel<<<kCtas, kThreads, C::kSmem, stream>>>(tmK, tmV, a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *why = "tree_attn launch";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(kCtas, (unsigned)(a.row_cap / 32));
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
  return p.d == 128 ? launch<128>(p, stream, why) : launch<64>(p, stream, why);
}

}  // namespace fa
