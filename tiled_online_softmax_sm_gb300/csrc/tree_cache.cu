// The small kernels around drafted token trees: the trees' ancestor bits and
// positions, the accepted path's rows moved behind the context, and page copies.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"
#include "paged_rows.cuh"

namespace fa {
namespace {

// ------------------------------------------------------------------ layout
// mask[i] = {i} and i's ancestors, positions[i] = seq_lens - n + depth.  One block
// per sequence; a thread makes one word of one node's row by following the parents
// from the node, which are in shared memory, down to the word's first node (a
// parent lies before its child), so no thread stores a row it would have to read
// again.  Word 0 walks to the context and counts the depth.
// Bound by latency: the offsets, the parents, and then the words that a thread makes,
// each a walk down its node's path, one after the other.  With a parent drawn from all
// earlier nodes, whose paths are short: 8 sequences of 24 nodes 1.8 us, 64 of 256 4.0, 64 of
// 1024 34 (the bytes take 0.1, 0.1 and 1.3).  Deep trees take time by words * depth, however
// few they are: one chain of 64 nodes 3.3 us, of 256 20, of 1024 938.
constexpr int kLayoutThreads = 512;
constexpr int kMaxNodes = 32 * 32;

__global__ void __launch_bounds__(kLayoutThreads)
tree_layout_kernel(const int* __restrict__ parents, const int* __restrict__ seq_lens,
                   const int* __restrict__ cu, int* __restrict__ mask, int* __restrict__ positions,
                   int total, int words, int* status) {
  __shared__ int up[kMaxNodes];
  const int s = blockIdx.x;
  const int q0 = __ldg(cu + s), n = __ldg(cu + s + 1) - q0, L = __ldg(seq_lens + s);
  if (q0 < 0 || n < 0 || (long long)q0 + n > total || L < n || n > 32 * words) {
    if (threadIdx.x == 0) atomicExch(status, kDevInvalidArg);
    return;
  }
  for (int t = threadIdx.x; t < n; t += kLayoutThreads) {
    int p = __ldg(parents + q0 + t);
    if (p < -1 || p >= t) {
      atomicExch(status, kDevInvalidArg);
      p = -1;
    }
    up[t] = p;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < n * words; x += kLayoutThreads) {
    const int i = x / words, w = x - i * words;
    uint32_t bits = 0u;
    int steps = 0;
    for (int t = i; t >= 32 * w; t = up[t]) {
      if (t < 32 * w + 32) bits |= 1u << (t & 31);
      ++steps;
    }
    const size_t at = (size_t)(q0 + i) * words + w;
    if (FA_IN_BOUNDS(at, (size_t)total * words, status)) mask[at] = (int)bits;
    if (w == 0 && positions != nullptr && FA_IN_BOUNDS(q0 + i, total, status))
      positions[q0 + i] = L - n + steps - 1;
  }
}

// ------------------------------------------------------------------ accept
// Row path[a] of the drafted tail moves to slot a.  The path increases, so a <=
// path[a], and slot a is the source of no later entry: b > a reads path[b] >= b.
// A thread owns 16 bytes of every row of a kv head and moves them in the path's
// order, eight entries at a time, loads before stores: the eight loads then come
// before every store that could reach them.  So rows move in place without a
// barrier.  The scale bytes (e4m3) have threads of their own.
// One block per (sequence, layer, 256 such columns); bound by latency: offsets,
// path, block table, rows (16 sequences 3.1 us, 64 with 8 layers 4.7 us, 2.5 of it
// bytes).
constexpr int kAcceptThreads = 256;
constexpr int kBatch = 8;

template <typename T>
__device__ __forceinline__ void move_rows(T* base, size_t stride, const int* from, const int* to,
                                          int count, size_t limit, int* status) {
  for (int a = 0; a < count; a += kBatch) {
    T x[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (a + e < count) x[e] = base[(size_t)from[a + e] * stride];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (a + e < count && FA_IN_BOUNDS(to[a + e], limit, status)) base[(size_t)to[a + e] * stride] = x[e];
  }
}

__global__ void __launch_bounds__(kAcceptThreads)
kv_accept_kernel(const KvAcceptParams p) {
  __shared__ int s_from[kMaxPath], s_to[kMaxPath];   // cache rows of kv head 0
  __shared__ int s_count[kAcceptThreads / 32 + 1];
  const int s = blockIdx.x / p.c.num_layers, layer = blockIdx.x - s * p.c.num_layers;
  const bool first_block = layer == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  const int q0 = __ldg(p.cu + s), n = __ldg(p.cu + s + 1) - q0, L = __ldg(p.seq_lens + s);
  const int k = __ldg(p.path_lens + s);
  const int* path = p.path + (size_t)s * p.max_path;
  bool good = q0 >= 0 && n >= 0 && (long long)q0 + n <= p.total && L >= n &&
              (long long)L <= (long long)p.max_blocks * kPage && k >= 0 && k <= p.max_path && k <= n;
  if (good)
    for (int a = threadIdx.x; a < k; a += kAcceptThreads) {
      const int t = __ldg(path + a);
      const int before = a > 0 ? __ldg(path + a - 1) : -1;
      if (t <= before || t >= n || before < -1) good = false;
    }
  good = !__syncthreads_or(!good);
  if (first_block) {
    if (!good) atomicExch(p.c.status, kDevInvalidArg);
    if (FA_IN_BOUNDS(s, p.num_seqs, p.c.status)) p.new_seq_lens[s] = good ? L - n + k : L;
  }
  if (!good) return;
  // the entries that move, in order (those in place already are skipped)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int a0 = 0; a0 < k; a0 += kAcceptThreads) {
    const int a = a0 + threadIdx.x;
    int from = 0, to = 0;
    bool moves = false;
    if (a < k) {
      const int t = __ldg(path + a);
      const int src = L - n + t, dst = L - n + a;
      const int* row = p.block_table + (size_t)s * p.max_blocks;
      const int ps = __ldg(row + src / kPage), pd = __ldg(row + dst / kPage);
      moves = t != a;
      if (moves && (ps < 0 || ps >= p.c.num_pages || pd < 0 || pd >= p.c.num_pages)) {
        atomicExch(p.c.status, kDevBadBlockTable);
        moves = false;
      }
      from = ps * p.c.Hkv * kPage + src % kPage;
      to = pd * p.c.Hkv * kPage + dst % kPage;
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, moves);
    if (lane == 0) s_count[warp] = __popc(vote);
    __syncthreads();
    int at = base + __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < kAcceptThreads / 32; ++w) {
      if (w < warp) at += s_count[w];
      base += s_count[w];
    }
    if (moves) {
      s_from[at] = from;
      s_to[at] = to;
    }
    __syncthreads();
  }
  const int units = p.c.row_bytes / 16;             // 16-byte columns of a row
  const int cols = p.c.Hkv * units;                 // of K, then as many of V
  const size_t rows = (size_t)p.c.num_pages * p.c.Hkv * kPage;
  const size_t limit = rows;
  for (int c = blockIdx.y * kAcceptThreads + threadIdx.x; c < 2 * cols + (p.c.k_scale ? 2 * p.c.Hkv : 0);
       c += gridDim.y * kAcceptThreads) {
    if (c < 2 * cols) {
      const int h = c % cols / units, u = c % units;
      uint4* cache = static_cast<uint4*>(c < cols ? p.c.k_cache : p.c.v_cache);
      move_rows(cache + ((size_t)layer * rows + h * kPage) * units + u, (size_t)units, s_from, s_to, base,
                limit - h * kPage, p.c.status);
    } else {
      const int h = (c - 2 * cols) % p.c.Hkv;
      uint8_t* scale = static_cast<uint8_t*>(c - 2 * cols < p.c.Hkv ? p.c.k_scale : p.c.v_scale);
      move_rows(scale + (size_t)layer * rows + h * kPage, (size_t)1, s_from, s_to, base, limit - h * kPage,
                p.c.status);
    }
  }
}

// -------------------------------------------------------------- page copies
// A page of a layer is Hkv * 16 * row_bytes contiguous bytes of K, as many of V,
// and Hkv * 16 scale bytes of each (e4m3).  One block per (pair, layer, kChunk
// bytes of K or of V); bound by HBM (512 pages, 8 layers, e4m3, 271 MB read and written:
// 42.5 us, 6.4 TB/s; 8 pages of one layer 2.1 us, launch and latency).
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;
constexpr int kChunk = kCopyThreads * kCopyLoads;   // 16-byte units

__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const KvMoveParams c, const int* __restrict__ pairs, int chunks) {
  const int part = blockIdx.x % (2 * chunks), item = blockIdx.x / (2 * chunks);
  const int pair = item / c.num_layers, layer = item - pair * c.num_layers;
  const int src = __ldg(pairs + 2 * (size_t)pair), dst = __ldg(pairs + 2 * (size_t)pair + 1);
  if (src < 0 || src >= c.num_pages || dst < 0 || dst >= c.num_pages) {
    if (threadIdx.x == 0) atomicExch(c.status, kDevBadBlockTable);
    return;
  }
  const int units = c.Hkv * c.row_bytes;            // 16-byte units of a page: 16 rows a head
  const size_t page0 = (size_t)layer * c.num_pages;
  uint4* cache = static_cast<uint4*>(part < chunks ? c.k_cache : c.v_cache);
  const uint4* from = cache + (page0 + src) * units;
  uint4* to = cache + (page0 + dst) * units;
  const int first = part % chunks * kChunk + threadIdx.x;
  uint4 x[kCopyLoads];
#pragma unroll
  for (int e = 0; e < kCopyLoads; ++e)
    if (first + e * kCopyThreads < units) x[e] = from[first + e * kCopyThreads];
#pragma unroll
  for (int e = 0; e < kCopyLoads; ++e)
    if (first + e * kCopyThreads < units && FA_IN_BOUNDS(dst, c.num_pages, c.status))
      to[first + e * kCopyThreads] = x[e];
  if (c.k_scale != nullptr && part % chunks == 0) {
    uint4* scale = static_cast<uint4*>(part < chunks ? c.k_scale : c.v_scale);
    for (int u = threadIdx.x; u < c.Hkv; u += kCopyThreads)
      if (FA_IN_BOUNDS(dst, c.num_pages, c.status))
        scale[(page0 + dst) * c.Hkv + u] = scale[(page0 + src) * c.Hkv + u];
  }
}

}  // namespace

cudaError_t launch_tree_layout(const TreeLayoutParams& p, cudaStream_t stream) {
  tree_layout_kernel<<<p.num_seqs, kLayoutThreads, 0, stream>>>(
      p.parents, p.seq_lens, p.cu, p.mask, p.positions, p.total, p.words, p.status);
  return cudaGetLastError();
}

cudaError_t launch_kv_accept(const KvAcceptParams& p, cudaStream_t stream) {
  const long long cols = 2ll * p.c.Hkv * (p.c.row_bytes / 16) + (p.c.k_scale ? 2 * p.c.Hkv : 0);
  const long long y = (cols + kAcceptThreads - 1) / kAcceptThreads;
  kv_accept_kernel<<<dim3((unsigned)(p.num_seqs * p.c.num_layers), (unsigned)(y < 1024 ? y : 1024)),
                     kAcceptThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const KvMoveParams& c, const int* pairs, int num_pairs,
                              cudaStream_t stream) {
  const int chunks = (c.Hkv * c.row_bytes + kChunk - 1) / kChunk;
  const long long blocks = 2ll * chunks * num_pairs * c.num_layers;
  copy_pages_kernel<<<(unsigned)blocks, kCopyThreads, 0, stream>>>(c, pairs, chunks);
  return cudaGetLastError();
}

}  // namespace fa
