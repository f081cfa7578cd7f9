// Internal launch interface between the C ABI layer (api.cu) and the kernel
// translation units.  Host-side only; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

namespace fa {

// Id of the CUDA context current on the calling thread (the runtime's primary
// context of the current device, unless the caller made another current).
// Device addresses of the library's __device__ variables belong to one
// context: cudaDeviceReset or another context gives the same variable another
// address, so a cached address is keyed by this id.  False when no live
// context is current.  The driver calls are fetched through the runtime, so
// the library does not link libcuda directly.
inline bool current_context_id(unsigned long long* id) {
  typedef CUresult (*GetCurrentFn)(CUcontext*);
  typedef CUresult (*GetIdFn)(CUcontext, unsigned long long*);
  struct Fns {
    GetCurrentFn get_current = nullptr;
    GetIdFn get_id = nullptr;
  };
  static const Fns fns = [] {   // looked up once, thread-safely
    Fns f;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      f.get_current = reinterpret_cast<GetCurrentFn>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      f.get_id = reinterpret_cast<GetIdFn>(p);
    return f;
  }();
  if (fns.get_current == nullptr || fns.get_id == nullptr) return false;
  CUcontext ctx = nullptr;
  if (fns.get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return false;
  return fns.get_id(ctx, id) == CUDA_SUCCESS;
}

// Device status codes written by kernels (same values as fa_status).
enum : int {
  kDevOk = 0,
  kDevInvalidArg = 1,
  kDevTimeout = 5,
  kDevBadBlockTable = 6,
  kDevDebugCheck = 7
};

// Debug builds (-DFA_DEBUG: libfa_gb300_debug.so) check each global store's
// index against the size of the buffer the kernel was given; a failed check
// records kDevDebugCheck in the status word and the store is skipped instead
// of landing outside the buffer.  In the normal build the check is the
// constant true and neither operand is evaluated.
#ifdef FA_DEBUG
#define FA_IN_BOUNDS(idx, limit, status)                     \
  (((size_t)(idx) < (size_t)(limit)) ? true                  \
                                     : (atomicExch((status), kDevDebugCheck), false))
#else
#define FA_IN_BOUNDS(idx, limit, status) true
#endif

// Failure-detection test hook of the forward and the e4m3 rows kernels, as the
// bf16 decode's: with FA_TEST_FORCE_WAIT_TIMEOUT=1 in the environment every warp
// that copies K and V skips its first tile or page, the bounded waits for it
// expire (after about 1 s) and FA_ERR_TIMEOUT is recorded.  Unset in normal use.
inline int skip_first_copy_for_tests() {
  const char* v = getenv("FA_TEST_FORCE_WAIT_TIMEOUT");
  return (v != nullptr && v[0] == '1') ? 1 : 0;
}

// Forward problem.  Dense BSHD when cu_q == nullptr; otherwise packed varlen
// (B = number of sequences, n/m = max lengths, token rows start at cu_q[b]).
struct FwdParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;          // may be null
  const int* cu_q;     // varlen only (device)
  const int* cu_k;     // varlen only (device)
  int B, H, Hkv, n, m, d, dv;
  int total_q, total_k;  // varlen: rows of the packed q/k tensors (0 if unknown)
  float scale;
  int causal;
  int* status;         // device status word
  // paged prefill (block_table != nullptr): k, v are caches [pages][Hkv][16][d],
  // seq_lens[b] keys per sequence, q packed by cu_q as for varlen
  const int* block_table = nullptr;
  const int* seq_lens = nullptr;
  int max_blocks = 0;
  int num_pages = 0;
  // e4m3 operands (q, k, v hold x / descale), bf16 output
  int fp8 = 0;
  float q_descale = 1.f, k_descale = 1.f, v_descale = 1.f;
  // sliding window (0: none; causal only) and sinks; e4m3 page caches' scale bytes
  int window = 0, sinks = 0;
  const void* k_scale = nullptr;
  const void* v_scale = nullptr;
  void* workspace = nullptr;   // e4m3 caches: parts of cut units (cache_parts_bytes), or null
};

// Heads that share a kv head and are rows of one query tile: the largest power
// of two that divides the group, at most 128 (its log2).
inline int packed_heads_log2(int H, int Hkv) {
  int gl = 0;
  while (gl < 7 && (H / Hkv) % (2 << gl) == 0) ++gl;
  return gl;
}

// Work units of a launch that packs heads: (sequence, head group, pair of query
// tiles).  The kernels number them in 32 bits.
inline long long packed_units(int num_seqs, int max_q, int H, int Hkv) {
  const int gl = packed_heads_log2(H, Hkv);
  const long long pair_q = 256 >> gl;
  return (long long)num_seqs * (H >> gl) * ((max_q + pair_q - 1) / pair_q);
}

// Parts that each unit of a chunk
// launch over the e4m3 cache is cut into: as many as fill the SMs where units
// are few, twice as many for several sequences (whose lengths may differ), and
// 1 from 152 units on.
inline int cache_parts(int num_seqs, int max_q, int H, int Hkv) {
  const long long units = packed_units(num_seqs, max_q, H, Hkv);
  if (units <= 0 || units > 152) return 1;
  return (int)((num_seqs == 1 ? 152 : 304) / units);
}
inline size_t cache_parts_bytes(int num_seqs, int max_q, int H, int Hkv, int d) {
  const int parts = cache_parts(num_seqs, max_q, H, Hkv);
  if (parts <= 1) return 0;
  return (size_t)packed_units(num_seqs, max_q, H, Hkv) * parts * 256 * (d + 4) * 4;
}

// The parts of a launch: no more than one per two K/V tiles (of 128 keys) that a
// unit can have.
inline int cache_parts_taken(int num_seqs, int max_q, int H, int Hkv, int max_blocks, int causal,
                             int window, int sinks) {
  long long keys = max_blocks * 16ll;
  if (causal && window > 0) {
    const long long seen = (long long)window + (256 >> packed_heads_log2(H, Hkv)) + sinks + 256;
    if (seen < keys) keys = seen;
  }
  const long long most = keys / 256, parts = cache_parts(num_seqs, max_q, H, Hkv);
  return (int)(most < 1 ? 1 : parts < most ? parts : most);
}

struct DecodeParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int* block_table;
  const int* seq_lens;
  int num_seqs, H, Hkv, d, dv, page_size, num_pages, max_blocks, num_splits;
  float scale;
  float* part_m;       // [S][H][X]
  float* part_l;       // [S][H][X]
  float* part_o;       // [S][H][X][dv]
  int* status;
  // fused form only: per (sequence, kv head) ticket counters, zero between
  // calls, and the outputs the merging split writes
  int* tickets = nullptr;
  void* o = nullptr;   // bf16 [S][H][dv]
  float* lse = nullptr;
};

struct CombineParams {
  const float* part_m;
  const float* part_l;
  const float* part_o;
  void* o;             // bf16 [S][H][dv]
  float* lse;          // [S][H], may be null
  int num_seqs, H, num_splits, dv;
};

struct GatherParams {
  const void* k_cache;
  const void* v_cache;
  const int* block_table;
  const int* seq_lens;
  void* k_out;         // bf16 [S][max_blocks * 16][Hkv][128]
  void* v_out;
  int num_seqs, Hkv, num_pages, max_blocks, num_splits;
  int* status;
};

// Rows written to, or read back from, the e4m3 paged cache.
struct KvRowsParams {
  const void* k;             // bf16 rows [total][Hkv][d] (written by the read-back)
  const void* v;
  long long k_stride, v_stride;  // write: elements from one token to the next
  void* k_cache;             // e4m3 [pages][Hkv][16][d]
  void* v_cache;
  void* k_scale;             // scale bytes [pages][Hkv][16]
  void* v_scale;
  const int* block_table;
  const int* seq_lens;
  const int* cu;
  int num_seqs, total, Hkv, d, num_pages, max_blocks;
  int* status;
};

// Attention of a few query rows per sequence over the e4m3 paged cache.
struct PagedE4m3Params {
  const void* q;             // bf16 [total_q][H][d]
  const void* k_cache;
  const void* v_cache;
  const void* k_scale;
  const void* v_scale;
  const int* block_table;
  const int* seq_lens;
  const int* cu_q;           // null: one query token per sequence
  void* o;                   // bf16 [total_q][H][d]
  float* lse;                // decode [S][H], chunk [H][total_q]; may be null
  int num_seqs, total_q, max_q, H, Hkv, d, num_pages, max_blocks;
  float scale;
  int causal, window, sinks; // window 0: none
  int* status;
  void* workspace = nullptr; // stream form's partials (rows_e4m3_workspace bytes), or null
};

cudaError_t launch_kv_write_e4m3(const KvRowsParams& p, cudaStream_t stream);
cudaError_t launch_kv_read_e4m3(const KvRowsParams& p, cudaStream_t stream);
// Query rows (tokens x grouped heads) of one kv head that the rows kernels can take.
constexpr int kRowsE4m3Max = 32;
// Whether a call takes the rows kernels: decode always, chunks of up to 16 rows
// a kv head, and of up to 32 except at d = 128 where the forward packs all heads
// of a group into one tile (a power of two of them; otherwise it reads K and V
// once more for each part of the group).  us of the rows kernels and of the
// forward, d = 128, 8 kv heads of 4, [512, 8192] tokens: 64 x 4 new tokens 147,
// 229; 64 x 8 253, 229; 16 x 8 89, 88; 1 x 8192 with 8 26, 27; 64 x 8 with
// groups of 3 253, 643; d = 64, 64 x 8 131, 209.
inline bool rows_e4m3_form(int max_q, int H, int Hkv, int d) {
  const int g = H / Hkv;
  const long long rows = (long long)max_q * g;
  if (max_q == 1 || rows <= 16) return true;
  return rows <= kRowsE4m3Max && (d == 64 || (g & (g - 1)) != 0);
}
// Bytes for any table width and window of these sizes, and whether the rows
// kernels use them for the given ones.
size_t rows_e4m3_workspace(int num_seqs, int max_q, int H, int Hkv, int d);
bool rows_e4m3_few_units(int num_seqs, int Hkv);   // false: never used, whatever the other sizes
bool rows_e4m3_uses_workspace(int num_seqs, int max_q, int H, int Hkv, int d, int max_blocks,
                              int causal, int window, int sinks);
cudaError_t launch_rows_e4m3(const PagedE4m3Params& p, cudaStream_t stream, const char** why);
cudaError_t launch_fwd_f32(const FwdParams& p, cudaStream_t stream);
cudaError_t launch_fwd_bf16(const FwdParams& p, cudaStream_t stream, const char** why);
cudaError_t launch_fwd_window(const FwdParams& p, cudaStream_t stream, const char** why);
cudaError_t launch_fwd_e4m3_cache(const FwdParams& p, cudaStream_t stream, const char** why);
// fused: partials and merge in one launch (p.tickets, p.o, p.lse set)
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream, bool fused);
cudaError_t launch_decode_partials(const DecodeParams& p, cudaStream_t stream);
// behind_partials: launched right after launch_decode_partials on the same
// stream, as a programmatic dependent of it
cudaError_t launch_split_combine(const CombineParams& p, cudaStream_t stream,
                                 bool behind_partials = false);
cudaError_t launch_decode_gather(const GatherParams& p, cudaStream_t stream);

}  // namespace fa
