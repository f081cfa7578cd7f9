// C ABI entries of drafted token trees over a paged cache: argument validation
// and workspace carving.  The kernels are in tree_attn.cu, tree_cache.cu and
// qkv_rows.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
fa_status api_fail(fa_status st, const char* msg);
fa_status api_status_ptr(int** out);
}  // namespace fa

namespace {

constexpr long long kInt = 0x7fffffffLL;

fa_status fail(fa_status st, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return fa::api_fail(st, msg);
}

fa_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FA_OK;
  return fail(FA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

fa_status check_dims(const char* fn, int d, int page_size) {
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "%s: d=%d (supported: 64, 128)", fn, d);
  if (page_size != 16) return fail(FA_ERR_UNSUPPORTED, "%s: page_size=%d (supported: 16)", fn, page_size);
  return FA_OK;
}

// The caches, their scales (both or none) and the sizes that number their rows in
// 32 bits.
fa_status check_caches(const char* fn, const void* k_cache, const void* v_cache, const void* k_scale,
                       const void* v_scale, int num_layers, int Hkv, int num_pages) {
  if (k_cache == nullptr || v_cache == nullptr) return fail(FA_ERR_INVALID_ARG, "%s: null cache", fn);
  if ((k_scale == nullptr) != (v_scale == nullptr))
    return fail(FA_ERR_INVALID_ARG, "%s: one of k_scale and v_scale is null", fn);
  if (num_pages == 0) return fail(FA_ERR_INVALID_ARG, "%s: empty page pool", fn);
  if ((long long)num_pages * Hkv * 16 > kInt || num_layers > 65535 || Hkv > 65536)
    return fail(FA_ERR_UNSUPPORTED, "%s: page pool or layers too large", fn);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  return FA_OK;
}

fa_status check_table(const char* fn, const int* block_table, const int* seq_lens, const int* cu,
                      int max_blocks) {
  if (block_table == nullptr || seq_lens == nullptr || cu == nullptr)
    return fail(FA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (max_blocks == 0) return fail(FA_ERR_INVALID_ARG, "%s: empty block table", fn);
  if (max_blocks > 0x3ffffff) return fail(FA_ERR_UNSUPPORTED, "%s: block table too large", fn);
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu, 4))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  return FA_OK;
}

// fa_paged_tree_attention, or (scales given) fa_paged_tree_attention_e4m3.
fa_status tree_attention(const char* fn, const void* q, const void* k_cache, const void* v_cache,
                         const void* k_scale, const void* v_scale, const int* block_table,
                         const int* seq_lens, const int* cu_seqlens_q, const int* mask, void* o,
                         float* lse, int num_seqs, int total_q, int max_seqlen_q, int mask_words, int H,
                         int Hkv, int d, int page_size, int num_pages, int max_blocks_per_seq,
                         float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || num_pages < 0 || max_blocks_per_seq < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H <= 0 || Hkv <= 0 || H % Hkv != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: H=%d Hkv=%d (need H %% Hkv == 0)", fn, H, Hkv);
  if (mask_words < 1) return fail(FA_ERR_INVALID_ARG, "%s: mask_words=%d", fn, mask_words);
  if (!(scale > 0.f) || scale == INFINITY)
    return fail(FA_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
  fa_status st = check_dims(fn, d, page_size);
  if (st != FA_OK) return st;
  if (H / Hkv > 128) return fail(FA_ERR_UNSUPPORTED, "%s: H/Hkv=%d > 128", fn, H / Hkv);
  if (num_seqs > fa::kMaxTreeSeqs)
    return fail(FA_ERR_UNSUPPORTED, "%s: num_seqs=%d > %d", fn, num_seqs, fa::kMaxTreeSeqs);
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return FA_OK;
  if (q == nullptr || o == nullptr || mask == nullptr) return fail(FA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if ((st = check_caches(fn, k_cache, v_cache, k_scale, v_scale, 1, Hkv, num_pages)) != FA_OK) return st;
  if ((st = check_table(fn, block_table, seq_lens, cu_seqlens_q, max_blocks_per_seq)) != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(mask, 4) || !aligned(lse, 4))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  const size_t need = fa::tree_attn_workspace(max_seqlen_q, H, Hkv, d);
  if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))
    return fail(FA_ERR_WORKSPACE, "%s: workspace %p of %zu bytes (need %zu, 256-byte aligned)", fn, workspace,
                workspace_bytes, need);
  if (max_seqlen_q > total_q) max_seqlen_q = total_q;   // no sequence has more
  // rows, mask words and positions in the list of K/V tiles (at most 4 a tile and 9 a
  // unit) are numbered in 32 bits
  const long long nodes = 2 * (128 / (H / Hkv));
  const double units = (double)num_seqs * Hkv * (double)((max_seqlen_q + nodes - 1) / nodes);
  if ((long long)total_q * H > kInt || (long long)total_q * mask_words > kInt ||
      units * (4.0 * ((max_blocks_per_seq + 7) / 8) + 9.0) > (double)kInt)
    return fail(FA_ERR_UNSUPPORTED, "%s: total_q*H, total_q*mask_words or the K/V tiles of all units exceed 2^31", fn);
  fa::TreeAttnParams p{q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens_q, mask, o, lse,
                       num_seqs, total_q, max_seqlen_q, mask_words, H, Hkv, d, num_pages, max_blocks_per_seq,
                       scale, workspace, nullptr};
  if ((st = fa::api_status_ptr(&p.status)) != FA_OK) return st;
  const char* why = "tree attention launch";
  const cudaError_t e = fa::launch_tree_attn(p, static_cast<cudaStream_t>(stream), &why);
  return launched(e, why);
}

// What fa_qk_norm_rope and fa_paged_qkv_write share; fills p.
fa_status rows_setup(const char* fn, const void* q, const void* k, const void* q_weight,
                     const void* k_weight, const float* cos_sin, const int* positions, void* q_out,
                     int total, int H, int Hkv, int d, long long q_stride, long long k_stride,
                     int rot_dim, int interleaved, int num_axes, const int* sections,
                     int max_positions, float eps, fa::QkvRowsParams* p, bool* nothing) {
  *nothing = false;
  if (total < 0) return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H <= 0 || Hkv <= 0) return fail(FA_ERR_INVALID_ARG, "%s: H=%d Hkv=%d", fn, H, Hkv);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "%s: d=%d (supported: 64, 128)", fn, d);
  if (rot_dim < 0 || rot_dim > d || rot_dim % 8 != 0)
    return fail(rot_dim < 0 || rot_dim > d ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED,
                "%s: rot_dim=%d (a multiple of 8 up to d)", fn, rot_dim);
  if (interleaved != 0 && interleaved != 1)
    return fail(FA_ERR_INVALID_ARG, "%s: interleaved=%d", fn, interleaved);
  if (num_axes < 1) return fail(FA_ERR_INVALID_ARG, "%s: num_axes=%d", fn, num_axes);
  if (num_axes > fa::kMaxAxes)
    return fail(FA_ERR_UNSUPPORTED, "%s: num_axes=%d > %d", fn, num_axes, fa::kMaxAxes);
  if (!(eps >= 0.f) || eps == INFINITY) return fail(FA_ERR_INVALID_ARG, "%s: eps must be finite, not negative", fn);
  if (sections == nullptr && num_axes > 1 && rot_dim > 0)
    return fail(FA_ERR_INVALID_ARG, "%s: several axes need sections", fn);
  int end = 0;
  for (int a = 0; a < fa::kMaxAxes; ++a) {
    if (a < num_axes) {
      const int n = sections != nullptr ? sections[a] : rot_dim / 2;
      if (n < 0 || n > rot_dim / 2 - end)
        return fail(FA_ERR_INVALID_ARG, "%s: sections do not add up to rot_dim/2", fn);
      end += n;
    }
    p->section_end[a] = a < num_axes ? end : rot_dim / 2;
  }
  if (end != rot_dim / 2) return fail(FA_ERR_INVALID_ARG, "%s: sections do not add up to rot_dim/2", fn);
  if (rot_dim > 0 && max_positions < 0) return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (total == 0) {
    *nothing = true;
    return FA_OK;
  }
  if (q == nullptr || k == nullptr || q_out == nullptr) return fail(FA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (rot_dim > 0 && (cos_sin == nullptr || positions == nullptr || max_positions == 0))
    return fail(FA_ERR_INVALID_ARG, "%s: a rotation needs cos_sin and positions", fn);
  if (H > 65536 || Hkv > 65536 || (long long)total * ((long long)H + 2ll * Hkv) > kInt)
    return fail(FA_ERR_UNSUPPORTED, "%s: H, Hkv <= 65536, total*(H + 2*Hkv) below 2^31", fn);
  if (q_stride < (long long)H * d || k_stride < (long long)Hkv * d || q_stride % 8 != 0 || k_stride % 8 != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: q_stride=%lld k_stride=%lld (multiples of 8, at least heads*d)", fn,
                q_stride, k_stride);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(cos_sin, 16) || !aligned(positions, 4) || !aligned(q_out, 16))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (q_out == q && q_stride != (long long)H * d)
    return fail(FA_ERR_INVALID_ARG, "%s: q_out is q, whose rows are not dense", fn);
  p->q = q;
  p->k = k;
  p->q_stride = q_stride;
  p->k_stride = k_stride;
  p->q_weight = q_weight;
  p->k_weight = k_weight;
  p->cos_sin = cos_sin;
  p->positions = positions;
  p->q_out = q_out;
  p->total = total;
  p->H = H;
  p->Hkv = Hkv;
  p->d = d;
  p->rot_dim = rot_dim;
  p->interleaved = interleaved;
  p->num_axes = num_axes;
  p->max_positions = max_positions;
  p->eps = eps;
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_tree_layout(const int* parents, const int* seq_lens, const int* cu_seqlens, int* mask,
                         int* positions, int num_seqs, int total, int mask_words, void* stream) {
  const char* fn = "fa_tree_layout";
  if (num_seqs < 0 || total < 0) return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (mask_words < 1) return fail(FA_ERR_INVALID_ARG, "%s: mask_words=%d", fn, mask_words);
  if (mask_words > 32 || (long long)total * mask_words > kInt)
    return fail(FA_ERR_UNSUPPORTED, "%s: mask_words=%d total=%d", fn, mask_words, total);
  if (num_seqs == 0 || total == 0) return FA_OK;
  if (parents == nullptr || seq_lens == nullptr || cu_seqlens == nullptr || mask == nullptr)
    return fail(FA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(parents, 4) || !aligned(seq_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(mask, 4) ||
      !aligned(positions, 4))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  fa::TreeLayoutParams p{parents, seq_lens, cu_seqlens, mask, positions, num_seqs, total, mask_words, nullptr};
  const fa_status st = fa::api_status_ptr(&p.status);
  if (st != FA_OK) return st;
  return launched(fa::launch_tree_layout(p, static_cast<cudaStream_t>(stream)), "fa_tree_layout launch");
}

fa_status fa_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                          const float* cos_sin, const int* positions, void* q_out, void* k_out,
                          int total, int H, int Hkv, int d, long long q_stride, long long k_stride,
                          int rot_dim, int interleaved, int num_axes, const int* sections,
                          int max_positions, float eps, void* stream) {
  const char* fn = "fa_qk_norm_rope";
  fa::QkvRowsParams p{};
  bool nothing = false;
  fa_status st = rows_setup(fn, q, k, q_weight, k_weight, cos_sin, positions, q_out, total, H, Hkv, d,
                            q_stride, k_stride, rot_dim, interleaved, num_axes, sections, max_positions, eps,
                            &p, &nothing);
  if (st != FA_OK || nothing) return st;
  if (k_out == nullptr || !aligned(k_out, 16))
    return fail(FA_ERR_INVALID_ARG, "%s: k_out is null or misaligned", fn);
  if (k_out == k && k_stride != (long long)Hkv * d)
    return fail(FA_ERR_INVALID_ARG, "%s: k_out is k, whose rows are not dense", fn);
  p.k_out = k_out;
  if ((st = fa::api_status_ptr(&p.status)) != FA_OK) return st;
  return launched(fa::launch_qkv_rows(p, static_cast<cudaStream_t>(stream)), "fa_qk_norm_rope launch");
}

fa_status fa_paged_qkv_write(const void* q, const void* k, const void* v, const void* q_weight,
                             const void* k_weight, const float* cos_sin, const int* positions,
                             void* q_out, void* k_cache, void* v_cache, const int* block_table,
                             const int* seq_lens, const int* cu_seqlens, int num_seqs, int total,
                             int H, int Hkv, int d, long long q_stride, long long k_stride,
                             long long v_stride, int rot_dim, int interleaved, int num_axes,
                             const int* sections, int max_positions, float eps, int page_size,
                             int num_pages, int max_blocks_per_seq, void* stream) {
  const char* fn = "fa_paged_qkv_write";
  fa::QkvRowsParams p{};
  bool nothing = false;
  if (num_seqs < 0 || num_pages < 0 || max_blocks_per_seq < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  fa_status st = check_dims(fn, d, page_size);
  if (st == FA_OK)
    st = rows_setup(fn, q, k, q_weight, k_weight, cos_sin, positions, q_out, total, H, Hkv, d, q_stride,
                    k_stride, rot_dim, interleaved, num_axes, sections, max_positions, eps, &p, &nothing);
  if (st != FA_OK || nothing || num_seqs == 0) return st;
  if ((st = check_caches(fn, k_cache, v_cache, nullptr, nullptr, 1, Hkv, num_pages)) != FA_OK) return st;
  if ((st = check_table(fn, block_table, seq_lens, cu_seqlens, max_blocks_per_seq)) != FA_OK) return st;
  if (v == nullptr || !aligned(v, 16)) return fail(FA_ERR_INVALID_ARG, "%s: v is null or misaligned", fn);
  if (v_stride < (long long)Hkv * d || v_stride % 8 != 0)
    return fail(FA_ERR_INVALID_ARG, "%s: v_stride=%lld (a multiple of 8, at least Hkv*d)", fn, v_stride);
  p.v = v;
  p.v_stride = v_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu = cu_seqlens;
  p.num_seqs = num_seqs;
  p.num_pages = num_pages;
  p.max_blocks = max_blocks_per_seq;
  if ((st = fa::api_status_ptr(&p.status)) != FA_OK) return st;
  return launched(fa::launch_qkv_rows(p, static_cast<cudaStream_t>(stream)), "fa_paged_qkv_write launch");
}

size_t fa_paged_tree_workspace_size(int num_seqs, int max_seqlen_q, int H, int Hkv, int d) {
  if (num_seqs <= 0 || max_seqlen_q <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || H / Hkv > 128 ||
      (d != 64 && d != 128))
    return 0;
  return fa::tree_attn_workspace(max_seqlen_q, H, Hkv, d);
}

fa_status fa_paged_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                  const int* block_table, const int* seq_lens,
                                  const int* cu_seqlens_q, const int* mask, void* o, float* lse,
                                  int num_seqs, int total_q, int max_seqlen_q, int mask_words, int H,
                                  int Hkv, int d, int page_size, int num_pages,
                                  int max_blocks_per_seq, float scale, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return tree_attention("fa_paged_tree_attention", q, k_cache, v_cache, nullptr, nullptr, block_table, seq_lens,
                        cu_seqlens_q, mask, o, lse, num_seqs, total_q, max_seqlen_q, mask_words, H, Hkv, d,
                        page_size, num_pages, max_blocks_per_seq, scale, workspace, workspace_bytes, stream);
}

fa_status fa_paged_tree_attention_e4m3(const void* q, const void* k_cache, const void* v_cache,
                                       const void* k_scale, const void* v_scale,
                                       const int* block_table, const int* seq_lens,
                                       const int* cu_seqlens_q, const int* mask, void* o, float* lse,
                                       int num_seqs, int total_q, int max_seqlen_q, int mask_words,
                                       int H, int Hkv, int d, int page_size, int num_pages,
                                       int max_blocks_per_seq, float scale, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const char* fn = "fa_paged_tree_attention_e4m3";
  if (num_seqs > 0 && total_q > 0 && max_seqlen_q > 0 && k_scale == nullptr && v_scale == nullptr)
    return fail(FA_ERR_INVALID_ARG, "%s: null scales", fn);
  return tree_attention(fn, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens_q, mask, o,
                        lse, num_seqs, total_q, max_seqlen_q, mask_words, H, Hkv, d, page_size, num_pages,
                        max_blocks_per_seq, scale, workspace, workspace_bytes, stream);
}

fa_status fa_paged_kv_accept(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                             const int* block_table, const int* seq_lens, const int* cu_seqlens,
                             const int* path, const int* path_lens, int* new_seq_lens, int num_seqs,
                             int total, int max_path, int num_layers, int Hkv, int d, int page_size,
                             int num_pages, int max_blocks_per_seq, void* stream) {
  const char* fn = "fa_paged_kv_accept";
  if (num_seqs < 0 || total < 0 || max_path < 0 || num_layers < 0 || num_pages < 0 || max_blocks_per_seq < 0)
    return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (Hkv <= 0) return fail(FA_ERR_INVALID_ARG, "%s: Hkv=%d", fn, Hkv);
  fa_status st = check_dims(fn, d, page_size);
  if (st != FA_OK) return st;
  if (max_path > fa::kMaxPath) return fail(FA_ERR_UNSUPPORTED, "%s: max_path=%d > %d", fn, max_path, fa::kMaxPath);
  if (num_seqs == 0 || num_layers == 0) return FA_OK;
  if ((st = check_caches(fn, k_cache, v_cache, k_scale, v_scale, num_layers, Hkv, num_pages)) != FA_OK) return st;
  if ((st = check_table(fn, block_table, seq_lens, cu_seqlens, max_blocks_per_seq)) != FA_OK) return st;
  if ((max_path > 0 && path == nullptr) || path_lens == nullptr || new_seq_lens == nullptr)
    return fail(FA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(path, 4) || !aligned(path_lens, 4) || !aligned(new_seq_lens, 4))
    return fail(FA_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
  if (new_seq_lens == seq_lens || new_seq_lens == cu_seqlens || new_seq_lens == path || new_seq_lens == path_lens)
    return fail(FA_ERR_INVALID_ARG, "%s: new_seq_lens is one of the inputs", fn);
  if ((long long)num_seqs * num_layers > kInt)
    return fail(FA_ERR_UNSUPPORTED, "%s: num_seqs*num_layers must stay below 2^31", fn);
  fa::KvAcceptParams p{{k_cache, v_cache, k_scale, v_scale, num_layers, Hkv, k_scale != nullptr ? d : 2 * d,
                        num_pages, nullptr},
                       block_table, seq_lens, cu_seqlens, path, path_lens, new_seq_lens, num_seqs, total,
                       max_path, max_blocks_per_seq};
  if ((st = fa::api_status_ptr(&p.c.status)) != FA_OK) return st;
  return launched(fa::launch_kv_accept(p, static_cast<cudaStream_t>(stream)), "fa_paged_kv_accept launch");
}

fa_status fa_paged_copy_pages(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                              const int* pairs, int num_pairs, int num_layers, int Hkv, int d,
                              int page_size, int num_pages, void* stream) {
  const char* fn = "fa_paged_copy_pages";
  if (num_pairs < 0 || num_layers < 0 || num_pages < 0) return fail(FA_ERR_INVALID_ARG, "%s: negative size", fn);
  if (Hkv <= 0) return fail(FA_ERR_INVALID_ARG, "%s: Hkv=%d", fn, Hkv);
  fa_status st = check_dims(fn, d, page_size);
  if (st != FA_OK) return st;
  if (num_pairs == 0 || num_layers == 0) return FA_OK;
  if ((st = check_caches(fn, k_cache, v_cache, k_scale, v_scale, num_layers, Hkv, num_pages)) != FA_OK) return st;
  if (pairs == nullptr || !aligned(pairs, 4)) return fail(FA_ERR_INVALID_ARG, "%s: pairs is null or misaligned", fn);
  if ((double)num_pairs * num_layers * Hkv > (double)(1 << 27))
    return fail(FA_ERR_UNSUPPORTED, "%s: num_pairs*num_layers*Hkv must stay below 2^27", fn);
  fa::KvMoveParams c{k_cache, v_cache, k_scale, v_scale, num_layers, Hkv, k_scale != nullptr ? d : 2 * d,
                     num_pages, nullptr};
  if ((st = fa::api_status_ptr(&c.status)) != FA_OK) return st;
  return launched(fa::launch_copy_pages(c, pairs, num_pairs, static_cast<cudaStream_t>(stream)),
                  "fa_paged_copy_pages launch");
}

}  // extern "C"
