// serve_checks.cpp — host checks of the serving operators' arguments
// (include/mk.h): everything that can be told without reading device memory.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "serve.hpp"

namespace mk {
namespace {

mk_status bad(std::string& err, const std::string& what) {
  err = what;
  return MK_ERR_INVALID_ARG;
}

constexpr long long kMaxKeys = 0x7ffffc00;  // a tile that begins before the last key stays below 2^31

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

// Rows of heads [rows][heads][d]: the vector loads and tensor maps need every
// row to start on 16 bytes.  Strides are bounded so that no offset leaves 63
// bits (rows and heads are ints) and a tensor map can hold them (2^40 bytes).
mk_status check_rows(const char* name, const void* p, long long row_stride, long long head_stride,
                     std::string& err) {
  const std::string n(name);
  if (!p) return bad(err, n + " is required");
  if (misaligned(p)) return bad(err, n + " must be 16-byte aligned");
  if (row_stride < 0 || head_stride < 0 || (row_stride & 7) || (head_stride & 7))
    return bad(err, n + ": strides must be multiples of 8 elements");
  if (row_stride >= (1ll << 38) || head_stride >= (1ll << 38)) return bad(err, n + ": stride too large");
  return MK_OK;
}

mk_status check_pages(const mk_kv_pages& p, bool table, std::string& err) {
  if (p.dtype != MK_DTYPE_BF16 && p.dtype != MK_DTYPE_FP16) return bad(err, "dtype must be MK_DTYPE_BF16 or MK_DTYPE_FP16");
  if (p.head_dim != 64 && p.head_dim != 128) {
    err = "head_dim must be 64 or 128";
    return MK_ERR_UNSUPPORTED;
  }
  if (p.n_kv_heads < 1 || p.n_kv_heads > 65535) return bad(err, "n_kv_heads out of range");
  if (p.n_pages < 0 || p.page_size < (table ? 1 : 0)) return bad(err, "n_pages or page_size out of range");
  if (p.n_pages > 0 && p.page_size > 0) {  // (an empty pool may have no address)
    mk_status s = check_rows("pages.k", p.k, p.row_stride, p.head_stride, err);
    if (s == MK_OK) s = check_rows("pages.v", p.v, p.row_stride, p.head_stride, err);
    if (s != MK_OK) return s;
  }
  if (p.page_stride < 0 || (p.page_stride & 7) || p.page_stride >= (1ll << 38))
    return bad(err, "page_stride must be a multiple of 8 elements, below 2^38");
  if (table) {
    if ((!p.page_table && p.table_width != 0) || misaligned4(p.page_table))
      return bad(err, "page_table is required, 4-byte aligned");
    if (p.table_width < 0 || p.table_stride < p.table_width) return bad(err, "table_stride must be >= table_width >= 0");
    if ((long long)p.table_width * p.page_size > kMaxKeys) return bad(err, "table_width * page_size exceeds 2^31 - 1024 positions");
  } else if (p.page_size > kMaxKeys) {
    return bad(err, "more than 2^31 - 1024 key rows");
  }
  return MK_OK;
}

// Whether rows of d elements along three dimensions lie on top of one another: from the smallest stride on, each must
// reach past all that the dimensions inside it span.  (A dimension of one entry has no stride.)
bool rows_overlap(int d, const long long (&count)[3], const long long (&stride)[3]) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return stride[x] < stride[y]; });
  long long span = d;
  for (int i : order) {
    if (count[i] <= 1) continue;
    if (stride[i] < span) return true;
    if (stride[i] > (1ll << 61) / count[i]) span = 1ll << 61;  // (longer than any stride can be)
    else span += (count[i] - 1) * stride[i];
  }
  return false;
}

mk_status check_heads(int n_q, int n_kv, std::string& err) {
  if (n_q < 1 || n_q > 65535 || n_q % n_kv) return bad(err, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
  return MK_OK;
}

mk_status check_scale(float s, std::string& err) {
  if (!std::isfinite(s) || s < 0.f) return bad(err, "scale must be finite and not negative");
  return MK_OK;
}

}  // namespace

mk_status check_append(const mk_append_args& a, std::string& err) {
  if (a.batch < 0 || a.n_tokens < 0 || a.n_q_heads < 0 || a.n_q_heads > 65535)
    return bad(err, "batch, n_tokens or n_q_heads out of range");
  mk_status s = check_pages(a.pages, true, err);
  if (s != MK_OK) return s;
  const mk_kv_pages& g = a.pages;
  if (rows_overlap(g.head_dim, {g.n_pages, g.n_kv_heads, g.page_size}, {g.page_stride, g.head_stride, g.row_stride}))
    return bad(err, "pages: rows that are written must not overlap");
  if (a.n_q_heads && !a.q) return bad(err, "n_q_heads without q");
  if (a.q) {
    if (a.n_q_heads < 1) return bad(err, "q without n_q_heads");
    s = check_rows("q", a.q, a.q_row_stride, a.q_head_stride, err);
    if (s == MK_OK) s = check_rows("q_out", a.q_out, a.qo_row_stride, a.qo_head_stride, err);
    if (s != MK_OK) return s;
    if (a.q == a.q_out && (a.q_row_stride != a.qo_row_stride || a.q_head_stride != a.qo_head_stride))
      return bad(err, "q_out on top of q must have q's strides");
  }
  s = check_rows("k", a.k, a.k_row_stride, a.k_head_stride, err);
  if (s == MK_OK) s = check_rows("v", a.v, a.v_row_stride, a.v_head_stride, err);
  if (s != MK_OK) return s;
  if (!a.cu_seqlens || !a.ctx_lens || misaligned4(a.cu_seqlens) || misaligned4(a.ctx_lens))
    return bad(err, "cu_seqlens and ctx_lens are required, 4-byte aligned");
  if (a.rope_theta != 0.0 && !(a.rope_theta >= 1.0 && std::isfinite(a.rope_theta)))
    return bad(err, "rope_theta must be 0 (no rotation) or at least 1");
  if (misaligned4(a.status)) return bad(err, "status must be 4-byte aligned");
  return MK_OK;
}

mk_status check_prompt(const mk_prompt_args& a, std::string& err) {
  if (a.batch < 0 || a.n_tokens < 0) return bad(err, "batch or n_tokens out of range");
  if (a.causal != 0 && a.causal != 1) return bad(err, "causal must be 0 or 1");
  const bool paged = a.pages.page_table != nullptr;
  mk_status s = check_pages(a.pages, paged, err);
  if (s == MK_OK) s = check_heads(a.n_q_heads, a.pages.n_kv_heads, err);
  if (s == MK_OK) s = check_scale(a.scale, err);
  if (s == MK_OK) s = check_rows("q", a.q, a.q_row_stride, a.q_head_stride, err);
  if (s == MK_OK) s = check_rows("out", a.out, a.o_row_stride, a.o_head_stride, err);
  if (s != MK_OK) return s;
  if (!a.cu_q || misaligned4(a.cu_q)) return bad(err, "cu_q is required, 4-byte aligned");
  if (paged) {
    if (!a.kv_lens || misaligned4(a.kv_lens)) return bad(err, "kv_lens is required with a page table, 4-byte aligned");
  } else {
    if (!a.cu_k || misaligned4(a.cu_k)) return bad(err, "cu_k is required with packed keys, 4-byte aligned");
    if (a.pages.n_pages != 1) return bad(err, "packed keys are one page: n_pages must be 1");
  }
  if (misaligned4(a.status)) return bad(err, "status must be 4-byte aligned");
  if (a.workspace && (reinterpret_cast<uintptr_t>(a.workspace) & 255)) {
    err = "workspace must be 256-byte aligned";
    return MK_ERR_WORKSPACE;
  }
  if (a.n_q_heads / a.pages.n_kv_heads > 128) {
    err = "more than 128 query heads per kv head";
    return MK_ERR_UNSUPPORTED;
  }
  const int ps = a.pages.page_size;
  if (paged && ps < 128 && ps != 16 && ps != 32 && ps != 64) {
    err = "prompt attention reads pages of 16, 32, 64 or at least 128 rows";
    return MK_ERR_UNSUPPORTED;
  }
  return MK_OK;
}

mk_status check_paged(const mk_paged_attn_args& a, std::string& err) {
  if (a.batch < 0) return bad(err, "batch out of range");
  mk_status s = check_pages(a.pages, true, err);
  if (s == MK_OK) s = check_heads(a.n_q_heads, a.pages.n_kv_heads, err);
  if (s == MK_OK) s = check_scale(a.scale, err);
  if (s == MK_OK) s = check_rows("q", a.q, a.q_row_stride, a.q_head_stride, err);
  if (s == MK_OK) s = check_rows("out", a.out, a.o_row_stride, a.o_head_stride, err);
  if (s != MK_OK) return s;
  if (!a.kv_lens || misaligned4(a.kv_lens)) return bad(err, "kv_lens is required, 4-byte aligned");
  if (misaligned4(a.status)) return bad(err, "status must be 4-byte aligned");
  if (a.batch > MK_PAGED_ATTN_MAX_BATCH) {
    err = "batch above MK_PAGED_ATTN_MAX_BATCH";
    return MK_ERR_UNSUPPORTED;
  }
  if (a.batch > 0) {
    if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255) ||
        a.workspace_bytes < paged_workspace_bytes(a.batch, a.n_q_heads, a.pages.n_kv_heads, a.pages.head_dim)) {
      err = "workspace missing, not 256-byte aligned or smaller than mk_paged_attention_workspace_bytes()";
      return MK_ERR_WORKSPACE;
    }
  }
  return MK_OK;
}

mk_status check_logits(const mk_logits_args& a, std::string& err) {
  if (a.rows < 0 || a.rows > 65535 || a.vocab < 1 || a.vocab > (1 << 30))
    return bad(err, "rows must be in [0, 65535], vocab in [1, 2^30]");
  if (a.dtype != MK_DTYPE_FP32 && a.dtype != MK_DTYPE_BF16 && a.dtype != MK_DTYPE_FP16) return bad(err, "unknown dtype");
  const int es = a.dtype == MK_DTYPE_FP32 ? 4 : 2;
  if (!a.logits || (reinterpret_cast<uintptr_t>(a.logits) & (es - 1))) return bad(err, "logits is required, aligned to its type");
  if (!a.out && !a.next_tokens) return bad(err, "out or next_tokens is required");
  if (a.rows > 1 && a.logits_stride < a.vocab) return bad(err, "logits_stride below vocab");
  if (a.out && a.rows > 1 && a.out_stride < a.vocab) return bad(err, "out_stride below vocab");
  if (a.out && static_cast<const void*>(a.out) == a.logits &&
      (a.dtype != MK_DTYPE_FP32 || (a.rows > 1 && a.out_stride != a.logits_stride)))
    return bad(err, "out on top of logits needs fp32 logits and the same stride");
  const void* words[] = {a.out, a.next_tokens, a.history, a.history_lens, a.prompt_lens, a.repetition, a.frequency,
                         a.presence, a.bias_indptr, a.bias_ids, a.bias_values, a.mask, a.status};
  for (const void* w : words)
    if (misaligned4(w)) return bad(err, "every array must be 4-byte aligned");
  if (a.history) {
    if (a.history_width < 0 || (a.rows > 1 && a.history_stride < a.history_width))
      return bad(err, "history_stride must be >= history_width >= 0");
    if (a.history_width >= (1 << 28)) return bad(err, "history_width must be below 2^28");
  } else if (a.repetition || a.frequency || a.presence || a.history_lens || a.prompt_lens) {
    return bad(err, "penalties and history lengths need a history");
  }
  if (a.bias_indptr || a.bias_ids || a.bias_values) {
    if (!a.bias_indptr || !a.bias_ids || !a.bias_values || a.bias_count < 0)
      return bad(err, "bias_indptr, bias_ids and bias_values go together");
  }
  const long long words_per_row = ((long long)a.vocab + 31) / 32;
  if (a.mask && a.mask_stride != 0 && a.mask_stride < words_per_row) return bad(err, "mask_stride below (vocab + 31) / 32");
  return MK_OK;
}

}  // namespace mk
