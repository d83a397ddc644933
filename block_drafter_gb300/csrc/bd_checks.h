// Host checks that the paged cache's and the target rows' entry points share.
#pragma once
#include <stdint.h>

#include <cmath>
#include <string>

#include "bd_paged.h"

namespace bd {

inline bd_status refuse(bd_status st, const std::string &msg) {
  set_last_error(msg);
  return st;
}
inline bd_status ran(const std::string &e) { return e.empty() ? BD_OK : refuse(BD_ERR_CUDA, e); }
inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether [p, p + np) and [q, q + nq) (bytes) share any.
inline bool overlap(const void *p, int64_t np, const void *q, int64_t nq) {
  const char *a = static_cast<const char *>(p), *b = static_cast<const char *>(q);
  return np > 0 && nq > 0 && a < b + nq && b < a + np;
}

inline bd_status check_heads(int n_q_heads, int n_kv_heads) {
  if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return refuse(BD_ERR_INVALID_ARG, "paged kv: n_q_heads must be a positive multiple of n_kv_heads");
  if (n_q_heads / n_kv_heads > BD_PAGED_MAX_GROUP || n_kv_heads > 1024)
    return refuse(BD_ERR_UNSUPPORTED, "paged kv: at most 128 query heads per KV head and 1024 KV heads");
  return BD_OK;
}

inline bd_status check_paged_batch(int page_size, const bd_paged_batch *t, bool rows) {
  if (!t) return refuse(BD_ERR_INVALID_ARG, "paged batch is NULL");
  if (t->n_requests < 1 || t->n_requests > BD_PAGED_MAX_REQUESTS)
    return refuse(BD_ERR_INVALID_ARG, "paged batch: n_requests must be in 1..1024");
  if (t->table_width < 1 || t->max_len < 0 ||
      t->max_len > static_cast<int64_t>(t->table_width) * page_size || t->max_len > (1 << 30))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: max_len must be within table_width * page_size (and 2^30)");
  if (!t->page_table || !t->seq_len || misaligned(t->page_table, 4) || misaligned(t->seq_len, 4))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: page_table and seq_len must be given");
  if (rows) {
    if (!t->row_start || misaligned(t->row_start, 4)) return refuse(BD_ERR_INVALID_ARG, "paged batch: row_start must be given");
    if (t->n_rows < 0 || t->max_rows < 0 || t->max_rows > t->n_rows || t->n_rows > (1 << 28))
      return refuse(BD_ERR_INVALID_ARG, "paged batch: 0 <= max_rows <= n_rows <= 2^28");
  }
  return BD_OK;
}

inline bd_status check_rows(const void *p, int64_t stride, int64_t width, int n_rows, const char *name, const char *who = "paged cache") {
  if (!p || misaligned(p, 16) || stride % 8 || (n_rows > 1 && stride < width))
    return refuse(BD_ERR_INVALID_ARG, std::string(who) + ": " + name +
                                          " must be 16-byte aligned rows with a stride that is a multiple of 8 and holds a row");
  return BD_OK;
}
inline int64_t row_bytes(int64_t stride, int64_t width, int n_rows) {
  return n_rows < 1 ? 0 : ((n_rows - 1) * stride + width) * 2;
}

inline bd_status check_mask(int window, int n_sink, float scale) {
  if (window < 0 || n_sink < 0) return refuse(BD_ERR_INVALID_ARG, "paged attention: window and n_sink must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(BD_ERR_INVALID_ARG, "paged attention: scale must be > 0 and finite");
  return BD_OK;
}

// The batch's part of the kernels' arguments.
inline void set_batch(PagedArgs &a, const bd_paged_batch *t) {
  a.n_requests = t->n_requests;
  a.table_width = t->table_width;
  a.n_rows = t->n_rows;
  a.max_rows = t->max_rows;
  a.max_len = t->max_len;
  a.page_table = t->page_table;
  a.seq_len = t->seq_len;
  a.row_start = t->row_start;
}

}  // namespace bd
