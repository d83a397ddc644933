// Paged K/V cache: arguments its kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "bd_internal.h"

namespace bd {

// One layer's pool and one batch of requests, as include/blockdrafter.h defines them.
struct PagedArgs {
  const void *k, *v;
  int64_t page_stride, head_stride, slot_stride;  // elements
  int n_kv_heads, group, head_dim, page_size, n_pages;
  int n_requests, table_width, n_rows, max_rows, max_len;
  const int32_t *page_table, *seq_len, *row_start;
  int window, n_sink;
  float scale_log2;  // scale * log2(e): scores in log2 units
  const void *q;
  int64_t q_stride;
};

struct PagedAttnArgs {
  PagedArgs p;
  void *out;
  int64_t out_stride;
  float *lse;  // [n_rows][n_q_heads] or null
  // workspace: where each block's share begins (many rows, long item lists only), the joins, and the
  // parts of items that several blocks work on: of the item that block g's share begins inside
  // (2g) and of the one that it ends inside (2g + 1)
  int64_t *units;       // units before each item of the list, and in all
  struct PagedShare *share;
  struct PagedJoin *join;
  float *part_o;        // [2 * n_ctas][part rows][head_dim] unnormalised sums
  float2 *part_ml;      // [2 * n_ctas][part rows] (reference in log2 units, row sum)
  int n_ctas;
  int whole;            // not 0: no shares, no joins, but every item (few rows: every KV head) is a cluster's,
                        // in so many rounds
  int cluster;          // blocks of it: 1 .. kMostCluster
  int item_rows;        // rows of an item (many rows)
};

struct PagedShare {  // item a block's share begins in, and the units before that item
  int64_t before;
  int item, pad;
};
// Rows from .. from + n - 1 (of the request's rows * group) of KV head h, joined from the parts of
// blocks g-1 .. g-2+np, g the place in the list; np = 0: none.
struct PagedJoin {
  int b, h, from, n, np, row0, len, rows;
};

constexpr int kMostCluster = 16;

// Query rows (of one KV head) a block of the few-rows attention takes.
constexpr int kFewRows = 16;
// Blocks of the few-rows attention: two on every SM.
inline int few_ctas() { return 2 * num_sms(); }

struct PagedWeightsArgs {
  PagedArgs p;
  const float *lse;
  const int32_t *rows_used;  // or null
  float decay;
  const float *score_in;     // or null
  float *score_out;
  int64_t score_stride;
};

struct PagedEvictArgs {
  PagedArgs p;
  const float *score;
  int64_t score_stride;
  int budget, n_sink, n_recent;
  const int32_t *dst_table;  // null: in place
  int dst_width;
  int32_t *kept, *len_out;
  float *score_out;          // or null
  int64_t score_out_stride;
};

// Bound on the slots that any rows of one request see.
inline int64_t visible_slots(const PagedArgs &a) {
  const int64_t seen = a.window > 0 ? static_cast<int64_t>(a.window) + a.max_rows + a.n_sink : a.max_len;
  return seen < a.max_len ? seen : a.max_len;
}
// Clusters of `size` blocks of a kernel that the current device holds at once; below 0: no answer.
template <typename... KArgs> int clusters_at_once(void (*kernel)(KArgs...), int threads, size_t smem, int size) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(size);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) == cudaSuccess &&
                  cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess;
  if (!ok) cudaGetLastError();  // the caller does without clusters: the error is not the next call's
  return ok ? n : -1;
}
// The same of 2, 4, 8 and 16 blocks, asked once on each device; a question that failed is asked again.
template <typename... KArgs> class ClustersAtOnce {
 public:
  ClustersAtOnce(void (*kernel)(KArgs...), int threads, size_t smem) : kernel_(kernel), threads_(threads), smem_(smem) {}
  int of(int size) const {
    if (size <= 1) return 1 << 30;
    int device = 0, x = 0;
    while (2 << x < size) ++x;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0) return 0;
    std::atomic<int> *kept = device < kDevices ? &n_[device][x] : nullptr;
    int n = kept ? kept->load(std::memory_order_relaxed) - 1 : -1;
    if (n < 0) {
      n = clusters_at_once(kernel_, threads_, smem_, size);
      if (n >= 0 && kept) kept->store(n + 1, std::memory_order_relaxed);
    }
    return n < 0 ? 0 : n;
  }

 private:
  static constexpr int kDevices = 64;
  void (*kernel_)(KArgs...);
  int threads_;
  size_t smem_;
  mutable std::atomic<int> n_[kDevices][4] = {};  // and one; 0: not asked yet
};
// Before a launch of clusters of `size` blocks: more than eight ask the function's leave, on every device.
template <typename... KArgs> cudaError_t allow_cluster(void (*kernel)(KArgs...), int size) {
  return size <= 8 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}
inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t few_bytes(int head_dim);
size_t many_bytes(int n_requests, int max_rows, int group, int head_dim);
std::string launch_attention_few(PagedAttnArgs a, void *workspace, int dtype, cudaStream_t s);
std::string launch_attention_many(PagedAttnArgs a, void *workspace, int dtype, cudaStream_t s);

bool weights_many_takes(const PagedArgs &a);
std::string launch_weights_many(const PagedWeightsArgs &A, int dtype, cudaStream_t s);

// The error words of the paged-cache kernels together; not read (a blocking copy each) before the first call of theirs.
unsigned take_error_words_paged();
unsigned take_error_word_paged_wt();
unsigned take_error_word_paged_attn();
unsigned take_error_word_paged_tc();

}  // namespace bd
