// Internal interface between the C-ABI layer (dsa_api.cpp) and the kernels.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dsa.h"

namespace dsa {

struct IndexerParams {
  const uint8_t *q_idx;     // bf16 [R, H_I, D_I]
  const float *w;           // [R, H_I]
  const uint8_t *idx_cache; // bf16 / e4m3 [NP, P, D_I]
  const float *idx_scale;   // [NP, P] or null
  const int32_t *page_table;
  const int32_t *row_req;
  const int32_t *row_len;
  const int32_t *block_first;
  const int32_t *block_nrows;
  float *scores;            // [row_hi - row_lo, W]: row r at (r - row_lo) * W
  uint32_t *status;
  uint32_t *row_hist;       // [R, 4096] key-bin counts for the top-k, or null
  int32_t idx_heads, idx_dim, max_rows, max_reqs, max_pages_per_req, score_width, num_pages;
  int32_t page_size, block_rows;
  int32_t row_lo, row_hi;   // the row window scored (0, max_rows for all rows)
  int32_t test_timeout;     // DSA_FLAG_TEST_WAIT_TIMEOUT: one wait that nothing completes
};

struct TopkParams {
  const float *scores;     // [rows of the window, W]
  const int32_t *row_len;
  int32_t *topk_idx;
  uint32_t *status;
  uint32_t *row_hist;  // [R, 4096] filled by the indexer (used, then zeroed), or null
  int32_t topk, score_width;
  int32_t row_lo;          // first row of the window; one cluster per row of it
  int32_t inputs_ready;    // see AttnParams
};

struct AttnParams {
  const uint8_t *q;        // bf16 [R, Hq, D]
  const uint8_t *k_cache;  // bf16 [NP, P, Hkv, D], or [NP, P, 2, Hkv, D] with V interleaved
  const uint8_t *v_cache;  // k_cache + Hkv * D * 2 when interleaved
  const int32_t *page_table;
  const int32_t *row_req;
  const int32_t *row_len;
  const int32_t *topk_idx; // [R, K]
  float *part_m;           // [R, Hq, S]
  float *part_l;
  float *part_acc;         // [R, Hq, S, D]
  uint32_t *status;
  int32_t num_q_heads, num_kv_heads, topk, num_splits;
  int32_t max_rows_attn, max_reqs, max_pages_per_req, score_width, num_pages, page_size;
  float sm_scale_log2;     // sm_scale * log2(e)
  int32_t kv_interleaved;  // 1: one copy moves a token's K and V rows
  int32_t page_shift;      // log2(page_size)
  const int32_t *grouped;  // [R] 1: the row is attended by the prefill-group kernel (null: no groups)
  int32_t skip_empty_rows; // 1: rows of length 0 get no partials (the step's merge never reads them)
  // 1: rows and page table may be read before the wait for the kernel before.
  // So inside dsa_step: its first kernel is an ordinary launch, behind
  // everything that wrote them.  A call of its own may follow one that does
  // (dsa_update_pages, dsa_compact_pages write the table and lengths).
  int32_t inputs_ready;
};

// Prefill row groups: the rows of one request in a slot of kGroupRows
// consecutive rows (at least kGroupMin of them) attend to the union of their
// selections on the tensor cores (group_attn.cu).
constexpr int kGroupRows = 16;
constexpr int kGroupMin = 8;

struct GroupParams {
  int32_t *grouped;  // [R] 1: the row is a group member
  int32_t *ntiles;   // [nslots] 128-position tiles holding a selected position (0: the slot is no group)
  int32_t *tiles;    // [nslots, umax / 128] those tiles' indices, ascending
  uint32_t *umask;   // [nslots, umax / 128, 16, 4] per tile and slot row j: bit b of word w set if
                     // row j selected position 128 * tile + 32 * w + b
  int32_t umax, nslots;  // umax: positions a group may span (a multiple of 128)
};

struct MergeParams {
  const float *part_m, *part_l, *part_acc;
  uint8_t *out;  // bf16 [R, Hq, D]
  float *lse;    // [R, Hq] or null
  const int32_t *row_len;  // [R] or null: a row of length 0 is written empty without reading its partials
  int32_t max_rows, num_q_heads, num_splits;
};

// Dense attention over the paged cache (dense_attn.cu).  Regions of its
// workspace past the status word; C = CTAs the split kernel runs on at most.
struct DenseParams {
  const uint8_t *q;        // bf16 [R, Hq, D]
  const int32_t *page_table;
  const int32_t *row_req;
  const int32_t *row_len;
  uint8_t *out;            // bf16 [R, Hq, D]
  float *lse;              // [R, Hq] or null
  uint32_t *status;
  // a bit a row: rows that no prompt tile has, rows without a visible
  // position (null: no tiles, every row is taken); see DensePromptParams
  const uint32_t *alone, *empty;
  int2 *tail;              // [C] the row that goes on past CTA c, row -1: none (dense_common.cuh)
  float2 *part_ml;         // [C, 2, Hq] (m, l) of a CTA's first and last row, log2 domain
  float *part_o;           // [C, 2, Hq, D]
  int32_t num_q_heads, num_kv_heads, max_rows, max_reqs, max_pages_per_req, max_len, num_pages, page_size;
  int32_t page_shift;      // log2(page_size)
  int32_t window, sinks;   // window 0: the whole prefix
  float sm_scale_log2;
};
// A step's new tokens (pages.cu).
struct AppendParams {
  const int32_t *page_table;
  const int32_t *row_req;
  const int32_t *row_len;
  const char *k_new, *v_new;  // bf16 [R, Hkv, D] or null
  const char *key_new;        // bf16 [R, idx_dim] or null
  char *k_cache, *v_cache;
  uint8_t *idx_cache;
  float *idx_scale;
  uint32_t *status;
  long long kv_stride;        // bytes from a token's K (V) row to the next token's
  int32_t kv_bytes, idx_dim, max_rows, max_reqs, max_pages_per_req, max_len, num_pages, page_size, page_shift;
};

// Page bookkeeping (pages.cu): the caller's state and its workspace's regions.
struct PagesParams {
  int32_t *page_table, *req_len, *page_refs;
  const int32_t *req_from, *req_add;
  int32_t *num_used, *page_map;  // outputs or null
  uint32_t *status;
  int32_t *head;       // [4] what a plan came to (see pages.cu)
  int32_t *slots;      // [8, 7, max_reqs] what each CTA of a plan knows of the slots (many slots only)
  int32_t *old_table;  // [max_reqs * max_pages_per_req] or [num_pages], the larger
  int32_t *delta;      // [num_pages]
  int32_t *list;       // [num_pages]
  int4 *apply;         // [max_reqs] each slot's old slot, pages kept, new length, first fresh page's rank
  int32_t max_reqs, max_pages_per_req, max_len, num_pages, page_shift;  // page_shift: log2(page_size)
};
constexpr int kCopyCaches = 128;  // caches of one copy launch
struct PageCopyParams {
  char *base[kCopyCaches];
  long long page_bytes[kCopyCaches];
  int first_piece[kCopyCaches];
  int n, pieces;
};

constexpr int kDenseMaxCtas = 256;  // the workspace holds partials for this many

// Prompt tiles of the dense attention (dense_prompt.cu): chunks of
// consecutive rows of one request, 2 * (128 / G) rows at most.
struct DenseChunk {
  int32_t first, rows;  // its rows
  int32_t lmin, lmax;   // shortest and longest of them
};
struct DensePromptParams {
  uint32_t *alone;     // [R / 32] a bit a row: in no chunk, not empty
  uint32_t *redo;      // [R / 32] a bit a row: its tiles met a value that is not finite, it is done again alone
  uint32_t *empty;     // [R / 32] a bit a row: a pad row, or refused
  int32_t *nchunks;    // [2] chunks, CTAs that take tiles (the others take single rows)
  int2 *shares;        // [C + 1] where each CTA's share begins: segment (chunk * Hkv + KV head), cost before it
  DenseChunk *chunks;  // [R]
  int32_t *before;     // [R + 1] cost of the chunks before each (all KV heads)
  int2 *tail;          // [C] the segment (chunk * Hkv + KV head) that goes on past CTA c, -1: none
  float2 *part_ml;     // [C, 2, 256] (m, l) of a CTA's first and last segment's queries, log2 domain
  float *part_o;       // [C, 2, 256, D]
};

// Launches `kernel` on `st` with programmatic stream serialization, so it may
// start while the previous kernel on the stream drains (the kernel itself
// waits with griddepcontrol.wait before reading that kernel's output).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t st, unsigned cluster_x, Args... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  lc.attrs = attr;
  lc.numAttrs = n;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

// The driver's tensor-map encoder (null: none).  It works on a host thread
// whose first call this is too: the driver's own call wants a context bound to
// the thread, which the runtime does only in calls that need one.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// SM count of the current device, asked for once per device.
cudaError_t sm_count(int *sms);
// Lets `kernel`, which has no static shared memory, use `bytes` of it on the
// current device.  The limit is a property of the loaded kernel, not of a call:
// it is always set to all that a CTA can have, so that calls of other configs,
// from other host threads too, never lower it under one another.  `done` (one
// per kernel, static) remembers the devices where it is set.
constexpr int kSmemOptIn = 227 * 1024;
struct SmemLimit {
  std::atomic<bool> set[64];
};
template <typename... KArgs>
inline cudaError_t allow_smem(void (*kernel)(KArgs...), int bytes, SmemLimit &done) {
  if (bytes > kSmemOptIn) return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done.set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOptIn);
  if (e == cudaSuccess && dev < 64) done.set[dev].store(true, std::memory_order_release);
  return e;
}

// Records the thread's last-error text (see dsa_last_error) and returns st.
dsa_status_t set_error(dsa_status_t st, const char *fmt, ...);

// Each launcher returns the launch error (cudaSuccess when queued).
cudaError_t launch_indexer_tc(const dsa_config_t &cfg, const IndexerParams &p, cudaStream_t st);
cudaError_t launch_topk(const dsa_config_t &cfg, const TopkParams &p, int rows, cudaStream_t st);
cudaError_t launch_sparse_attn(const dsa_config_t &cfg, const AttnParams &p, cudaStream_t st);
cudaError_t launch_dense_attn(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                              const void *k_cache, const void *v_cache, cudaStream_t st);
bool dense_prompt_enabled(const dsa_config_t &cfg);
cudaError_t launch_append(const AppendParams &p, bool fp8, cudaStream_t st);
cudaError_t launch_update_pages(const PagesParams &p, const dsa_page_cache_t *caches, int n, cudaStream_t st);
cudaError_t launch_compact_pages(const PagesParams &p, const dsa_page_cache_t *caches, int n, cudaStream_t st);
cudaError_t launch_merge(const dsa_config_t &cfg, const MergeParams &p, cudaStream_t st);
// The prefill-group path: whether a config uses it, the union capacity per
// slot (positions, a multiple of 128), and its two kernels.
bool group_path_enabled(const dsa_config_t &cfg);
int32_t group_union_capacity(const dsa_config_t &cfg);
cudaError_t launch_group_union(const dsa_config_t &cfg, const AttnParams &p, const GroupParams &gp, cudaStream_t st);
cudaError_t launch_group_attn(const dsa_config_t &cfg, const AttnParams &p, const GroupParams &gp, cudaStream_t st);

}  // namespace dsa
