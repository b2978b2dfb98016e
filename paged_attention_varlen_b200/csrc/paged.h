// paged.h -- host plan and launches of the paged serving operators: the step's tables and slot map, the
// cache write, and attention / differential attention whose lengths are read on the device.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ala.h"

namespace ala {

// A planned ala_paged_attention / ala_paged_diff_attention call.  Nothing in it depends on the lengths,
// which the kernel reads from device memory at every execution.
struct PagedPlan {
  int32_t dtype = 0, maps = 1;                     // maps: softmax maps per head (2: differential)
  int32_t heads = 0, kv_heads = 0, d = 0;          // query heads (both maps counted), query head size
  int32_t row = 0;                                 // elements of one K / V row of a kv head: maps * d
  int32_t batch = 0, max_blocks = 0, block_size = 0, num_blocks = 0, mask_type = 0;
  int64_t n_tokens = 0, q_stride = 0;
  float qk_scale = 1.f, norm_eps = 0.f, out_scale = 1.f;
  void *q = nullptr, *k = nullptr, *v = nullptr, *out = nullptr;
  const int32_t *block_tables = nullptr, *seq_len = nullptr, *kv_seq_len = nullptr;
  const float *slopes = nullptr, *lambda = nullptr, *norm_weight = nullptr;
  float* lse = nullptr;
  uint64_t ws_size = 0, off_desc = 0, off_ml = 0, off_part = 0;
  bool maps_ready = false;
  CUtensorMap tmK, tmV;
  const void* bound_ws = nullptr;  // a workspace whose status words are clear (ala_op_bind_workspace)
};

// The workspace starts with the status words and, from byte 256, a counter for each CTA; both start out as zeros, and
// an execution leaves the counters so.  The rest needs no initial values.
constexpr uint64_t kPagedHeaderBytes = 1024;

// Kernel head size (columns of a K / V row: 64, 128 or 256) that serves rows of `row` elements; 0: none.
int paged_kernel_d(int64_t row);
// Sizes the workspace of a filled-in plan.
void paged_layout(PagedPlan* plan);
// Checks the arguments of both attention operators and fills in the plan; `lambda` selects the differential
// form.  Nothing touches the GPU.
struct PagedAttnArgs {
  const ala_tensor *query, *key, *value, *block_tables, *seq_len, *kv_seq_len, *slopes, *lambda, *norm_weight;
  int64_t query_stride;
  int mask_type;
  int32_t heads, kv_heads;
  float qk_scale, norm_eps, out_scale;
  const ala_tensor *out, *lse;
  bool diff;
};
int paged_plan(PagedPlan* plan, const PagedAttnArgs& a, char* err, size_t errlen);
int paged_run(PagedPlan* plan, void* workspace, cudaStream_t stream, char* err, size_t errlen);

struct PagedStepArgs {
  const int32_t *seq_len, *finished, *context_len;
  int32_t* block_tables;
  int32_t* free_blocks;
  const int32_t* free_count;
  int32_t *kv_seq_len, *free_count_out, *cu_seq_len, *slot_mapping, *positions, *status;
  int32_t batch, max_blocks, block_size, capacity, n_tokens;
};
// Most requests of a step: their sums stay in one CTA's shared memory.
constexpr int32_t kPagedStepMaxBatch = 8192;
cudaError_t launch_paged_step(const PagedStepArgs& a, cudaStream_t stream);

struct PagedWriteArgs {
  const uint8_t *key, *value;       // value may be null
  uint8_t *key_cache, *value_cache;
  const int32_t* slots;
  int64_t key_stride, value_stride;  // bytes between tokens
  int64_t key_row, value_row;        // bytes of one token's row
  int64_t n_tokens, n_slots;
};
cudaError_t launch_paged_write(const PagedWriteArgs& a, cudaStream_t stream);

}  // namespace ala
