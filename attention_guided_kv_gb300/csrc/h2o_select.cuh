// The H2O select and truncate launches, shared by the evictions of the bf16
// and the 4-bit cache (h2o_evict.cu, h2o_select_long.cu).
#pragma once

#include "common.cuh"
#include "h2o_link.cuh"

namespace kvsel_host {

struct H2OSelectArgs {
  const int32_t* seq_lens;
  const float* cum;
  const int32_t* pos_map;
  int32_t* keep_slots;  // [batch][num_kv_heads][budget]: kept slots, ascending, -1 padded
  int32_t* keep_out;    // the same as original positions, or null
  int32_t* first_move;  // [batch][num_kv_heads]: first slot whose content changes
  kvsel::H2OLink link;
  int* status;
  int batch, num_kv_heads, max_len, budget, n_sink, window;
};
kvsel_status launch_h2o_select(const char* fn, const H2OSelectArgs& a, cudaStream_t st);

// The same for long rows, each spread over many CTAs (h2o_select_long.cu); rows
// = batch * num_kv_heads at most 65535, scratch of h2o_long_bytes(rows).
size_t h2o_long_bytes(int rows);
kvsel_status launch_h2o_select_long(const char* fn, const H2OSelectArgs& a, void* scratch, cudaStream_t st);

struct H2OTruncateArgs {
  int32_t* seq_lens;
  int32_t* block_table;
  int32_t* freed;  // or null
  int batch, max_pages, budget, max_len, page_shift;
};
kvsel_status launch_h2o_truncate(const char* fn, const H2OTruncateArgs& a, cudaStream_t st);

}  // namespace kvsel_host
