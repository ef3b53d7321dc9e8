// Declarations of the paged-cache bookkeeping kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace mla {

constexpr int kTablesMaxRequests = 16384;  // two prefix sums per request in shared memory

struct TablesArgs {
  const int* ctx_lens;
  const int* new_lens;
  const int* pages_held;  // or null
  int* block_table;
  const int* free_pages;
  const int* free_used;
  int* free_used_out;
  int* seqlens;
  int* cu_new;
  int* pages_held_out;  // or null
  int* seq_ids;
  int* pos;
  int* slots;
  const int* parents;      // or null
  long long* tree_mask;    // with parents
  int* err;
  int B, max_pages, n_free, max_tokens, page_size, num_pages;
  int page_shift;  // log2 of a page size that is a power of two, else -1
};
cudaError_t tables_prepare();
cudaError_t launch_build_tables(const TablesArgs& a, int sm_count, cudaStream_t s);

struct AcceptArgs {
  uint8_t* kv_cache;
  const int* block_table;
  const int* seqlens;
  const int* cu_q;
  const long long* tree_mask;
  const int* accepted;
  int* seqlens_out;
  int* path;
  int* err;
  int B, T, row_bytes, max_pages, page_size, num_pages;
};
cudaError_t launch_accept_tree(const AcceptArgs& a, cudaStream_t s);

}  // namespace mla
