// Declarations shared by the kernels of the speculative-decoding operators
// (tree attention, block tables and slot maps, accepted branches).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mla {

constexpr int kTreeTile = 64;      // cache rows per attention tile
constexpr int kTreeMaxNodes = 64;  // drafted tokens of one sequence: the bits of a mask word
constexpr int kTreeRows = 128;     // (token, head) rows of one row block

// Cost of one more segment inside a KV chunk (the next rows' queries, the
// output of the last), in 64-token tiles.
constexpr int kTreeSegTiles = 4;

// Workspace of mla_decode_tree.  seqs: the sequences with work, in order, 4 ints
// each (first token, drafted tokens, length, place in the batch).  rec: 8 ints
// per chunk boundary (G + 1 of them): place on that list, row block and tile
// where the chunk starts, 0, then the list's entry; the last one is (list's
// length, 0, ...).  up / cp: prefix sums of the plan over the list, used there
// only when the batch is too large for shared memory.  part_u / part_lse: the
// partial results of pieces of row blocks, 128 rows per slot: chunk c writes a
// piece that continues a block into slot 2c and one that begins a block in
// slot 2c + 1 (fp32).
struct TreeWsLayout {
  size_t rec = 0, seqs = 0, up = 0, cp = 0, part_lse = 0, part_u = 0, total = 0;
};
TreeWsLayout tree_ws_layout(int B, int d_c, int num_chunks);

struct TreeArgs {
  const void* q;
  const void* kv;
  const int* block_table;
  const int* seqlens;
  const int* cu_q;
  const unsigned long long* mask;
  void* u;
  float* lse;
  int* rec;
  int4* seqs;
  long long* up;
  int* cp;
  float* part_u;
  float* part_lse;
  int* err;
  int B, T, n_h, d_c, d_R, page_size, max_pages, num_pages, num_chunks;
  float scale;
  bool bf16;     // q and the cache (else fp32)
  bool out_f32;  // u
};

cudaError_t launch_tree_plan(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t s);

// The DeepSeek-V3-shape attend kernel: bf16, d_c = 512, d_R = 64.  The rows of
// q [T, n_h, 576] and u [T, n_h, 512] are flat: row t n_h + h.
//   k: 32 cache rows, all nine 64-column blocks; v: one CTA's four latent blocks
//     of 64 cache rows; q: 64 rows, three 64-column blocks (a copy each);
//   u_out: 32 rows of u, 128 bytes of columns; part_out the same of part_u.
struct TreeMaps {
  CUtensorMap k, v, q, u_out, part_out;
};
int tree_sm100_prepare();  // co-resident clusters, 0 if the kernel cannot run
cudaError_t launch_tree_sm100(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s);

// The small-latent attend kernel (bf16 or fp32; decode_small_sm100_supported
// says which widths).  q_map: the flat rows [T n_h, d_c + d_R], box 128 bytes x
// 128 rows; kv_map: the cache, box 128 bytes x 64 rows, 128-byte swizzle;
// kv_pv_map (fp32): the cache with 128-byte swizzle of 32-byte atoms.
cudaError_t launch_tree_small_sm100(const TreeArgs& a, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                                    const CUtensorMap& kv_pv_map, cudaStream_t s);

}  // namespace mla
