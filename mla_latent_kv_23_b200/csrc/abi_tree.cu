// C ABI of the speculative-decoding operators: argument validation, workspace
// sizing, TMA descriptors and launches.
#include <climits>
#include <cmath>
#include <cstring>

#include "abi_common.h"
#include "append_slots.h"
#include "internal.h"
#include "mla.h"
#include "tables.h"
#include "tree.h"

namespace mla {
namespace {

// A tensor map of 2- or 4-byte elements; strides in bytes, innermost first.
bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* ptr, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw,
            CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return g_encode(m, type, rank, const_cast<void*>(ptr), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, promotion,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

mla_status validate_tree(const mla_tree_params* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 0 || p->n_h < 1) return MLA_ERR_INVALID_ARG;
  if (p->n_h > 128) return MLA_ERR_UNSUPPORTED;
  if (p->d_c < 8 || p->d_c % 8 != 0 || p->d_R < 0 || p->d_R % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (p->d_c > 512 || p->d_R > 64) return MLA_ERR_UNSUPPORTED;
  if (p->page_size <= 0 || p->page_size % kTreeTile != 0) return MLA_ERR_INVALID_ARG;
  if (p->max_pages_per_seq < 1 || p->num_pages < 1) return MLA_ERR_INVALID_ARG;
  if ((long long)p->num_pages * p->page_size > INT_MAX ||
      (long long)p->max_pages_per_seq * p->page_size > INT_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->softmax_scale) || !(p->softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (!valid_dtype(p->dtype) || p->num_splits < 0) return MLA_ERR_INVALID_ARG;
  // flat rows and partial slots are 32-bit coordinates; one grid row per chunk
  if ((long long)p->T * p->n_h > INT_MAX - 2 * kTreeRows || p->num_splits > 65535)
    return MLA_ERR_UNSUPPORTED;
  if (p->B == 0 || p->T == 0) return MLA_OK;
  if (!p->q || !p->kv_cache || !p->block_table || !p->seqlens || !p->cu_q || !p->tree_mask || !p->u)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->kv_cache) || !aligned16(p->block_table) ||
      !aligned16(p->seqlens) || !aligned16(p->cu_q) || !aligned16(p->tree_mask) || !aligned16(p->u) ||
      (p->lse && !aligned16(p->lse)))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// The attend kernels: paired CTAs for the DeepSeek-V3 shape (bf16, d_c = 512,
// d_R = 64), one CTA for the small latent widths.
enum class TreeKernel { kNone, kV3, kSmall };

TreeKernel tree_kernel(const mla_tree_params* p, const DeviceInfo* d) {
  if (d->cc_major != 10 || g_encode == nullptr) return TreeKernel::kNone;
  const bool bf16 = p->dtype == MLA_DTYPE_BF16;
  if (bf16 && p->d_c == 512 && p->d_R == 64 && d->tree_clusters > 0) return TreeKernel::kV3;
  if (d->small_tc && decode_small_sm100_supported(bf16, p->d_c, p->d_R)) return TreeKernel::kSmall;
  return TreeKernel::kNone;
}

// One chunk per resident cluster, but no more than the batch can have tiles by
// what the host knows (the most row blocks times the block table's width): starting and
// retiring 148 CTAs of 226 KB takes longer than the work of a small call.
int tree_chunks(const mla_tree_params* p, const DeviceInfo* d) {
  if (p->num_splits > 0) return p->num_splits;
  const long long blocks = ((long long)p->T * p->n_h + (kTreeRows - 1LL) * p->B) / kTreeRows;
  const long long tiles = (long long)p->max_pages_per_seq * p->page_size / kTreeTile;
  const long long most = blocks * tiles;
  const int resident = tree_kernel(p, d) == TreeKernel::kV3 ? d->tree_clusters : d->sm_count;
  return most < resident ? (int)(most < 1 ? 1 : most) : resident;
}

mla_status plan_and_attend_small(const mla_tree_params* p, const TreeArgs& a, cudaStream_t s) {
  const cuuint64_t es = a.bf16 ? 2 : 4, W = (cuuint64_t)p->d_c + p->d_R;
  const auto type = a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const cuuint64_t qdims[2] = {W, (cuuint64_t)p->T * p->n_h};
  const cuuint64_t kdims[2] = {W, (cuuint64_t)p->num_pages * p->page_size};
  const cuuint64_t strides[1] = {W * es};
  const cuuint32_t qbox[2] = {static_cast<cuuint32_t>(128 / es), 128};
  const cuuint32_t kbox[2] = {static_cast<cuuint32_t>(128 / es), kTreeTile};
  CUtensorMap q, kv, kv_pv;
  memset(&kv_pv, 0, sizeof(kv_pv));
  if (!encode(&q, type, 2, p->q, qdims, strides, qbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&kv, type, 2, p->kv_cache, kdims, strides, kbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      // an MN-major tf32 operand: 128-byte swizzle of 32-byte atoms
      (!a.bf16 && !encode(&kv_pv, type, 2, p->kv_cache, kdims, strides, kbox,
                          CU_TENSOR_MAP_SWIZZLE_128B_ATOM_32B)))
    return MLA_ERR_CUDA;
  const mla_status st = cuda_status(launch_tree_plan(a, s));
  return st != MLA_OK ? st : cuda_status(launch_tree_small_sm100(a, q, kv, kv_pv, s));
}

mla_status encode_tree(TreeMaps* m, const mla_tree_params* p, const TreeArgs& a) {
  const cuuint64_t rows = (cuuint64_t)p->T * p->n_h;
  const cuuint64_t kvrows = (cuuint64_t)p->num_pages * p->page_size;
  constexpr cuuint64_t kRow = 576 * 2;  // bytes of a cache or query row
  constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr auto k128 = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = true;
  {  // (column, row, 64-column block)
    const cuuint64_t dims[3] = {64, kvrows, 9}, strides[2] = {kRow, 128};
    const cuuint32_t box[3] = {64, 32, 9};
    ok &= encode(&m->k, kBf16, 3, p->kv_cache, dims, strides, box, k128);
  }
  {  // (column, row, block & 1, block >> 1): a CTA's columns 128 r + {0, 64, 256, 320} in one copy
    const cuuint64_t dims[4] = {192, kvrows, 2, 2}, strides[3] = {kRow, 128, 512};
    const cuuint32_t box[4] = {64, 64, 2, 2};
    ok &= encode(&m->v, kBf16, 4, p->kv_cache, dims, strides, box, k128);
  }
  {
    const cuuint64_t dims[3] = {64, rows, 9}, strides[2] = {kRow, 128};
    const cuuint32_t box[3] = {64, 64, 3};
    ok &= encode(&m->q, kBf16, 3, p->q, dims, strides, box, k128);
  }
  {  // 128-byte lines of 32 rows
    const cuuint64_t dims[2] = {512, rows}, strides[1] = {512u * (a.out_f32 ? 4 : 2)};
    const cuuint32_t box[2] = {a.out_f32 ? 32u : 64u, 32};
    ok &= encode(&m->u_out, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : kBf16, 2, p->u, dims, strides,
                 box, k128, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    const cuuint64_t pdims[2] = {512, 2ull * a.num_chunks * kTreeRows}, pstrides[1] = {512 * 4};
    const cuuint32_t pbox[2] = {32, 32};
    ok &= encode(&m->part_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.part_u, pdims, pstrides, pbox,
                 k128, CU_TENSOR_MAP_L2_PROMOTION_NONE);
  }
  return ok ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status mla_decode_tree_workspace_size(const mla_tree_params* p, size_t* bytes) {
  if (bytes == nullptr) return MLA_ERR_INVALID_ARG;
  mla_status st = validate_tree(p);
  if (st != MLA_OK) return st;
  const DeviceInfo* d = nullptr;
  if ((st = device_info(&d)) != MLA_OK) return st;
  if (tree_kernel(p, d) == TreeKernel::kNone) return MLA_ERR_UNSUPPORTED;
  *bytes = tree_ws_layout(p->B, p->d_c, tree_chunks(p, d)).total;
  return MLA_OK;
}

mla_status mla_decode_tree(const mla_tree_params* p, void* workspace, size_t workspace_bytes,
                           void* stream) {
  mla_status st = validate_tree(p);
  if (st != MLA_OK || p->B == 0 || p->T == 0) return st;
  const DeviceInfo* d = nullptr;
  if ((st = device_info(&d)) != MLA_OK) return st;
  if (tree_kernel(p, d) == TreeKernel::kNone) return MLA_ERR_UNSUPPORTED;
  const int G = tree_chunks(p, d);
  const TreeWsLayout L = tree_ws_layout(p->B, p->d_c, G);
  if (workspace_bytes < L.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MLA_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  TreeArgs a = {};
  a.q = p->q;
  a.kv = p->kv_cache;
  a.block_table = p->block_table;
  a.seqlens = p->seqlens;
  a.cu_q = p->cu_q;
  a.mask = reinterpret_cast<const unsigned long long*>(p->tree_mask);
  a.u = p->u;
  a.lse = p->lse;
  a.rec = reinterpret_cast<int*>(w + L.rec);
  a.seqs = reinterpret_cast<int4*>(w + L.seqs);
  a.up = reinterpret_cast<long long*>(w + L.up);
  a.cp = reinterpret_cast<int*>(w + L.cp);
  a.part_lse = reinterpret_cast<float*>(w + L.part_lse);
  a.part_u = reinterpret_cast<float*>(w + L.part_u);
  a.err = d->flags;
  a.B = p->B;
  a.T = p->T;
  a.n_h = p->n_h;
  a.d_c = p->d_c;
  a.d_R = p->d_R;
  a.page_size = p->page_size;
  a.max_pages = p->max_pages_per_seq;
  a.num_pages = p->num_pages;
  a.num_chunks = G;
  a.scale = p->softmax_scale;
  a.bf16 = p->dtype == MLA_DTYPE_BF16;
  a.out_f32 = p->u_fp32 != 0 || p->dtype == MLA_DTYPE_FP32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tree_kernel(p, d) == TreeKernel::kV3) {
    TreeMaps maps;
    if ((st = encode_tree(&maps, p, a)) != MLA_OK) return st;
    if ((st = cuda_status(launch_tree_plan(a, s))) != MLA_OK) return st;
    if ((st = cuda_status(launch_tree_sm100(a, maps, s))) != MLA_OK) return st;
  } else if ((st = plan_and_attend_small(p, a, s)) != MLA_OK) {
    return st;
  }
  return cuda_status(launch_tree_combine(a, s));
}

mla_status mla_build_tables(const mla_tables_params* p, void* stream) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->B < 0 || p->max_tokens < 0 || p->n_free < 0 || p->page_size < 1 ||
      p->max_pages_per_seq < 1 || p->num_pages < 1)
    return MLA_ERR_INVALID_ARG;
  if (p->B > kTablesMaxRequests || p->max_tokens > INT_MAX - 1024 || (long long)p->num_pages * p->page_size > INT_MAX ||
      (long long)p->max_pages_per_seq * p->page_size > INT_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (!p->free_used || !p->free_used_out || !p->cu_new || (p->n_free > 0 && !p->free_pages))
    return MLA_ERR_INVALID_ARG;
  if (p->B > 0 && (!p->ctx_lens || !p->new_lens || !p->block_table || !p->seqlens))
    return MLA_ERR_INVALID_ARG;
  if (p->max_tokens > 0 && (!p->seq_ids || !p->pos || !p->slots)) return MLA_ERR_INVALID_ARG;
  if ((p->parents != nullptr) != (p->tree_mask != nullptr)) return MLA_ERR_INVALID_ARG;
  if ((p->pages_held != nullptr) != (p->pages_held_out != nullptr)) return MLA_ERR_INVALID_ARG;
  const void* all[] = {p->ctx_lens, p->new_lens, p->pages_held, p->block_table, p->free_pages,
                       p->free_used, p->free_used_out, p->seqlens, p->cu_new, p->pages_held_out,
                       p->seq_ids, p->pos, p->slots, p->parents, p->tree_mask};
  for (const void* x : all)
    if (!aligned16(x)) return MLA_ERR_INVALID_ARG;
  // every block of the kernel reads the inputs while others write the outputs
  struct Range {
    const void* at;
    long long n;
    int size;
  };
  const long long B = p->B, N = p->max_tokens;
  const Range in[] = {{p->ctx_lens, B, 4}, {p->new_lens, B, 4}, {p->pages_held, B, 4},
                      {p->free_pages, p->n_free, 4}, {p->free_used, 1, 4}, {p->parents, N, 4}};
  const Range out[] = {{p->free_used_out, 1, 4}, {p->seqlens, B, 4}, {p->cu_new, B + 1, 4},
                       {p->pages_held_out, B, 4}, {p->seq_ids, N, 4}, {p->pos, N, 4},
                       {p->slots, N, 4}, {p->tree_mask, N, 8},
                       {p->block_table, B * p->max_pages_per_seq, 4}};
  for (const Range& x : in)
    for (const Range& y : out) {
      const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.at), y0 = reinterpret_cast<uintptr_t>(y.at);
      if (x0 != 0 && y0 != 0 && x0 < y0 + y.n * y.size && y0 < x0 + x.n * x.size)
        return MLA_ERR_INVALID_ARG;
    }
  const DeviceInfo* d = nullptr;
  mla_status st = device_info(&d);
  if (st != MLA_OK) return st;
  TablesArgs a = {};
  a.ctx_lens = p->ctx_lens;
  a.new_lens = p->new_lens;
  a.pages_held = p->pages_held;
  a.block_table = p->block_table;
  a.free_pages = p->free_pages;
  a.free_used = p->free_used;
  a.free_used_out = p->free_used_out;
  a.seqlens = p->seqlens;
  a.cu_new = p->cu_new;
  a.pages_held_out = p->pages_held_out;
  a.seq_ids = p->seq_ids;
  a.pos = p->pos;
  a.slots = p->slots;
  a.parents = p->parents;
  a.tree_mask = reinterpret_cast<long long*>(p->tree_mask);
  a.err = d->flags;
  a.B = p->B;
  a.max_pages = p->max_pages_per_seq;
  a.n_free = p->n_free;
  a.max_tokens = p->max_tokens;
  a.page_size = p->page_size;
  a.num_pages = p->num_pages;
  a.page_shift = -1;
  if ((p->page_size & (p->page_size - 1)) == 0)
    for (a.page_shift = 0; (1 << a.page_shift) < p->page_size;) ++a.page_shift;
  return cuda_status(launch_build_tables(a, d->sm_count, static_cast<cudaStream_t>(stream)));
}

mla_status mla_accept_tree(const mla_accept_params* p, void* stream) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 0 || p->width < 1 || !valid_dtype(p->dtype) || p->page_size < 1 ||
      p->max_pages_per_seq < 1 || p->num_pages < 1)
    return MLA_ERR_INVALID_ARG;
  const long long row_bytes = (long long)p->width * (p->dtype == MLA_DTYPE_BF16 ? 2 : 4);
  if (row_bytes % 16 != 0) return MLA_ERR_INVALID_ARG;
  if (row_bytes > INT_MAX || (long long)p->num_pages * p->page_size > INT_MAX ||
      (long long)p->max_pages_per_seq * p->page_size > INT_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (p->B == 0) return MLA_OK;
  if (!p->kv_cache || !p->block_table || !p->seqlens || !p->cu_q || !p->accepted || !p->seqlens_out ||
      (p->T > 0 && (!p->tree_mask || !p->path)))
    return MLA_ERR_INVALID_ARG;
  const void* all[] = {p->kv_cache, p->block_table, p->seqlens, p->cu_q, p->tree_mask, p->accepted,
                       p->seqlens_out, p->path};
  for (const void* x : all)
    if (!aligned16(x)) return MLA_ERR_INVALID_ARG;
  const DeviceInfo* d = nullptr;
  mla_status st = device_info(&d);
  if (st != MLA_OK) return st;
  AcceptArgs a = {};
  a.kv_cache = static_cast<uint8_t*>(p->kv_cache);
  a.block_table = p->block_table;
  a.seqlens = p->seqlens;
  a.cu_q = p->cu_q;
  a.tree_mask = reinterpret_cast<const long long*>(p->tree_mask);
  a.accepted = p->accepted;
  a.seqlens_out = p->seqlens_out;
  a.path = p->path;
  a.err = d->flags;
  a.B = p->B;
  a.T = p->T;
  a.row_bytes = (int)row_bytes;
  a.max_pages = p->max_pages_per_seq;
  a.page_size = p->page_size;
  a.num_pages = p->num_pages;
  return cuda_status(launch_accept_tree(a, static_cast<cudaStream_t>(stream)));
}

mla_status mla_append_latent_slots(const void* h, const void* W_DKV, const void* W_KR,
                                   const int* slots, const int* pos, void* kv_cache, int cache_rows,
                                   int T, int d_model, int d_c, int d_R, float rope_base,
                                   mla_dtype dtype, void* stream) {
  if (!valid_dtype(dtype) || T < 0 || cache_rows < 1 || d_model < 1 || d_c < 8 || d_c % 8 != 0 ||
      d_R < 0 || d_R % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  if (!(rope_base > 0.f) || !std::isfinite(rope_base)) return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  if (!h || !W_DKV || !slots || !kv_cache || (d_R > 0 && (!W_KR || !pos))) return MLA_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(W_DKV) || !aligned16(W_KR) || !aligned16(slots) || !aligned16(pos) ||
      !aligned16(kv_cache))
    return MLA_ERR_INVALID_ARG;
  // the grids' limits: 65535 tiles of 128 tokens, as many of 32 features
  if (T > 65535 * 128 || (long long)d_c + d_R > 65535 * 32 - 64) return MLA_ERR_UNSUPPORTED;
  const DeviceInfo* d = nullptr;
  mla_status st = device_info(&d);
  if (st != MLA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AppendSlotsArgs a = {};
  a.cache = kv_cache;
  a.slots = slots;
  a.pos = pos;
  a.err = d->flags;
  a.T = T;
  a.d_model = d_model;
  a.d_c = d_c;
  a.d_R = d_R;
  a.rows = cache_rows;
  a.max_clusters = d->append_clusters;
  a.rope_base = rope_base;
  if (dtype == MLA_DTYPE_FP32)
    return cuda_status(launch_append_slots_f32(a, static_cast<const float*>(h),
                                               static_cast<const float*>(W_DKV),
                                               static_cast<const float*>(W_KR), s));
  if (!d->append_tc || g_encode == nullptr || d_model % 64 != 0) return MLA_ERR_UNSUPPORTED;
  auto rows_map = [&](CUtensorMap* m, const void* ptr, int rows, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)d_model, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d_model * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap w_dkv, w_kr, x;
  if (!rows_map(&w_dkv, W_DKV, d_c, 32) || !rows_map(&x, h, T, append_slots_rows(T)))
    return MLA_ERR_CUDA;
  w_kr = w_dkv;
  if (d_R > 0 && !rows_map(&w_kr, W_KR, d_R, 32)) return MLA_ERR_CUDA;
  return cuda_status(launch_append_slots(a, w_dkv, w_kr, x, s));
}

}  // extern "C"
