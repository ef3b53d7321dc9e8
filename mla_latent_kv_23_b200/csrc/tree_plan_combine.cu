// Plan and combine stages of mla_decode_tree.
//
// plan (one block): validates every sequence, and cuts the line of all row
// blocks' tiles into chunks.  Two cuts:
//   * pieces: with no more row blocks than chunks, block v of t tiles gets
//     1 + floor((chunks - blocks) t / (all tiles)) chunks of its own (at
//     most one per two tiles, and one up to kWholeTiles), so that no chunk holds two blocks; the sum stays within the chunks;
//   * line: every block takes kTreeSegTiles + t units (a chunk that enters one
//     more block pays for its queries and its output), the line is cut into
//     equal units, and a cut that would leave kSnap tiles or fewer of a block
//     on one side moves to that block's edge.
// The pieces are taken where their longest is no longer than a chunk of the
// line plus one block's start charge.
//
// combine: the pieces of a block that several chunks share are merged by their
// log-sum-exp (exact algebra of the softmax): lse = log sum exp(lse_s),
// u = sum exp(lse_s - lse) u_s, in fp32.  One CTA takes 8 rows of the block
// that is cut at the end of "its" chunk and begins there; the number of pieces
// is read off the chunk records.  Rows of a sequence whose length is out of
// range get u = 0 and lse = -inf.
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include "sm100_ptx.cuh"
#include "tree.h"
#include "tree_schedule.cuh"

namespace mla {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanSmemSeqs = 2048;  // batches up to this size keep the prefix sums on chip
constexpr int kSnap = 2;
// A block of up to four tiles is not cut into pieces, and pieces have two tiles
// or more: a tile takes 1 us, partial results and their merge 2 to 4 (one block
// of 2 tiles: 12.8 us whole, 14.1 cut; 4 tiles: 14.7 either way; 8 tiles: 18.7
// whole, 15.3 in four pieces, 15.8 in eight).
constexpr int kWholeTiles = 4;

// Inclusive scan of one value per thread; *total gets the block's sum.
__device__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  __syncthreads();
  return before + x;
}

__global__ void __launch_bounds__(kPlanThreads)
    tree_plan_kernel(const int* __restrict__ cu_q, const int* __restrict__ seqlens, int B, int T,
                     int n_h, long long max_len, int num_chunks, int* rec, int4* seqs,
                     long long* up_ws, int* cp_ws, int* err) {
  ptx::pdl_launch_dependents();
  __shared__ long long warp_sums[kPlanThreads / 32];
  __shared__ long long up_s[kPlanSmemSeqs + 1];
  __shared__ int cp_s[kPlanSmemSeqs + 1];
  __shared__ int longest_piece;
  constexpr int K = kTreeSegTiles;
  const bool on_chip = B <= kPlanSmemSeqs;
  long long* up = on_chip ? up_s : up_ws;  // units before place k of the list on the line
  int* cp = on_chip ? cp_s : cp_ws;        // chunks before place k when cut into pieces
  long long units_all = 0, blocks_all = 0, total;
  int listed = 0;
  int flags = 0;
  if (threadIdx.x == 0) longest_piece = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    TreeSeq s = {};
    if (i < B) s = tree_seq(cu_q, seqlens, i, T, n_h, max_len);
    flags |= s.flag;
    const long long units = (long long)s.blocks * (s.tiles + K);
    const long long incl = block_scan(units, warp_sums, &total);
    const int work = s.blocks > 0;
    // row blocks (high half) and sequences with work (low half)
    long long both;
    const long long at = block_scan(((long long)s.blocks << 32) | work, warp_sums, &both);
    if (work) {
      const int k = listed + (int)(at & 0xffffffff) - 1;
      seqs[k] = make_int4(s.row0, s.n, s.L, i);
      up[k] = units_all + incl - units;
    }
    units_all += total;
    blocks_all += both >> 32;
    listed += (int)(both & 0xffffffff);
  }
  if (flags) atomicOr(err, flags);
  if (threadIdx.x == 0) up[listed] = units_all;
  __syncthreads();
  const long long tiles_all = units_all - K * blocks_all;
  const long long per = units_all > 0 ? (units_all + num_chunks - 1) / num_chunks : 1;
  const bool fits = blocks_all > 0 && blocks_all <= num_chunks;
  // pieces of each of a sequence's blocks
  auto pieces = [&](const TreeSeq& s) -> int {
    if (s.tiles <= kWholeTiles) return 1;
    const long long n = 1 + (num_chunks - blocks_all) * s.tiles / tiles_all;
    return (int)min(n, (long long)(s.tiles + 1) / 2);
  };
  if (fits) {
    long long chunks = 0;
    for (int base = 0; base < listed; base += kPlanThreads) {
      const int k = base + threadIdx.x;
      int n = 0;
      if (k < listed) {
        const TreeSeq s = tree_listed(seqs[k], n_h);
        const int p = pieces(s);
        n = p * s.blocks;
        atomicMax(&longest_piece, (s.tiles + p - 1) / p);
      }
      const long long incl = block_scan(n, warp_sums, &total);
      if (k < listed) cp[k] = (int)(chunks + incl - n);
      chunks += total;
    }
    if (threadIdx.x == 0) cp[listed] = (int)chunks;
  }
  __syncthreads();
  const bool cut_pieces = fits && longest_piece <= per + K;
  for (int c = threadIdx.x; c <= num_chunks; c += kPlanThreads) {
    int k = listed, g = 0, t = 0;
    int4 first = make_int4(0, 0, 0, 0);
    if (cut_pieces ? c < cp[listed] : c * per < units_all) {
      const long long x = cut_pieces ? c : c * per;
      int lo = 0, hi = listed;  // the largest k that starts at or before x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((cut_pieces ? (long long)cp[mid] : up[mid]) <= x) lo = mid; else hi = mid;
      }
      k = lo;
      first = seqs[k];
      const TreeSeq s = tree_listed(first, n_h);
      if (cut_pieces) {
        const int p = pieces(s), i = c - cp[k];
        g = i / p;
        t = (int)((long long)(i % p) * s.tiles / p);
      } else {
        const long long off = x - up[k];
        g = (int)(off / (s.tiles + K));
        t = (int)(off % (s.tiles + K)) - K;
        if (t <= kSnap) {
          t = 0;
        } else if (s.tiles - t <= kSnap) {
          t = 0;
          ++g;  // past the sequence's last block: the walk goes on to the next one
        }
      }
    }
    int4* r = reinterpret_cast<int4*>(rec) + 2 * c;
    r[0] = make_int4(k, g, t, 0);
    r[1] = first;
  }
}

constexpr int kCombineWarps = 8;
constexpr int kCombineThreads = 32 * kCombineWarps;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool kOutBf16>
__device__ __forceinline__ void store4(void* u, size_t at, float4 v) {
  if (kOutBf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(u) + at) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(u) + at) = v;
  }
}

// Grid (16, chunks): 8 rows of the block that begins in chunk y and is cut at
// its end.  One warp per row; lane l owns columns 4 l + 128 j, j < kVecs, below
// d_c.
template <bool kOutBf16, int kVecs>
__global__ void __launch_bounds__(kCombineThreads)
    tree_combine_kernel(const int* __restrict__ rec, const int* __restrict__ cu_q,
                        const int* __restrict__ seqlens, const float* __restrict__ part_u,
                        const float* __restrict__ part_lse, void* __restrict__ u_out,
                        float* __restrict__ lse_out, int B, int T, int n_h, int d_c,
                        long long max_len, int num_chunks) {
  constexpr int kGroup = 4;  // partial rows requested at a time
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.y;
  auto mine = [&](int j) { return 4 * lane + 128 * j < d_c; };
  // sequences whose length is out of range
  for (long long b = (long long)c * gridDim.x + blockIdx.x; b < B; b += (long long)gridDim.x * gridDim.y) {
    const TreeSeq s = tree_seq(cu_q, seqlens, (int)b, T, n_h, max_len);
    if (s.flag != MLA_DEVFLAG_BAD_SEQLEN) continue;
    for (int r = warp; r < s.n * n_h; r += kCombineWarps) {
      const size_t row = (size_t)s.row0 * n_h + r;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (mine(j)) store4<kOutBf16>(u_out, row * d_c + 4 * lane + 128 * j, make_float4(0.f, 0.f, 0.f, 0.f));
      if (lane == 0 && lse_out != nullptr) lse_out[row] = -INFINITY;
    }
  }
  const int4* r = reinterpret_cast<const int4*>(rec);
  const int4 start = r[2 * c], end = r[2 * c + 2], seq = r[2 * c + 3];
  if (end.z == 0) return;  // not cut inside a block
  if (start.x == end.x && start.y == end.y && start.z > 0) return;  // it began in an earlier chunk
  // the chunks after this one that also end inside the block
  int pieces = 2;
  for (int d0 = c + 2; d0 <= num_chunks; d0 += 32) {
    int4 e = make_int4(-1, 0, 0, 0);
    if (d0 + lane <= num_chunks) e = r[2 * (d0 + lane)];
    const uint32_t same =
        __ballot_sync(0xffffffffu, e.x == end.x && e.y == end.y && e.z > 0);
    const int run = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
    pieces += run;
    if (run < 32) break;
  }
  const int i = blockIdx.x * kCombineWarps + warp;  // row of the block
  if (i >= min(kTreeRows, seq.y * n_h - end.y * kTreeRows)) return;
  // slot of piece k: 2c + 1, then 2 (c + 1), 2 (c + 2), ...
  auto prow = [&](int k) -> size_t {
    return (size_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * kTreeRows + i;
  };
  float4 v[kGroup][kVecs];
  auto load_group = [&](int k0) {
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
      if (k0 + k < pieces) {
        const float* src = part_u + prow(k0 + k) * d_c + 4 * lane;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
          if (mine(j)) v[k][j] = *reinterpret_cast<const float4*>(src + 128 * j);
      }
  };
  // the first partial rows are requested together with the statistics
  load_group(0);
  float m = -INFINITY, z = 0.f;
  for (int k = lane; k < pieces; k += 32) {
    const float x = part_lse[prow(k)];
    if (x > m) {
      z = z * expf(m - x) + 1.f;
      m = x;
    } else if (x != -INFINITY) {
      z += expf(x - m);
    }
  }
  const float m_all = warp_max(m);
  // (a NaN statistic of a row with non-finite scores stays in z)
  z = warp_sum(m == -INFINITY ? z : z * expf(m - m_all));
  const float lse = z == 0.f ? -INFINITY : m_all + logf(z);
  float4 acc[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lse != -INFINITY)
    for (int k0 = 0; k0 < pieces; k0 += kGroup) {
      if (k0 > 0) load_group(k0);
      const float w_me = lane < kGroup && k0 + lane < pieces ? expf(part_lse[prow(k0 + lane)] - lse) : 0.f;
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        const float w = __shfl_sync(0xffffffffu, w_me, k);
        if (k0 + k < pieces) {
#pragma unroll
          for (int j = 0; j < kVecs; ++j) {
            acc[j].x += w * v[k][j].x;
            acc[j].y += w * v[k][j].y;
            acc[j].z += w * v[k][j].z;
            acc[j].w += w * v[k][j].w;
          }
        }
      }
    }
  const size_t row = (size_t)seq.x * n_h + (size_t)end.y * kTreeRows + i;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (mine(j)) store4<kOutBf16>(u_out, row * d_c + 4 * lane + 128 * j, acc[j]);
  if (lane == 0 && lse_out != nullptr) lse_out[row] = lse;
}

}  // namespace

TreeWsLayout tree_ws_layout(int B, int d_c, int num_chunks) {
  auto up256 = [](size_t x) { return (x + 255) / 256 * 256; };
  TreeWsLayout L;
  size_t off = 0;
  L.rec = off;
  off = up256(off + sizeof(int) * 8 * ((size_t)num_chunks + 1));
  L.seqs = off;
  off = up256(off + sizeof(int) * 4 * (size_t)B);
  L.up = off;
  off = up256(off + sizeof(long long) * ((size_t)B + 1));
  L.cp = off;
  off = up256(off + sizeof(int) * ((size_t)B + 1));
  L.part_lse = off;
  off = up256(off + sizeof(float) * 2 * (size_t)num_chunks * kTreeRows);
  L.part_u = off;
  off = up256(off + sizeof(float) * 2 * (size_t)num_chunks * kTreeRows * d_c);
  L.total = off;
  return L;
}

cudaError_t launch_tree_plan(const TreeArgs& a, cudaStream_t s) {
  tree_plan_kernel<<<1, kPlanThreads, 0, s>>>(a.cu_q, a.seqlens, a.B, a.T, a.n_h,
                                              (long long)a.max_pages * a.page_size, a.num_chunks,
                                              a.rec, a.seqs, a.up, a.cp, a.err);
  return cudaGetLastError();
}

cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kTreeRows / kCombineWarps, a.num_chunks, 1);
  cfg.blockDim = dim3(kCombineThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, (const int*)a.rec, a.cu_q, a.seqlens,
                              (const float*)a.part_u, (const float*)a.part_lse, a.u, a.lse, a.B,
                              a.T, a.n_h, a.d_c, (long long)a.max_pages * a.page_size, a.num_chunks);
  };
  if (a.d_c <= 256) return a.out_f32 ? go(tree_combine_kernel<false, 2>) : go(tree_combine_kernel<true, 2>);
  return a.out_f32 ? go(tree_combine_kernel<false, 4>) : go(tree_combine_kernel<true, 4>);
}

}  // namespace mla
