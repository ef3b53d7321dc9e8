// Paged-cache bookkeeping of a speculative-decoding step, on the GPU:
//   mla_build_tables  pages for the requests' new tokens from a free list, and a
//                     cache row, a position and (for drafted trees) an ancestor
//                     mask for every new token;
//   mla_accept_tree   the cache rows of an accepted branch moved to the front
//                     of its tree's rows.
// Both are bound by latency: a few KB to a few MB of integers or rows.
#include <climits>

#include "mla.h"
#include "tables.h"
#include "tree.h"
#include "tree_schedule.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------------ tables
// One launch without any exchange between blocks: every block computes the
// prefix sums over all requests (new tokens and new pages; 512 threads, a run
// of consecutive requests each) into shared memory, and its warps then take
// jobs of two kinds:
//   request b:     its new block-table entries and, if it is a drafted tree,
//                  positions and masks of its tokens (a prompt: masks of 0);
//   token slice k: sequence, row and (where the request is no tree) position of
//                  tokens [128 k, 128 k + 128), four per lane.
// A new page is read from the free list wherever it is needed, so no job waits
// for another's block-table entry.
constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kSlice = 128;

struct Request {
  int ctx, n;       // cached and new tokens (a refused request: its cached ones, if those are in order, and 0)
  int have, want;   // pages before and after
  bool bad;
};

// Page of a position (a shift where the page size is a power of two: a
// division is a tenth of the small calls' time on the GPU).
__device__ __forceinline__ int page_of(const TablesArgs& a, int p) {
  return a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size;
}

// A refused request is as it was, so that the step's outputs can be the next
// one's inputs: the pages that it holds stay its own (without pages_held nothing
// says which those are), and so does its length where that is in order itself.
__device__ __forceinline__ Request request(const TablesArgs& a, int b) {
  Request r;
  r.ctx = a.ctx_lens[b];
  r.n = a.new_lens[b];
  const int max_len = a.max_pages * a.page_size;
  bool keep = r.ctx >= 0 && r.ctx <= max_len;  // the length is in order
  r.bad = !keep || r.n < 0 || r.n > max_len - r.ctx;
  r.have = !keep || r.ctx == 0 ? 0 : page_of(a, r.ctx - 1) + 1;
  if (a.pages_held != nullptr) {
    const int held = a.pages_held[b];
    keep = keep && held >= r.have && held <= a.max_pages;
    r.bad = r.bad || !keep;
    r.have = held;
  }
  if (!r.bad) {
    const int L = r.ctx + r.n;
    r.want = max(r.have, L == 0 ? 0 : page_of(a, L - 1) + 1);
    return r;
  }
  if (a.pages_held == nullptr) {
    keep = false;
    r.have = 0;
  } else if (r.have < 0 || r.have > a.max_pages) {
    r.have = 0;
  }
  if (!keep) r.ctx = 0;
  r.n = 0;
  r.want = r.have;
  return r;
}

// Inclusive block scan of a pair.
__device__ void scan2(long long& x, long long& y, long long (*sums)[2], long long* tx, long long* ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    sums[warp][0] = x;
    sums[warp][1] = y;
  }
  __syncthreads();
  long long bx = 0, by = 0;
  *tx = *ty = 0;
#pragma unroll
  for (int w = 0; w < kTabWarps; ++w) {
    if (w < warp) {
      bx += sums[w][0];
      by += sums[w][1];
    }
    *tx += sums[w][0];
    *ty += sums[w][1];
  }
  x += bx;
  y += by;
}

// Entry k of a request's block table, k below its page count: as it is, or
// from the free list.  -1 where the list ran out or the id is out of range.
__device__ __forceinline__ int page_at(const TablesArgs& a, int b, int k, int have, long long first,
                                       int& flags) {
  int page;
  if (k < have) {
    page = a.block_table[(size_t)b * a.max_pages + k];
  } else {
    const long long f = first + (k - have);
    if (f >= a.n_free) {
      flags |= MLA_DEVFLAG_NO_PAGES;
      return -1;
    }
    page = a.free_pages[f];
  }
  if (page < 0 || page >= a.num_pages) {
    flags |= MLA_DEVFLAG_BAD_PAGE;
    return -1;
  }
  return page;
}

__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int smem[];
  int* cu = smem;               // [B + 1] new tokens before request b (saturated)
  int* pg = smem + a.B + 1;     // [B] new pages before request b (saturated)
  __shared__ long long sums[kTabWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.B + kTabThreads - 1) / kTabThreads;
  const int i0 = min(a.B, (int)threadIdx.x * per), i1 = min(a.B, i0 + per);
  int flags = 0;
  int used = *a.free_used;
  long long tok = 0, pages = 0;
  for (int i = i0; i < i1; ++i) {
    const Request r = request(a, i);
    if (r.bad) flags |= MLA_DEVFLAG_BAD_SEQLEN;
    tok += r.n;
    pages += r.want - r.have;
  }
  long long it = tok, ip = pages, all_tok, all_pages;
  scan2(it, ip, sums, &all_tok, &all_pages);
  it -= tok;
  ip -= pages;
  for (int i = i0; i < i1; ++i) {
    const Request r = request(a, i);
    cu[i] = (int)min(it, (long long)INT_MAX);
    pg[i] = (int)min(ip, (long long)INT_MAX);
    it += r.n;
    ip += r.want - r.have;
  }
  if (threadIdx.x == 0) cu[a.B] = (int)min(all_tok, (long long)INT_MAX);
  __syncthreads();
  if (used < 0 || used > a.n_free) {
    if (all_pages > 0) flags |= MLA_DEVFLAG_NO_PAGES;
    used = a.n_free;  // nothing is free
  }
  const int total = (int)min(all_tok, (long long)a.max_tokens);  // tokens that are written
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      *a.free_used_out = (int)min((long long)a.n_free, used + all_pages);
      if (all_tok > a.max_tokens) flags |= MLA_DEVFLAG_NO_ROOM;
    }
    for (int i = threadIdx.x; i <= a.B; i += kTabThreads) {
      a.cu_new[i] = cu[i];
      if (i < a.B) {
        const Request r = request(a, i);
        a.seqlens[i] = r.ctx + r.n;
        // held are the pages that the list had; the request's other new
        // entries are -1 and taken by a later step
        if (a.pages_held_out != nullptr)
          a.pages_held_out[i] = r.have + (int)min((long long)(r.want - r.have), max(0ll, a.n_free - ((long long)used + pg[i])));
      }
    }
  }
  const bool trees = a.parents != nullptr;
  const int slices = (total + kSlice - 1) / kSlice;
  const long long jobs = (long long)a.B + slices;
  for (long long job = (long long)warp * gridDim.x + blockIdx.x; job < jobs; job += (long long)kTabWarps * gridDim.x) {
    if (job < a.B) {
      const int b = (int)job;
      const Request r = request(a, b);
      const int t0 = cu[b];
      const bool tree = trees && t0 < total && r.n <= kTreeMaxNodes;
      // tokens lane and lane + 32 of a tree: their parents are on their way
      // while the pages are looked up
      int up[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        up[h] = tree && i < r.n && t0 + i < total ? a.parents[t0 + i] : -1;
      }
      const long long first = (long long)used + pg[b];
      for (int k = r.have + lane; k < r.want; k += 32) {
        const int page = page_at(a, b, k, r.have, first, flags);
        a.block_table[(size_t)b * a.max_pages + k] = page;
      }
      if (!trees || t0 >= total) continue;
      if (!tree) {  // a prompt: no branches
        for (int i = lane; i < min(r.n, total - t0); i += 32) a.tree_mask[t0 + i] = 0;
        continue;
      }
      // branches of 1, 2, 4 ... 64 tokens, joined with the branch that ends
      // where they begin.  A token without a parent points at itself.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        if (up[h] < -1 || up[h] >= i) {
          flags |= MLA_DEVFLAG_BAD_TREE;
          up[h] = -1;
        }
        if (up[h] < 0) up[h] = i;
      }
      unsigned long long m[2];
      if (r.n <= 32) {
        uint32_t mask = 1u << lane;
        int u = up[0];
        for (int d = 1; d < r.n; d <<= 1) {
          mask |= __shfl_sync(0xffffffffu, mask, u);
          u = __shfl_sync(0xffffffffu, u, u);
        }
        m[0] = mask;
        m[1] = 0;
      } else {
        m[0] = 1ull << lane;
        m[1] = 1ull << (lane + 32);
        for (int d = 1; d < r.n; d <<= 1) {
          unsigned long long jm[2];
          int ju[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned long long lo = __shfl_sync(0xffffffffu, m[0], up[h] & 31);
            const unsigned long long hi = __shfl_sync(0xffffffffu, m[1], up[h] & 31);
            const int ulo = __shfl_sync(0xffffffffu, up[0], up[h] & 31);
            const int uhi = __shfl_sync(0xffffffffu, up[1], up[h] & 31);
            jm[h] = up[h] < 32 ? lo : hi;
            ju[h] = up[h] < 32 ? ulo : uhi;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            m[h] |= jm[h];
            up[h] = ju[h];
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        if (i < r.n && t0 + i < total) {
          a.tree_mask[t0 + i] = (long long)m[h];
          a.pos[t0 + i] = r.ctx + __popcll(m[h]) - 1;
        }
      }
      continue;
    }
    // four consecutive tokens per lane
    const int t0 = (int)(job - a.B) * kSlice + 4 * lane;
    if (t0 >= total) continue;
    int lo = 0, hi = a.B;  // the largest b with cu[b] <= t0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t0) lo = mid; else hi = mid;
    }
    int b = lo;
    Request r = request(a, b);
    int page = -1, page_k = -1;
    int seq[4], row[4], pos[4];
    bool tree[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + e;
      if (t < total) {
        if (t >= cu[b + 1]) {
          do ++b; while (t >= cu[b + 1]);
          r = request(a, b);
          page_k = -1;
        }
        const int q = r.ctx + (t - cu[b]), k = page_of(a, q);
        if (k != page_k) {
          page = page_at(a, b, k, r.have, (long long)used + pg[b], flags);
          page_k = k;
        }
        seq[e] = b;
        pos[e] = q;
        row[e] = page < 0 ? -1 : page * a.page_size + (q - k * a.page_size);
        tree[e] = trees && r.n <= kTreeMaxNodes;
      }
    }
    if (t0 + 4 <= total) {
      *reinterpret_cast<int4*>(a.seq_ids + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(row[0], row[1], row[2], row[3]);
      if (!(tree[0] || tree[1] || tree[2] || tree[3])) {
        *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!tree[e]) a.pos[t0 + e] = pos[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t0 + e < total) {
          a.seq_ids[t0 + e] = seq[e];
          a.slots[t0 + e] = row[e];
          if (!tree[e]) a.pos[t0 + e] = pos[e];
        }
    }
  }
  if (flags) atomicOr(a.err, flags);
}

// ------------------------------------------------------------------ accept
// One block per sequence.  Thread (i, k) holds 16-byte chunk k of the 128-byte
// slices of tree row i: all its reads come before the block's barrier and all
// its writes after it, so that a row may be both a source and a target.  Row i
// goes to the place of bit i among the accepted token's mask bits.
constexpr int kAccThreads = kTreeMaxNodes * 8;
constexpr int kAccSlices = 9;  // 1152 bytes a pass: a bf16 row of 576 values

__global__ void __launch_bounds__(kAccThreads) accept_tree_kernel(const __grid_constant__ AcceptArgs a) {
  const int b = blockIdx.x;
  const int i = threadIdx.x >> 3, k = threadIdx.x & 7;
  const TreeSeq seq = tree_seq(a.cu_q, a.seqlens, b, a.T, 1, (long long)a.max_pages * a.page_size);
  const int node = a.accepted[b];
  const int row0 = seq.row0, n = seq.n, L = seq.L;
  int flags = seq.flag;
  const bool good = flags != MLA_DEVFLAG_BAD_SEQLEN;
  if (node < -1 || node >= n) flags |= MLA_DEVFLAG_BAD_TREE;
  unsigned long long mask = 0;
  if (good && node >= 0 && node < n) mask = (unsigned long long)a.tree_mask[row0 + node];
  if (n < 64) mask &= (1ull << n) - 1;
  const int kept = __popcll(mask);
  const int to = __popcll(mask & ((1ull << i) - 1));
  const bool mine = (mask >> i) & 1;
  // the cache row of a position
  auto row_of = [&](int p) -> long long {
    const int page = a.block_table[(size_t)b * a.max_pages + p / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      flags |= MLA_DEVFLAG_BAD_PAGE;
      return -1;
    }
    return (long long)page * a.page_size + p % a.page_size;
  };
  long long src = -1, dst = -1;
  if (mine && to != i) {
    src = row_of(L - n + i);
    dst = row_of(L - n + to);
  }
  const bool move = src >= 0 && dst >= 0;
  const int chunks = a.row_bytes / 16;
  for (int c0 = 0; c0 < chunks; c0 += 8 * kAccSlices) {
    uint4 v[kAccSlices];
    if (move) {
      const uint4* from = reinterpret_cast<const uint4*>(a.kv_cache + src * a.row_bytes);
#pragma unroll
      for (int s = 0; s < kAccSlices; ++s)
        if (c0 + 8 * s + k < chunks) v[s] = from[c0 + 8 * s + k];
    }
    __syncthreads();
    if (move) {
      uint4* into = reinterpret_cast<uint4*>(a.kv_cache + dst * a.row_bytes);
#pragma unroll
      for (int s = 0; s < kAccSlices; ++s)
        if (c0 + 8 * s + k < chunks) into[c0 + 8 * s + k] = v[s];
    }
  }
  if (k == 0 && n > 0) {
    // the branch, then -1: token i takes place `to`, and the last n - kept
    // places are free
    if (mine) a.path[row0 + to] = i;
    if (i >= kept && i < n) a.path[row0 + i] = -1;
  }
  if (threadIdx.x == 0) a.seqlens_out[b] = good ? L - n + kept : L;
  if (flags) atomicOr(a.err, flags);
}

}  // namespace

cudaError_t tables_prepare() {
  return cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (2 * kTablesMaxRequests + 1) * (int)sizeof(int));
}

cudaError_t launch_build_tables(const TablesArgs& a, int sm_count, cudaStream_t s) {
  const long long jobs = (long long)a.B + (a.max_tokens + kSlice - 1) / kSlice;
  // one warp per job up to two blocks per SM (a block more costs one more
  // computation of the prefix sums)
  const long long blocks = (jobs + kTabWarps - 1) / kTabWarps;
  const int grid = (int)(blocks < 1 ? 1 : blocks < 2 * sm_count ? blocks : 2 * sm_count);
  build_tables_kernel<<<grid, kTabThreads, (2 * (size_t)a.B + 1) * sizeof(int), s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_accept_tree(const AcceptArgs& a, cudaStream_t s) {
  accept_tree_kernel<<<a.B, kAccThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
