// Attend stage of mla_decode_tree on the 5th-generation tensor cores (sm_100a)
// at the DeepSeek-V3 shape: latent d_c = 512, RoPE key d_R = 64, bf16.
//
// Math ("MLA deep compression", absorption section, both equations, and its
// decoupled-RoPE section), for token r of a tree of n drafted tokens that are
// the last n of a sequence's L cached ones, and for every head:
//     s_j = q . [c_j || k^R_j],  seen where j < L - n or bit j - (L - n) of mask_r
//     u   = sum_j softmax(scale s)_j c_j
// The n n_h query rows of a sequence are flat (token-major) and taken in
// blocks of 128: all rows of a block share every cached row, so they are the M
// dimension of two dense contractions per 64-token tile,
//     S = Q . [C || K^R]^T      (K = 576)
//     O = O * alpha + P . C     (N = 512 latent)
// with an online softmax between them; u = O / l at the end.  Few heads fill a
// block with several tokens of the tree, so that a cached row is read once
// for them.
//
// What bounds it: 128 rows take 278.5 kflop for each 1152-byte cached row,
// 242 flop/B, the ridge of this part: at one block a sequence the HBM and the
// tensor roofline meet, at more blocks the tile comes from L2 and the tensor
// cores bound it; long calls run at the power limit, where energy does.  O of
// 128 rows and 512 columns in fp32 fills the tensor memory of one SM, so a pair
// of CTAs (one 2-CTA cluster) shares a block, CTA r owning rows [64r, 64r + 64),
// and all tensor work is paired (cta_group::2):
//  * P . C is one MMA per 16 tokens and 256 columns (M = 128, N = 256): CTA r
//    supplies latent columns [128r, 128r + 128) and [256 + 128r, 256 + 128r +
//    128) of all 64 tokens of the tile (the V copy, 32 KB).
//  * S takes all 576 columns (M = 128, N = 64, 36 steps): CTA r supplies tokens
//    [32r, 32r + 32) of the tile (the K copy, 36 KB).
// An MMA reads its B operand at one shared-memory address in both CTAs, so the
// two copies cannot share their common part: a tile comes from L2 twice.  The
// form with one copy (S split by columns alone, the halves' sums added in the
// softmax) discards half of S's products and reads three fifths of the bytes: 16
// trees of 64 tokens over 4096 took 1378 us in that form and 1210 in this one, 6
// tokens over 4 x 128 Ki 1132 and 1027, 37 over 32 Ki 362 and 328, 16 single
// tokens over 4096 42.9 and 42.8.
//
// The mask is one 64-bit word per token: a tile that reaches into the drafted
// tokens shifts it to the tile's positions.  A drafted token's cache row may
// hold infinities or NaN that a row which does not see it must not meet (0 x
// NaN in P . C): every row's raw score of such a token is then non-finite, so
// the softmax finds it there and clears the non-finite values of that cache
// row in shared memory before P . C; rows that see the token get NaN by their
// weight.
//
// TMEM per CTA (512 columns): S 2 x 32 | O 256.  S and O have the layout of a
// paired MMA with M = 128: lane l holds row l % 64, of columns (tokens) in
// half l / 64 of N.  So a softmax thread has one row and 32 of a tile's tokens,
// and the same row's O.
// Shared memory per CTA: Q (64 rows x 576 values, the S operand A) 72 KB; two K
// slots of 36 KB (read by S alone, refilled at once); two V slots of 32 KB
// (loaded one tile behind); two P slots of 8 KB (64 rows x 64 tokens bf16).
//
// Roles (384 threads): warp 0 = queries and K copies; warp 1 = S issuer and
// warp 2 = P . C issuer (even CTA); warp 3 = V copies; warps 4-11 = softmax, two
// groups of four that take alternate tiles.
//
// Epilogue: u = O / l leaves TMEM through the V slots by TMA stores of whole
// 128-byte lines, or row by row where fewer than a warp's 32 rows exist (the
// rows behind belong to the next sequence).  Pieces of split blocks are written
// in fp32.  The next segment's queries, its first K copies and their S go on
// meanwhile; what waits is its first V copy, for the stores to have read the
// slots, and its first P . C, for every softmax warp to have read O.
#include <cuda_bf16.h>
#include <math.h>

#include "sm100_ptx.cuh"
#include "tree.h"
#include "tree_schedule.cuh"

namespace mla {
namespace {
using namespace ptx;

constexpr int kThreads = 384;
constexpr int kWarpK = 0, kWarpMma = 1, kWarpAlloc = 2, kWarpV = 3, kWarpSoftmax0 = 4;
constexpr int kDc = 512;

constexpr uint32_t kQBlk = 64 * 128;            // 64 rows x 64 columns
constexpr uint32_t kQBytes = 9 * kQBlk;         // 73728
constexpr uint32_t kKBlk = 32 * 128;            // 32 tokens x 64 columns
constexpr uint32_t kKBytes = 9 * kKBlk;         // 36864
constexpr uint32_t kVBlk = 64 * 128;            // 64 tokens x 64 columns
constexpr uint32_t kVBytes = 4 * kVBlk;         // 32768
constexpr uint32_t kPBytes = 64 * 128;          // 64 rows x 64 tokens
// (all with 128-byte swizzle)

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + kQBytes;              // [2]
constexpr uint32_t kOffV = kOffK + 2 * kKBytes;          // [2]
constexpr uint32_t kOffP = kOffV + 2 * kVBytes;          // [2]
constexpr uint32_t kOffMax = kOffP + 2 * kPBytes;        // float [2 tile parity][64 rows]
constexpr uint32_t kOffEx = kOffMax + 2 * 64 * 4;        // float [2][2 group][2 half][64 rows]
constexpr uint32_t kOffScratch = kOffEx + 2 * 2 * 2 * 64 * 4;  // 16 words written by the odd CTA's signals
constexpr uint32_t kOffBar = kOffScratch + 64;

// Barriers of the even CTA that the odd CTA signals ("paired" below) count
// the even CTA's own arrivals, and the odd CTA's signals as 4-byte
// transactions (st.async) that one of the even CTA's arrivals announces.
// Tile g uses slot g & 1 of everything.
enum Bar {
  K_FULL = 0,           // [2] even CTA: both CTAs' TMA bytes of a K slot
  K_EMPTY = K_FULL + 2, // [2] S of the slot's tile done (paired commit)
  V_FULL = K_EMPTY + 2, // [2] even CTA: both CTAs' TMA bytes of a V slot (tiles without drafted tokens)
  V_LOCAL = V_FULL + 2, // [2] this CTA's TMA bytes of a V slot (tiles with drafted tokens)
  V_EMPTY = V_LOCAL + 2,// [2] P . C of the slot's tile done (paired commit)
  S_FULL = V_EMPTY + 2, // [2] per S buffer (paired commit)
  S_EMPTY = S_FULL + 2, // [2] even CTA, paired: softmax warps read the S buffer
  P_FULL = S_EMPTY + 2, // [2] even CTA, paired: softmax warps wrote P
  PV_DONE = P_FULL + 2, // [2] (paired commit)
  Q_FULL = PV_DONE + 2, // even CTA: both CTAs' TMA bytes of the queries
  Q_EMPTY,              // last S of a segment done (paired commit)
  DEC,                  // [2] per softmax group: its 2 publishing warps decided a tile's maximum
  GRP = DEC + 2,        // the 8 softmax warps of this CTA
  EPI_FREE,             // the 8 softmax warps' output stores have read the V slots
  O_FREE,               // even CTA, paired: the softmax warps have read a segment's O
  MMA_FINAL,            // even CTA: all S issued so far are complete
  MMA_FINAL_PV,         // even CTA: all P . C issued so far are complete
  BAR_COUNT
};
constexpr uint32_t kOffTmemSlot = kOffBar + BAR_COUNT * 8;
constexpr uint32_t kSmemUsed = kOffTmemSlot + 16;
constexpr size_t kSmemBytes = kSmemUsed;  // the base is 1024-byte aligned (checked at entry)

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;     // 2 x 32 columns
constexpr uint32_t kTmemO = 256;   // 2 x 128 columns (latent blocks 0-255, 256-511)
constexpr float kRescaleThreshold = 30.0f;  // log2 units: rescale O only if the max grows by > 2^30
constexpr int kPrefetchAhead = 4;           // tiles between an L2 prefetch and the tile's TMA load
constexpr uint16_t kBothCtas = 3;

static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "align");
static_assert(kSmemBytes <= 232448, "shared memory");

struct Params {
  TreeMaps maps;
  const __nv_bfloat16* q;   // for L2 prefetch of the next segment's rows
  const __nv_bfloat16* kv;  // for L2 prefetch of tiles ahead of their loads
  const int* block_table;
  const unsigned long long* mask;
  const int* rec;
  const int4* seqs;
  float* part_lse;
  void* u;
  float* lse;
  int* err;
  int n_h, max_pages, page_size, num_pages;
  int out_f32;       // u is fp32 (else bf16)
  float scale_log2;  // softmax_scale * log2(e)
};

// 2D tiled store of a shared-memory box; tracked by bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}

// 32 lanes x 8 consecutive columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
// 3D tiled loads with an L2 policy into this CTA's shared memory, complete on
// a barrier of this CTA or (pair) of the even CTA of the pair.  No multicast.
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                                 int y, int z, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_to_pair_hint(uint32_t dst, const CUtensorMap* m, uint32_t cluster_bar,
                                                         int x, int y, int z, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z), "l"(pol)
      : "memory");
}

// One thread of a converged warp, always the same.  Instructions that take
// uniform registers (MMA, TMA, commits) come from an elected thread: behind
// `lane == 0` the compiler cannot keep their operands uniform, and a warp that
// waits as a whole needs no shuffle after it.  Both together, against lane 0
// waiting and issuing: 16 trees of 64 tokens over 4096 1556 -> 1440 us, 37 over
// 256 355 -> 313, one token over 70 23.4 -> 20.5.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Waits of a whole converged warp; a failed one (its time ran out) fails for
// every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, MLA_DEVFLAG_TIMEOUT));
}

// The same for the copies' warps, which mostly wait and are ahead of the rest:
// the warp is suspended instead of polling.  Long calls run at the power limit,
// where what the polls burn is missing elsewhere (16 trees of 64 tokens over 4096
// 1225 -> 1211 us, 64 ragged sequences 329 -> 323, 16 single tokens over 4096
// 42.5 -> 41.6).
__device__ __forceinline__ bool warp_sleep(uint32_t bar, uint32_t parity, int* err) {
  const uint64_t t0 = cycles();
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, done)) return true;
    if (__any_sync(0xffffffffu, cycles() - t0 > kWaitLimitCycles)) {
      atomicOr(err, MLA_DEVFLAG_TIMEOUT);
      return false;
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_sm100_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  uint8_t* base = smem_raw;
  if (sbase & 1023u) {  // the swizzled layouts need it; nothing has been started yet
    if (threadIdx.x == 0) atomicOr(p.err, MLA_DEVFLAG_LAYOUT);
    return;
  }
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = blockIdx.x >> 1;
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
  // Signal a paired barrier of the even CTA: from the even CTA a local
  // arrival (with `announce`, the one arrival per phase that also expects the
  // odd CTA's `odd_bytes` of signals); from the odd CTA a non-blocking 4-byte
  // st.async into scratch word `scratch_word` of the even CTA.
  auto signal_lead = [&](int i, bool announce, uint32_t odd_bytes, int scratch_word) {
    if (leader) {
      if (announce)
        mbar_arrive_expect_tx(bar(i), odd_bytes);
      else
        mbar_arrive(bar(i));
    } else {
      st_async_b32(mapa(sbase + kOffScratch + 4u * scratch_word, 0), 0u, mapa(bar(i), 0));
    }
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(K_FULL + i), 1);
      mbar_init(bar(K_EMPTY + i), 1);
      mbar_init(bar(V_FULL + i), 1);
      mbar_init(bar(V_LOCAL + i), 1);
      mbar_init(bar(V_EMPTY + i), 1);
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(S_EMPTY + i), 4);
      mbar_init(bar(P_FULL + i), 4);
      mbar_init(bar(PV_DONE + i), 1);
      mbar_init(bar(DEC + i), 2);
    }
    mbar_init(bar(Q_FULL), 1);
    mbar_init(bar(Q_EMPTY), 1);
    mbar_init(bar(GRP), 8);
    mbar_init(bar(EPI_FREE), 8);
    mbar_init(bar(O_FREE), 8);
    mbar_init(bar(MMA_FINAL), 1);
    mbar_init(bar(MMA_FINAL_PV), 1);
    fence_mbar_init();
  }
  if (warp == kWarpAlloc) {
    tmem_alloc_pair(sbase + kOffTmemSlot, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kWarpK && lane == 0) {
    prefetch_tmap(&p.maps.k);
    prefetch_tmap(&p.maps.q);
  }
  if (warp == kWarpV && lane == 0) prefetch_tmap(&p.maps.v);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and TMEM exist before either uses the other's
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + kOffTmemSlot);
  // everything above overlaps the plan kernel; its results are read below
  pdl_wait_previous();
  pdl_launch_dependents();

  // Cache rows of tiles [t0, t0 + 32): lane i looks up the page of tile t0 + i.
  auto page_of = [&](const TreeSegment& sg, int t0) {
    int page = 0;
    if (t0 + lane < sg.t1) {
      page = p.block_table[(size_t)sg.seq.b * p.max_pages + ((t0 + lane) * kTreeTile) / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        atomicOr(p.err, MLA_DEVFLAG_BAD_PAGE);
        page = 0;
      }
    }
    return page;
  };
  // tiles from here on reach into the drafted tokens
  auto drafted = [&](const TreeSegment& sg, int t) { return t * kTreeTile > sg.seq.L - sg.seq.n - kTreeTile; };

  if (warp == kWarpK) {
    // ---------------------------------------------------- queries and K copies
    const uint64_t pol = l2_policy_evict_normal();  // the V copy reads the same lines
    TreeWalk walk;
    walk.init(p.rec, p.seqs, p.n_h, chunk);
    TreeSegment sg;
    int g = 0, seg_i = 0;
    bool ok = true;
    // This CTA's 64 rows of the block, 24 KB at a time.  Rows past the block's
    // last belong to the next sequence, or read as zero behind q's end: nothing
    // of theirs is written.
    auto load_q = [&](const TreeSegment& sg) {
      if (seg_i > 0) ok = ok && warp_wait(bar(Q_EMPTY), (seg_i - 1) & 1, p.err);
      if (ok && elect_one()) {
        const int y = sg.first + 64 * (int)rank;
        if (leader) mbar_arrive_expect_tx(bar(Q_FULL), 2 * kQBytes);
        for (int c = 0; c < 9; c += 3) {
          if (leader)
            tma_load_3d_hint(sbase + kOffQ + c * kQBlk, &p.maps.q, bar(Q_FULL), 0, y, c, pol);
          else
            tma_load_3d_to_pair_hint(sbase + kOffQ + c * kQBlk, &p.maps.q, mapa(bar(Q_FULL), 0), 0, y, c, pol);
        }
      }
      __syncwarp();
    };
    // the next segment's rows go to L2
    auto prefetch_next_q = [&]() {
      TreeWalk peek = walk;
      TreeSegment nx;
      if (peek.next(nx) && nx.rows > 64 * (int)rank && elect_one()) {
        const __nv_bfloat16* src = p.q + ((size_t)nx.first + 64 * rank) * (kDc + 64);
        const uint32_t bytes = static_cast<uint32_t>(min(64, nx.rows - 64 * (int)rank)) * (kDc + 64) * 2;
        for (uint32_t off = 0; off < bytes; off += 16384)
          bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(src) + off, min(16384u, bytes - off));
      }
      __syncwarp();
    };
    // 64 rows of a page that a 64-token tile reads: contiguous bytes
    auto prefetch_tile = [&](int page, int t) {
      const int tok = t * kTreeTile;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          p.kv + ((size_t)page * p.page_size + tok % p.page_size) * (kDc + 64));
      constexpr uint32_t kTile = kTreeTile * (kDc + 64) * 2;
      for (uint32_t off = 0; off < kTile; off += 16384) bulk_prefetch_l2(src + off, min(16384u, kTile - off));
    };
    while (ok && walk.next(sg)) {
      // (after the first segment a K slot is free before the query area)
      if (seg_i == 0) load_q(sg);
      for (int t0 = sg.t0; ok && t0 < sg.t1; t0 += 32) {
        const int my_page = page_of(sg, t0);
        const int n_here = min(32, sg.t1 - t0);
        for (int i = 0; ok && i < n_here; ++i, ++g) {
          const int page = __shfl_sync(0xffffffffu, my_page, i);
          // The tile kPrefetchAhead tiles later goes to L2 now: its copies are
          // issued only when a slot frees, and an L2 hit then lands in a
          // fraction of the HBM latency.  The even CTA fetches all of it.  At the
          // start of a chunk every SM is already loading its queries and first
          // tiles: the first prefetch comes behind those, below.
          const int page_ahead = __shfl_sync(0xffffffffu, my_page, (i + kPrefetchAhead) & 31);
          if (leader && g >= 2 && i + kPrefetchAhead < n_here && elect_one())
            prefetch_tile(page_ahead, t0 + i + kPrefetchAhead);
          const int s = g & 1;
          if (!(ok = warp_sleep(bar(K_EMPTY + s), ((g >> 1) & 1) ^ 1, p.err))) break;
          if (elect_one()) {
            const int tok = (t0 + i) * kTreeTile;
            const int y = page * p.page_size + tok % p.page_size + 32 * (int)rank;
            const uint32_t dst = sbase + kOffK + s * kKBytes;
            if (leader) {
              mbar_arrive_expect_tx(bar(K_FULL + s), 2 * kKBytes);
              tma_load_3d_hint(dst, &p.maps.k, bar(K_FULL + s), 0, y, 0, pol);
            } else {
              tma_load_3d_to_pair_hint(dst, &p.maps.k, mapa(bar(K_FULL + s), 0), 0, y, 0, pol);
            }
          }
          __syncwarp();
          if (seg_i > 0 && t0 + i == sg.t0) load_q(sg);
          if (t0 + i == min(sg.t0 + 1, sg.t1 - 1)) {
            if (seg_i == 0) {  // (i = 1 here if there are more tiles)
              for (int k = 1; k <= kPrefetchAhead; ++k) {
                const int pg = __shfl_sync(0xffffffffu, my_page, (i + k) & 31);
                if (leader && i + k < n_here && elect_one()) prefetch_tile(pg, t0 + i + k);
              }
            }
            prefetch_next_q();
          }
        }
      }
      ++seg_i;
    }
    // commits of the last tiles and of the last segment, on their way to this CTA
    for (int k = max(0, g - 2); ok && k < g; ++k) ok = warp_sleep(bar(K_EMPTY + (k & 1)), (k >> 1) & 1, p.err);
    if (ok && seg_i > 0) warp_sleep(bar(Q_EMPTY), (seg_i - 1) & 1, p.err);
  } else if (warp == kWarpV) {
    // ------------------------------------------------------------ V copies
    // a sequence of one row block reads each of its tiles for the last time
    // here: those lines leave L2 first
    const uint64_t pol_once = l2_policy_evict_first(), pol_shared = l2_policy_evict_normal();
    TreeWalk walk;
    walk.init(p.rec, p.seqs, p.n_h, chunk);
    TreeSegment sg;
    int g = 0, seg_i = 0;
    uint32_t local_used = 0, local_phase = 0;  // slots that had a V_LOCAL phase; parity of the next
    bool ok = true;
    while (ok && walk.next(sg)) {
      const uint64_t pol = sg.seq.blocks == 1 ? pol_once : pol_shared;
      // the last segment's output stores have read the slots
      if (seg_i > 0 && !(ok = warp_wait(bar(EPI_FREE), (seg_i - 1) & 1, p.err))) break;
      for (int t0 = sg.t0; ok && t0 < sg.t1; t0 += 32) {
        const int my_page = page_of(sg, t0);
        const int n_here = min(32, sg.t1 - t0);
        for (int i = 0; i < n_here; ++i, ++g) {
          const int page = __shfl_sync(0xffffffffu, my_page, i);
          const int s = g & 1;
          if (!(ok = warp_sleep(bar(V_EMPTY + s), ((g >> 1) & 1) ^ 1, p.err))) break;
          const bool local = drafted(sg, t0 + i);
          if (elect_one()) {
            const int tok = (t0 + i) * kTreeTile;
            const int y = page * p.page_size + tok % p.page_size;
            const uint32_t dst = sbase + kOffV + s * kVBytes;
            if (local) {
              // the softmax clears what must not meet P . C before it hands P over
              mbar_arrive_expect_tx(bar(V_LOCAL + s), kVBytes);
              tma_load_4d_hint(dst, &p.maps.v, bar(V_LOCAL + s), 128 * (int)rank, y, 0, 0, pol);
            } else if (leader) {
              mbar_arrive_expect_tx(bar(V_FULL + s), 2 * kVBytes);
              tma_load_4d_hint(dst, &p.maps.v, bar(V_FULL + s), 0, y, 0, 0, pol);
            } else {
              tma_load_4d_to_pair_hint(dst, &p.maps.v, mapa(bar(V_FULL + s), 0), 128, y, 0, 0, pol);
            }
          }
          __syncwarp();
          if (local) {
            local_used |= 1u << s;
            local_phase ^= 1u << s;
          }
        }
      }
      ++seg_i;
    }
    // this CTA's own copies land before it may exit (the paired ones are
    // consumed by the MMAs before the final cluster barrier)
    for (int s = 0; s < 2; ++s)
      if ((local_used >> s) & 1) warp_wait(bar(V_LOCAL + s), ((local_phase >> s) & 1) ^ 1, p.err);
    // and the commits of the last tiles
    for (int k = max(0, g - 2); ok && k < g; ++k)
      ok = warp_sleep(bar(V_EMPTY + (k & 1)), (k >> 1) & 1, p.err) && warp_sleep(bar(PV_DONE + (k & 1)), (k >> 1) & 1, p.err);
  } else if (warp == kWarpMma || warp == kWarpAlloc) {
    // ------------------------------------------------------------ MMA issuers
    // Warp 1 issues every S, warp 2 (done allocating) every P . C.  The two
    // streams touch disjoint TMEM and shared memory, and each commit tracks
    // only its own thread's MMAs, so a P . C whose P is ready never waits
    // behind an S being issued (issuing blocks while the tensor pipe's queue
    // is full) and vice versa.
    // One elected thread per warp does all of it, waits included: between two
    // products no other lane has to be met again.
    if (leader && elect_one()) {
      constexpr uint32_t kIdS = idesc_bf16(128, 64, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, 256, true);
      TreeWalk walk;
      walk.init(p.rec, p.seqs, p.n_h, chunk);
      TreeSegment sg;
      int g0 = 0, seg_i = 0;
      bool ok = true;
      // Descriptors are the first tile's plus a distance in 16-byte units: the
      // one thread that issues has 36 products a tile to keep the pipe fed
      const uint64_t q0 = smem_desc(sbase + kOffQ, 16, 1024, kLayoutSW128);
      const uint64_t k0 = smem_desc(sbase + kOffK, 16, 1024, kLayoutSW128);
      const uint64_t v0 = smem_desc(sbase + kOffV, kVBlk, 1024, kLayoutSW128);
      const uint64_t p0 = smem_desc(sbase + kOffP, 16, 1024, kLayoutSW128);
      // S for global tile g: 36 steps over the columns
      auto issue_s = [&](int g, bool last) {
        tc_fence_after();
        const uint64_t k = k0 + (g & 1) * (kKBytes >> 4);
        const uint32_t dS = tmem + kTmemS + (g & 1) * 32;
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ss_pair(dS, q0 + c * (kQBlk >> 4) + ks * 2, k + c * (kKBlk >> 4) + ks * 2, kIdS,
                             c + ks > 0 ? 1u : 0u);
        umma_commit_pair(bar(S_FULL + (g & 1)), kBothCtas);
        umma_commit_pair(bar(K_EMPTY + (g & 1)), kBothCtas);
        if (last) umma_commit_pair(bar(Q_EMPTY), kBothCtas);
      };
      // O (+)= P . C for global tile g; `first` = first tile of its segment
      auto issue_pv = [&](int g, bool first) {
        tc_fence_after();
        const uint64_t v = v0 + (g & 1) * (kVBytes >> 4), a = p0 + (g & 1) * (kPBytes >> 4);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 tokens per MMA
            umma_f16_ss_pair(tmem + kTmemO + blk * 128, a + kk * 2,
                             v + 2 * blk * (kVBlk >> 4) + kk * (2048 >> 4), kIdPV,
                             (first && kk == 0) ? 0u : 1u);
        umma_commit_pair(bar(V_EMPTY + (g & 1)), kBothCtas);
        umma_commit_pair(bar(PV_DONE + (g & 1)), kBothCtas);
      };
      // S runs up to two tiles ahead of P . C (its two buffers), so the softmax
      // of a tile has two S of tensor work to hide behind.
      auto wait = [&](int b, uint32_t parity) {
        return mbar_wait(bar(b), parity, p.err, MLA_DEVFLAG_TIMEOUT);
      };
      const bool s_issuer = warp == kWarpMma;
      uint32_t v_phase = 0;  // parity of each slot's next V_FULL phase
      while (ok && walk.next(sg)) {
        const int n_t = sg.t1 - sg.t0;
        if (s_issuer) {
          // S(g) once its K copy is loaded and its S buffer has been read
          if (!(ok = wait(Q_FULL, seg_i & 1))) break;
          for (int j = 0; ok && j < n_t; ++j) {
            const int g = g0 + j;
            if (!(ok = wait(S_EMPTY + (g & 1), ((g >> 1) & 1) ^ 1) &&
                       wait(K_FULL + (g & 1), (g >> 1) & 1)))
              break;
            issue_s(g, j == n_t - 1);
          }
        } else {
          // P . C(g) once P(g) is written and its V copy is there (which P says
          // of a tile with drafted tokens)
          for (int j = 0; ok && j < n_t; ++j) {
            const int g = g0 + j;
            if (!drafted(sg, sg.t0 + j)) {
              if (!(ok = wait(V_FULL + (g & 1), (v_phase >> (g & 1)) & 1))) break;
              v_phase ^= 1u << (g & 1);
            }
            if (!(ok = wait(P_FULL + (g & 1), (g >> 1) & 1))) break;
            // the segment's first P . C overwrites O: every softmax warp of
            // both CTAs must have read the last segment's
            if (j == 0 && seg_i > 0 && !(ok = wait(O_FREE, (seg_i - 1) & 1))) break;
            issue_pv(g, j == 0);
          }
        }
        g0 += n_t;
        ++seg_i;
      }
      // The odd CTA's last signals: no product waits for them, but they are
      // writes to this CTA's shared memory, and a cluster barrier does not wait
      // for those (st.async)
      if (s_issuer) {
        for (int k = max(0, g0 - 2); ok && k < g0; ++k) ok = wait(S_EMPTY + (k & 1), (k >> 1) & 1);
      } else if (ok && seg_i > 0) {
        wait(O_FREE, (seg_i - 1) & 1);
      }
      // every MMA issued by this thread has completed before TMEM is freed
      const int fin = s_issuer ? MMA_FINAL : MMA_FINAL_PV;
      umma_commit_pair(bar(fin), 1);
      wait(fin, 0);
    }
    __syncwarp();
  } else if (warp >= kWarpSoftmax0) {
    // ------------------------------------------------------------ softmax
    // Two groups of four warps take alternate tiles (group = g & 1, which is
    // also the tile's S buffer and P slot).  Thread (warp q, lane l) of a group
    // has row (32 q + l) % 64 and half (32 q + l) / 64 of the tile's tokens; the
    // halves exchange their maxima through shared memory.  The running maximum
    // after tile g is published per row (slot g & 1); a group decides tile g
    // from the maximum after tile g - 1, which the other group published.
    const int sw_warp = warp - kWarpSoftmax0;       // 0..7
    const int grp = sw_warp >> 2;                   // softmax group; also the O block it drains
    const int gw = sw_warp & 3;                     // warp within the group
    const int qd = warp & 3;                        // TMEM lanes [32 qd, 32 qd + 32)
    const int row = (32 * qd + lane) & 63;          // this thread's row of this CTA's 64, of S and of O
    const int half = qd >> 1;                       // its tokens: 32 half + [0, 32)
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    float* mx_pub = reinterpret_cast<float*>(base + kOffMax);  // [tile parity][row]
    // maxima [tile turn][group][half][row]; between segments the sums
    // [kind][group][half][row]
    float* ex = reinterpret_cast<float*>(base + kOffEx);
    auto ex_at = [&](int k, int group, int h) -> float& { return ex[((k * 2 + group) * 2 + h) * 64 + row]; };
    uint32_t local_phase = 0;  // parity of V_LOCAL's next phase (this group's slot)
    const float c_log2 = p.scale_log2;
    uint32_t grp_phase = 0;
    // A failed wait (a broken protocol) sets the device flag; the warp then
    // skips its later waits but still runs every step, so that the group's
    // named barriers and the other roles' waits stay matched and the kernel
    // ends.
    auto rendezvous = [&](bool live) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(GRP));
      const uint32_t ph = (grp_phase++) & 1;
      return live && warp_wait(bar(GRP), ph, p.err);
    };

    TreeWalk walk;
    walk.init(p.rec, p.seqs, p.n_h, chunk);
    TreeSegment sg;
    int g = 0;
    bool ok = true;
    while (walk.next(sg)) {
      const int n = sg.seq.n, P0 = sg.seq.L - n;  // P0: position of the first drafted token
      const int n_t = sg.t1 - sg.t0;
      const int g0 = g;
      // this group's sums over its own tiles of the segment, in the scale of
      // m_used (the maximum it last applied)
      float m_used = -INFINITY, l = 0.f, l_exact = 0.f;
      for (int jt = (grp - g0) & 1; jt < n_t; jt += 2) {
        const int gt = g0 + jt;
        const int tok0 = (sg.t0 + jt) * kTreeTile;
        // a tile that reaches into the drafted tokens: which of them this
        // thread's row sees (none for rows past the block's last, whose results
        // are not written), read while S of the tile runs
        const bool tail = drafted(sg, sg.t0 + jt);
        unsigned long long seen = 0;
        if (tail && 64 * (int)rank + row < sg.rows)
          seen = p.mask[sg.seq.row0 + (sg.g * kTreeRows + 64 * (int)rank + row) / p.n_h];
        // ---- scores of tile gt -> registers; free the S buffer
        ok = ok && warp_wait(bar(S_FULL + grp), (gt >> 1) & 1, p.err);
        tc_fence_after();
        float sc[32];  // token 32 half + k
        tmem_ld32(tmem + lane_base + kTmemS + grp * 32, sc);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) signal_lead(S_EMPTY + grp, gw == 0, 16u, gw);
        uint32_t clear = 0, past = 0;  // tokens of this half with non-finite values; behind the sequence's end
        if (tail) {
          // bit k = position tok0 + k: the context, then the drafted tokens
          const int sh = tok0 - P0;  // > -64; at most n - 1
          const unsigned long long ctx = sh >= 0 ? 0 : (1ull << -sh) - 1;
          const unsigned long long all = n < 64 ? (1ull << n) - 1 : ~0ull;
          auto place = [&](unsigned long long m) {  // of drafted tokens
            return static_cast<uint32_t>((sh >= 0 ? m >> sh : (m << -sh) | ctx) >> (32 * half));
          };
          const uint32_t vis = place(seen & all);
          past = ~place(all);
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!(fabsf(sc[k]) <= 3.402823466e38f)) bad |= 1u << k;
            if (!((vis >> k) & 1)) sc[k] = -INFINITY;
          }
          // a non-finite cache row makes every row's score so: one warp of each
          // half finds it
          clear = __reduce_or_sync(0xffffffffu, bad) & ~past;
        }
        float mx;
        {
          float m4[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
          for (int k = 4; k < 32; ++k) m4[k & 3] = fmaxf(m4[k & 3], sc[k]);
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        const int turn = (gt >> 1) & 1;
        ex_at(turn, grp, half) = mx;
        // ---- the maximum after this tile.  The running maximum may go
        // stale: it moves only when a tile's maximum exceeds it by more than
        // 2^kRescaleThreshold (weights stay below that factor), which keeps O
        // rescales rare.  Raw scores: scale > 0 commutes with max.
        float m_prev = -INFINITY;
        if (jt > 0) {  // tile gt - 1 (the other group's) is in this segment
          ok = ok && warp_wait(bar(DEC + (grp ^ 1)), ((gt - 1) >> 1) & 1, p.err);
          m_prev = mx_pub[((gt - 1) & 1) * 64 + row];
        }
        named_bar_sync(1 + grp, 128);
        const float t_s = fmaxf(mx, ex_at(turn, grp, half ^ 1)) * c_log2;
        const float m_new = (m_prev == -INFINITY || t_s > m_prev + kRescaleThreshold) ? fmaxf(m_prev, t_s) : m_prev;
        if (half == 0) {  // publish
          mx_pub[(gt & 1) * 64 + row] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(DEC + grp));
        }
        // O's row: rescale if its maximum moved at this tile
        const bool resc_o = jt > 0 && m_new != m_prev;
        // this group's sums move to the new scale
        if (m_new != m_used) {
          const float f = m_used == -INFINITY ? 0.f : ex2_approx(m_used - m_new);
          l *= f;
          l_exact *= f;
          m_used = m_new;
        }
        const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
        // the weights, in pairs.  u is normalised by the sum of the rounded
        // weights it was built from; lse uses the unrounded ones
        uint32_t pk[16];
        {
          float r0 = 0.f, r1 = 0.f, e0 = 0.f, e1 = 0.f;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float a = ex2_approx(fmaf(sc[k], c_log2, neg_m));
            const float b = ex2_approx(fmaf(sc[k + 1], c_log2, neg_m));
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
            const float2 pf = __bfloat1622float2(h2);
            r0 += pf.x;
            r1 += pf.y;
            e0 += a;
            e1 += b;
            pk[k >> 1] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          l += r0 + r1;
          l_exact += e0 + e1;
        }

        // P slot grp was last read by PV(gt - 2); O may be rescaled
        // only after PV(gt - 1) (tiles of an earlier segment were retired by
        // that segment's epilogue, and the first P . C of a segment
        // overwrites O)
        if (gt >= 2) ok = ok && warp_wait(bar(PV_DONE + grp), ((gt - 2) >> 1) & 1, p.err);
        if (__any_sync(0xffffffffu, resc_o)) {
          ok = ok && warp_wait(bar(PV_DONE + (grp ^ 1)), ((gt - 1) >> 1) & 1, p.err);
          tc_fence_after();
          // both O blocks of these lanes, 8 columns at a time: this is rare, and
          // its registers are the loop's
          const float alpha_o = resc_o ? ex2_approx(m_prev - m_new) : 1.f;  // m_prev = -inf: O holds only zeros
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 8) {
            float o[8];
            tmem_ld8(tmem + lane_base + kTmemO + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= alpha_o;
            tmem_st8(tmem + lane_base + kTmemO + c0, o);
          }
          tmem_wait_st();
        }
        // P's row: 64 tokens, 128 bytes, 16-byte chunk c at c ^ (row & 7)
        const uint32_t prow = sbase + kOffP + grp * kPBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          st_shared_v4(prow + (static_cast<uint32_t>((4 * half + c) ^ (row & 7)) << 4), pk[4 * c], pk[4 * c + 1],
                       pk[4 * c + 2], pk[4 * c + 3]);
        if (tail && (gw & 1) == 0) {
          // The P . C of a tile with drafted tokens waits for these warps, one
          // per half, to have seen its V copy land and cleared in it rows behind
          // the sequence's end, which may hold anything, and the non-finite
          // values of drafted tokens.  16 bytes per lane: a token's 256 columns.
          ok = ok && warp_wait(bar(V_LOCAL + grp), local_phase, p.err);
          local_phase ^= 1;
          uint8_t* tile = base + kOffV + grp * kVBytes + (lane >> 3) * kVBlk + (lane & 7) * 16 + half * 32 * 128;
          for (uint32_t todo = past; todo != 0; todo &= todo - 1)
            *reinterpret_cast<uint4*>(tile + (__ffs(todo) - 1) * 128) = make_uint4(0, 0, 0, 0);
          for (uint32_t todo = clear; todo != 0; todo &= todo - 1) {
            uint4* at = reinterpret_cast<uint4*>(tile + (__ffs(todo) - 1) * 128);
            uint4 v = *at;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
              if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
            }
            *at = v;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) signal_lead(P_FULL + grp, gw == 0, 16u, gw);
      }
      g = g0 + n_t;

      // ---- epilogue: u = O / l for this thread's O lane (one row, 128
      // consecutive latent columns of O block grp)
      // the maximum after the segment's last tile (published by half a group)
      ok = ok && warp_wait(bar(DEC + ((g - 1) & 1)), ((g - 1) >> 1) & 1, p.err);
      const float m_fin = mx_pub[((g - 1) & 1) * 64 + row];
      // (P . C of the last tile done: every warp has handed over its last P, so
      // none still reads the maxima that the sums now take the place of)
      ok = ok && warp_wait(bar(PV_DONE + ((g - 1) & 1)), ((g - 1) >> 1) & 1, p.err);
      tc_fence_after();
      {
        // this thread's sums in the scale of the final maximum
        const float f = m_used == m_fin ? 1.f : m_used == -INFINITY ? 0.f : ex2_approx(m_used - m_fin);
        ex_at(0, grp, half) = l * f;
        ex_at(1, grp, half) = l_exact * f;
      }
      ok = rendezvous(ok);
      const float l_o = (ex_at(0, 0, 0) + ex_at(0, 0, 1)) + (ex_at(0, 1, 0) + ex_at(0, 1, 1));
      const float le_o = (ex_at(1, 0, 0) + ex_at(1, 0, 1)) + (ex_at(1, 1, 0) + ex_at(1, 1, 1));
      // no token seen: u = 0 (a NaN sum, of non-finite scores, stays)
      const float inv = l_o == 0.f ? 0.f : 1.f / l_o;
      const int c = grp;                          // O block drained by this group
      const int col0 = 256 * c + 128 * (qd >> 1);  // latent column of TMEM column kTmemO + 128c
      // The output is staged in the V slots (every P . C is done), 8 KB per
      // warp: its 32 rows x 128 columns as boxes of 128-byte lines (64 bf16 or
      // 32 fp32 columns) in the 128-byte-swizzled layout of the output tensor
      // map (16-byte chunk k of row r at k ^ (r & 7)).
      const uint32_t stg = sbase + kOffV + sw_warp * 8192u;
      const int y_w = 64 * (int)rank + 32 * (qd & 1);  // this warp's first row of the block
      const int y_out = sg.whole ? sg.first + y_w : sg.slot * kTreeRows + y_w;
      const bool full = !sg.whole || y_w + 32 <= sg.rows;
      if (y_w >= sg.rows) {
        // none of this warp's rows exist
      } else if (full && (p.out_f32 || !sg.whole)) {
        const CUtensorMap* omap = sg.whole ? &p.maps.u_out : &p.maps.part_out;
        // fp32: four boxes of 32 columns, two at a time through the 8 KB
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float o[32];
          tmem_ld32(tmem + lane_base + kTmemO + c * 128 + c0, o);
          tmem_wait_ld();
          const uint32_t box = stg + static_cast<uint32_t>((c0 >> 5) & 1) * 4096u;
          if (c0 == 64) {  // the first two boxes must have left before reuse
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            st_shared_v4(box + lane * 128u + ((static_cast<uint32_t>(e ^ (lane & 7))) << 4),
                         __float_as_uint(o[4 * e] * inv), __float_as_uint(o[4 * e + 1] * inv),
                         __float_as_uint(o[4 * e + 2] * inv), __float_as_uint(o[4 * e + 3] * inv));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(omap, box, col0 + c0, y_out);
            bulk_commit();
          }
        }
      } else {
        const bool live = y_w + lane < sg.rows;
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float o[32];
          tmem_ld32(tmem + lane_base + kTmemO + c * 128 + c0, o);
          tmem_wait_ld();
          const size_t at = ((size_t)y_out + lane) * kDc + col0 + c0;
          if (p.out_f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.u) + at);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (live)
                dst[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
            continue;
          }
          const uint32_t line = stg + static_cast<uint32_t>(c0 >> 6) * 4096u + lane * 128u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[8 * e + 2 * k] * inv, o[8 * e + 2 * k + 1] * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            if (full) {
              const uint32_t chunk16 = static_cast<uint32_t>(((c0 & 63) >> 3) + e);
              st_shared_v4(line + ((chunk16 ^ static_cast<uint32_t>(lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            } else if (live) {
              reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.u) + at)[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (full && !p.out_f32) {  // both boxes
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.maps.u_out, stg, col0, y_out);
            tma_store_2d(&p.maps.u_out, stg + 4096u, col0 + 64, y_out);
            bulk_commit();
          }
        }
      }
      if (y_w + lane < sg.rows && qd < 2 && c == 0) {
        const float lse = le_o == 0.f ? -INFINITY : (m_fin + log2f(le_o)) * 0.69314718055994531f;
        if (!sg.whole)
          p.part_lse[y_out + lane] = lse;
        else if (p.lse != nullptr)
          p.lse[y_out + lane] = lse;
      }
      // O has been read: the next segment's P . C may overwrite it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        signal_lead(O_FREE, sw_warp == 0, 32u, 10);
        // the staging area may take the next tiles once the stores have read it
        bulk_wait_read_all();
        mbar_arrive(bar(EPI_FREE));
      }
      // every warp has read the sums, and the maxima of this segment, before any
      // starts the next one
      ok = rendezvous(ok);
    }
    // the last stores complete before the CTA exits
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  // all paired MMAs are complete, and every signal and commit between the CTAs
  // has been waited for by its receiver: none is still on its way to a CTA that ends
  cluster_sync();
  if (warp == kWarpAlloc) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  cluster_sync();
}

}  // namespace

// Per device, once: opt in to the shared-memory size and count how many
// 2-CTA clusters of this kernel can be resident at the same time.
int tree_sm100_prepare() {
  if (cudaFuncSetAttribute(tree_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kSmemBytes) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, tree_sm100_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_tree_sm100(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s) {
  Params p;
  p.maps = maps;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kv = static_cast<const __nv_bfloat16*>(a.kv);
  p.block_table = a.block_table;
  p.mask = a.mask;
  p.rec = a.rec;
  p.seqs = a.seqs;
  p.part_lse = a.part_lse;
  p.u = a.u;
  p.lse = a.lse;
  p.err = a.err;
  p.n_h = a.n_h;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.num_pages = a.num_pages;
  p.out_f32 = a.out_f32 ? 1 : 0;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * a.num_chunks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_sm100_kernel, p);
}

}  // namespace mla
