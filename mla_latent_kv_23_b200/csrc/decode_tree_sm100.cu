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
// cores bound it.  O of 128 rows and 512 columns in fp32 fills the tensor
// memory of one SM, so a pair of CTAs (one 2-CTA cluster) shares a block, and
// the operands are split as in the decode kernel of this shape:
//  * CTA r loads, for every cached row, latent columns [128r, 128r + 128) and
//    [256 + 128r, 256 + 128r + 128) plus RoPE columns [32r, 32r + 32).
//  * CTA r owns rows [64r, 64r + 64) of the block and their O in its TMEM.
//  * P . C is one paired MMA (cta_group::2) per 16 tokens and 256 columns.
//  * S is a paired MMA with M = 256: rows (query row i, column half j) against
//    B = [CTA 0's columns of the tile | CTA 1's]; row (i, j) counts against
//    half j, so half of the products are discarded and one shuffle adds the two
//    partial scores.  Per tile 1673 tensor cycles are issued where 1095 would
//    do; passing data between the CTAs instead costs more than it saves.
//
// The mask is one 64-bit word per token: a tile that reaches into the drafted
// tokens shifts it to the tile's positions.  A drafted token's cache row may
// hold infinities or NaN that a row which does not see it must not meet (0 x
// NaN in P . C): every row's raw score of such a token is then non-finite, so
// the softmax finds it there and clears the non-finite values of that cache
// row in shared memory before P . C; rows that see the token get NaN by their
// weight.
//
// TMEM per CTA (512 columns): S 2 x 128 (double-buffered) | O 256.
// Shared memory per CTA: Q (128 rows x 288 values, the S operand A) 72 KB;
// 4 tile stages of 36 KB; P (64 rows x 64 tokens bf16) as two 32-token halves:
// tokens 0-31 in the tile's own RoPE block (free once S of the tile is done),
// tokens 32-63 in a two-slot 4 KB ring.
//
// Roles (384 threads): warp 0 = TMA producer; warp 1 = S issuer and warp 2 =
// P . C issuer (even CTA); warp 3 = relay (the segment's queries, rows past a
// sequence's end zeroed, signals to the even CTA); warps 4-11 = softmax, two
// groups of four that take alternate tiles.
//
// Epilogue: u = O / l leaves TMEM through the query area (free once the
// segment's last S is done) by TMA stores of whole 128-byte lines, or row by
// row where fewer than a warp's 32 rows exist (the rows behind belong to the
// next sequence).  Pieces of split blocks are written in fp32.
#include <cuda_bf16.h>
#include <math.h>

#include "sm100_ptx.cuh"
#include "tree.h"
#include "tree_schedule.cuh"

namespace mla {
namespace {
using namespace ptx;

constexpr int kThreads = 384;
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpAlloc = 2, kWarpRelay = 3, kWarpSoftmax0 = 4;
constexpr int kStages = 4;
constexpr int kDc = 512;

constexpr uint32_t kKvBlk = 64 * 128;                    // tile: 64 rows x 64 cols, SW128
constexpr uint32_t kKvRope = 64 * 64;                    // tile: 64 rows x 32 cols, SW64
constexpr uint32_t kStageBytes = 4 * kKvBlk + kKvRope;   // 36864
constexpr uint32_t kQBlk = 128 * 128;                    // Q: 128 rows x 64 cols, SW128
constexpr uint32_t kQRope = 128 * 64;                    // Q: 128 rows x 32 cols, SW64
constexpr uint32_t kQBytes = 4 * kQBlk + kQRope;         // 73728
constexpr uint32_t kPHalf = 64 * 64;                     // 64 rows x 32 tokens bf16, SW64

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKv = kOffQ + kQBytes;
constexpr uint32_t kOffP = kOffKv + kStages * kStageBytes;   // [2] second halves of P
constexpr uint32_t kOffMax = kOffP + 2 * kPHalf;             // float [2 tile parity][64 rows]
constexpr uint32_t kOffSum = kOffMax + 2 * 64 * 4;           // float [2 segment parity][2 kind][2 group][64 rows]
constexpr uint32_t kOffScratch = kOffSum + 2 * 2 * 2 * 64 * 4;    // 16 words written by the odd CTA's signals
constexpr uint32_t kOffBar = kOffScratch + 64;

// Barriers of the even CTA that the odd CTA signals ("paired" below) count
// the even CTA's own arrivals, and the odd CTA's signals as 4-byte
// transactions (st.async) that one of the even CTA's arrivals announces.
enum Bar {
  LOCAL_FULL = 0,                  // [stage] this CTA's TMA bytes of a stage (tail tiles)
  KV_FULL = LOCAL_FULL + kStages,  // [stage] even CTA: both CTAs' stage ready; full tiles count
                                   //     both CTAs' TMA bytes, tail tiles the relays' signals
  KV_EMPTY = KV_FULL + kStages,    // [stage] P . C of the stage's tile done (paired commit)
  S_FULL = KV_EMPTY + kStages,     // [2] per S buffer (paired commit)
  S_EMPTY = S_FULL + 2,            // [2] even CTA, paired: softmax warps read the S buffer
  P_FULL = S_EMPTY + 2,            // [2] even CTA, paired: softmax warps wrote P
  PV_DONE = P_FULL + 2,            // [2] (paired commit)
  Q_LOCAL = PV_DONE + 2,           // this CTA's query bytes
  Q_FULL,                          // even CTA, paired: both queries in place (relays)
  Q_EMPTY,                         // last S of a segment done (paired commit)
  DEC,                             // [2] per softmax group: its 4 warps decided a tile's maximum
  GRP = DEC + 2,                   // the 8 softmax warps of this CTA
  EPI_FREE,                        // [4] per segment (mod 4): the 8 softmax warps' output stores have
                                   //     read the two stages that they are staged in
  O_FREE = EPI_FREE + 4,           // even CTA, paired: the softmax warps have read a segment's O
  MMA_FINAL,                       // even CTA: all S issued so far are complete
  MMA_FINAL_PV,                    // even CTA: all P . C issued so far are complete
  BAR_COUNT
};
constexpr uint32_t kOffTmemSlot = kOffBar + BAR_COUNT * 8;
constexpr uint32_t kSmemUsed = kOffTmemSlot + 16;
constexpr size_t kSmemBytes = kSmemUsed;  // the base is 1024-byte aligned (checked at entry)

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;     // 2 x 128 columns
constexpr uint32_t kTmemO = 256;   // 2 x 128 columns (latent blocks 0-255, 256-511)
constexpr float kRescaleThreshold = 30.0f;  // log2 units: rescale O only if the max grows by > 2^30
constexpr int kPrefetchAhead = 4;           // tiles between an L2 prefetch and the tile's TMA load
constexpr uint16_t kBothCtas = 3;

static_assert(kOffKv % 1024 == 0 && kStageBytes % 1024 == 0 && kOffP % 1024 == 0, "align");
static_assert(kSmemBytes <= 232448, "shared memory");

// First latent column of 64-column block kc (0..3) of the columns CTA `half`
// owns; the RoPE columns of that CTA start at 512 + 32 half.
__device__ __forceinline__ int lat_col(int kc, int half) {
  return (kc >> 1) * 256 + half * 128 + (kc & 1) * 64;
}

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

// 16 lanes x 64 consecutive fp32 columns of TMEM, as the accumulator fragments
// of 8 tiles of 16 x 8: v[4 i + 2 e + f] = (lane l / 4 + 8 e, column 8 i +
// 2 (l % 4) + f) for thread l.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
// Four 8 x 8 matrices of 16-bit values to shared memory; lane l gives the
// address of row l % 8 of matrix l / 8 (16 bytes) and holds of each matrix the
// pair (row l / 4, columns 2 (l % 4) + {0, 1}).
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
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
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(LOCAL_FULL + s), 1);
      mbar_init(bar(KV_FULL + s), 1);
      mbar_init(bar(KV_EMPTY + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(S_EMPTY + i), 4);
      mbar_init(bar(P_FULL + i), 4);
      mbar_init(bar(DEC + i), 4);
      mbar_init(bar(PV_DONE + i), 1);
    }
    mbar_init(bar(Q_LOCAL), 1);
    mbar_init(bar(Q_FULL), 1);
    mbar_init(bar(Q_EMPTY), 1);
    mbar_init(bar(GRP), 8);
    for (int i = 0; i < 4; ++i) mbar_init(bar(EPI_FREE + i), 8);
    mbar_init(bar(O_FREE), 8);
    mbar_init(bar(MMA_FINAL), 1);
    mbar_init(bar(MMA_FINAL_PV), 1);
    fence_mbar_init();
  }
  if (warp == kWarpAlloc) {
    tmem_alloc_pair(sbase + kOffTmemSlot, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&p.maps.kv_lat4);
    prefetch_tmap(&p.maps.kv_rope);
  }
  if (warp == kWarpRelay && lane == 0) {
    prefetch_tmap(p.maps.has_q4 ? &p.maps.q_lat4 : &p.maps.q_lat);
    prefetch_tmap(p.maps.has_q4 ? &p.maps.q_rope4 : &p.maps.q_rope);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and TMEM exist before either uses the other's
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + kOffTmemSlot);
  // everything above overlaps the plan kernel; its results are read below
  pdl_wait_previous();
  pdl_launch_dependents();

  if (warp == kWarpTma) {
    // ------------------------------------------------------------ producer
    // a sequence of one row block reads each of its tiles once: those are
    // evicted from L2 first; with more blocks other clusters read the same
    // tiles, from L2 if they are still there
    const uint64_t pol_once = l2_policy_evict_first(), pol_shared = l2_policy_evict_normal();
    TreeWalk walk;
    walk.init(p.rec, p.seqs, p.n_h, chunk);
    TreeSegment sg;
    int g = 0;
    // A segment that ends before tile e stages its output in the stages of
    // tiles e - 2 and e - 1, which tiles e + 2 and e + 3 take next: those wait
    // for its stores.  epi: segments waited for; e0, e1, e2: the ends of the
    // `open` ones after them (at most e = g - 2, g - 1 and g)
    int epi = 0, open = 0, e0 = 0, e1 = 0, e2 = 0;
    uint32_t tail_used = 0, tail_phase = 0;  // stages that held a tail tile; parity of its LOCAL_FULL's next phase
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int* bt = p.block_table + (size_t)sg.seq.b * p.max_pages;
      const int L = sg.seq.L;
      const uint64_t pol_stream = sg.seq.blocks == 1 ? pol_once : pol_shared;
      for (int t0 = sg.t0; ok && t0 < sg.t1; t0 += 32) {
        // each lane fetches the page of one upcoming tile
        int my_page = 0;
        if (t0 + lane < sg.t1) {
          my_page = bt[((t0 + lane) * kTreeTile) / p.page_size];
          if (my_page < 0 || my_page >= p.num_pages) {
            atomicOr(p.err, MLA_DEVFLAG_BAD_PAGE);
            my_page = 0;
          }
        }
        const int n_here = min(32, sg.t1 - t0);
        for (int i = 0; i < n_here; ++i, ++g) {
          const int page = __shfl_sync(0xffffffffu, my_page, i);
          // The tile kPrefetchAhead tiles later goes to L2 now: its TMA load is
          // issued only when a stage frees (after this tile's P . C), and an
          // L2 hit then lands in a fraction of the HBM latency, which would
          // otherwise keep every stage busy that much longer.  A 64-token
          // tile of one page is 64 x 1152 contiguous bytes; the even CTA
          // fetches all of it.
          // At the start of a chunk every SM is already loading its query and
          // first stages; fetching more then only delays those, so the first
          // kStages tiles of the chunk prefetch nothing.
          const int page_ahead = __shfl_sync(0xffffffffu, my_page, (i + kPrefetchAhead) & 31);
          if (leader && g >= kStages && i + kPrefetchAhead < n_here && elect_one()) {
            const int tok_a = (t0 + i + kPrefetchAhead) * kTreeTile;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(
                p.kv + ((size_t)page_ahead * p.page_size + tok_a % p.page_size) * (kDc + 64));
            constexpr uint32_t kTile = kTreeTile * (kDc + 64) * 2;
            for (uint32_t off = 0; off < kTile; off += 16384)
              bulk_prefetch_l2(src + off, min(16384u, kTile - off));
          }
          while (open > 0 && g >= e0 + 2) {
            ok = ok && warp_wait(bar(EPI_FREE + (epi & 3)), (epi >> 2) & 1, p.err);
            ++epi;
            --open;
            e0 = e1;
            e1 = e2;
          }
          const int s = g % kStages;
          if (!(ok = ok && warp_wait(bar(KV_EMPTY + s), ((g / kStages) & 1) ^ 1, p.err))) break;
          const int tok = (t0 + i) * kTreeTile;
          const int y = page * p.page_size + tok % p.page_size;
          const uint32_t st = sbase + kOffKv + s * kStageBytes;
          const bool tail = L - tok < kTreeTile;
          if (elect_one()) {
            if (tail) {
              // this CTA's relay zeroes the rows past the end once they land,
              // then signals the even CTA
              mbar_arrive_expect_tx(bar(LOCAL_FULL + s), kStageBytes);
              tma_load_4d_hint(st, &p.maps.kv_lat4, bar(LOCAL_FULL + s), 128 * (int)rank, y, 0, 0,
                               pol_stream);
              tma_load_2d_hint(st + 4 * kKvBlk, &p.maps.kv_rope, bar(LOCAL_FULL + s),
                               kDc + 32 * (int)rank, y, pol_stream);
            } else if (leader) {
              // full tile: both CTAs' bytes complete on the even CTA's barrier
              mbar_arrive_expect_tx(bar(KV_FULL + s), 2 * kStageBytes);
              tma_load_4d_hint(st, &p.maps.kv_lat4, bar(KV_FULL + s), 0, y, 0, 0, pol_stream);
              tma_load_2d_hint(st + 4 * kKvBlk, &p.maps.kv_rope, bar(KV_FULL + s), kDc, y, pol_stream);
            } else {
              const uint32_t full = mapa(bar(KV_FULL + s), 0);
              tma_load_4d_to_pair_hint(st, &p.maps.kv_lat4, full, 128, y, 0, 0, pol_stream);
              tma_load_2d_to_pair_hint(st + 4 * kKvBlk, &p.maps.kv_rope, full, kDc + 32, y, pol_stream);
            }
          }
          __syncwarp();
          if (tail) {
            tail_used |= 1u << s;
            tail_phase ^= 1u << s;
          }
        }
      }
      (open == 0 ? e0 : open == 1 ? e1 : e2) = g;
      ++open;
    }
    // this CTA's tail copies land before it may exit (full tiles are consumed
    // by the paired MMAs before the final cluster barrier)
    for (int s = 0; s < kStages; ++s)
      if ((tail_used >> s) & 1) warp_wait(bar(LOCAL_FULL + s), ((tail_phase >> s) & 1) ^ 1, p.err);
  } else if (warp == kWarpRelay) {
    // ------------------------------------------------------------ relay
    TreeWalk walk;
    walk.init(p.rec, p.seqs, p.n_h, chunk);
    TreeSegment sg;
    int g = 0, seg_i = 0;
    uint32_t tail_phase = 0;  // parity of each stage's next LOCAL_FULL phase
    bool ok = true;
    bool q_in_flight = false;
    while (ok && walk.next(sg)) {
      // this segment's query rows (i, j) = Q[64 rank + 16 qd + i, columns of
      // CTA j], stored as row 32 qd + 16 j + i.  Rows past the block's last
      // belong to the next sequence, or read as zero behind q's end: nothing
      // of theirs is written.
      // the query area is free once the previous segment's last S has read it
      if (seg_i > 0 && !(ok = warp_wait(bar(Q_EMPTY), (seg_i - 1) & 1, p.err))) break;
      if (elect_one()) {
        const int y0 = sg.first + 64 * (int)rank;
        mbar_arrive_expect_tx(bar(Q_LOCAL), kQBytes);
        if (p.maps.has_q4) {
          // one copy per 64-column block: rows 32 qd + 16 j + i at once
          for (int kc = 0; kc < 4; ++kc)
            tma_load_4d(sbase + kOffQ + kc * kQBlk, &p.maps.q_lat4, bar(Q_LOCAL), lat_col(kc, 0), 0,
                        0, y0 >> 4);
          tma_load_4d(sbase + kOffQ + 4 * kQBlk, &p.maps.q_rope4, bar(Q_LOCAL), kDc, 0, 0, y0 >> 4);
        } else {
          for (int qd = 0; qd < 4; ++qd)
            for (int j = 0; j < 2; ++j) {
              const uint32_t r0 = static_cast<uint32_t>(32 * qd + 16 * j);
              for (int kc = 0; kc < 4; ++kc)
                tma_load_2d(sbase + kOffQ + kc * kQBlk + r0 * 128, &p.maps.q_lat, bar(Q_LOCAL),
                            lat_col(kc, j), y0 + 16 * qd);
              tma_load_2d(sbase + kOffQ + 4 * kQBlk + r0 * 64, &p.maps.q_rope, bar(Q_LOCAL),
                          kDc + 32 * j, y0 + 16 * qd);
            }
        }
      }
      q_in_flight = true;
      // the next segment's query rows go to L2 now, so that its TMA load
      // after this segment's last S is an L2 hit
      if (lane == 0) {
        TreeWalk peek = walk;
        TreeSegment nx;
        if (peek.next(nx) && nx.rows > 64 * (int)rank) {
          const __nv_bfloat16* src = p.q + ((size_t)nx.first + 64 * rank) * (kDc + 64);
          const uint32_t bytes =
              static_cast<uint32_t>(min(64, nx.rows - 64 * (int)rank)) * (kDc + 64) * 2;
          for (uint32_t off = 0; off < bytes; off += 16384)
            bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(src) + off, min(16384u, bytes - off));
        }
      }
      if (!(ok = warp_wait(bar(Q_LOCAL), seg_i & 1, p.err))) break;
      q_in_flight = false;
      if (lane == 0) signal_lead(Q_FULL, true, 4u, 8);
      __syncwarp();

      const int L = sg.seq.L;
      for (int t = sg.t0; t < sg.t1; ++t, ++g) {
        const int s = g % kStages;
        const int rows_valid = L - t * kTreeTile;
        if (rows_valid >= kTreeTile) continue;  // full tile: no relay
        if (!(ok = warp_wait(bar(LOCAL_FULL + s), (tail_phase >> s) & 1, p.err))) break;
        tail_phase ^= 1u << s;
        // rows past the sequence end may hold anything; make them zero so
        // that 0-probability x garbage cannot turn into NaN in P . C
        uint8_t* tile = base + kOffKv + s * kStageBytes;
        // 16 bytes per lane: a row's 4 x 128 latent bytes, 8 rows' 64 RoPE bytes
        for (int r = rows_valid; r < kTreeTile; ++r)
          *reinterpret_cast<uint4*>(tile + (lane >> 3) * kKvBlk + r * 128 + (lane & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        for (int r = rows_valid + (lane >> 2); r < kTreeTile; r += 8)
          *reinterpret_cast<uint4*>(tile + 4 * kKvBlk + r * 64 + (lane & 3) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) signal_lead(KV_FULL + s, true, 4u, 9);
        __syncwarp();
      }
      ++seg_i;
    }
    // a query copy still in flight must land before the CTA may exit
    if (q_in_flight) warp_wait(bar(Q_LOCAL), seg_i & 1, p.err);
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
      constexpr uint32_t kIdS = idesc_bf16(256, 128, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, 256, true);
      TreeWalk walk;
      walk.init(p.rec, p.seqs, p.n_h, chunk);
      TreeSegment sg;
      int g0 = 0, seg_i = 0;
      bool ok = true;
      // Descriptors are the first tile's plus a distance in 16-byte units: the
      // one thread that issues has 18 products a tile to keep the pipe fed
      const uint64_t q_lat = smem_desc(sbase + kOffQ, 16, 1024, kLayoutSW128);
      const uint64_t q_rope = smem_desc(sbase + kOffQ + 4 * kQBlk, 16, 512, kLayoutSW64);
      const uint64_t k_lat = smem_desc(sbase + kOffKv, 16, 1024, kLayoutSW128);
      const uint64_t k_rope = smem_desc(sbase + kOffKv + 4 * kKvBlk, 16, 512, kLayoutSW64);
      const uint64_t v_lat = smem_desc(sbase + kOffKv, kKvBlk, 1024, kLayoutSW128);
      const uint64_t p_ring = smem_desc(sbase + kOffP, 16, 512, kLayoutSW64);
      // S for global tile g: 16 steps over the latent columns, 2 over RoPE
      auto issue_s = [&](int g, bool last) {
        tc_fence_after();
        const uint32_t st = (g % kStages) * (kStageBytes >> 4);
        const uint32_t dS = tmem + kTmemS + (g & 1) * 128;
#pragma unroll
        for (int kc = 0; kc < 4; ++kc)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ss_pair(dS, q_lat + kc * (kQBlk >> 4) + ks * 2,
                             k_lat + st + kc * (kKvBlk >> 4) + ks * 2, kIdS, kc + ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          umma_f16_ss_pair(dS, q_rope + ks * 2, k_rope + st + ks * 2, kIdS, 1u);
        umma_commit_pair(bar(S_FULL + (g & 1)), kBothCtas);
        if (last) umma_commit_pair(bar(Q_EMPTY), kBothCtas);
      };
      // O (+)= P . C for global tile g; `first` = first tile of its segment
      auto issue_pv = [&](int g, bool first) {
        tc_fence_after();
        const uint32_t st = (g % kStages) * (kStageBytes >> 4);
        // P tokens 0-31 sit in the stage's RoPE block (S is done with it),
        // tokens 32-63 in the second-half ring
        const uint64_t pa[2] = {k_rope + st, p_ring + (g & 1) * (kPHalf >> 4)};
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 tokens per MMA
            umma_f16_ss_pair(tmem + kTmemO + blk * 128, pa[kk >> 1] + (kk & 1) * 2,
                             v_lat + st + 2 * blk * (kKvBlk >> 4) + kk * (2048 >> 4), kIdPV,
                             (first && kk == 0) ? 0u : 1u);
        umma_commit_pair(bar(KV_EMPTY + g % kStages), kBothCtas);
        umma_commit_pair(bar(PV_DONE + (g & 1)), kBothCtas);
      };
      // S runs up to two tiles ahead of P . C (its two buffers), so the softmax
      // of a tile has two S of tensor work to hide behind.
      auto wait = [&](int b, uint32_t parity) {
        return mbar_wait(bar(b), parity, p.err, MLA_DEVFLAG_TIMEOUT);
      };
      const bool s_issuer = warp == kWarpMma;
      while (ok && walk.next(sg)) {
        const int n_t = sg.t1 - sg.t0;
        if (s_issuer) {
          // S(g) once its stage is loaded and its S buffer has been read
          if (!(ok = wait(Q_FULL, seg_i & 1))) break;
          for (int j = 0; ok && j < n_t; ++j) {
            const int g = g0 + j;
            if (!(ok = wait(S_EMPTY + (g & 1), ((g >> 1) & 1) ^ 1) &&
                       wait(KV_FULL + g % kStages, (g / kStages) & 1)))
              break;
            issue_s(g, j == n_t - 1);
          }
        } else {
          // P . C(g) once P(g) is written
          for (int j = 0; ok && j < n_t; ++j) {
            const int g = g0 + j;
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
      // every MMA issued by this thread has completed before TMEM is freed
      const int fin = s_issuer ? MMA_FINAL : MMA_FINAL_PV;
      umma_commit_pair(bar(fin), 1);
      wait(fin, 0);
    }
    __syncwarp();
  } else if (warp >= kWarpSoftmax0) {
    // ------------------------------------------------------------ softmax
    // Two groups of four warps take alternate tiles (group = g & 1, which is
    // also the tile's S buffer and P ring slot); warp q of a group reads TMEM
    // lanes [32q, 32q + 32) for all 64 tokens, so a row's tile maximum needs
    // no exchange between warps.  The running maximum after tile g is
    // published per row in shared memory (slot g & 1); a group decides tile
    // g from the maximum after tile g - 1, which the other group published.
    const int sw_warp = warp - kWarpSoftmax0;       // 0..7
    const int grp = sw_warp >> 2;                   // softmax group; also the O block it drains
    const int gw = sw_warp & 3;                     // warp within the group
    const int qd = warp & 3;                        // TMEM lanes [32 qd, 32 qd + 32)
    const int rl = 16 * qd + (lane >> 2);           // this thread's S rows (of this CTA's 64): rl and rl + 8
    const int tk = 2 * (lane & 3);                  // and their tokens: 8 i + tk + {0, 1}, i < 8
    const int hO = (32 * qd + lane) & 63;           // row of this thread's O lane
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    // stmatrix addresses: lane l gives row l % 8 of 8 x 8 matrix l / 8 (rows
    // rl, rl + 8 of token group i, then of group i + 1)
    const int pr = 16 * qd + (lane & 15), pg = lane >> 4;
    const uint32_t sw64 = static_cast<uint32_t>((pr >> 1) & 3);  // 64-byte swizzle of row pr
    float* mx_pub = reinterpret_cast<float*>(base + kOffMax);  // [tile parity][row]
    // [kind][group][row], of two segments in turn
    float* sums = reinterpret_cast<float*>(base + kOffSum);
    int seg_i = 0;
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
      float m_used[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, l_exact[2] = {0.f, 0.f};
      for (int jt = (grp - g0) & 1; jt < n_t; jt += 2) {
        const int gt = g0 + jt;
        const int tok0 = (sg.t0 + jt) * kTreeTile;
        // a tile that reaches into the drafted tokens: which of them this
        // thread's rows see (none for rows past the block's last, whose
        // results are not written), read while S of the tile runs
        const bool tail = tok0 > P0 - kTreeTile;
        unsigned long long seen[2] = {0, 0};
        if (tail) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 64 * (int)rank + rl + 8 * e;
            if (r < sg.rows) seen[e] = p.mask[sg.seq.row0 + (sg.g * kTreeRows + r) / p.n_h];
          }
        }
        // ---- partial scores of tile gt -> registers; free the S buffer
        ok = ok && warp_wait(bar(S_FULL + grp), (gt >> 1) & 1, p.err);
        tc_fence_after();
        // sc[4 i + 2 e + f]: row rl + 8 e, token 8 i + tk + f.  The two partials
        // of 16 rows sit in lanes 32 qd + {0 .. 15} (CTA 0's columns, first half
        // of the buffer's columns) and 32 qd + {16 .. 31} (CTA 1's, second
        // half): two loads of 16 lanes put both in the same thread.
        float sc[32];
        {
          const uint32_t sb = tmem + lane_base + kTmemS + grp * 128;
          float other[32];
          tmem_ld_16x64(sb, sc);
          tmem_ld_16x64(sb + (16u << 16) + 64, other);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) sc[k] += other[k];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) signal_lead(S_EMPTY + grp, gw == 0, 16u, gw);
        uint32_t clear_lo = 0, clear_hi = 0;  // tokens whose non-finite values must not meet P . C
        if (tail) {
          // bit k = position tok0 + k: the context, then the drafted tokens
          const int sh = tok0 - P0;  // > -64; at most n - 1
          const unsigned long long ctx = sh >= 0 ? 0 : (1ull << -sh) - 1;
          const unsigned long long drafted = n < 64 ? (1ull << n) - 1 : ~0ull;
          uint32_t bad[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const unsigned long long bits = seen[e] & drafted;
            const unsigned long long vis = (sh >= 0 ? bits >> sh : (bits << -sh) | ctx) >> tk;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                float& x = sc[4 * i + 2 * e + f];
                // (rows past the sequence's end are zero: their scores are finite)
                if (!(fabsf(x) <= 3.402823466e38f)) bad[i >> 2] |= 1u << (8 * (i & 3) + f);
                if (!((vis >> (8 * i + f)) & 1)) x = -INFINITY;
              }
          }
          if (gw == 0 && __any_sync(0xffffffffu, (bad[0] | bad[1]) != 0)) {
            clear_lo = __reduce_or_sync(0xffffffffu, bad[0] << tk);
            clear_hi = __reduce_or_sync(0xffffffffu, bad[1] << tk);
          }
        }
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m0 = sc[2 * e], m1 = sc[2 * e + 1];
#pragma unroll
          for (int i = 1; i < 8; ++i) {
            m0 = fmaxf(m0, sc[4 * i + 2 * e]);
            m1 = fmaxf(m1, sc[4 * i + 2 * e + 1]);
          }
          mx[e] = fmaxf(m0, m1);
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1)
#pragma unroll
          for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        // ---- the maximum after this tile.  The running maximum may go
        // stale: it moves only when a tile's maximum exceeds it by more than
        // 2^kRescaleThreshold (weights stay below that factor), which keeps O
        // rescales rare.  Raw scores: scale > 0 commutes with max.
        if (jt > 0)  // tile gt - 1 (the other group's) is in this segment
          ok = ok && warp_wait(bar(DEC + (grp ^ 1)), ((gt - 1) >> 1) & 1, p.err);
        float m_new[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float t_s = mx[e] * c_log2;
          const float m_prev = jt > 0 ? mx_pub[((gt - 1) & 1) * 64 + rl + 8 * e] : -INFINITY;
          m_new[e] = (m_prev == -INFINITY || t_s > m_prev + kRescaleThreshold) ? fmaxf(m_prev, t_s) : m_prev;
          if ((lane & 3) == 0) mx_pub[(gt & 1) * 64 + rl + 8 * e] = m_new[e];
        }
        named_bar_sync(1 + grp, 128);
        // O lane hO: rescale if its row's maximum moved at this tile
        float alpha_o = 1.f;
        bool resc_o = false;
        if (jt > 0) {
          const float mo_prev = mx_pub[((gt - 1) & 1) * 64 + hO];
          const float mo_new = mx_pub[(gt & 1) * 64 + hO];
          if (mo_new != mo_prev) {
            alpha_o = ex2_approx(mo_prev - mo_new);  // mo_prev = -inf: O holds only zeros
            resc_o = true;
          }
        }
        // the decision of tile gt is published (and slot (gt - 1) & 1 read)
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DEC + grp));
        // this group's sums move to the new scale
        float neg_m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (m_new[e] != m_used[e]) {
            const float f = m_used[e] == -INFINITY ? 0.f : ex2_approx(m_used[e] - m_new[e]);
            l[e] *= f;
            l_exact[e] *= f;
            m_used[e] = m_new[e];
          }
          neg_m[e] = m_new[e] == -INFINITY ? 0.f : -m_new[e];
        }
        // pk[2 i + e]: the weights of row rl + 8 e, tokens 8 i + tk + {0, 1}.  u
        // is normalised by the sum of the rounded weights it was built from;
        // lse uses the unrounded weights
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float r0 = 0.f, r1 = 0.f, e0 = 0.f, e1 = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = ex2_approx(fmaf(sc[4 * i + 2 * e], c_log2, neg_m[e]));
            const float b = ex2_approx(fmaf(sc[4 * i + 2 * e + 1], c_log2, neg_m[e]));
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
            const float2 pf = __bfloat1622float2(h2);
            r0 += pf.x;
            r1 += pf.y;
            e0 += a;
            e1 += b;
            pk[2 * i + e] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          l[e] += r0 + r1;
          l_exact[e] += e0 + e1;
        }

        // P's ring slot grp was last read by PV(gt - 2); O may be rescaled
        // only after PV(gt - 1) (tiles of an earlier segment were retired by
        // that segment's epilogue, and the first P . C of a segment
        // overwrites O)
        if (gt >= 2) ok = ok && warp_wait(bar(PV_DONE + grp), ((gt - 2) >> 1) & 1, p.err);
        if (__any_sync(0xffffffffu, resc_o)) {
          ok = ok && warp_wait(bar(PV_DONE + (grp ^ 1)), ((gt - 1) >> 1) & 1, p.err);
          tc_fence_after();
          // both O blocks of these lanes, 8 columns at a time: this is rare, and
          // its registers are the loop's
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
        // P: row r, token group i (8 tokens, 16 bytes): half i / 4 of the row (32
        // tokens = 64 B, 64-byte swizzle) lives in the stage's RoPE block or in
        // ring slot grp
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t half = i < 4 ? sbase + kOffKv + (gt % kStages) * kStageBytes + 4 * kKvBlk
                                      : sbase + kOffP + grp * kPHalf;
          const uint32_t ch = static_cast<uint32_t>((i & 3) + pg);
          stmatrix_x4(half + pr * 64 + ((ch ^ sw64) << 4), pk[2 * i], pk[2 * i + 1], pk[2 * i + 2], pk[2 * i + 3]);
        }
        if (clear_lo | clear_hi) {
          // (uniform in the warp) S of this tile is done, its P . C waits for
          // this warp: clear the non-finite latent values of those tokens in
          // this CTA's columns, 16 bytes per lane and token
          unsigned long long todo = clear_lo | (static_cast<unsigned long long>(clear_hi) << 32);
          uint8_t* tile = base + kOffKv + (gt % kStages) * kStageBytes + (lane >> 3) * kKvBlk + (lane & 7) * 16;
          while (todo) {
            const int k = __ffsll(todo) - 1;
            todo &= todo - 1;
            uint4 v = *reinterpret_cast<uint4*>(tile + k * 128);
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
              if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
            }
            *reinterpret_cast<uint4*>(tile + k * 128) = v;
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
      // the maximum after the segment's last tile (decided by either group)
      if (((g - 1) & 1) != grp) ok = ok && warp_wait(bar(DEC + (grp ^ 1)), ((g - 1) >> 1) & 1, p.err);
      const float mO_fin = mx_pub[((g - 1) & 1) * 64 + hO];
      {
        // this group's sums in the scale of the final maximum
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m_fin = mx_pub[((g - 1) & 1) * 64 + rl + 8 * e];
          const float f = m_used[e] == m_fin ? 1.f : m_used[e] == -INFINITY ? 0.f : ex2_approx(m_used[e] - m_fin);
          float lf = l[e] * f, lef = l_exact[e] * f;
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            lf += __shfl_xor_sync(0xffffffffu, lf, o);
            lef += __shfl_xor_sync(0xffffffffu, lef, o);
          }
          if ((lane & 3) == 0) {
            sums[(0 * 2 + grp) * 64 + rl + 8 * e] = lf;
            sums[(1 * 2 + grp) * 64 + rl + 8 * e] = lef;
          }
        }
      }
      // every warp has read the published maxima of this segment, and the sums
      // of the last, before any starts the next one
      ok = rendezvous(ok);
      const float l_o = sums[(0 * 2 + 0) * 64 + hO] + sums[(0 * 2 + 1) * 64 + hO];
      const float le_o = sums[(1 * 2 + 0) * 64 + hO] + sums[(1 * 2 + 1) * 64 + hO];
      ok = ok && warp_wait(bar(PV_DONE + ((g - 1) & 1)), ((g - 1) >> 1) & 1, p.err);
      tc_fence_after();
      // no token seen: u = 0 (a NaN sum, of non-finite scores, stays)
      const float inv = l_o == 0.f ? 0.f : 1.f / l_o;
      const int c = grp;                          // O block drained by this group
      const int col0 = 256 * c + 128 * (qd >> 1);  // latent column of TMEM column kTmemO + 128c
      // The output is staged in the stages of the segment's last tiles (those
      // of tiles g - 2 and g - 1, whose P . C are done), 8 KB per warp: its 32
      // rows x 128 columns as boxes of 128-byte lines (64 bf16 or 32 fp32
      // columns) in the 128-byte-swizzled layout of the output tensor map
      // (16-byte chunk k of row r at k ^ (r & 7)).  The next segment's queries
      // and first two tiles load meanwhile.
      const uint32_t stg = sbase + kOffKv + static_cast<uint32_t>((g + 2 + grp) % kStages) * kStageBytes +
                           gw * 8192u;
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
          const uint32_t row = stg + static_cast<uint32_t>(c0 >> 6) * 4096u + lane * 128u;
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
              st_shared_v4(row + ((chunk16 ^ static_cast<uint32_t>(lane & 7)) << 4), w[0], w[1], w[2], w[3]);
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
        const float lse = le_o == 0.f ? -INFINITY : (mO_fin + log2f(le_o)) * 0.69314718055994531f;
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
        mbar_arrive(bar(EPI_FREE + (seg_i & 3)));
      }
      __syncwarp();
      ++seg_i;
      sums = reinterpret_cast<float*>(base + kOffSum) + (seg_i & 1) * 256;
    }
    // the last stores complete before the CTA exits
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // all paired MMAs are complete and no arrival is still on its way
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
