// Latent append through a slot map (mla_append_latent_slots): for token t
//     kv_cache[slots[t]] = [ W_DKV . h[t]  ||  RoPE(W_KR . h[t], pos[t]) ]
// ("MLA deep compression", low-rank projection and decoupled-RoPE sections).
//
// bf16, on the tensor cores (sm_100a): up to 128 tokens are the M dimension,
// 32 j features (rows of W_DKV, then of W_KR) the N dimension, K = d_model.
// What bounds it is the operands' way into shared memory: few tokens read the
// weights once (8.3 MB at the DeepSeek-V3 shape), many re-read both operands
// from L2, and an SM gets about 130 B/ns with all of its stages in flight.  So
// K is split over the CTAs of a cluster until every SM loads, and with few
// tokens all of a CTA's blocks are in flight at once.  The partial tiles (fp32)
// meet through distributed shared memory: a rank sums its share of the tile over
// the ranks in order (the result does not depend on timing, and no scratch
// memory is needed), rotates the RoPE features and writes runs of four features
// (8 bytes a thread, neighbours side by side) of cache rows.
//
// fp32: one CTA per token and 32 features on the CUDA cores.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <cstring>

#include "append_slots.h"
#include "mla.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {
using namespace ptx;

constexpr int kThreads = 256;
constexpr int kTokens = 128;            // tokens per CTA, the MMA's M
constexpr int kBox = 32;                // features per weight copy
constexpr int kMaxBoxes = 9;            // feature boxes per CTA (N = 288 as two MMAs)
constexpr uint32_t kBoxBytes = kBox * 128;
constexpr int kProducers = kThreads / 32 - 1;  // warps that issue copies: all but warp 1
constexpr int kMaxStages = 16;
// pipeline stages, then the fp32 partial tile.  An MMA reads 128 token rows
// from a stage's start, also where fewer were loaded (what it reads there
// only reaches rows of D that are not used): 16 KB behind the last stage
constexpr uint32_t kArea = 212992;
constexpr int kPad = 4;                 // floats between rows of the partial tile
static_assert(1 + kMaxBoxes <= 2 * kProducers && kTokens <= kThreads, "copies per producer");
static_assert(kTokens * (kMaxBoxes * kBox + kPad) * 4 <= kArea, "the partial tile");
static_assert(2 * (kTokens * 128 + kMaxBoxes * kBoxBytes) + kTokens * 128 <= kArea, "two stages");

enum Bar { FULL = 0, EMPTY = FULL + kMaxStages, DONE = EMPTY + kMaxStages, BAR_COUNT };
constexpr uint32_t kOffBar = kArea;
constexpr uint32_t kOffTmem = kOffBar + BAR_COUNT * 8;
constexpr uint32_t kOffSlots = kOffTmem + 16;                    // int [128]
constexpr uint32_t kOffPos = kOffSlots + kTokens * 4;            // int [128]
constexpr uint32_t kOffTurn = kOffPos + kTokens * 4;             // double [144]
constexpr size_t kSmem = kOffTurn + kMaxBoxes * kBox / 2 * 8 + 1024;  // + alignment slack
static_assert(kOffTurn % 8 == 0 && kSmem <= 232448, "shared memory");

struct Params {
  CUtensorMap w_map[2];  // W_DKV, W_KR: box 64 x 32 rows
  CUtensorMap x_map;     // h [T, K]: box 64 x x_rows
  __nv_bfloat16* cache;
  const int* slots;
  const int* pos;
  int* err;
  int K, T, x_rows, boxes, stages, tmem_cols, d_c, d_R, rows;
  double log_base;
};

// One thread of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// A whole converged warp waits; a failed wait fails for every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, MLA_DEVFLAG_TIMEOUT));
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// (x0, x1) rotated by pos * turn full turns.  Positions reach 10^5 radians, so
// the turns are reduced in fp64; what is left, under half a turn, is good to
// 2^-25 of a turn in fp32.
__device__ __forceinline__ void rotate(float& x0, float& x1, int pos, double turn) {
  const double t = (double)pos * turn;
  float s, c;
  sincospif(2.f * (float)(t - rint(t)), &s, &c);
  const float y = x0 * c - x1 * s;
  x1 = x0 * s + x1 * c;
  x0 = y;
}

// Grid (kCs, feature tiles, token tiles), cluster (kCs, 1, 1) along K.
template <int kCs>
__global__ void __launch_bounds__(kThreads, 1) append_slots_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x;
  const int t0 = blockIdx.z * kTokens, nt = min(kTokens, p.T - t0);
  // boxes [box0, box0 + boxes) of W_DKV's nd and W_KR's nr
  const int nd = (p.d_c + kBox - 1) / kBox, nr = (p.d_R + kBox - 1) / kBox;
  const int box0 = blockIdx.y * p.boxes, boxes = min(p.boxes, nd + nr - box0);
  const int kb_all = p.K / 64;
  const int kb0 = (int)((long long)kb_all * rank / kCs), kb1 = (int)((long long)kb_all * (rank + 1) / kCs);
  const uint32_t xblk = p.x_rows * 128, stage = xblk + p.boxes * kBoxBytes;
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
  int* slots = reinterpret_cast<int*>(base + kOffSlots);
  int* pos = reinterpret_cast<int*>(base + kOffPos);
  double* turns = reinterpret_cast<double*>(base + kOffTurn);

  // what the epilogue needs of this thread's token, read ahead
  const int my_slot = (int)threadIdx.x < nt ? p.slots[t0 + threadIdx.x] : -1;
  const int my_pos = (int)threadIdx.x < nt && p.d_R > 0 ? p.pos[t0 + threadIdx.x] : 0;
  if (threadIdx.x == 64) {
    prefetch_tmap(&p.x_map);
    prefetch_tmap(&p.w_map[box0 < nd ? 0 : 1]);
  }
  const int copies = 1 + boxes;  // a block: the tokens, then the weight boxes
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(FULL + s), min(copies, kProducers));
      mbar_init(bar(EMPTY + s), 1);
    }
    mbar_init(bar(DONE), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + kOffTmem, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + kOffTmem);

  bool ok = true;
  if (warp != 1) {
    // ---------------------------------------------------------- producers
    // A block's copies and products are a few instructions, so what is done
    // around them counts: 0.49 us a block with both behind `lane == 0`, a
    // division per block and descriptors built anew; 0.22 with an elected
    // thread for the products (its operands stay in uniform registers) and the
    // copies of a block spread over seven warps, copy k on warp k % 7.
    const int w = warp == 0 ? 0 : warp - 1;
    if (w < copies) {
      uint32_t phase = 0;
      for (int kb = kb0, s = 0; kb < kb1; ++kb) {
        if (kb - kb0 >= p.stages) {
          if (!(ok = warp_wait(bar(EMPTY + s), phase, p.err))) break;
        }
        if (elect_one()) {
          const uint32_t st = sbase + s * stage, full = bar(FULL + s);
          const int second = w + kProducers < copies;
          mbar_arrive_expect_tx(full, (w == 0 ? xblk : kBoxBytes) + second * kBoxBytes);
          for (int k = w; k < copies; k += kProducers) {
            if (k == 0) {
              tma_load_2d(st, &p.x_map, full, kb * 64, t0);
            } else {
              const int box = box0 + k - 1;
              tma_load_2d(st + xblk + (k - 1) * kBoxBytes, &p.w_map[box < nd ? 0 : 1], full, kb * 64,
                          (box < nd ? box : box - nd) * kBox);
            }
          }
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          if (kb - kb0 >= p.stages) phase ^= 1;
        }
      }
    }
    // meanwhile: the turns of the tile's RoPE pairs, by pair within the tile
    for (int i = w * 32 + lane; i < boxes * kBox / 2; i += kProducers * 32) {
      const int f = (box0 - nd) * kBox + 2 * i;  // of the RoPE key
      if (f >= 0) turns[i] = exp(-(double)f / (double)p.d_R * p.log_base) * 0.15915494309189535;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const int n = p.boxes * kBox, parts = n > 256 ? 2 : 1;  // (N is at most 256)
    const uint32_t idesc = idesc_bf16(kTokens, n / parts, false);
    const uint64_t x0 = smem_desc(sbase, 16, 1024, kLayoutSW128);
    const uint64_t w0 = smem_desc(sbase + xblk, 16, 1024, kLayoutSW128);
    const uint32_t step = stage >> 4, half = (n / 2 * 128) >> 4;  // in a descriptor's 16-byte units
    uint32_t phase = 0, at = 0;
    if (elect_one()) {
      for (int kb = kb0, s = 0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(bar(FULL + s), phase, p.err, MLA_DEVFLAG_TIMEOUT))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t acc = ks > 0 || kb > kb0;
          umma_f16_ss(tmem, x0 + at + 2 * ks, w0 + at + 2 * ks, idesc, acc);
          if (parts == 2) umma_f16_ss(tmem + n / 2, x0 + at + 2 * ks, w0 + at + half + 2 * ks, idesc, acc);
        }
        umma_commit(bar(EMPTY + s));
        at += step;
        if (++s == p.stages) s = 0, phase ^= 1, at = 0;
      }
      umma_commit(bar(DONE));
      ok = mbar_wait(bar(DONE), 0, p.err, MLA_DEVFLAG_TIMEOUT) && ok;
    }
  }
  if ((int)threadIdx.x < nt) {
    slots[threadIdx.x] = my_slot;
    pos[threadIdx.x] = my_pos;
  }
  __syncwarp();
  ok = __syncthreads_and(ok);
  tc_fence_after();
  // the partial tile as [token][feature] in the pipeline's area (every load
  // has been consumed): TMEM lane = token, column = feature; the four spare
  // floats per row keep eight lanes' 16-byte stores on different banks
  const int ld = p.boxes * kBox + kPad;
  {
    const int t = (warp & 3) * 32 + lane;
    float* row = reinterpret_cast<float*>(base) + t * ld;
    const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if ((warp & 3) * 32 < nt)
      for (int c0 = (warp >> 2) * 32; c0 < boxes * kBox; c0 += 64) {
        float v[32];
        tmem_ld32(at + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          *reinterpret_cast<float4*>(row + c0 + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      }
  }
  tc_fence_before();
  cluster_sync();
  // this rank's share of the tile: runs of four features, token-major
  const int quads = boxes * kBox / 4, all = nt * quads;
  const int share = (all + kCs - 1) / kCs, end = min(all, share * (rank + 1));
  const int width = p.d_c + p.d_R;
  for (int i = share * rank + (int)threadIdx.x; i < end; i += kThreads) {
    const int t = i / quads, q = i - t * quads;
    const uint32_t at = sbase + (t * ld + 4 * q) * 4;
    float4 y[kCs];
#pragma unroll
    for (int r = 0; r < kCs; ++r) y[r] = ld_cluster_v4(mapa(at, r));
    float4 x = y[0];
#pragma unroll
    for (int r = 1; r < kCs; ++r) {
      x.x += y[r].x;
      x.y += y[r].y;
      x.z += y[r].z;
      x.w += y[r].w;
    }
    const int slot = slots[t];
    const bool rope = box0 + q / 8 >= nd;
    const int f = 4 * q + (rope ? (box0 - nd) * kBox : box0 * kBox);
    if (!ok || slot < 0 || f >= (rope ? p.d_R : p.d_c)) continue;
    if (slot >= p.rows) {
      atomicOr(p.err, MLA_DEVFLAG_BAD_PAGE);
      continue;
    }
    if (rope) {
      rotate(x.x, x.y, pos[t], turns[2 * q]);
      rotate(x.z, x.w, pos[t], turns[2 * q + 1]);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&lo);
    w.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p.cache + (size_t)slot * width + (rope ? p.d_c : 0) + f) = w;
  }
  cluster_sync();  // the other ranks have read this CTA's partial tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// Grid (tokens, groups of 32 features): warp w takes feature pairs of its group.
__global__ void __launch_bounds__(256)
    append_slots_f32_kernel(const float* __restrict__ h, const float* __restrict__ w_dkv,
                            const float* __restrict__ w_kr, const int* __restrict__ slots,
                            const int* __restrict__ pos, float* __restrict__ cache, int K, int d_c,
                            int d_R, int rows, double log_base, int* err) {
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = slots[t];
  if (slot < 0) return;
  if (slot >= rows) {
    if (threadIdx.x == 0) atomicOr(err, MLA_DEVFLAG_BAD_PAGE);
    return;
  }
  const float* x = h + (size_t)t * K;
  const int width = d_c + d_R;
  for (int f = blockIdx.y * 32 + 2 * warp; f < min(width, (int)blockIdx.y * 32 + 32); f += 16) {
    const float* w = f < d_c ? w_dkv + (size_t)f * K : w_kr + (size_t)(f - d_c) * K;
    float a = 0.f, b = 0.f;
    for (int k = lane; k < K; k += 32) {
      a = fmaf(x[k], w[k], a);
      b = fmaf(x[k], w[K + k], b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) {
      if (f >= d_c) {
        const double ang = (double)pos[t] * exp(-(double)(f - d_c) / (double)d_R * log_base);
        double s, c;
        sincos(ang - 6.283185307179586 * floor(ang / 6.283185307179586), &s, &c);
        const float a1 = a * (float)c - b * (float)s;
        b = a * (float)s + b * (float)c;
        a = a1;
      }
      *reinterpret_cast<float2*>(cache + (size_t)slot * width + f) = make_float2(a, b);
    }
  }
}

}  // namespace

bool append_slots_prepare(int (&max_clusters)[kClusterSizes]) {
  auto prepare = [&](auto kernel, int e) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
      return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1 << e, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1 << e;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(&max_clusters[e], kernel, &cfg) == cudaSuccess && max_clusters[e] > 0;
  };
  if (!prepare(append_slots_kernel<1>, 0) || !prepare(append_slots_kernel<2>, 1) ||
      !prepare(append_slots_kernel<4>, 2) || !prepare(append_slots_kernel<8>, 3)) {
    cudaGetLastError();
    return false;
  }
  return true;
}

// Token rows of one copy: T up to a whole 8-row group, 128 at most.
int append_slots_rows(int T) { return std::min(kTokens, (T + 7) / 8 * 8); }

cudaError_t launch_append_slots(const AppendSlotsArgs& a, const CUtensorMap& w_dkv,
                                const CUtensorMap& w_kr, const CUtensorMap& x, cudaStream_t s) {
  Params p;
  p.w_map[0] = w_dkv;
  p.w_map[1] = w_kr;
  p.x_map = x;
  p.cache = static_cast<__nv_bfloat16*>(a.cache);
  p.slots = a.slots;
  p.pos = a.pos;
  p.err = a.err;
  p.K = a.d_model;
  p.T = a.T;
  p.x_rows = append_slots_rows(a.T);
  p.d_c = a.d_c;
  p.d_R = a.d_R;
  p.rows = a.rows;
  p.log_base = log(a.rope_base);
  const int total = (a.d_c + kBox - 1) / kBox + (a.d_R + kBox - 1) / kBox;
  const int token_tiles = (a.T + kTokens - 1) / kTokens, kb = a.d_model / 64;
  // Boxes per CTA and CTAs along K, by what was measured (us): a block of 64
  // columns takes 0.22 or its bytes at 130 per ns, the exchange of the partial
  // tile its bytes at 25 per ns, the rest 5.  At d_model = 7168 it comes within
  // 15 % of what one wave of CTAs takes and of what several do, and takes the
  // fastest of these: 37 tokens 7.5 with (2 boxes, 8 CTAs), 8.2 with (3, 8),
  // 9.8 with (6, 8), 9.9 with (1, 4); 1024 tokens 16.1 with (5, 4), 18.0 with
  // (6, 4), 19.2 with (2, 2), 21.5 with (9, 4), 27.7 with (6, 2); 4096 tokens
  // 38.3 with (9, 2), 45.9 with (9, 4), 47.3 with (5, 2).
  int cs = 1;
  p.boxes = 1;
  double best = 0;
  for (int j = 1; j <= std::min(kMaxBoxes, total); ++j)
    for (int e = 0; e < kClusterSizes && (1 << e) <= kb; ++e) {
      const int clusters = (total + j - 1) / j * token_tiles;
      const int waves = (clusters + a.max_clusters[e] - 1) / a.max_clusters[e];
      const double block = std::max(0.22, (p.x_rows * 128 + j * kBoxBytes) / 130e3);
      const double t = waves * (((kb + (1 << e) - 1) >> e) * block +
                                std::min(a.T, kTokens) * j * kBox * 4 / 25e3 + 5);
      if (best == 0 || t < best) {
        best = t;
        p.boxes = j;
        cs = 1 << e;
      }
    }
  const uint32_t stage = p.x_rows * 128 + p.boxes * kBoxBytes;
  p.stages = std::min<int>(kMaxStages, (kArea - kTokens * 128) / stage);
  p.tmem_cols = 32;
  while (p.tmem_cols < p.boxes * kBox) p.tmem_cols *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (total + p.boxes - 1) / p.boxes, token_tiles);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cs == 8   ? cudaLaunchKernelEx(&cfg, append_slots_kernel<8>, p)
         : cs == 4 ? cudaLaunchKernelEx(&cfg, append_slots_kernel<4>, p)
         : cs == 2 ? cudaLaunchKernelEx(&cfg, append_slots_kernel<2>, p)
                   : cudaLaunchKernelEx(&cfg, append_slots_kernel<1>, p);
}

cudaError_t launch_append_slots_f32(const AppendSlotsArgs& a, const float* h, const float* w_dkv,
                                    const float* w_kr, cudaStream_t s) {
  const dim3 grid(a.T, (a.d_c + a.d_R + 31) / 32);
  append_slots_f32_kernel<<<grid, 256, 0, s>>>(h, w_dkv, w_kr, a.slots, a.pos,
                                               static_cast<float*>(a.cache), a.d_model, a.d_c, a.d_R,
                                               a.rows, log(a.rope_base), a.err);
  return cudaGetLastError();
}

}  // namespace mla
