// Latent append through a slot map (mla_append_latent_slots): for token t
//     kv_cache[slots[t]] = [ W_DKV . h[t]  ||  RoPE(W_KR . h[t], pos[t]) ]
// ("MLA deep compression", low-rank projection and decoupled-RoPE sections).
//
// bf16, on the tensor cores (sm_100a): a dense product with the 576 features
// (128 rows of W_DKV or W_KR per tile) as M, up to 256 tokens as N and K =
// d_model.  Few tokens are bound by reading the weights once (8.3 MB at the
// DeepSeek-V3 shape), many by the operands' way from L2 to the SMs; both want
// every SM at work, which five feature tiles are not.  So K is split over the
// CTAs of a cluster, whose partial tiles (fp32) meet through distributed
// shared memory: rank r sums the tokens r, r + cs, ... over the ranks in order
// (the result does not depend on timing, and no scratch memory is needed),
// rotates the RoPE features and writes whole rows of 128 features.
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
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kWBlk = 128 * 128;  // 128 features x 64 bf16
constexpr int kMaxTokens = 256;        // tokens per CTA
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 8;
constexpr uint32_t kArea = 196608;     // pipeline stages, then the fp32 partial tile
static_assert(kArea >= kMaxTokens * 128 * 4 && kArea >= 4 * (kWBlk + kMaxTokens * 128), "area");

enum Bar { FULL = 0, EMPTY = FULL + kMaxStages, DONE = EMPTY + kMaxStages, BAR_COUNT };
constexpr uint32_t kOffBar = kArea;
constexpr uint32_t kOffSlot = kOffBar + BAR_COUNT * 8;
constexpr size_t kSmem = kOffSlot + 16 + 1024;  // + alignment slack

struct Params {
  CUtensorMap w_map[2];  // W_DKV, W_KR: box 64 x 128 rows
  CUtensorMap x_map;     // h [T, K]: box 64 x n_blk rows
  __nv_bfloat16* cache;
  const int* slots;
  const int* pos;
  int* err;
  int tiles0, K, T, n_blk, stages, tmem_cols, d_c, d_R, rows;
  double log_base;
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// (x0, x1) rotated by pos * base^(-k2 / d).  Positions reach 10^5 radians, so
// the angle is reduced in fp64.
__device__ __forceinline__ float2 rope_pair(float x0, float x1, int pos, double freq) {
  const double ang = (double)pos * freq;
  const float red = (float)(ang - 6.283185307179586 * floor(ang / 6.283185307179586));
  float s, c;
  sincosf(red, &s, &c);
  return make_float2(x0 * c - x1 * s, x0 * s + x1 * c);
}

// Grid (kCs, token blocks, feature tiles), cluster (kCs, 1, 1) along K.
template <int kCs>
__global__ void __launch_bounds__(kThreads, 1) append_slots_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int cs = kCs;
  const int rank = blockIdx.x;
  const int t0 = blockIdx.y * p.n_blk;
  const bool rope = (int)blockIdx.z >= p.tiles0;
  const int row0 = ((int)blockIdx.z - (rope ? p.tiles0 : 0)) * 128;
  const int kb_all = p.K / 64;
  const int kb0 = (int)((long long)kb_all * rank / cs), kb1 = (int)((long long)kb_all * (rank + 1) / cs);
  const uint32_t xblk = p.n_blk * 128, stage = kWBlk + xblk;
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(FULL + s), 2);  // the two producers
      mbar_init(bar(EMPTY + s), 1);
    }
    mbar_init(bar(DONE), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + kOffSlot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + kOffSlot);

  // this warp's tokens of the epilogue, one per lane: token `lane` of them is
  // (warp + kWarps lane) cs + rank of the block
  const int nt = min(p.n_blk, p.T - t0);
  const int my_t = (warp + kWarps * lane) * cs + rank;
  const int my_slot = my_t < nt ? p.slots[t0 + my_t] : -1;
  const int my_pos = my_t < nt && rope ? p.pos[t0 + my_t] : 0;

  bool ok = true;
  if ((warp == 0 || warp == 2) && lane == 0) {
    // producers: warp 0 the weights, warp 2 the tokens
    const CUtensorMap* m = warp == 2 ? &p.x_map : &p.w_map[rope ? 1 : 0];
    const uint32_t bytes = warp == 2 ? xblk : kWBlk, off = warp == 2 ? kWBlk : 0;
    const int y = warp == 2 ? t0 : row0;
    for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
      const int s = i % p.stages;
      if (i >= p.stages &&
          !(ok = mbar_wait(bar(EMPTY + s), ((i / p.stages) & 1) ^ 1, p.err, MLA_DEVFLAG_TIMEOUT)))
        break;
      mbar_arrive_expect_tx(bar(FULL + s), bytes);
      tma_load_2d(sbase + s * stage + off, m, bar(FULL + s), kb * 64, y);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16(128, p.n_blk, false);
    uint32_t acc = 0;
    for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
      const int s = i % p.stages;
      if (!(ok = mbar_wait(bar(FULL + s), (i / p.stages) & 1, p.err, MLA_DEVFLAG_TIMEOUT))) break;
      tc_fence_after();
      const uint32_t st = sbase + s * stage;
      for (int ks = 0; ks < 4; ++ks) {
        umma_f16_ss(tmem, smem_desc(st + ks * 32, 16, 1024, kLayoutSW128),
                    smem_desc(st + kWBlk + ks * 32, 16, 1024, kLayoutSW128), idesc, acc);
        acc = 1;
      }
      umma_commit(bar(EMPTY + s));
    }
    umma_commit(bar(DONE));
  }
  __syncwarp();
  if (threadIdx.x == 0) ok = mbar_wait(bar(DONE), 0, p.err, MLA_DEVFLAG_TIMEOUT) && ok;
  ok = __syncthreads_and(ok);
  tc_fence_after();
  // the partial tile as [token][128 features] in the pipeline's area (every
  // load has been consumed): TMEM lane = feature, column = token
  float* part = reinterpret_cast<float*>(base);
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  for (int c0 = (warp >> 2) * 32; c0 < p.n_blk; c0 += 64) {
    float v[32];
    tmem_ld32(tmem + lane_base + c0, v);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (c0 + k < p.n_blk) part[(c0 + k) * 128 + (warp & 3) * 32 + lane] = v[k];
  }
  tc_fence_before();
  cluster_sync();
  // one warp per token, four features per lane
  const int f = row0 + 4 * lane;
  const int width = p.d_c + p.d_R;
  const bool live = ok && f < (rope ? p.d_R : p.d_c);
  const double freq0 = rope ? exp(-(double)f / (double)p.d_R * p.log_base) : 0.0;
  const double freq1 = rope ? exp(-(double)(f + 2) / (double)p.d_R * p.log_base) : 0.0;
  for (int k = 0; k < (kMaxTokens + kWarps * cs - 1) / (kWarps * cs); ++k) {
    const int t = (warp + kWarps * k) * cs + rank;
    if (t >= nt) break;
    const int slot = __shfl_sync(0xffffffffu, my_slot, k), pos = __shfl_sync(0xffffffffu, my_pos, k);
    if (slot < 0) continue;
    if (slot >= p.rows) {
      if (lane == 0) atomicOr(p.err, MLA_DEVFLAG_BAD_PAGE);
      continue;
    }
    const uint32_t at = sbase + (t * 128 + 4 * lane) * 4;
    float4 y[cs];
#pragma unroll
    for (int r = 0; r < cs; ++r) y[r] = ld_cluster_v4(mapa(at, r));
    float4 x = y[0];
#pragma unroll
    for (int r = 1; r < cs; ++r) {
      x.x += y[r].x;
      x.y += y[r].y;
      x.z += y[r].z;
      x.w += y[r].w;
    }
    if (!live) continue;
    if (rope) {
      const float2 a = rope_pair(x.x, x.y, pos, freq0), b = rope_pair(x.z, x.w, pos, freq1);
      x = make_float4(a.x, a.y, b.x, b.y);
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

int append_slots_prepare() {
  auto prepare = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) == cudaSuccess;
  };
  if (!prepare(append_slots_kernel<1>) || !prepare(append_slots_kernel<2>) ||
      !prepare(append_slots_kernel<4>) || !prepare(append_slots_kernel<8>)) {
    cudaGetLastError();
    return 0;
  }
  return 1;
}

// Tokens per CTA: T in as few blocks of up to 256 as there have to be, all
// alike, in steps of 16 (the MMA's N).
int append_slots_tokens(int T) {
  const int blocks = (T + kMaxTokens - 1) / kMaxTokens;
  return ((T + blocks - 1) / blocks + 15) / 16 * 16;
}

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
  p.tiles0 = (a.d_c + 127) / 128;
  p.K = a.d_model;
  p.T = a.T;
  p.n_blk = append_slots_tokens(a.T);
  p.stages = std::min<int>(kMaxStages, kArea / (kWBlk + p.n_blk * 128));
  p.tmem_cols = 32;
  while (p.tmem_cols < p.n_blk) p.tmem_cols *= 2;
  p.d_c = a.d_c;
  p.d_R = a.d_R;
  p.rows = a.rows;
  p.log_base = log(a.rope_base);
  const int tiles = p.tiles0 + (a.d_R > 0 ? (a.d_R + 127) / 128 : 0);
  const int blocks = (a.T + p.n_blk - 1) / p.n_blk;
  // K over as many CTAs as fill the SMs once (powers of two: a cluster sits in
  // one GPC, and others would leave SMs of it idle), each with 4 blocks of 64
  // columns or more
  int cs = 1;
  while (2 * cs <= kMaxCluster && 2 * cs * tiles * blocks <= a.sm_count && 2 * cs * 256 <= a.d_model) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, blocks, tiles);
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
