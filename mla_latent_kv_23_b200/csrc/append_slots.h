// Declarations of the latent append through a slot map.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

namespace mla {

constexpr int kClusterSizes = 4;  // 1, 2, 4, 8 CTAs along K

struct AppendSlotsArgs {
  void* cache;  // [rows, d_c + d_R]
  const int* slots;
  const int* pos;
  int* err;
  int T, d_model, d_c, d_R, rows;
  const int* max_clusters;  // [kClusterSizes] co-resident clusters of each size
  double rope_base;
};
bool append_slots_prepare(int (&max_clusters)[kClusterSizes]);
int append_slots_rows(int T);  // token rows of the x map's box
// w maps: box 64 x 32 rows; x map: box 64 x append_slots_rows(T); bf16, 128-byte swizzle
cudaError_t launch_append_slots(const AppendSlotsArgs& a, const CUtensorMap& w_dkv,
                                const CUtensorMap& w_kr, const CUtensorMap& x, cudaStream_t s);
cudaError_t launch_append_slots_f32(const AppendSlotsArgs& a, const float* h, const float* w_dkv,
                                    const float* w_kr, cudaStream_t s);

}  // namespace mla
