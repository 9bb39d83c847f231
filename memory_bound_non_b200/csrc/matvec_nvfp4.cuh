// What the kernels of the NVFP4 matrix-vector product share.
#pragma once

#include "frt_device.cuh"
#include "frt_fragments.cuh"
#include "frt_launch.h"
#include "frt_tensor.cuh"

namespace frt {

constexpr int kGroup = 128;  // k of a step, and of a factor of x

// How x enters: 16 bits without factors (f16), with a power of two per group
// (bf16), codes.
enum XForm { kX16, kXScaled16, kXE4M3, kXE4M3Block, kXNvfp4 };

struct MatvecArgs {
  const void* x;
  const float* x_scales;
  const uint8_t* x_sf;
  const uint8_t* w_codes;
  const uint8_t* w_sf;
  const float* w_scale;
  const uint16_t* bias;
  uint16_t* y;
  int M, N, K;
  int m0, rows;    // rows of x of this launch: m0 .. m0 + rows - 1
  int groups;      // ceil(K / 128)
  int seg_groups;  // groups of x in shared memory at a time
  int kw, kw_log2; // warps that share a weight tile (a power of two)
  int tiles;       // weight tiles of 16 rows
  int cluster;     // CTAs that split k
  int swizzled;
  XForm form;
  int dt;
};

__device__ __forceinline__ int64_t sf_bytes(const MatvecArgs& a, int64_t n_rows) {
  const int cols = a.K >> 4;
  return a.swizzled ? ((n_rows + 127) >> 7) * (int64_t)((cols + 3) >> 2) * 512 : n_rows * cols;
}

template <int DT>
__device__ __forceinline__ float value16(uint16_t w) {
  return Pack16<DT>::to_float2((uint32_t)w).x;
}

// y[row r][n] from its sum, scaled and with the bias.
__device__ __forceinline__ void store_y1(const MatvecArgs& a, int r, int n, float sum, float scale) {
  const bool half = a.dt == FRT_F16;
  float b = 0.0f;
  if (a.bias != nullptr && FRT_IDX_OK(n, a.N)) b = half ? value16<FRT_F16>(a.bias[n]) : value16<FRT_BF16>(a.bias[n]);
  const float v = fmaf(sum, scale, b);
  const int64_t at = (int64_t)(a.m0 + r) * a.N + n;
  if (FRT_IDX_OK(at, (int64_t)a.M * a.N))
    a.y[at] = (uint16_t)(half ? Pack16<FRT_F16>::from_float2(v, 0.0f) : Pack16<FRT_BF16>::from_float2(v, 0.0f));
}
// Rows of x that one launch of the tile kernel takes.
constexpr int kTileXRows = 128;
frt_status launch_matvec_tiles(const MatvecArgs& a, cudaStream_t stream);

}  // namespace frt
