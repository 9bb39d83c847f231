// y = x w^T + bias with NVFP4 weights, for few rows of x.
//
// What bounds it: the weights, 0.5625 B each, read once; against that stand one
// cvt and one multiply per two weights and one mma.m16n8k16 per 256 weights and
// 8 rows.
//
// Mapping.  16 weight rows on the 16-row side of the mma, 8 NT rows of x on
// the other.  The order of k inside a product is free: with g = lane / 4 and t
// = lane % 4 a lane holds weight rows g and g + 8 at k = 32 t .. 32 t + 31 of a
// group of 128, one 16-byte load a row, and two factors a row.  A warp keeps
// four groups of weights on their way (4 KB and their factors), which is what
// covers the HBM latency; the KW warps of a CTA that share a weight tile split
// k, and their sums are joined in shared memory in a fixed order.
//
// x lies in shared memory as binary16 in the order in which the lanes read it.
// FP16 rows, e4m3 codes and NVFP4 code * factor are exact there.  bf16 rows are
// scaled by a power of two per row and group, and like the block-scaled FP8
// rows keep a factor per row and group that is applied to the group's fp32
// sums.
#include "frt_device.cuh"
#include "frt_host.h"

namespace frt {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 128;   // k of one load
constexpr int kItem = 4;      // groups a warp has on their way
constexpr int kSMs = 148;
constexpr int kXBytes = 80 * 1024;  // of x in shared memory at a time

// how x enters: 16-bit without a scale (f16), with a power of two per group
// (bf16), codes
constexpr int kXF16 = 0, kXBF16 = 1, kXE4M3 = 2, kXE4M3Block = 3, kXNvfp4 = 4;
__host__ __device__ constexpr bool group_scaled(int xf) { return xf == kXBF16 || xf == kXE4M3Block; }

struct Args {
  const void* x;
  const float* x_scales;
  const uint8_t* x_sf;
  const uint8_t* w_codes;
  const uint8_t* w_sf;
  const float* w_scale;
  const uint16_t* bias;
  uint16_t* y;
  int M, N, K;
  int m0, rows;      // rows of x of this launch: m0 .. m0 + rows - 1
  int groups;        // ceil(K / 128)
  int seg_items;     // items of x in shared memory at a time
  int kw;            // warps that share a weight tile (a power of two)
  int units;         // sets of kWarps / kw weight tiles
  int swizzled;
  int dt;
};

__device__ __forceinline__ int64_t sf_at(const Args& a, int64_t row, int col) {
  return a.swizzled ? sf_offset_swizzled(row, col, a.K >> 4) : row * (a.K >> 4) + col;
}
__device__ __forceinline__ int64_t sf_bytes(const Args& a, int64_t n_rows) {
  const int cols = a.K >> 4;
  return a.swizzled ? ((n_rows + 127) >> 7) * (int64_t)((cols + 3) >> 2) * 512 : n_rows * cols;
}

// Weights of one group: rows g and g + 8, 32 codes and two factors each.
struct WFrag {
  uint32_t c[2][4];
  uint32_t sf[2];
};
// A lane's loads of an item (kItem groups): the item's start in rows g and g +
// 8, and where its 32 codes of each group lie from there.  Every load is made:
// rows behind the last are row N - 1 again, their sums are dropped; codes
// behind K are the last ones again, x is zero there.
// LAY: 0 any K, 1 K % 32 == 0 with row-major factors, 2 with swizzled ones;
// K % 32 == 0 has 16-byte loads of codes and 2-byte loads of factors.
template <int LAY>
struct WLoader {
  const uint8_t* c[2];
  int row[2];
  int col[kItem];  // first of the two 16-blocks, from the start of the row

  __device__ __forceinline__ void set_rows(const Args& a, int row0, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row[h] = min(row0 + g + 8 * h, a.N - 1);
      c[h] = a.w_codes + (int64_t)row[h] * (a.K >> 1);
    }
  }
  __device__ __forceinline__ void set_item(const Args& a, int item, int t) {
    const int last = (a.K >> 4) - (LAY == 0 ? 1 : 2);
#pragma unroll
    for (int u = 0; u < kItem; ++u) col[u] = min((item * kItem + u) * (kGroup / 16) + 2 * t, last);
  }
  __device__ __forceinline__ void load(const Args& a, int u, WFrag& f) const {
    const int64_t bytes = (int64_t)a.N * (a.K >> 1), n_sf = sf_bytes(a, a.N);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* p = c[h] + 8 * col[u];
      f.sf[h] = 0;
      if (LAY == 0) {
        const int next = min(col[u] + 1, (a.K >> 4) - 1);
        const uint8_t* p1 = c[h] + 8 * next;
        const int64_t s0 = sf_at(a, row[h], col[u]), s1 = sf_at(a, row[h], next);
        uint2 v = make_uint2(0, 0), w = v;
        if (FRT_SPAN_OK(p - a.w_codes, 8, bytes)) v = ld_stream(reinterpret_cast<const uint2*>(p));
        if (FRT_SPAN_OK(p1 - a.w_codes, 8, bytes)) w = ld_stream(reinterpret_cast<const uint2*>(p1));
        if (FRT_IDX_OK(s0, n_sf) && FRT_IDX_OK(s1, n_sf)) f.sf[h] = __ldg(a.w_sf + s0) | __ldg(a.w_sf + s1) << 8;
        f.c[h][0] = v.x;
        f.c[h][1] = v.y;
        f.c[h][2] = w.x;
        f.c[h][3] = w.y;
      } else {
        const int64_t s = LAY == 2 ? sf_offset_swizzled(row[h], col[u], a.K >> 4)
                                   : (int64_t)row[h] * (a.K >> 4) + col[u];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (FRT_SPAN_OK(p - a.w_codes, 16, bytes)) v = ld_stream(reinterpret_cast<const uint4*>(p));
        if (FRT_SPAN_OK(s, 2, n_sf)) f.sf[h] = __ldg(reinterpret_cast<const uint16_t*>(a.w_sf + s));
        f.c[h][0] = v.x;
        f.c[h][1] = v.y;
        f.c[h][2] = v.z;
        f.c[h][3] = v.w;
      }
    }
  }
};

// Four elements of row r (0 based within the launch) at column k as two
// binary16 pairs, and the factor of (row, group): a warp holds the 128 elements
// of a group.
template <int XF>
__device__ __forceinline__ uint2 load_x4(const Args& a, int r, int k, float* scale) {
  const int64_t row = a.m0 + r;
  const bool on = r < a.rows && k < a.K;
  const int64_t at = row * a.K + k;
  const int64_t n = (int64_t)a.M * a.K;
  uint2 o = make_uint2(0, 0);
  *scale = 1.0f;
  if (XF == kXF16 || XF == kXBF16) {
    if (on && FRT_SPAN_OK(at, 4, n)) o = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + at);
    if (XF == kXBF16) {
      float2 u = Pack16<FRT_BF16>::to_float2(o.x), v = Pack16<FRT_BF16>::to_float2(o.y);
      const float s = pow2_to_half_range(warp_max_abs(absmax4(u.x, u.y, v.x, v.y)));
      o.x = Pack16<FRT_F16>::from_float2(u.x * s, u.y * s);
      o.y = Pack16<FRT_F16>::from_float2(v.x * s, v.y * s);
      *scale = 1.0f / s;
    }
  } else if (XF == kXE4M3 || XF == kXE4M3Block) {
    uint32_t w = 0;
    if (on && FRT_SPAN_OK(at, 4, n)) w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.x) + at);
    e4m3x4_to_half2(w, &o.x);
    const int64_t sa = row * a.groups + k / kGroup;
    if (XF == kXE4M3Block && on && FRT_IDX_OK(sa, (int64_t)a.M * a.groups)) *scale = a.x_scales[sa];
  } else {
    uint32_t w = 0, s = 0;
    if (on && FRT_SPAN_OK(at >> 1, 2, n >> 1))
      w = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.x) + (at >> 1));
    if (on) {
      const int64_t sa = sf_at(a, row, k >> 4);
      if (FRT_IDX_OK(sa, sf_bytes(a, a.M))) s = a.x_sf[sa];
    }
    uint32_t h[4], f[2];
    e2m1x8_to_half2(w, h);
    e4m3x4_to_half2(s * 0x0101u, f);
    o = make_uint2(hmul2(h[0], f[0]), hmul2(h[1], f[0]));
  }
  return o;
}

template <int NT, int XF, int LAY>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) matvec_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int mr = NT == 1 ? min(a.rows, 8) : 8;  // rows of x that shared memory holds per 8
  const int step_words = NT * mr * 4;           // 16-byte words of 32 k
  constexpr int kRed = NT * 8 * 17;             // a warp's sums, [row of x][weight row]
  float* red = reinterpret_cast<float*>(smem);
  uint2* xf = reinterpret_cast<uint2*>(smem + sizeof(float) * kWarps * kRed);
  float* xs = reinterpret_cast<float*>(xf + (size_t)a.seg_items * kItem * 8 * step_words);

  const int kw = a.kw, ks = warp & (kw - 1), rw = warp / kw, tiles_at_once = kWarps / kw;
  const int items = (a.groups + kItem - 1) / kItem;
  const bool one_seg = a.seg_items >= items;
  // rows of x that are not there: the last one again, its sums are dropped
  const uint4* x_lane = reinterpret_cast<const uint4*>(xf) + min(g, mr - 1) * 4 + t;

  // This warp's items: of each unit the items ks, ks + kw, ... of its weight
  // tile, unit after unit.
  struct Cursor {
    int unit, item;
  };
  auto advance = [&](Cursor c) {
    c.item += kw;
    if (c.item >= items) {
      c.item = ks;
      c.unit += gridDim.x;
    }
    return c;
  };
  WFrag w[kItem];
  WLoader<LAY> loader;
  Cursor cur = {(int)blockIdx.x, ks};  // (kw <= items)
  loader.set_rows(a, (cur.unit * tiles_at_once + rw) * 16, g);
  loader.set_item(a, ks, t);
#pragma unroll
  for (int u = 0; u < kItem; ++u) loader.load(a, u, w[u]);  // constant inputs: before the wait
  const float w_scale = __ldg(a.w_scale);
  pdl_enter();
  const float scale = w_scale * (XF == kXE4M3 || XF == kXNvfp4 ? a.x_scales[0] : 1.0f);

  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    for (int seg = 0; seg < items; seg += a.seg_items) {
      const int seg_end = min(seg + a.seg_items, items);
      if (!one_seg || unit == (int)blockIdx.x) {
        if (!one_seg) __syncthreads();  // the last segment is read
        const int rows = NT == 1 ? mr : 8 * NT;
        const int n_groups = min(seg_end * kItem, a.groups) - seg * kItem;
        for (int i = warp; i < rows * n_groups; i += kWarps) {
          const int r = i % rows, c = i / rows;
          float s;
          const uint2 v = load_x4<XF>(a, r, (seg * kItem + c) * kGroup + 4 * lane, &s);
          // steps 2p and 2p + 1 of a lane side by side
          const int pair = (lane & 7) >> 1;
          xf[((c * 4 + pair) * step_words + ((r >> 3) * mr + (r & 7)) * 4 + (lane >> 3)) * 2 + (lane & 1)] = v;
          if (group_scaled(XF) && lane == 0) xs[c * (8 * NT) + r] = s;
        }
        __syncthreads();
      }
      while (cur.unit == unit && cur.item < seg_end) {
        const Cursor next = advance(cur);
        if (next.unit != unit) loader.set_rows(a, (next.unit * tiles_at_once + rw) * 16, g);
        loader.set_item(a, next.item, t);
#pragma unroll
        for (int u = 0; u < kItem; ++u) {
          const int group = cur.item * kItem + u;
          if (group < a.groups) {
            const int c = group - seg * kItem;
            float part[NT][4];
            if (group_scaled(XF)) {
#pragma unroll
              for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.0f;
            }
            uint32_t sc[4];
            e4m3x4_to_half2(__byte_perm(w[u].sf[0], 0, 0x1100), sc);
            e4m3x4_to_half2(__byte_perm(w[u].sf[1], 0, 0x1100), sc + 2);
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // words of 8 codes
              uint32_t h0[4], h1[4];
              e2m1x8_to_half2(w[u].c[0][q], h0);
              e2m1x8_to_half2(w[u].c[1][q], h1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                h0[e] = hmul2(h0[e], sc[q >> 1]);
                h1[e] = hmul2(h1[e], sc[2 + (q >> 1)]);
              }
              const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
              const uint4* xb = x_lane + (c * 4 + q) * step_words;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 bv = xb[n * 32];
                mma_16816(group_scaled(XF) ? part[n] : acc[n], a0, bv.x, bv.y);
                mma_16816(group_scaled(XF) ? part[n] : acc[n], a1, bv.z, bv.w);
              }
            }
            if (group_scaled(XF)) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float s = xs[c * (8 * NT) + 8 * n + 2 * t + e];
                  acc[n][e] = fmaf(part[n][e], s, acc[n][e]);
                  acc[n][2 + e] = fmaf(part[n][2 + e], s, acc[n][2 + e]);
                }
            }
          }
          loader.load(a, u, w[u]);
        }
        cur = next;
      }
    }
    // sums of the warps that share a weight tile
    float* mine = red + warp * kRed;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mine[(8 * n + 2 * t + e) * 17 + g] = acc[n][e];
        mine[(8 * n + 2 * t + e) * 17 + g + 8] = acc[n][2 + e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < tiles_at_once * 16 * a.rows; i += kThreads) {
      const int col = i & 15, tile = (i >> 4) % tiles_at_once, r = (i >> 4) / tiles_at_once;
      const int n = (unit * tiles_at_once + tile) * 16 + col;
      if (n >= a.N) continue;
      float sum = 0.0f;
      for (int k = 0; k < kw; ++k) sum += red[(tile * kw + k) * kRed + r * 17 + col];
      sum *= scale;
      const bool half = a.dt == FRT_F16;
      if (a.bias != nullptr && FRT_IDX_OK(n, a.N)) {
        const uint32_t bw = a.bias[n];
        sum += half ? Pack16<FRT_F16>::to_float2(bw).x : Pack16<FRT_BF16>::to_float2(bw).x;
      }
      const int64_t at = (int64_t)(a.m0 + r) * a.N + n;
      if (FRT_IDX_OK(at, (int64_t)a.M * a.N))
        a.y[at] = (uint16_t)(half ? Pack16<FRT_F16>::from_float2(sum, 0.0f)
                                  : Pack16<FRT_BF16>::from_float2(sum, 0.0f));
    }
    __syncthreads();
  }
}

template <int NT, int XF, int LAY>
frt_status launch_one(Args a, cudaStream_t stream) {
  const int items = (a.groups + kItem - 1) / kItem;
  a.kw = 1;
  while (a.kw < kWarps && a.kw * 2 <= items) a.kw *= 2;
  const int tiles = (a.N + 15) / 16, at_once = kWarps / a.kw;
  a.units = (tiles + at_once - 1) / at_once;
  const size_t mr = NT == 1 && a.rows < 8 ? a.rows : 8;
  const size_t item_bytes = (size_t)kItem * (8 * NT * mr * 4 * 8 + (group_scaled(XF) ? 8 * NT * 4 : 0));
  const size_t red = sizeof(float) * kWarps * NT * 8 * 17;
  int64_t seg = kXBytes / item_bytes;
  if (seg < 1) seg = 1;
  if (seg > a.kw) seg -= seg % a.kw;
  a.seg_items = (int)(seg < items ? seg : items);
  const size_t smem = red + a.seg_items * item_bytes;
  static std::atomic<int> opted{48 * 1024};
  const frt_status st = opt_in_smem(matvec_kernel<NT, XF, LAY>, smem, opted);
  if (st != FRT_OK) return st;
  const int resident = kSMs * (NT <= 2 ? 2 : 1);
  const unsigned grid = (unsigned)(a.units < resident ? a.units : resident);
  return launch(matvec_kernel<NT, XF, LAY>, dim3(grid), dim3(kThreads), smem, stream, a);
}
template <int NT, int XF>
frt_status launch_wide(const Args& a, cudaStream_t stream) {
  if (a.K % 32 != 0) return launch_one<NT, XF, 0>(a, stream);
  return a.swizzled ? launch_one<NT, XF, 2>(a, stream) : launch_one<NT, XF, 1>(a, stream);
}
template <int XF>
frt_status launch_rows(Args a, cudaStream_t stream) {
  for (a.m0 = 0; a.m0 < a.M; a.m0 += 64) {
    a.rows = a.M - a.m0 < 64 ? a.M - a.m0 : 64;
    const frt_status st = a.rows <= 8    ? launch_wide<1, XF>(a, stream)
                          : a.rows <= 16 ? launch_wide<2, XF>(a, stream)
                          : a.rows <= 32 ? launch_wide<4, XF>(a, stream)
                          : a.rows <= 48 ? launch_wide<6, XF>(a, stream)
                                         : launch_wide<8, XF>(a, stream);
    if (st != FRT_OK) return st;
  }
  return FRT_OK;
}

}  // namespace
}  // namespace frt

using namespace frt;

extern "C" frt_status frt_matvec_nvfp4(const void* x, const float* x_scales, const uint8_t* x_sf,
                                       const uint8_t* w_codes, const uint8_t* w_sf, const float* w_scale,
                                       const void* bias, void* y, int M, int N, int K, frt_x_format x_format,
                                       frt_sf_layout sf_layout, frt_dtype dt, cudaStream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0 || x_format < FRT_X_16BIT || x_format > FRT_X_NVFP4 ||
      (sf_layout != FRT_SF_ROW_MAJOR && sf_layout != FRT_SF_SWIZZLED_128X4) || !valid_dtype(dt))
    return FRT_ERR_INVALID_ARG;
  if (M == 0) return FRT_OK;
  for (const void* p : {x, (const void*)w_codes, (const void*)w_sf})
    if (p == nullptr || !aligned(p, 16)) return FRT_ERR_INVALID_ARG;
  if (w_scale == nullptr || !aligned(w_scale, 4) || y == nullptr || !aligned(y, 2) || !aligned(bias, 2))
    return FRT_ERR_INVALID_ARG;
  if (x_format != FRT_X_16BIT && (x_scales == nullptr || !aligned(x_scales, 4))) return FRT_ERR_INVALID_ARG;
  if (x_format == FRT_X_NVFP4 && (x_sf == nullptr || !aligned(x_sf, 16))) return FRT_ERR_INVALID_ARG;
  Args a = {};
  a.x = x;
  a.x_scales = x_scales;
  a.x_sf = x_sf;
  a.w_codes = w_codes;
  a.w_sf = w_sf;
  a.w_scale = w_scale;
  a.bias = static_cast<const uint16_t*>(bias);
  a.y = static_cast<uint16_t*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.groups = K / kGroup + (K % kGroup != 0);
  a.swizzled = sf_layout == FRT_SF_SWIZZLED_128X4;
  a.dt = dt;
  switch (x_format) {
    case FRT_X_16BIT: return dt == FRT_F16 ? launch_rows<kXF16>(a, stream) : launch_rows<kXBF16>(a, stream);
    case FRT_X_E4M3: return launch_rows<kXE4M3>(a, stream);
    case FRT_X_E4M3_BLOCK: return launch_rows<kXE4M3Block>(a, stream);
    default: return launch_rows<kXNvfp4>(a, stream);
  }
}
