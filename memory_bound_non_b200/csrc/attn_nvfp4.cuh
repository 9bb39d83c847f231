// What the kernels of the attention over an NVFP4 KV cache share: arguments,
// sequences, query rows and pages.
#pragma once

#include "frt_device.cuh"
#include "frt_fragments.cuh"
#include "frt_launch.h"
#include "frt_tensor.cuh"

namespace frt {

struct AttnArgs {
  const void* q;
  const uint8_t* k_codes;
  const uint8_t* k_sf;
  const uint8_t* v_codes;
  const uint8_t* v_sf;
  const float* kv_scales;
  const int32_t* kv_len;
  const int32_t* q_indptr;
  const int32_t* page_table;
  void* out;
  float2* part_ml;  // [chunk][M Hq] (maximum, sum)
  float* part_o;    // [chunk][M Hq][hd]
  int32_t* part_n;  // [M Hq] chunks that hold a part of the row
  int32_t* status;
  int M, n_seqs, Hq, Hkv, hd, group;
  int capacity, page_size, max_pages, n_pages;
  int max_q_len, max_len;  // max_len: the largest length a token may have
  int window;
  // p / d = (p + umulhi(p, mul)) >> shift for 0 <= p < 2^31
  uint32_t page_mul, group_mul;
  int page_shift, group_shift;
  // The keys of a row tile are cut into `chunks`: with cluster != 0 evenly, for
  // the CTAs of a cluster, which join their parts through distributed shared
  // memory; else chunk_tiles tiles each, joined by a second kernel.
  int row_tiles, chunks, chunk_tiles, cluster;
  float scale_log2;
  int dt;
};

// Tokens [t0, t0 + n) of a sequence.
struct Seq {
  int t0, n;
  bool bad;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
  int s0 = 0, s1 = a.M;
  if (a.q_indptr != nullptr && FRT_SPAN_OK(b, 2, a.n_seqs + 1)) {
    s0 = __ldg(a.q_indptr + b);
    s1 = __ldg(a.q_indptr + b + 1);
  }
  Seq s;
  s.bad = s0 < 0 || s1 > a.M || s1 < s0;
  s0 = min(max(s0, 0), a.M);
  s1 = min(max(s1, s0), a.M);
  s.t0 = s0;
  s.n = s1 - s0;
  if (s.n > a.max_q_len) {
    s.n = a.max_q_len;
    s.bad = true;
  }
  return s;
}

__device__ __forceinline__ int fast_div(int p, uint32_t mul, int shift) {
  return (int)((__umulhi((uint32_t)p, mul) + (uint32_t)p) >> shift);
}

// Row r of a sequence (token-major, then the heads of the KV head's group) and
// the positions [lo, hi) that it sees; tok < 0: no such row.
struct QueryRow {
  int tok, head, lo, hi;
  bool bad;
};
__device__ __forceinline__ QueryRow query_row(const AttnArgs& a, const Seq& s, int r, int kvh) {
  QueryRow o = {-1, 0, 0, 0, false};
  const int i = fast_div(r, a.group_mul, a.group_shift);
  if (i >= s.n) return o;
  o.tok = s.t0 + i;
  o.head = kvh * a.group + (r - i * a.group);
  if (FRT_IDX_OK(o.tok, a.M)) {
    const int len = __ldg(a.kv_len + o.tok);
    o.hi = min(max(len, 0), a.max_len);
    o.bad = o.hi != len;
    o.lo = a.window > 0 ? max(0, o.hi - a.window) : 0;
  }
  return o;
}

// What the R rows from row0 on see together, computed by every warp for itself.
struct RowRange {
  int all_lo, all_hi;    // the positions that any row sees (empty: all_hi <= all_lo)
  int full_lo, full_hi;  // the positions that every row sees
  bool any, bad;         // is there a row; is an argument out of range
  __device__ __forceinline__ int first() const { return all_lo & ~3; }
  __device__ __forceinline__ int tiles(int keys) const {
    const int span = all_hi - first();
    return span / keys + (span % keys != 0);
  }
};
template <int R>
__device__ __forceinline__ RowRange row_range(const AttnArgs& a, const Seq& s, int row0, int kvh) {
  RowRange o = {0x7FFFFFFF, 0, 0, 0x7FFFFFFF, false, s.bad};
  constexpr int kEach = (R + 31) / 32;
  QueryRow q[kEach];  // (their loads in flight together)
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = 32 * i + (threadIdx.x & 31);
    q[i] = query_row(a, s, r < R ? row0 + r : 0x7FFFFFFF, kvh);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (q[i].tok < 0) continue;
    o.any = true;
    o.bad |= q[i].bad;
    if (q[i].hi > q[i].lo) {
      o.all_lo = min(o.all_lo, q[i].lo);
      o.all_hi = max(o.all_hi, q[i].hi);
    }
    o.full_lo = max(o.full_lo, q[i].lo);
    o.full_hi = min(o.full_hi, q[i].hi);
  }
  o.all_lo = __reduce_min_sync(0xFFFFFFFFu, o.all_lo);
  o.all_hi = __reduce_max_sync(0xFFFFFFFFu, o.all_hi);
  o.full_lo = __reduce_max_sync(0xFFFFFFFFu, o.full_lo);
  o.full_hi = __reduce_min_sync(0xFFFFFFFFu, o.full_hi);
  o.any = __any_sync(0xFFFFFFFFu, o.any);
  if (o.all_hi <= o.all_lo) o.all_lo = o.all_hi = 0;
  return o;
}

// First slot of the quad of positions pos .. pos + 3, or -1 (behind the end, or
// on a page that does not exist).
__device__ __forceinline__ int quad_slot(const AttnArgs& a, int b, int pos, const RowRange& range) {
  if (pos >= range.all_hi) return -1;
  if (a.page_table == nullptr) return pos;
  const int page = fast_div(pos, a.page_mul, a.page_shift);
  const int64_t at = (int64_t)b * a.max_pages + page;
  if (!FRT_IDX_OK(at, (int64_t)a.n_seqs * a.max_pages)) return -1;
  const int entry = __ldg(a.page_table + at);
  if (entry < 0 || entry >= a.n_pages) {
    if (a.status != nullptr && pos + 3 >= range.all_lo) atomicOr(a.status, 1);
    return -1;
  }
  return entry * a.page_size + (pos - page * a.page_size);
}

// Bytes that hold the NaN factor, marked in their top bits.
__device__ __forceinline__ uint32_t nan_factors(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Four outputs from d on, and the part of a chunk.
__device__ __forceinline__ void store_out4(const AttnArgs& a, int64_t at, float4 v, float f) {
  const uint2 w = a.dt == FRT_F16 ? make_uint2(Pack16<FRT_F16>::from_float2(v.x * f, v.y * f),
                                               Pack16<FRT_F16>::from_float2(v.z * f, v.w * f))
                                  : make_uint2(Pack16<FRT_BF16>::from_float2(v.x * f, v.y * f),
                                               Pack16<FRT_BF16>::from_float2(v.z * f, v.w * f));
  if (FRT_SPAN_OK(at, 4, (int64_t)a.M * a.Hq * a.hd))
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = w;
}
// Joining the parts that the CTAs of a cluster hold of a row: their factors
// from (maximum, sum) at ml in each CTA's shared memory, to factor[k * stride]
// (0 behind the last CTA) ...
__device__ __forceinline__ void cluster_factors(const AttnArgs& a, uint32_t ml, float gs_v, float* factor, int stride) {
  const float kInf = __int_as_float(0x7F800000);
  float2 part[8];
  float top = -kInf, sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    part[k] = k < a.chunks ? ld_cluster2(cluster_addr(ml, k)) : make_float2(-kInf, 0.0f);
    top = fmaxf(top, part[k].x);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    part[k].x = part[k].x == -kInf ? 0.0f : ex2_approx(part[k].x - top);
    sum = fmaf(part[k].y, part[k].x, sum);
  }
  const float f = sum == 0.0f ? 0.0f : gs_v / sum;
#pragma unroll
  for (int k = 0; k < 8; ++k) factor[k * stride] = part[k].x * f;
}
// ... and four dimensions of the row, in fp32 at o.
__device__ __forceinline__ float4 join_cluster4(const AttnArgs& a, uint32_t o, int rank, const float* factor,
                                                int stride) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int k = 0; k < a.chunks; k += 4) {
    float4 u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = ld_cluster4(cluster_addr(o, k + e < a.chunks ? k + e : rank));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = factor[(k + e) * stride];
      v.x = fmaf(u[e].x, f, v.x);
      v.y = fmaf(u[e].y, f, v.y);
      v.z = fmaf(u[e].z, f, v.z);
      v.w = fmaf(u[e].w, f, v.w);
    }
  }
  return v;
}
__device__ __forceinline__ void store_part4(const AttnArgs& a, int chunk, int64_t at, float4 v) {
  const int64_t n = (int64_t)a.M * a.Hq * a.hd;
  if (FRT_SPAN_OK(chunk * n + at, 4, n * a.chunks)) *reinterpret_cast<float4*>(a.part_o + chunk * n + at) = v;
}

// The CTA's place in the grid and its tiles [tile0, tile1) of `tiles`.
struct Place {
  int kvh, rt, chunk;
};
__device__ __forceinline__ Place place_of(const AttnArgs& a) {
  // heads are neighbours in the grid: CTAs that run at the same time read
  // neighbouring bytes of a slot
  Place p;
  int x = blockIdx.x;
  if (a.cluster) {
    p.chunk = x % a.chunks;
    x /= a.chunks;
    p.kvh = x % a.Hkv;
    p.rt = x / a.Hkv;
  } else {
    p.kvh = x % a.Hkv;
    x /= a.Hkv;
    p.rt = x % a.row_tiles;
    p.chunk = x / a.row_tiles;
  }
  return p;
}
__device__ __forceinline__ int2 tiles_of(const AttnArgs& a, int chunk, int tiles) {
  if (a.cluster) return make_int2((int)((int64_t)tiles * chunk / a.chunks), (int)((int64_t)tiles * (chunk + 1) / a.chunks));
  const int t0 = min((int64_t)chunk * a.chunk_tiles, (int64_t)tiles);
  return make_int2(t0, min(t0 + a.chunk_tiles, tiles));
}

// How many chunks a row's tiles fill, written by the CTA of the first one.
__device__ __forceinline__ void store_chunks(const AttnArgs& a, int64_t row, int tiles) {
  if (a.chunks > 1 && FRT_IDX_OK(row, (int64_t)a.M * a.Hq)) a.part_n[row] = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
}

// Query rows of a CTA of the tile kernel, and keys of one of its tiles.
constexpr int kTileRows = 128;
__host__ __device__ constexpr int tile_keys(int hd) { return hd <= 128 ? 128 : 64; }
frt_status launch_attn_tiles(const AttnArgs& a, cudaStream_t stream);

}  // namespace frt
