// y = x w^T + bias with NVFP4 weights, for few rows of x.
//
// What bounds it: the weights, 0.5625 B each, read once; against that stand one
// cvt and one multiply per two weights and one mma.m16n8k16 per 256 weights and
// 8 rows.  1 x 4096 -> 32768: 75.6 MB, 11.5 us at the copy rate, 19 us measured
// (4.0 TB/s; a plain read of 67 MB by bulk copies takes 14.6 us, launch
// included).  Small ones are bound by the launch and three dependent steps: 1 x
// 1024 -> 2560 3.6 us.
//
// Mapping.  16 weight rows on the 16-row side of the mma, 8 NT rows of x on
// the other.  The order of k inside a product is free: with g = lane / 4 and t
// = lane % 4 a lane holds weight rows g and g + 8 at k = 32 t .. 32 t + 31 of a
// group of 128, one 16-byte load a row, and two factors a row.  A warp keeps
// four groups of weights on their way (4 KB and their factors), which is what
// covers the HBM latency.  Tiles are dealt to the CTAs in turn, so that the SMs'
// shares differ by one tile at most; a warp takes a tile alone, or kw warps
// split its k and join their sums in shared memory in a fixed order.  Laying x
// out costs every CTA its whole share of k: with many rows of x or few tiles the
// CTAs of a cluster split k too, and join through distributed shared memory.
//
// x lies in shared memory as binary16 in the order in which the lanes read it
// (16 bytes are a lane's part of two products).  FP16 rows, e4m3 codes and
// NVFP4 code * factor are exact there.  bf16 rows are scaled by a power of two
// per row and group, and like the block-scaled FP8 rows keep a factor per row
// and group that is applied to the group's fp32 sums.  That factor, w_scale over
// the power of two, is kept a normal number: for tiny groups the power is smaller
// and binary16 cuts x at 2^-151 / w_scale, which is below 2^-139 in y.
#include <algorithm>

#include "matvec_nvfp4.cuh"

namespace frt {
namespace {

// groups a warp has on their way (with the sums of 32 rows no registers are left
// for more than two)
__host__ __device__ constexpr int ahead_of(int nt) { return nt == 4 ? 2 : 4; }
// CTAs that share an SM and their warps: up to 8 rows of x (NT 1) two, above (NT
// 2 and 4) one of twice the warps, which lays its many rows out once.
__host__ __device__ constexpr int ctas_of(int nt) { return nt == 1 ? 2 : 1; }
__host__ __device__ constexpr int warps_of(int nt) { return 16 / ctas_of(nt); }

using Args = MatvecArgs;

// Weights of one group: rows g and g + 8, 32 codes and two factors each.
struct WFrag {
  uint32_t c[2][4];
  uint32_t sf[2];
};
// A lane's rows g and g + 8 of a weight tile.  Rows behind the last are row N -
// 1 again, their sums are dropped; codes behind K are the last ones again, x is
// zero there.
// LAY: 0 any K, 1 K % 32 == 0 with row-major factors, 2 with swizzled ones;
// K % 32 == 0 has 16-byte loads of codes and 2-byte loads of factors.
template <int LAY>
struct WRows {
  const uint8_t* c[2];
  const uint8_t* sf[2];

  __device__ __forceinline__ void set(const Args& a, int row0, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min(row0 + g + 8 * h, a.N - 1);
      c[h] = a.w_codes + (int64_t)row * (a.K >> 1);
      sf[h] = a.w_sf + (LAY == 2 || (LAY == 0 && a.swizzled) ? sf_offset_swizzled(row, 0, a.K >> 4)
                                                              : (int64_t)row * (a.K >> 4));
    }
  }
  // (swizzled: 128 bytes a column, past 32 bits from K = 2^28 on)
  __device__ __forceinline__ int64_t sf_at(const Args& a, int col) const {
    return LAY == 2 || (LAY == 0 && a.swizzled) ? (int64_t)(col >> 2) * 512 + (col & 3) : col;
  }
  // Group `base` + u; whole: the sets' four groups lie inside K.
  __device__ __forceinline__ void load(const Args& a, int base, int u, bool whole, int t, WFrag& f) const {
    const int64_t bytes = (int64_t)a.N * (a.K >> 1), n_sf = sf_bytes(a, a.N);
    if (LAY == 0) {
      const int last = (a.K >> 4) - 1;
      const int c0 = min((base + u) * (kGroup / 16) + 2 * t, last), c1 = min(c0 + 1, last);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t *p0 = c[h] + 8 * c0, *p1 = c[h] + 8 * c1;
        const uint8_t *s0 = sf[h] + sf_at(a, c0), *s1 = sf[h] + sf_at(a, c1);
        uint2 v = make_uint2(0, 0), w = v;
        if (FRT_SPAN_OK(p0 - a.w_codes, 8, bytes)) v = ld_stream(reinterpret_cast<const uint2*>(p0));
        if (FRT_SPAN_OK(p1 - a.w_codes, 8, bytes)) w = ld_stream(reinterpret_cast<const uint2*>(p1));
        f.sf[h] = 0;
        if (FRT_IDX_OK(s0 - a.w_sf, n_sf) && FRT_IDX_OK(s1 - a.w_sf, n_sf)) f.sf[h] = __ldg(s0) | __ldg(s1) << 8;
        f.c[h][0] = v.x;
        f.c[h][1] = v.y;
        f.c[h][2] = w.x;
        f.c[h][3] = w.y;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t *p, *s;
        if (whole) {
          const int col = base * (kGroup / 16) + 2 * t;
          p = c[h] + 8 * col + u * (kGroup / 2);
          s = sf[h] + sf_at(a, col) + u * (LAY == 2 ? 1024 : 8);
        } else {
          const int col = min((base + u) * (kGroup / 16) + 2 * t, (a.K >> 4) - 2);
          p = c[h] + 8 * col;
          s = sf[h] + sf_at(a, col);
        }
        uint4 v = make_uint4(0, 0, 0, 0);
        if (FRT_SPAN_OK(p - a.w_codes, 16, bytes)) v = ld_stream(reinterpret_cast<const uint4*>(p));
        f.sf[h] = 0;
        if (FRT_SPAN_OK(s - a.w_sf, 2, n_sf)) f.sf[h] = __ldg(reinterpret_cast<const uint16_t*>(s));
        f.c[h][0] = v.x;
        f.c[h][1] = v.y;
        f.c[h][2] = v.z;
        f.c[h][3] = v.w;
      }
    }
  }
};

// Lays rows of x out in shared memory as binary16, groups seg .. seg + len - 1
// of n_rows rows (those behind the last are zeros): xf in the lanes' order, xs
// the factors times the weights' scale.  16 lanes take a group of a row, eight elements each; a row is
// shared by `split` of these half-warps, whose loads go out in batches.
template <XForm FORM, int NT, int kWarps>
__device__ __forceinline__ void stage_x(const Args& a, int seg, int len, int n_rows, int mr, int step, float w_scale,
                                        uint4* xf, float* xs) {
  constexpr bool kScaled = FORM == kXScaled16 || FORM == kXE4M3Block;
  constexpr int kBatch = 4;
  constexpr int kBytes = FORM == kX16 || FORM == kXScaled16 ? 16 : FORM == kXNvfp4 ? 4 : 8;  // of eight elements
  const int l = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int split = max(2 * kWarps / n_rows, 1), row_step = 2 * kWarps / split;
  const int r0 = h / split, part = h - r0 * split;
  const int64_t x_bytes = (int64_t)a.M * (a.K / 8) * kBytes;
  // (trip counts are the same for both halves of a warp)
  for (int j = 0; j < n_rows; j += row_step) {
    const int r = r0 + j;
    const bool row_on = r0 < row_step && r < n_rows, data = row_on && r < a.rows;
    const int64_t row = a.m0 + min(r, a.rows - 1);
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * (a.K / 8) * kBytes + l * kBytes;
    for (int c0 = part; c0 - part < len; c0 += kBatch * split) {
      uint4 v[kBatch];
      uint32_t sf[kBatch];
      float scale[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + b * split, k = (seg + c) * kGroup + 8 * l;
        v[b] = make_uint4(0, 0, 0, 0);
        sf[b] = 0;
        scale[b] = 1.0f;
        if (data && c < len && k < a.K) {
          const uint8_t* p = x + (int64_t)(seg + c) * (16 * kBytes);
          if (!FRT_SPAN_OK(p - static_cast<const uint8_t*>(a.x), kBytes, x_bytes)) continue;
          if (kBytes == 16) {
            v[b] = *reinterpret_cast<const uint4*>(p);
          } else if (kBytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            v[b].x = u.x;
            v[b].y = u.y;
          } else {
            v[b].x = *reinterpret_cast<const uint32_t*>(p);
          }
          if (FORM == kXNvfp4) {
            const int64_t at = a.swizzled ? sf_offset_swizzled(row, k >> 4, a.K >> 4) : row * (a.K >> 4) + (k >> 4);
            if (FRT_IDX_OK(at, sf_bytes(a, a.M))) sf[b] = a.x_sf[at];
          }
          if (FORM == kXE4M3Block) {
            const int64_t at = row * a.groups + seg + c;
            if (FRT_IDX_OK(at, (int64_t)a.M * a.groups)) scale[b] = a.x_scales[at];
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int c = c0 + b * split;
        uint4 o = v[b];
        if (FORM == kXScaled16) {
          float2 f[4];
          unpack_pairs<FRT_BF16, 4>(&o.x, f);
          const float amax = fmaxf(absmax4(f[0].x, f[0].y, f[1].x, f[1].y), absmax4(f[2].x, f[2].y, f[3].x, f[3].y));
          const float s = pow2_to_half_range(half_warp_max_abs(amax), most_pow2(w_scale));
          mul_pairs<4>(f, s);
          pack_pairs<FRT_F16, 4>(f, &o.x);
          scale[b] = 1.0f / s;
        } else if (FORM == kXE4M3 || FORM == kXE4M3Block) {
          e4m3x4_to_half2(v[b].x, &o.x);
          e4m3x4_to_half2(v[b].y, &o.z);
        } else if (FORM == kXNvfp4) {
          uint32_t f[2];
          e2m1x8_to_half2(v[b].x, &o.x);
          e4m3x4_to_half2(sf[b] * 0x0101u, f);
          o = make_uint4(hmul2(o.x, f[0]), hmul2(o.y, f[0]), hmul2(o.z, f[0]), hmul2(o.w, f[0]));
        }
        if (row_on && c < len) {
          xf[(c * 4 + (l & 3)) * step + ((r >> 3) * mr + (r & 7)) * 4 + (l >> 2)] = o;
          if (kScaled && l == 0) xs[c * (8 * NT) + r] = scale[b] * w_scale;
        }
      }
    }
  }
}

constexpr int kRedStride = 20;  // floats between two rows of x of a warp's sums

// y[row r][n .. n + 7]; N % 8 == 0 and y 16-byte aligned.
__device__ __forceinline__ void store_y8(const Args& a, int r, int n, float* sum, float scale) {
  const bool half = a.dt == FRT_F16;
  float b[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (a.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (FRT_IDX_OK(n + e, a.N)) b[e] = half ? value16<FRT_F16>(a.bias[n + e]) : value16<FRT_BF16>(a.bias[n + e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = fmaf(sum[e], scale, b[e]);
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    out[e] = half ? Pack16<FRT_F16>::from_float2(sum[2 * e], sum[2 * e + 1])
                  : Pack16<FRT_BF16>::from_float2(sum[2 * e], sum[2 * e + 1]);
  const int64_t at = (int64_t)(a.m0 + r) * a.N + n;
  if (FRT_SPAN_OK(at, 8, (int64_t)a.M * a.N))
    *reinterpret_cast<uint4*>(a.y + at) = make_uint4(out[0], out[1], out[2], out[3]);
}

__device__ __forceinline__ void add8(float* sum, const float4& u, const float4& v) {
  sum[0] += u.x;
  sum[1] += u.y;
  sum[2] += u.z;
  sum[3] += u.w;
  sum[4] += v.x;
  sum[5] += v.y;
  sum[6] += v.z;
  sum[7] += v.w;
}

// Floats of a warp's sums of a tile, [row of x][weight row].
__host__ __device__ constexpr int sum_floats(int nt, int mr) { return (nt == 1 ? mr : 8 * nt) * kRedStride; }

// SCALED: x has a factor per row and group.
template <int NT, bool SCALED, int LAY>
__global__ void __launch_bounds__(32 * warps_of(NT), ctas_of(NT)) matvec_kernel(const Args a) {
  constexpr int kWarps = warps_of(NT), kAhead = ahead_of(NT);
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int mr = NT == 1 ? min(a.rows, 8) : 8;  // rows of x that shared memory holds per 8
  const int step = NT * mr * 4;                 // 16-byte words of 32 k
  const int red_warp = sum_floats(NT, mr);
  const int ranks = a.cluster, rank = (int)blockIdx.x % ranks;
  const int cta = (int)blockIdx.x / ranks, ctas = (int)gridDim.x / ranks;  // (clusters, if there are any)
  const int kw = a.kw, ks = warp & (kw - 1), rw = warp >> a.kw_log2, at_once = kWarps >> a.kw_log2;
  // the tile of this warp in a round (tiles are dealt to the CTAs in turn)
  auto tile_of = [&](int round) { return (round * at_once + rw) * ctas + cta; };
  const int per_round = at_once * ctas;
  const int rounds = a.tiles / per_round + (a.tiles % per_round > cta);  // of this CTA's first warp
  const int group0 = a.groups * rank / ranks, group1 = a.groups * (rank + 1) / ranks;

  // sums [round, or its parity where there is no cluster][warp][row of x][weight row]
  float* red = reinterpret_cast<float*>(smem);
  const int sum_sets = ranks > 1 ? (a.tiles + per_round - 1) / per_round : 2;
  uint4* xf = reinterpret_cast<uint4*>(smem + sizeof(float) * sum_sets * kWarps * red_warp);
  float* xs = reinterpret_cast<float*>(xf + (size_t)a.seg_groups * 4 * step);
  // rows of x that are not there: the last one again, its sums are dropped
  const uint4* x_lane = xf + min(g, mr - 1) * 4 + t;

  // This warp's groups: of each tile and segment of k a contiguous share, in
  // sets of kAhead.  end == 0: no more.
  struct Cursor {
    int round, seg, base, end;
  };
  auto share = [&](Cursor& c) {
    const int len = min(a.seg_groups, group1 - c.seg);
    c.base = c.seg + (len * ks >> a.kw_log2);
    c.end = c.seg + (len * (ks + 1) >> a.kw_log2);
    if (tile_of(c.round) >= a.tiles) c.end = 0;
  };
  auto settle = [&](Cursor& c) {  // past empty shares
    while (c.base >= c.end && c.end > 0) {
      c.seg += a.seg_groups;
      if (c.seg >= group1) {
        c.seg = group0;
        ++c.round;
      }
      share(c);
    }
  };
  auto advance = [&](Cursor c) {
    c.base += kAhead;
    settle(c);
    return c;
  };
  auto is_whole = [&](const Cursor& c) { return LAY != 0 && (c.base + kAhead) * kGroup <= a.K; };
  WFrag w[kAhead];
  WRows<LAY> rows;
  Cursor cur = {0, group0, 0, 0};
  share(cur);
  settle(cur);
  rows.set(a, tile_of(cur.round) * 16, g);
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (cur.base + u < cur.end) rows.load(a, cur.base, u, is_whole(cur), t, w[u]);  // constant inputs: before the wait
  const float w_scale = __ldg(a.w_scale);
  pdl_enter();
  const bool wide = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  // (the weights' scale is in xs where there are such factors: sums of large rows stay finite)
  const float scale = SCALED ? 1.0f : w_scale * (a.form == kX16 ? 1.0f : a.x_scales[0]);

  for (int round = 0; round < rounds; ++round) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    for (int seg = group0; seg < group1; seg += a.seg_groups) {
      if (a.seg_groups < group1 - group0 || round == 0) {
        if (seg > group0 || round > 0) __syncthreads();  // the last segment is read
        const int n_rows = NT == 1 ? mr : 8 * NT, len = min(a.seg_groups, group1 - seg);
        if (SCALED) {
          if (a.form == kXScaled16)
            stage_x<kXScaled16, NT, kWarps>(a, seg, len, n_rows, mr, step, w_scale, xf, xs);
          else
            stage_x<kXE4M3Block, NT, kWarps>(a, seg, len, n_rows, mr, step, w_scale, xf, xs);
        } else if (a.form == kX16) {
          stage_x<kX16, NT, kWarps>(a, seg, len, n_rows, mr, step, w_scale, xf, xs);
        } else if (a.form == kXE4M3) {
          stage_x<kXE4M3, NT, kWarps>(a, seg, len, n_rows, mr, step, w_scale, xf, xs);
        } else {
          stage_x<kXNvfp4, NT, kWarps>(a, seg, len, n_rows, mr, step, w_scale, xf, xs);
        }
        __syncthreads();
      }
      while (cur.end > 0 && cur.round == round && cur.seg == seg) {
        const Cursor next = advance(cur);
        if (next.round != round && next.end > 0) rows.set(a, tile_of(next.round) * 16, g);
        const bool next_whole = is_whole(next);
        const uint4* xb = x_lane + (cur.base - seg) * 4 * step;
        const float* xsb = xs + (cur.base - seg) * 8 * NT + 2 * t;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (cur.base + u < cur.end) {
            float part[NT][4];
            if (SCALED) {
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
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 bv = xb[n * 32];
                mma_16816(SCALED ? part[n] : acc[n], a0, bv.x, bv.y);
                mma_16816(SCALED ? part[n] : acc[n], a1, bv.z, bv.w);
              }
              xb += step;
            }
            if (SCALED) {
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const float2 s = *reinterpret_cast<const float2*>(xsb + u * 8 * NT + 8 * n);
                acc[n][0] = fmaf(part[n][0], s.x, acc[n][0]);
                acc[n][1] = fmaf(part[n][1], s.y, acc[n][1]);
                acc[n][2] = fmaf(part[n][2], s.x, acc[n][2]);
                acc[n][3] = fmaf(part[n][3], s.y, acc[n][3]);
              }
            }
          }
          if (next.base + u < next.end) rows.load(a, next.base, u, next_whole, t, w[u]);
        }
        cur = next;
      }
    }
    // The sums through shared memory: of the warp's own tile, or of the kw warps
    // that share one.  Two sets of them, so that one barrier a round is enough;
    // a cluster keeps those of every round.
    float* sums = red + (size_t)(ranks > 1 ? round : round & 1) * kWarps * red_warp;
    float* mine = sums + warp * red_warp + g;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        if (NT > 1 || r < mr) {
          mine[r * kRedStride] = acc[n][e];
          mine[r * kRedStride + 8] = acc[n][2 + e];
        }
      }
    if (ranks > 1) continue;
    if (kw == 1)
      __syncwarp();
    else
      __syncthreads();
    if (NT == 1 || !wide) {  // one output to a lane, neighbours along n: two tiles, or two rows of a warp's own
      const int two = lane >> 4, col = lane & 15;
      const int r0 = kw == 1 ? two : warp, r_step = kw == 1 ? 2 : kWarps;
      for (int r = r0; r < a.rows; r += r_step) {
        for (int q = kw == 1 ? rw : two; q < at_once; q += kw == 1 ? kWarps : 2) {
          const int n = ((round * at_once + q) * ctas + cta) * 16 + col;
          if (n >= a.N) break;
          const float* p = sums + (q << a.kw_log2) * red_warp + r * kRedStride + col;
          float sum = 0.0f;
          for (int k = 0; k < kw; ++k) sum += p[k * red_warp];
          store_y1(a, r, n, sum, scale);
        }
      }
      continue;
    }
    // eight outputs to a lane: two lanes a tile and row of x, the rows dealt to
    // the warps (of a warp's own tile to its lanes)
    const int q = kw == 1 ? rw : lane >> 1, o = lane & 1;
    const int n = ((round * at_once + q) * ctas + cta) * 16 + 8 * o;
    if (q < at_once && n < a.N) {
      const float* p = sums + (q << a.kw_log2) * red_warp + 8 * o;
      for (int r = kw == 1 ? lane >> 1 : warp; r < a.rows; r += kw == 1 ? 16 : kWarps) {
        float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < kw; ++k) {
          const float* pk = p + k * red_warp + r * kRedStride;
          add8(sum, *reinterpret_cast<const float4*>(pk), *reinterpret_cast<const float4*>(pk + 4));
        }
        store_y8(a, r, n, sum, scale);
      }
    }
  }
  if (ranks == 1) return;

  // ---- a cluster's sums: its tiles are dealt to the CTAs in turn; a lane reads
  // the sums of one CTA (eight outputs), the lanes of a row are added as a tree
  cluster_sync();
  const int slots = rounds * at_once;
  const int c = (lane >> 1) & (ranks - 1), lanes = 2 * ranks;
  const uint32_t red_at = cluster_addr(smem_addr(red), c);
  for (int j0 = 0; j0 * ranks + rank < slots; j0 += 32 / lanes) {
    const int slot = (j0 + lane / lanes) * ranks + rank, n = (slot * ctas + cta) * 16 + 8 * (lane & 1);
    const bool on = slot < slots && n < a.N;
    for (int r = warp; r < a.rows; r += kWarps) {
      const uint32_t at = red_at + (slot * kw * red_warp + r * kRedStride + 8 * (lane & 1)) * 4;
      float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (on)
        for (int k = 0; k < kw; ++k) {
          const float4 u = ld_cluster4(at + k * red_warp * 4), v = ld_cluster4(at + k * red_warp * 4 + 16);
          add8(sum, u, v);
        }
      for (int d = 2; d < lanes; d *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], d);
      if (on && c == 0) {
        if (wide) {
          store_y8(a, r, n, sum, scale);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) store_y1(a, r, n + e, sum[e], scale);
        }
      }
    }
  }
  cluster_sync();  // the sums are read
}

template <int NT, bool SCALED, int LAY>
frt_status launch_one(Args a, cudaStream_t stream) {
  constexpr int kPerSM = ctas_of(NT), kWarps = warps_of(NT), kAhead = ahead_of(NT);
  a.tiles = (int)(((int64_t)a.N + 15) / 16);
  const int mr = NT == 1 && a.rows < 8 ? a.rows : 8;
  const int x_rows = NT == 1 ? mr : 8 * NT;
  const size_t group_bytes = (size_t)4 * NT * mr * 4 * 16 + (SCALED ? 8 * NT * 4 : 0);
  const size_t set_bytes = sizeof(float) * kWarps * sum_floats(NT, mr);
  const size_t most = 225 * 1024, half = 112 * 1024;
  // How k is split, over the kw warps that share a tile and the CTAs of a
  // cluster: the cheapest of the plans that fit, in microseconds.  Measured: a
  // batch of x 0.8; a group (0.25 + 0.1 NT)
  // for a warp among up to 16 of the SM; a round 0.5; joining a cluster's sums 2.5
  // and 0.2 (1 + kw) for every turn of a warp.
  double best = 0;
  size_t smem = 0;
  int64_t grid_ctas = 1;  // (or clusters) that run at once: the sums' place in shared memory goes by it
  a.cluster = 0;
  for (int ranks = 1; ranks <= 8; ranks *= 2) {
    if (ranks > 1 && ranks > a.groups) break;
    const int k_groups = (a.groups + ranks - 1) / ranks;
    for (int kw = 1, log2 = 0; kw <= kWarps && kw <= k_groups; kw *= 2, ++log2) {
      for (int sm = kPerSM; sm >= 1; --sm) {
        const int64_t ctas = cluster_room(sm, ranks);
        const int64_t used = a.tiles < ctas ? a.tiles : ctas;
        const int64_t per_round = used * (kWarps / kw);
        const int64_t rounds = (a.tiles + per_round - 1) / per_round;
        const size_t red = set_bytes * (ranks > 1 ? (size_t)rounds : 2);
        const size_t limit = sm == 2 ? half : most;
        int seg = k_groups;
        if (red + k_groups * group_bytes > limit) {
          // x in segments, whole sets for every warp; not in a cluster
          if (ranks > 1 || sm == 2 || red + kw * kAhead * group_bytes > limit) continue;
          seg = (int)((limit - red) / group_bytes) / (kw * kAhead) * (kw * kAhead);
        }
        const int split = 2 * kWarps / x_rows > 1 ? 2 * kWarps / x_rows : 1;
        const int turns_x = (x_rows + 2 * kWarps / split - 1) / (2 * kWarps / split);
        const double batches = (double)turns_x * ((seg + 4 * split - 1) / (4 * split));
        const double staging = 0.8 * batches * (seg < k_groups ? (double)((k_groups + seg - 1) / seg * rounds) : 1.0);
        const double group = 0.25 + 0.1 * NT;
        const double turns = (double)((a.rows + kWarps - 1) / kWarps) * (double)((rounds * (kWarps / kw) + 15) / 16);
        const double cost = staging + rounds * (((k_groups + kw - 1) / kw) * group + 0.5) +
                            (ranks > 1 ? 2.5 + turns * (0.2 + 0.2 * kw) : 0.0);
        if (a.cluster == 0 || cost < best) {
          best = cost;
          a.cluster = ranks;
          a.kw = kw;
          a.kw_log2 = log2;
          a.seg_groups = seg;
          grid_ctas = used;
          smem = red + seg * group_bytes;
        }
      }
    }
  }
  if (a.cluster == 0) return FRT_ERR_UNSUPPORTED;  // (never: a segment of one set always fits)
  static SmemOptIn opted;
  const frt_status st = opt_in_smem(matvec_kernel<NT, SCALED, LAY>, smem, opted);
  if (st != FRT_OK) return st;
  const dim3 grid((unsigned)(grid_ctas * a.cluster)), block(32 * kWarps);
  if (a.cluster > 1) return launch_cluster(matvec_kernel<NT, SCALED, LAY>, grid, block, smem, stream, a.cluster, a);
  return launch(matvec_kernel<NT, SCALED, LAY>, grid, block, smem, stream, a);
}
template <int NT, bool SCALED>
frt_status launch_layout(const Args& a, cudaStream_t stream) {
  if (a.K % 32 != 0) return launch_one<NT, SCALED, 0>(a, stream);
  return a.swizzled ? launch_one<NT, SCALED, 2>(a, stream) : launch_one<NT, SCALED, 1>(a, stream);
}
template <bool SCALED>
frt_status launch_few(const Args& a, cudaStream_t stream) {
  return a.rows <= 8    ? launch_layout<1, SCALED>(a, stream)
         : a.rows <= 16 ? launch_layout<2, SCALED>(a, stream)
                        : launch_layout<4, SCALED>(a, stream);
}
// Up to kFewRows rows of x the warps' products win: 16 rows of 4096 to 32768
// 23.5-32 us against the tiles' 53-64 (the forms of x), of 8192 to 8192 16-19
// against 28-33, of 1024 to 4096 3.9-4.4 against 5.3-5.8, of 4096 to 1024 6.2-6.6
// against 6.9-7.5, where only bf16 rows take 8.0 against 7.5.  Up to kMoreRows,
// which is what they carry at most, they win where the weights are more than
// kManyWeights: 32 rows of 4096 to 32768 35-46 against 54-65, of 5120 to 5120
// 13.6-15.9 against 18.2-21.6, of 2048 to 16384 13.1-15.4 against 14.9-17.1; at
// kManyWeights, 4096 to 4096, 17 rows 10.2-11.3 against 10.5-11.2 and 32 rows
// 10.9-12.2 against 10.6-11.4; of 256 to 11682 4.6-5.0 against 3.9-4.0.
constexpr int kFewRows = 16, kMoreRows = 32;
constexpr int64_t kManyWeights = 1 << 24;
bool warps_win(const Args& a) {
  return a.rows <= kFewRows || (a.rows <= kMoreRows && (int64_t)a.N * a.K > kManyWeights);
}
constexpr int kMaxSize = 0x7FFF0000;  // (32-bit indices reach past M, N and K by less than 65536)
frt_status launch_rows(Args a, cudaStream_t stream) {
  for (a.m0 = 0; a.m0 < a.M; a.m0 += kTileXRows) {
    a.rows = std::min(a.M - a.m0, kTileXRows);
    const bool scaled = a.form == kXScaled16 || a.form == kXE4M3Block;
    const frt_status st = !warps_win(a) ? launch_matvec_tiles(a, stream)
                          : scaled      ? launch_few<true>(a, stream)
                                        : launch_few<false>(a, stream);
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
  if (M > kMaxSize || N > kMaxSize || K > kMaxSize) return FRT_ERR_UNSUPPORTED;
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
    case FRT_X_16BIT: a.form = dt == FRT_F16 ? kX16 : kXScaled16; break;
    case FRT_X_E4M3: a.form = kXE4M3; break;
    case FRT_X_E4M3_BLOCK: a.form = kXE4M3Block; break;
    default: a.form = kXNvfp4; break;
  }
  return launch_rows(a, stream);
}
