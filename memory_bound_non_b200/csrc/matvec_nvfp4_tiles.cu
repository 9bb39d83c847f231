// y = x w^T + bias with NVFP4 weights for more rows of x than the warps'
// products carry: 128 weight rows to a CTA, on the 5th-generation tensor cores.
//
// What bounds it: up to 128 rows of x the weights' bytes still take longer than
// the products (2 operations per weight and row), so the codes' conversion
// counts, one cvt and one multiply per two weights, and laying x out, which
// every CTA does for itself.
//
// Steps of 128 k, two buffers: all warps bring the step's weights (A, 128 rows)
// and rows of x (B) to binary16 in shared memory (64 k to a region of 128-byte
// lines, 128-byte swizzle), one thread issues the eight products of the step
// into tensor memory while the warps convert the next one.  Weights are loaded
// kAhead steps ahead of their conversion.  Where x has a factor per row and
// step (bf16, block-scaled FP8) the sums of a step go to one of two accumulators
// and are added to registers with their factors while the next step runs.
// With few tiles the CTAs of a cluster split k and join their sums through
// distributed shared memory.  Measured: 41 rows of 2048 (block-scaled FP8) to
// 16384 18 us (3.1 us of bytes, 1.7 of products), 62 of 256 to 11682 5.0 us; a
// step takes 1600 clocks, a chain of conversion, barrier and sums in which no
// single part stands out (without x 16 % less, without the factors' sums 14 %,
// without the products 2 %).  At 65 to 128 rows with such factors the sums in
// registers spill (240 bytes a thread for bf16 rows, 372 for block-scaled FP8).
#include <algorithm>

#include "matvec_nvfp4.cuh"

namespace frt {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;              // weight rows
constexpr int kRegionA = kRows * 128;   // bytes of 64 k
constexpr int kAhead = 3;

// NX: rows of x that the build carries (32, 64 or 128).
template <int NX>
struct Tile {
  static constexpr int kA = 2 * kRegionA, kB = 2 * NX * 128, kStage = kA + kB;
  static constexpr size_t kSmem = 1024 + 2 * kStage + 3 * NX * 4 + 64;
  static_assert(kSmem >= tmem_smem(2 * NX), "tensor memory is never waited for");
};

struct RawX {
  uint4 v;
  uint32_t sf;
  float scale;
};
// Where a half-warp's lane l reads row r, step after step; FORM as
// MatvecArgs::form.
template <XForm FORM>
struct XRow {
  static constexpr int kBytes = FORM == kX16 || FORM == kXScaled16 ? 16 : FORM == kXNvfp4 ? 4 : 8;  // of eight elements
  const uint8_t* p;
  const uint8_t* sf;
  const float* scale;
  __device__ __forceinline__ void set(const MatvecArgs& a, int r, int group, int l) {
    const int64_t row = a.m0 + min(r, a.rows - 1);
    const int k8 = group * (kGroup / 8) + l;
    p = static_cast<const uint8_t*>(a.x) + (row * (a.K / 8) + k8) * kBytes;
    if (FORM == kXNvfp4)
      sf = a.x_sf + (a.swizzled ? sf_offset_swizzled(row, k8 >> 1, a.K >> 4) : row * (a.K >> 4) + (k8 >> 1));
    if (FORM == kXE4M3Block) scale = a.x_scales + row * a.groups + group;
  }
  // reads (on: row and column are there) and moves on to the next step
  __device__ __forceinline__ RawX next(const MatvecArgs& a, bool on) {
    RawX o = {make_uint4(0, 0, 0, 0), 0, 1.0f};
    if (on && FRT_SPAN_OK(p - static_cast<const uint8_t*>(a.x), kBytes, (int64_t)a.M * (a.K / 8) * kBytes)) {
      if (kBytes == 16) {
        o.v = *reinterpret_cast<const uint4*>(p);
      } else if (kBytes == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        o.v.x = u.x;
        o.v.y = u.y;
      } else {
        o.v.x = *reinterpret_cast<const uint32_t*>(p);
      }
      if (FORM == kXNvfp4 && FRT_IDX_OK(sf - a.x_sf, sf_bytes(a, a.M))) o.sf = *sf;
      if (FORM == kXE4M3Block && FRT_IDX_OK(scale - a.x_scales, (int64_t)a.M * a.groups)) o.scale = *scale;
    }
    p += 16 * kBytes;
    if (FORM == kXNvfp4) sf += a.swizzled ? 1024 : 8;
    if (FORM == kXE4M3Block) ++scale;
    return o;
  }
};
// The same as binary16; 16 lanes hold a group of a row.  `most`: most_pow2 of the
// weights' scale.
template <XForm FORM>
__device__ __forceinline__ uint4 convert_x(RawX& raw, int most) {
  uint4 o = raw.v;
  if (FORM == kXScaled16) {
    float2 f[4];
    unpack_pairs<FRT_BF16, 4>(&o.x, f);
    const float amax = fmaxf(absmax4(f[0].x, f[0].y, f[1].x, f[1].y), absmax4(f[2].x, f[2].y, f[3].x, f[3].y));
    const float s = pow2_to_half_range(half_warp_max_abs(amax), most);
    mul_pairs<4>(f, s);
    pack_pairs<FRT_F16, 4>(f, &o.x);
    raw.scale = 1.0f / s;
  } else if (FORM == kXE4M3 || FORM == kXE4M3Block) {
    const uint2 u = make_uint2(raw.v.x, raw.v.y);
    e4m3x4_to_half2(u.x, &o.x);
    e4m3x4_to_half2(u.y, &o.z);
  } else if (FORM == kXNvfp4) {
    const uint32_t f = e4m3_to_both(raw.sf);
    e2m1x8_to_half2(raw.v.x, &o.x);
    o = make_uint4(hmul2(o.x, f), hmul2(o.y, f), hmul2(o.z, f), hmul2(o.w, f));
  }
  return o;
}

// Four columns of this thread's lane.
__device__ __forceinline__ void tc_ld4(uint32_t addr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(addr));
}

template <int NX, XForm FORM>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const MatvecArgs a, int polls) {
  using T = Tile<NX>;
  constexpr bool kScaled = FORM == kXScaled16 || FORM == kXE4M3Block;
  constexpr int kCols = kScaled ? 2 * NX : NX;  // TMEM columns
  constexpr int kQ = NX / 4;                    // columns of a thread
  constexpr int kXEach = NX / 32;               // rows of x of a half-warp
  extern __shared__ unsigned char raw_smem[];
  const uint32_t base = (smem_addr(raw_smem) + 1023) & ~1023u;
  unsigned char* smem = raw_smem + (base - smem_addr(raw_smem));
  float* xs = reinterpret_cast<float*>(smem + 2 * T::kStage);  // [3][NX]
  uint64_t* bar = reinterpret_cast<uint64_t*>(xs + 3 * NX);    // [2]
  uint64_t* drained = bar + 2;  // the products behind a wait that ran out
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar + 3);
  int* gave_up_at = reinterpret_cast<int*>(tmem_at + 1);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ranks = a.cluster, rank = (int)blockIdx.x % ranks, tile = (int)blockIdx.x / ranks;
  const int g0 = a.groups * rank / ranks, g1 = a.groups * (rank + 1) / ranks;
  const int nx = (a.rows + 15) & ~15;  // rows of x in the products

  // This thread's weights: of row wrow the blocks lane % 4 and 4 + lane % 4 of a
  // step.
  const int wrow = 8 * warp + 2 * (lane >> 3) + ((lane >> 2) & 1);
  const int64_t w_at = (int64_t)min(tile * kRows + wrow, a.N - 1);
  const uint8_t* w_c = a.w_codes + w_at * (a.K >> 1) + 8 * (g0 * 8 + (lane & 3));
  const uint8_t* w_f = a.w_sf + (a.swizzled ? sf_offset_swizzled(w_at, g0 * 8 + (lane & 3), a.K >> 4)
                                            : w_at * (a.K >> 4) + g0 * 8 + (lane & 3));
  const int f_half = a.swizzled ? 512 : 4;  // four blocks on: an atom, or 4 bytes
  struct RawW {
    uint2 c[2];
    uint32_t sf[2];
  };
  int cols_left = min(a.K >> 4, g1 * 8) - g0 * 8 - (lane & 3);  // from this thread's first block of a step on
  auto load_w = [&](RawW& w) {  // and on to the next step
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w.c[j] = make_uint2(0, 0);
      w.sf[j] = 0;
      if (4 * j < cols_left) {
        if (FRT_SPAN_OK(w_c + 32 * j - a.w_codes, 8, (int64_t)a.N * (a.K >> 1)))
          w.c[j] = ld_stream(reinterpret_cast<const uint2*>(w_c + 32 * j));
        if (FRT_IDX_OK(w_f + f_half * j - a.w_sf, sf_bytes(a, a.N))) w.sf[j] = __ldg(w_f + f_half * j);
      }
    }
    w_c += 64;
    w_f += 2 * f_half;
    cols_left -= 8;
  };
  RawW w[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(w[u]);  // constant inputs: before the wait
  const float w_scale = __ldg(a.w_scale);
  const int most = most_pow2(w_scale);
  if (threadIdx.x == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    mbar_init(drained, 1);
    mbar_init_fence();
    *gave_up_at = 0;
  }
  pdl_wait();

  // x: half-warp h takes rows h, h + 32, ..
  const int h = threadIdx.x >> 4, l = threadIdx.x & 15;
  RawX x[kXEach];
  XRow<FORM> x_row[kXEach];
  int k_left = min(a.K, g1 * kGroup) - g0 * kGroup - 8 * l;  // columns from this lane's first of the next step on
#pragma unroll
  for (int i = 0; i < kXEach; ++i) {
    x_row[i].set(a, h + 32 * i, g0, l);
    x[i] = x_row[i].next(a, h + 32 * i < a.rows && k_left > 0);
  }
  if (warp == 0) {
    __syncwarp();
    tc_alloc<kCols>(tmem_at);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t my_tmem = tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * kQ;
  pdl_release();

  bool gave_up = false;
  auto wait = [&](int b, int phase) {
    if (!gave_up && !mbar_wait_bounded(&bar[b], phase, polls)) {
      gave_up = true;
      *gave_up_at = 1;
    }
  };
  float acc[kQ];
#pragma unroll
  for (int i = 0; i < kQ; ++i) acc[i] = 0.0f;
  // adds step i's sums with their factors
  static_assert(kAhead == 3, "a step's place in the unrolled loop is its place in xs");
  auto add_step = [&](int i, int third) {  // third: i % 3
    wait(i & 1, (i >> 1) & 1);
    __syncwarp();
    tc_fence_after();
    float d[kQ];
#pragma unroll
    for (int c = 0; c < kQ; c += 4) tc_ld4(my_tmem + (i & 1) * NX + c, d + c);
    tc_wait_ld();
    const float4* f = reinterpret_cast<const float4*>(xs + third * NX + (warp >> 2) * kQ);
#pragma unroll
    for (int c = 0; c < kQ; c += 4) {
      const float4 u = f[c / 4];
      acc[c] = fmaf(d[c], u.x, acc[c]);
      acc[c + 1] = fmaf(d[c + 1], u.y, acc[c + 1]);
      acc[c + 2] = fmaf(d[c + 2], u.z, acc[c + 2]);
      acc[c + 3] = fmaf(d[c + 3], u.w, acc[c + 3]);
    }
    tc_fence_before();
  };

  const int steps = g1 - g0;
  const uint32_t line0 = wrow * 128 + (((2 * (lane & 3)) ^ (wrow & 7)) << 4);
  const uint32_t line1 = wrow * 128 + (((2 * (lane & 3) + 1) ^ (wrow & 7)) << 4);
  for (int i0 = 0; i0 < steps; i0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u, b = i & 1;
      if (i >= steps) break;
      const uint32_t to_a = base + b * T::kStage, to_b = to_a + T::kA;
      if (!kScaled && i >= 2) wait(b, ((i >> 1) - 1) & 1);  // (with factors: add_step has waited)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t f = e4m3_to_both(w[u].sf[j]), to = to_a + j * kRegionA;
        uint32_t v[8];
        e2m1x8_to_half2(w[u].c[j].x, v);
        e2m1x8_to_half2(w[u].c[j].y, v + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = hmul2(v[e], f);
        st_shared16(to + line0, make_uint4(v[0], v[1], v[2], v[3]));
        st_shared16(to + line1, make_uint4(v[4], v[5], v[6], v[7]));
      }
      k_left -= kGroup;
#pragma unroll
      for (int n = 0; n < kXEach; ++n) {
        const int r = h + 32 * n;
        const uint4 v = convert_x<FORM>(x[n], most);
        st_shared16(to_b + (l >> 3) * (NX * 128) + r * 128 + (((l & 7) ^ (r & 7)) << 4), v);
        if (kScaled && l == 0) xs[u * NX + r] = x[n].scale * w_scale;
        x[n] = x_row[n].next(a, r < a.rows && k_left > 0);
      }
      load_w(w[u]);  // (behind x, which is wanted sooner)
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (threadIdx.x == 0) {
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_smem(tmem + (kScaled ? b * NX : 0), smem_operand(to_a + (k >> 2) * kRegionA + (k & 3) * 32, 16, 1024),
                      smem_operand(to_b + (k >> 2) * (NX * 128) + (k & 3) * 32, 16, 1024), product_desc(nx, false),
                      kScaled ? k > 0 : i > 0 || k > 0);
        tc_commit(&bar[b]);
      }
      __syncwarp();
      if (kScaled && i > 0) add_step(i - 1, (u + 2) % 3);
    }
  }
  if (kScaled) {
    add_step(steps - 1, (steps - 1) % 3);
  } else {
    if (steps > 1) wait(steps & 1, ((steps - 2) >> 1) & 1);
    wait((steps - 1) & 1, ((steps - 1) >> 1) & 1);
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < kQ; c += 4) tc_ld4(my_tmem + c, acc + c);
    tc_wait_ld();
  }
  tc_fence_before();
  __syncthreads();
  if (*gave_up_at != 0) {  // a wait that ran out: the rows become NaN; the products end before TMEM is freed
    if (threadIdx.x == 0) {
      tc_commit(drained);
      (void)mbar_wait_bounded(drained, 0, 1 << 14);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kQ; ++c) acc[c] = __int_as_float(0x7FC00000);
  }
  __syncwarp();
  if (warp == 0) tc_free<kCols>(tmem);

  const float scale = kScaled ? 1.0f : w_scale * (FORM == kX16 ? 1.0f : a.x_scales[0]);
  const int n = tile * kRows + 32 * (warp & 3) + lane, col0 = (warp >> 2) * kQ;
  if (ranks == 1) {
    if (n < a.N) {
#pragma unroll
      for (int c = 0; c < kQ; ++c)
        if (col0 + c < a.rows) store_y1(a, col0 + c, n, acc[c], scale);
    }
    return;
  }
  // a cluster's sums over the operands that nothing reads any more: [row of x][weight row]
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int c = 0; c < kQ; ++c) sums[(col0 + c) * kRows + 32 * (warp & 3) + lane] = acc[c];
  cluster_sync();
  const int q = (threadIdx.x & 31) * 4;  // four weight rows to a lane, a row of x to a warp
  for (int r = rank * (kThreads / 32) + warp; r < a.rows; r += ranks * (kThreads / 32)) {
    const uint32_t at = base + (r * kRows + q) * 4;
    float4 s[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < ranks) s[c] = ld_cluster4(cluster_addr(at, c));
#pragma unroll
    for (int c = 1; c < 8; ++c)
      if (c < ranks) {
        s[0].x += s[c].x;
        s[0].y += s[c].y;
        s[0].z += s[c].z;
        s[0].w += s[c].w;
      }
    const float y[4] = {s[0].x, s[0].y, s[0].z, s[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (tile * kRows + q + e < a.N) store_y1(a, r, tile * kRows + q + e, y[e], scale);
  }
  cluster_sync();  // the sums are read
}

template <int NX, XForm FORM>
frt_status launch_tiles(MatvecArgs a, cudaStream_t stream) {
  static SmemOptIn opted;
  const frt_status st = opt_in_smem(tiles_kernel<NX, FORM>, Tile<NX>::kSmem, opted);
  if (st != FRT_OK) return st;
  a.tiles = (int)(((int64_t)a.N + kRows - 1) / kRows);
  // k is split while that fills the SMs better and leaves a CTA two steps
  a.cluster = 1;
  while (a.cluster < 8 && a.tiles <= cluster_room(1, 2 * a.cluster) && a.groups >= 4 * a.cluster) a.cluster *= 2;
  const dim3 grid((unsigned)(a.tiles * a.cluster)), block(kThreads);
  if (a.cluster > 1)
    return launch_cluster(tiles_kernel<NX, FORM>, grid, block, Tile<NX>::kSmem, stream, a.cluster, a, wait_polls());
  return launch(tiles_kernel<NX, FORM>, grid, block, Tile<NX>::kSmem, stream, a, wait_polls());
}
template <XForm FORM>
frt_status launch_form(const MatvecArgs& a, cudaStream_t stream) {
  return a.rows <= 32   ? launch_tiles<32, FORM>(a, stream)
         : a.rows <= 64 ? launch_tiles<64, FORM>(a, stream)
                        : launch_tiles<128, FORM>(a, stream);
}

}  // namespace

frt_status launch_matvec_tiles(const MatvecArgs& a, cudaStream_t stream) {
  switch (a.form) {
    case kX16: return launch_form<kX16>(a, stream);
    case kXScaled16: return launch_form<kXScaled16>(a, stream);
    case kXE4M3: return launch_form<kXE4M3>(a, stream);
    case kXE4M3Block: return launch_form<kXE4M3Block>(a, stream);
    default: return launch_form<kXNvfp4>(a, stream);
  }
}

}  // namespace frt
