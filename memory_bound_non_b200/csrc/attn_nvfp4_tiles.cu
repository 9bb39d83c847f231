// Attention over an NVFP4 KV cache for many query rows (a chunk of a prefill, a
// wide group): 128 rows of one KV head to a CTA, on the 5th-generation tensor
// cores.
//
// What bounds it: 4 hd operations per row and key on the tensor cores and one
// exponential per row and key on the special-function units (16 a clock and
// SM: 1024 clocks for a tile of 128 x 128, the products take 1024 together at
// hd 128); the cache is read from L2 by the row tiles of a head.
//
// One tile of KT keys:
//   K codes -> binary16 in shared memory (all warps)      | P V of the tile before
//   S = Q K^T                        (tcgen05, S in TMEM)  | V codes -> binary16
//   p = 2^(s - m + 11) in registers, two threads a row
//   P -> TMEM (binary16, over S), O += P V  (tcgen05, P from TMEM, O in TMEM)
// Two CTAs share an SM (hd <= 192), so that one's products run beside the
// other's conversions and exponentials.  Inside a CTA only the warp that issues P V
// waits for all of P and V; the others go on to the next tile's K.
// Measured, 512 tokens of 16/8 heads of 128 over 4608 positions: 47 us, 390
// TFLOP/s (46.6 to 47.1 in repeats; the warps' products took 142; with block-wide
// barriers in those places and one exponential's argument to an instruction
// 47.9); a tile takes 3600 clocks of an SM against the 1024 of its bound, in the
// latency of its dependent steps; a call costs 10 us before and behind its tiles.
//
// Operand layouts: Q and K as rows of 64 dimensions (128 bytes) with the
// 128-byte swizzle, k-major; V in the same form, which read as the B operand of
// P V is mn-major (dimensions contiguous, keys eight to a group of 1024 bytes).
// The 16-byte pieces are written by lanes that hold 4 blocks of 2 keys, which
// is free of bank conflicts.
//
// m is renewed when a score passes it by more than 4 (as in the kernel for few
// rows); O is then rescaled in TMEM.  c >= 0: a negative scale is moved into Q.
#include "attn_nvfp4.cuh"
#include "frt_tensor.cuh"

namespace frt {
namespace {

constexpr int kThreads = 256;
constexpr size_t kSmallBytes = 9 * 1024;     // struct Small
constexpr int kQRegion = kTileRows * 128;  // bytes of 64 dimensions of all rows

template <int HD>
struct Tile {
  static constexpr int C = HD / 64;          // regions of 64 dimensions
  static constexpr int KT = tile_keys(HD);   // keys
  static constexpr int kRegion = KT * 128;   // bytes of 64 dimensions of all keys
  static constexpr int U = KT * C / 64;      // 16-element blocks a thread converts
  static constexpr int kCols = KT + HD <= 256 ? 256 : 512;  // TMEM columns: S (P over it), O
  static constexpr int kO = KT;                             // first column of O
  // (a cluster's parts, 128 rows of HD floats, fit over the operands)
  static_assert(kTileRows * HD * 4 <= C * (kQRegion + 2 * kRegion), "parts over the operands");
  static constexpr size_t kUsed = 1024 + C * (kQRegion + 2 * kRegion) + kSmallBytes;
  static constexpr size_t kSmem = kUsed > tmem_smem(kCols) ? kUsed : tmem_smem(kCols);
};

// x plus both halves of w, one rounding each.
__device__ __forceinline__ float add_halves(float x, uint32_t w) {
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
      "add.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %0, hi, %0;\n\t}"
      : "+f"(x)
      : "r"(w));
  return x;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy_async16(uint32_t to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

struct Small {  // behind the operands
  float top[2][kTileRows];    // each half's largest score of a row; at the end its sum
  float scale[kTileRows];     // score -> log2 units
  int tok[kTileRows], head[kTileRows];
  int slot[2][32];            // quad slots of a tile, by tile parity
  int holes[2];               // a tile has quads that are not there
  uint32_t nan[4];            // keys of the tile with a NaN factor in V
  float2 ml[kTileRows];       // (maximum, sum) of a row, for the cluster
  float factor[8][kTileRows];
  uint64_t s_done, o_done, drained;  // products
  uint64_t v_ready, p_ready;         // a tile's V and P, an arrival of each warp
  uint32_t tmem;
  int gave_up;
};
static_assert(sizeof(Small) <= kSmallBytes, "fits behind the operands");

template <int HD>
__global__ void __launch_bounds__(kThreads, HD > 192 ? 1 : 2) tiles_kernel(const AttnArgs a, int polls) {
  using T = Tile<HD>;
  constexpr int C = T::C, KT = T::KT, U = T::U, kRegion = T::kRegion;
  extern __shared__ unsigned char raw_smem[];
  const uint32_t base = (smem_addr(raw_smem) + 1023) & ~1023u;
  const uint32_t q_smem = base, k_smem = base + C * kQRegion, v_smem = k_smem + C * kRegion;
  Small& sm = *reinterpret_cast<Small*>(raw_smem + (v_smem + C * kRegion - smem_addr(raw_smem)));

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  const Place place = place_of(a);
  const int kvh = place.kvh, rt = place.rt, chunk = place.chunk;

  pdl_wait();
  const Seq seq = sequence(a, b);
  const RowRange range = row_range<kTileRows>(a, seq, rt * kTileRows, kvh);
  if (range.bad && a.status != nullptr) atomicOr(a.status, 1);
  const int tiles = range.tiles(KT);
  const int2 part = tiles_of(a, chunk, tiles);
  const int tile0 = part.x, tile1 = part.y;
  if (!range.any || (!a.cluster && chunk > 0 && tile0 >= tiles)) return;  // no rows, or no work

  // this thread's row and half of the columns (TMEM lanes are split by warp % 4)
  const int row = 32 * (warp & 3) + lane, half = warp >> 2;
  const QueryRow mine = query_row(a, seq, rt * kTileRows + row, kvh);
  if (half == 0) {
    sm.tok[row] = mine.tok;
    sm.head[row] = mine.head;
  }
  if (threadIdx.x == 0) {
    mbar_init(&sm.s_done, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.drained, 1);
    mbar_init(&sm.v_ready, kThreads / 32);
    mbar_init(&sm.p_ready, kThreads / 32);
    mbar_init_fence();
    sm.gave_up = 0;
  }
  if (warp == 0) {
    __syncwarp();
    tc_alloc<T::kCols>(&sm.tmem);
  }

  const int nblk = a.hd >> 4;
  auto find_slots = [&](int tile) {  // warp 0
    const int slot = tile < tile1 && lane < KT / 4 ? quad_slot(a, b, range.first() + tile * KT + 4 * lane, range) : -1;
    sm.slot[tile & 1][lane] = slot;
    const bool hole = __any_sync(0xFFFFFFFFu, lane < KT / 4 && slot < 0);
    if (lane == 0) sm.holes[tile & 1] = hole;
  };
  if (warp == 0) find_slots(tile0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();
  const uint32_t tmem = sm.tmem;
  const uint32_t s_tmem = tmem + ((uint32_t)(warp & 3) << 21), o_tmem = s_tmem + T::kO;

  // The blocks that this thread converts: of unit i key key0 + 64 (i / C), region
  // i % C, block lane % 4 of it.
  const int key0 = 8 * warp + 2 * (lane >> 3) + ((lane >> 2) & 1);
  struct Raw {
    uint2 c[U];
    uint32_t sf[U];
  };
  const int row_bytes = a.Hkv * (a.hd >> 1), sf_row = a.Hkv * nblk;
  const int code0 = (key0 & 3) * row_bytes + kvh * (a.hd >> 1) + 8 * (lane & 3);
  const int sf0 = (kvh * nblk + (lane & 3)) * 4 + (key0 & 3);
  auto load = [&](const uint8_t* codes, const uint8_t* sf, int tile, Raw& r) {
    const int left = range.all_hi - (range.first() + tile * KT) - key0;
#pragma unroll
    for (int j = 0; j < U / C; ++j) {
      const int quad = tile < tile1 ? sm.slot[tile & 1][(key0 >> 2) + 16 * j] : -1;
      const bool on = quad >= 0 && 64 * j < left;
      const uint8_t* pc = codes + code0 + (int64_t)quad * row_bytes;
      const uint8_t* ps = sf + sf0 + (int64_t)quad * sf_row;
#pragma unroll
      for (int kc = 0; kc < C; ++kc) {
        const int i = j * C + kc;
        r.c[i] = make_uint2(0, 0);
        r.sf[i] = 0;
        if (on && 4 * kc + (lane & 3) < nblk) {
          if (FRT_SPAN_OK(pc + 32 * kc - codes, 8, (int64_t)a.capacity * row_bytes))
            r.c[i] = ld_stream(reinterpret_cast<const uint2*>(pc + 32 * kc));
          if (FRT_IDX_OK(ps + 16 * kc - sf, (int64_t)((a.capacity + 3) >> 2) * sf_row * 4)) r.sf[i] = __ldg(ps + 16 * kc);
        }
      }
    }
  };
  const int line0 = key0 * 128 + (((2 * (lane & 3)) ^ (key0 & 7)) << 4);
  const int line1 = key0 * 128 + (((2 * (lane & 3) + 1) ^ (key0 & 7)) << 4);
  auto convert = [&](const Raw& r, uint32_t to, bool is_v) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      uint32_t sf = r.sf[i];
      if (is_v && (sf & 0x7F) == 0x7F) {
        const int key = key0 + 64 * (i / C);
        sf = 0;
        atomicOr(&sm.nan[key >> 5], 1u << (key & 31));
      }
      const uint32_t f = e4m3_to_both(sf);
      uint32_t h[8];
      e2m1x8_to_half2(r.c[i].x, h);
      e2m1x8_to_half2(r.c[i].y, h + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = hmul2(h[e], f);
      const uint32_t at = to + (i % C) * kRegion + (i / C) * 64 * 128;
      st_shared16(at + line0, make_uint4(h[0], h[1], h[2], h[3]));
      st_shared16(at + line1, make_uint4(h[4], h[5], h[6], h[7]));
    }
  };
  bool gave_up = false;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!gave_up && !mbar_wait_bounded(bar, phase, polls)) {
      gave_up = true;
      sm.gave_up = 1;
    }
  };

  Raw k_raw;
  load(a.k_codes, a.k_sf, tile0, k_raw);

  // ---- Q: 16 lanes a row (32 above 128 dimensions)
  {
    constexpr int kLanes = HD <= 128 ? 16 : 32, kRows = 32 / kLanes;
    const float c = a.scale_log2 * __ldg(a.kv_scales);
    const uint32_t flip = c < 0.0f ? 0x80008000u : 0u;
    const int l = lane % kLanes;
    // Copied as they are to where they belong, then converted there: short
    // loops, since code that runs once costs its instruction fetches.
    auto q_row = [&](int i) { return (i * 8 + warp) * kRows + lane / kLanes; };
    auto q_at = [&](int r) { return q_smem + (l >> 3) * kQRegion + r * 128 + (((l & 7) ^ (r & 7)) << 4); };
    constexpr int kIters = kTileRows / (8 * kRows);
#pragma unroll 2
    for (int i = 0; i < kIters; ++i) {
      const int r = q_row(i), tok = sm.tok[r];
      const int64_t at = ((int64_t)max(tok, 0) * a.Hq + sm.head[r]) * (a.hd / 8) + min(l, a.hd / 8 - 1);
      const bool on = tok >= 0 && l < a.hd / 8 && FRT_IDX_OK(at, (int64_t)a.M * a.Hq * (a.hd / 8));
      if (l < HD / 8) copy_async16(q_at(r), static_cast<const uint4*>(a.q) + at, on);
    }
    copy_async_wait();
#pragma unroll 1
    for (int i = 0; i < kIters; ++i) {
      const int r = q_row(i);
      float s = 1.0f;
      if (a.dt == FRT_BF16 || flip != 0) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (l < HD / 8) v = ld_shared16(q_at(r));
        if (a.dt == FRT_BF16) {
          float2 f[4];
          unpack_pairs<FRT_BF16, 4>(&v.x, f);
          const float amax = fmaxf(absmax4(f[0].x, f[0].y, f[1].x, f[1].y), absmax4(f[2].x, f[2].y, f[3].x, f[3].y));
          s = pow2_to_half_range(kLanes == 16 ? half_warp_max_abs(amax) : warp_max_abs(amax));
          mul_pairs<4>(f, s);
          pack_pairs<FRT_F16, 4>(f, &v.x);
        }
        if (l < HD / 8) st_shared16(q_at(r), make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
      }
      // (never 0, which would make a masked score NaN)
      if (l == 0) sm.scale[r] = fmaxf(fabsf(c) / s, 0x1p-120f);
    }
  }

  const float kInf = __int_as_float(0x7F800000);
  float m = -kInf, sum = 0.0f;
  for (int tile = tile0; tile < tile1; ++tile) {
    const int nth = tile - tile0;
    Raw v_raw;
    load(a.v_codes, a.v_sf, tile, v_raw);
    if (warp == 0) find_slots(tile + 1);
    if (threadIdx.x < 4) sm.nan[threadIdx.x] = 0;
    convert(k_raw, k_smem, false);
    fence_proxy_async_smem();
    if (nth > 0) wait(&sm.o_done, (nth - 1) & 1);  // V and P of the tile before are read
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
        tc_mma_smem(tmem, smem_operand(q_smem + (k >> 2) * kQRegion + (k & 3) * 32, 16, 1024),
                    smem_operand(k_smem + (k >> 2) * kRegion + (k & 3) * 32, 16, 1024), product_desc(KT, false), k > 0);
      tc_commit(&sm.s_done);
    }
    __syncwarp();
    convert(v_raw, v_smem, true);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.v_ready);
    load(a.k_codes, a.k_sf, tile + 1, k_raw);

    wait(&sm.s_done, nth & 1);
    __syncwarp();
    tc_fence_after();
    uint32_t s[KT / 2];
#pragma unroll
    for (int i = 0; i < KT / 64; ++i) tc_ld32(s_tmem + half * (KT / 2) + 32 * i, s + 32 * i);
    tc_wait_ld();
    // masks
    const int pos = range.first() + tile * KT + half * (KT / 2);
    const int pos0 = range.first() + tile * KT;
    if (pos0 < range.full_lo || range.full_hi - pos0 < KT || sm.holes[tile & 1] != 0) {
      const int from = mine.lo - pos, to = mine.hi - pos;
#pragma unroll
      for (int i = 0; i < KT / 2; ++i) {
        const bool there = sm.slot[tile & 1][(half * (KT / 2) + i) >> 2] >= 0;
        if (i < from || i >= to || !there) s[i] = 0xFF800000u;
      }
    }
    float top = __uint_as_float(s[0]);
#pragma unroll
    for (int i = 1; i < KT / 2; ++i) top = fmaxf(top, __uint_as_float(s[i]));
    sm.top[half][row] = top;
    tc_fence_before();
    pair_sync(1 + (warp & 3));  // the other half's maxima are there, and its part of S is read (P lies over S)
    const float c = sm.scale[row];
    top = fmaxf(top, sm.top[half ^ 1][row]) * c;
    wait(&sm.v_ready, nth & 1);
    // a NaN factor in V: the weight of its key turns NaN for the rows that see it
#pragma unroll
    for (int w = 0; w < KT / 64; ++w) {
      const uint32_t nan = sm.nan[half * (KT / 64) + w];
      if (nan != 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if ((nan >> i & 1) && s[32 * w + i] != 0xFF800000u) s[32 * w + i] = 0x7FC00000u;
      }
    }
    const bool renew = top > m + 4.0f;
    float f = 1.0f;
    if (renew) {
      f = ex2_approx(m - top);
      m = top;
      sum *= f;
    }
    __syncwarp();
    tc_fence_after();
    if (nth > 0 && __any_sync(0xFFFFFFFFu, renew)) {
#pragma unroll 1
      for (int i = 0; i < HD / 64; ++i) {
        uint32_t o[32];
        const uint32_t at = o_tmem + half * (HD / 2) + 32 * i;
        tc_ld32(at, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tc_st32(at, o);
      }
    }
    const float shift = 11.0f - (m == -kInf ? 0.0f : m);
    uint32_t p[KT / 4];
    // (the tile's weights by themselves: one by one, those below half a step of the
    // running sum would all be rounded alike, 0.3 % of it over 131072 positions)
    float tile_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < KT / 4; ++i) {
      const float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                                  make_float2(c, c), make_float2(shift, shift));
      p[i] = Pack16<FRT_F16>::from_float2(ex2_approx(e.x), ex2_approx(e.y));
      tile_sum = add_halves(tile_sum, p[i]);
    }
    sum += tile_sum;
    if constexpr (KT == 128)
      tc_st32(s_tmem + half * 32, p);
    else
      tc_st16(s_tmem + half * 16, p);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.p_ready);
    if (warp == 0) {  // (the others go on to the next tile's K)
      wait(&sm.p_ready, nth & 1);
      __syncwarp();
      if (lane == 0) {
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          tc_mma_tmem(tmem + T::kO, tmem + 8 * k, smem_operand(v_smem + k * 2048, kRegion, 1024),
                      product_desc(HD, true), nth > 0 || k > 0);
        tc_commit(&sm.o_done);
      }
      __syncwarp();
    }
  }

  // ---- output
  const int n = tile1 - tile0;
  if (n > 0) wait(&sm.o_done, (n - 1) & 1);
  sm.top[half][row] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  sum += sm.top[half ^ 1][row];
  const bool whole = !a.cluster && tiles <= a.chunk_tiles;  // this CTA saw all of the keys
  const float gs_v = __ldg(a.kv_scales + 1);
  // The sums go through shared memory, over the operands that nothing reads any
  // more (128 rows of HD floats, their 16-byte pieces swizzled by row), so that
  // neighbouring threads write neighbouring dimensions and the CTAs of a cluster
  // can read one another's.
#pragma unroll 1
  for (int i = 0; i < HD / 64; ++i) {
    uint32_t o[32];
    const int d0 = half * (HD / 2) + 32 * i;
    if (n > 0) {
      tc_ld32(o_tmem + d0, o);
      tc_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      st_shared16(base + row * (HD * 4) + ((((d0 + e) >> 2) ^ (row & 7)) << 4),
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
  }
  if (half == 0) {
    sm.ml[row] = make_float2(m, sum);
    if (!a.cluster && mine.tok >= 0) {
      const int64_t q_row = (int64_t)mine.tok * a.Hq + mine.head;
      if (chunk == 0) store_chunks(a, q_row, tiles);
      const int64_t at = (int64_t)chunk * a.M * a.Hq + q_row;
      if (!whole && FRT_IDX_OK(at, (int64_t)a.M * a.Hq * a.chunks)) a.part_ml[at] = make_float2(m, sum);
    }
  }
  if (a.cluster)
    cluster_sync();
  else
    __syncthreads();
  // each row's factors for the parts
  const int ctas = a.cluster ? a.chunks : 1, rank = a.cluster ? chunk : 0;
  if (threadIdx.x < kTileRows) {
    const int r = threadIdx.x;
    if (a.cluster) {
      cluster_factors(a, smem_addr(sm.ml + r), gs_v, &sm.factor[0][r], kTileRows);
    } else {
      const float total = sm.ml[r].y;
      sm.factor[0][r] = !whole ? 1.0f : total == 0.0f ? 0.0f : gs_v / total;
    }
  }
  __syncthreads();
  // pieces of four dimensions, dealt to the CTAs of a cluster
#pragma unroll 1
  for (int i = rank * kThreads + threadIdx.x; i < kTileRows * (HD / 4); i += ctas * kThreads) {
    const int r = i / (HD / 4), d = i % (HD / 4) * 4;
    const int tok = sm.tok[r];
    if (tok < 0 || d >= a.hd) continue;
    const int64_t at = ((int64_t)tok * a.Hq + sm.head[r]) * a.hd + d;
    const uint32_t piece = base + r * (HD * 4) + (((d >> 2) ^ (r & 7)) << 4);
    float4 v;
    if (a.cluster) {
      v = join_cluster4(a, piece, rank, &sm.factor[0][r], kTileRows);
    } else {
      const float4 u = ld_shared4(piece);
      const float f = sm.factor[0][r];
      v = make_float4(u.x * f, u.y * f, u.z * f, u.w * f);
    }
    if (a.cluster || whole)
      store_out4(a, at, v, 1.0f);
    else
      store_part4(a, chunk, at, v);
  }
  if (a.cluster) cluster_sync();  // the parts are read
  // a wait that ran out: report it, and let the products end before TMEM is freed
  if (sm.gave_up != 0 && threadIdx.x == 0) {
    if (a.status != nullptr) atomicOr(a.status, 2);
    tc_commit(&sm.drained);
    (void)mbar_wait_bounded(&sm.drained, 0, 1 << 16);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tc_free<T::kCols>(tmem);
}

template <int HD>
frt_status launch_tiles(const AttnArgs& a, cudaStream_t stream) {
  static SmemOptIn opted;
  const frt_status st = opt_in_smem(tiles_kernel<HD>, Tile<HD>::kSmem, opted);
  if (st != FRT_OK) return st;
  const dim3 grid((unsigned)(a.Hkv * a.row_tiles * a.chunks), a.n_seqs), block(kThreads);
  if (a.cluster)
    return launch_cluster(tiles_kernel<HD>, grid, block, Tile<HD>::kSmem, stream, a.chunks, a, wait_polls());
  return launch(tiles_kernel<HD>, grid, block, Tile<HD>::kSmem, stream, a, wait_polls());
}

}  // namespace

frt_status launch_attn_tiles(const AttnArgs& a, cudaStream_t stream) {
  return a.hd <= 64    ? launch_tiles<64>(a, stream)
         : a.hd <= 128 ? launch_tiles<128>(a, stream)
         : a.hd <= 192 ? launch_tiles<192>(a, stream)
                       : launch_tiles<256>(a, stream);
}

}  // namespace frt
