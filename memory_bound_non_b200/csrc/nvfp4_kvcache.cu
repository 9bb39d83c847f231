// NVFP4 KV cache: the writer (op (b) with a 4-bit store) and the reader.
//
// Writer.  Per head of hd elements: RMSNorm, rotate-half RoPE, then for K and
// V blocks of 16 with an e4m3 factor sf = e4m3(amax / (6 gs)) and codes
// e2m1(y / (sf gs)) (scaled by rounded reciprocals, as the NVFP4 producers).
// 2 B an element are read, 2 B of Q or 0.5625 B of K and V written.
//
// Mapping: hd/16 lanes hold a head, each 8 elements of the lower half and
// their 8 rotation partners of the upper half (two 16-byte loads), so RoPE
// needs no exchange, a block is two neighbouring 8-element units and the head
// reduction is a few shuffles inside a group of P >= hd/16 lanes.  A warp
// holds heads of one kind (Q, K or V) only; of Q a lane group takes two heads
// of a token, which share its RoPE rows.
//
// What bounds it: 4096 tokens of 32/8 heads of 128 take about 27 us, 2.1 times
// their bytes at the copy rate: half the issue slots (K's exact products and the
// 16-bit unpacking) and the wait for rows at random positions of the tables.
// With one head to a lane group and 64-bit index arithmetic it took 39 us.  A
// few tokens are bound by the launch (ten: 5.6 us with the reader, two launches).
//
// K decides its codes next to e2m1 borders, so y has to be the exact value
// rounded once: products as exact pairs (p, e) by FMA, their difference by
// TwoSum, rstd as a pair from an fp64 sum: 16 fp32 operations an element on K
// alone (a sixth of the heads of a 32/8 layer).
#include "frt_device.cuh"
#include "frt_fragments.cuh"
#include "frt_host.h"

namespace frt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// head kinds
constexpr int kQ = 0, kK = 1, kV = 2;

struct WriteArgs {
  const uint4* qkv;
  const uint4* q_norm_w;
  const uint4* k_norm_w;
  const float4* cos_tab;
  const float4* sin_tab;
  const int32_t* positions;
  const int32_t* slots;
  uint4* q_out;
  uint32_t* codes[2];  // K, V
  uint8_t* sf[2];
  const float* kv_scales;
  int32_t* status;
  int M, Hq, Hkv, L;  // L = hd / 16: lanes of a head, and 16-byte chunks of half a head
  int max_pos, capacity;
  float eps, inv_hd;
  double inv_hd64;
  int q_units;                // units of kQHeads Q heads of a token
  uint32_t q_mul, kv_mul;     // i / d = (i + umulhi(i, mul)) >> shift, 0 <= i < 2^31
  int q_shift, kv_shift;
  int64_t warps_q, warps_kv;  // warps that hold Q units, and K (or V) heads
};
constexpr int kQHeads = 2;

__device__ __forceinline__ int divide(int i, uint32_t mul, int shift) {
  return (int)((__umulhi((uint32_t)i, mul) + (uint32_t)i) >> shift);
}
void divisor(int d, uint32_t* mul, int* shift) {
  *shift = 0;
  while ((1LL << *shift) < d) ++*shift;
  *mul = (uint32_t)((((1ULL << *shift) - d) << 32) / d + 1);
}

// Exact a * b - c * d of fp32 numbers as an unevaluated pair (to ~2^-48 of the
// larger product).
__device__ __forceinline__ void diff_of_products(float a, float b, float c, float d, float* hi, float* lo) {
  const float p = a * b, q = c * d;
  const float ep = fmaf(a, b, -p), eq = fmaf(c, d, -q);
  const float s = p - q;
  const float t = s - p;
  *hi = s;
  *lo = ((p - (s - t)) - (q + t)) + (ep - eq);
}
// (hi + lo) * (r.hi + r.lo), rounded once to fp32.
__device__ __forceinline__ float pair_mul(float hi, float lo, const Split32& r) {
  const float p = hi * r.hi;
  const float e = fmaf(hi, r.hi, -p);
  return p + fmaf(hi, r.lo, fmaf(lo, r.hi, e));
}

__device__ __forceinline__ float amax8(const float* y) {
  return fmaxf(absmax4(y[0], y[1], y[2], y[3]), absmax4(y[4], y[5], y[6], y[7]));
}
// Largest magnitude of 8 elements; +inf if one of them is not finite.
__device__ __forceinline__ float amax8_or_inf(const float* y) {
  bool fine = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) fine = fine && (fabsf(y[e]) < __int_as_float(0x7F800000));
  return fine ? amax8(y) : __int_as_float(0x7F800000);
}

// P: lanes of a head, the next power of two from L (4, 8 or 16; 1 and 2 for
// the smallest heads).
template <int DT, int P>
__global__ void __launch_bounds__(kThreads, 4) write_kernel(WriteArgs a) {
  const int lane = threadIdx.x & 31;
  // K's heads first, which take longest
  int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int kind = kK;
  if (w >= a.warps_kv) {
    w -= a.warps_kv;
    kind = kV;
    if (w >= a.warps_kv) {
      w -= a.warps_kv;
      kind = kQ;
    }
  }
  const int64_t count = (int64_t)a.M * (kind == kQ ? a.q_units : a.Hkv);  // (below 2^31)
  const int64_t item = w * (32 / P) + lane / P;                           // of this lane group
  bool on = item < count && lane % P < a.L;
  // Lanes without work load what the last one loads; nothing is stored for them.
  const int l = min(lane % P, a.L - 1);
  const int it = (int)min(item, count - 1);
  const int i = kind == kQ ? divide(it, a.q_mul, a.q_shift) : divide(it, a.kv_mul, a.kv_shift);
  const int h = kind == kQ ? (it - i * a.q_units) * kQHeads : it - i * a.Hkv;
  const int heads = a.Hq + 2 * a.Hkv;
  const int C = 2 * a.L;  // chunks of a head

  // constant inputs before the wait
  const uint4* norm_w = kind == kQ ? a.q_norm_w : a.k_norm_w;
  const bool normed = kind != kV && norm_w != nullptr;
  uint4 w_lo = make_uint4(0, 0, 0, 0), w_hi = w_lo;
  if (normed && FRT_IDX_OK(l + a.L, C)) {
    w_lo = __ldg(norm_w + l);
    w_hi = __ldg(norm_w + l + a.L);
  }
  const float gs = kind == kQ ? 1.0f : __ldg(a.kv_scales + (kind - kK));
  pdl_enter();

  int p = 0, slot = 0;
  if (FRT_IDX_OK(i, a.M)) {
    p = __ldg(a.positions + i);
    slot = a.slots != nullptr ? __ldg(a.slots + i) : p;
  }
  // x of the head (of both heads of a Q unit): issued before the position is
  // looked at, which the RoPE rows follow
  const int64_t x_chunks = (int64_t)a.M * heads * C;
  const int64_t in0 = (int64_t)i * heads * C + (kind == kQ ? h : kind == kK ? a.Hq + h : a.Hq + a.Hkv + h) * C + l;
  const bool second = kind == kQ && h + 1 < a.Hq;
  uint4 x_lo = make_uint4(0, 0, 0, 0), x_hi = x_lo, x2_lo = x_lo, x2_hi = x_lo;
  if (FRT_IDX_OK(in0 + a.L, x_chunks)) {
    x_lo = ld_stream(a.qkv + in0);
    x_hi = ld_stream(a.qkv + in0 + a.L);
  }
  if (second && FRT_IDX_OK(in0 + C + a.L, x_chunks)) {
    x2_lo = ld_stream(a.qkv + in0 + C);
    x2_hi = ld_stream(a.qkv + in0 + C + a.L);
  }
  if (p < 0 || p >= a.max_pos || slot < 0 || slot >= a.capacity) {
    if (a.status != nullptr && on && l == 0) atomicOr(a.status, 1);
    on = false;
    p = 0;
  }
  float2 cs[4], sn[4], nsn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) cs[e] = sn[e] = nsn[e] = make_float2(0.0f, 0.0f);
  if (kind != kV && FRT_SPAN_OK((int64_t)p * C + 2 * l, 2, (int64_t)a.max_pos * C)) {
    const float* c = reinterpret_cast<const float*>(a.cos_tab + (int64_t)p * C + 2 * l);
    const float* s = reinterpret_cast<const float*>(a.sin_tab + (int64_t)p * C + 2 * l);
    load_rope_pairs<4>(c, s, cs, sn, nsn);
  }

  if (kind == kQ) {
    const int64_t q0 = (int64_t)i * a.Hq * C + h * C + l;
#pragma unroll
    for (int n = 0; n < kQHeads; ++n) {
      float2 lo[4], hi[4];
      unpack_pairs<DT, 4>(n == 0 ? &x_lo.x : &x2_lo.x, lo);
      unpack_pairs<DT, 4>(n == 0 ? &x_hi.x : &x2_hi.x, hi);
      if (normed) {
        const float ss = group_sum<P>(lane % P < a.L ? sum_squares_pairs<4>(lo, hi) : 0.0f);
        const float r = head_rstd(ss, a.inv_hd, a.eps);
        float2 wl[4], wh[4];
        unpack_pairs<DT, 4>(&w_lo.x, wl);
        unpack_pairs<DT, 4>(&w_hi.x, wh);
        scale_pairs<4>(lo, r, wl);
        scale_pairs<4>(hi, r, wh);
      }
      float2 o1[4], o2[4];
      rope_pairs<4>(lo, hi, cs, sn, nsn, o1, o2);
      uint4 s1, s2;
      pack_pairs<DT, 4>(o1, &s1.x);
      pack_pairs<DT, 4>(o2, &s2.x);
      if (on && (n == 0 || second) && FRT_IDX_OK(q0 + n * C + a.L, (int64_t)a.M * a.Hq * C)) {
        a.q_out[q0 + n * C] = s1;
        a.q_out[q0 + n * C + a.L] = s2;
      }
    }
    return;
  }
  float2 lo[4], hi[4];
  unpack_pairs<DT, 4>(&x_lo.x, lo);
  unpack_pairs<DT, 4>(&x_hi.x, hi);

  // y of this lane's two 8-element units
  float y1[8], y2[8];
  if (kind == kK) {
    Split32 r;
    r.hi = 1.0f;
    if (normed) {
      // squared in fp64: bf16 values reach past the square root of fp32's range, both ways
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ss = fma((double)lo[e].x, (double)lo[e].x, ss);
        ss = fma((double)lo[e].y, (double)lo[e].y, ss);
        ss = fma((double)hi[e].x, (double)hi[e].x, ss);
        ss = fma((double)hi[e].y, (double)hi[e].y, ss);
      }
      if (lane % P >= a.L) ss = 0.0;  // (a copy of another lane)
#pragma unroll
      for (int o = P / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      r = Split32(rsqrt_f64(fma(ss, a.inv_hd64, (double)a.eps)));
      float2 wl[4], wh[4];
      unpack_pairs<DT, 4>(&w_lo.x, wl);
      unpack_pairs<DT, 4>(&w_hi.x, wh);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // products of two 16-bit values: exact
        lo[e] = __fmul2_rn(lo[e], wl[e]);
        hi[e] = __fmul2_rn(hi[e], wh[e]);
      }
    }
    const float* fa = &lo[0].x;
    const float* fb = &hi[0].x;
    const float* fc = &cs[0].x;
    const float* fs = &sn[0].x;
    const float* fn = &nsn[0].x;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s, t;
      diff_of_products(fa[e], fc[e], fb[e], fs[e], &s, &t);
      y1[e] = pair_mul(s, t, r);
      diff_of_products(fb[e], fc[e], fa[e], fn[e], &s, &t);
      y2[e] = pair_mul(s, t, r);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y1[2 * e] = lo[e].x;
      y1[2 * e + 1] = lo[e].y;
      y2[2 * e] = hi[e].x;
      y2[2 * e + 1] = hi[e].y;
    }
  }

  // Block c is units 2c and 2c + 1; unit u sits in lane u % L, lower (u < L) or
  // upper half.  With an even L the partner of a unit is in the next lane's
  // same half; with an odd one a block can straddle the halves.
  const float m1 = amax8_or_inf(y1), m2 = amax8_or_inf(y2);
  const int u1 = l, u2 = l + a.L;
  const int pu1 = u1 ^ 1, pu2 = u2 ^ 1;
  const int base = lane - l;
  const int pl1 = base + (pu1 < a.L ? pu1 : pu1 - a.L), pl2 = base + (pu2 < a.L ? pu2 : pu2 - a.L);
  const float f1 = __shfl_sync(0xFFFFFFFFu, m1, pl1 & 31), g1 = __shfl_sync(0xFFFFFFFFu, m2, pl1 & 31);
  const float f2 = __shfl_sync(0xFFFFFFFFu, m1, pl2 & 31), g2 = __shfl_sync(0xFFFFFFFFu, m2, pl2 & 31);
  const float b1 = fmaxf(m1, pu1 < a.L ? f1 : g1), b2 = fmaxf(m2, pu2 < a.L ? f2 : g2);
  const float rden = __frcp_rn(6.0f * gs);
  const float inf = __int_as_float(0x7F800000);
  float r1, r2;
  uint32_t sf1 = nvfp4_scale(b1, rden, gs, &r1), sf2 = nvfp4_scale(b2, rden, gs, &r2);
  uint32_t c1 = nvfp4_codes<8>(y1, r1), c2 = nvfp4_codes<8>(y2, r2);
  if (b1 == inf) sf1 = 0x7F, c1 = 0;
  if (b2 == inf) sf2 = 0x7F, c2 = 0;

  const int t = kind - kK;
  if (!on) return;
  const int64_t row = (int64_t)slot * a.Hkv + h;
  const int64_t quad = ((int64_t)(slot >> 2) * a.Hkv + h) * a.L;
  if (FRT_IDX_OK(row * C + u2, (int64_t)a.capacity * a.Hkv * C)) {
    a.codes[t][row * C + u1] = c1;
    a.codes[t][row * C + u2] = c2;
    const int64_t sf_bytes = (int64_t)((a.capacity + 3) >> 2) * a.Hkv * a.L * 4;
    const int64_t s1 = (quad + (u1 >> 1)) * 4 + (slot & 3), s2 = (quad + (u2 >> 1)) * 4 + (slot & 3);
    if ((u1 & 1) == 0 && FRT_IDX_OK(s1, sf_bytes)) a.sf[t][s1] = (uint8_t)sf1;
    if ((u2 & 1) == 0 && FRT_IDX_OK(s2, sf_bytes)) a.sf[t][s2] = (uint8_t)sf2;
  }
}

template <int DT>
frt_status launch_write(const WriteArgs& a0, cudaStream_t stream) {
  WriteArgs a = a0;
  const int P = a.L > 8 ? 16 : a.L > 4 ? 8 : a.L > 2 ? 4 : a.L;
  const int per = 32 / P;
  a.inv_hd64 = 1.0 / (16 * a.L);
  a.inv_hd = (float)a.inv_hd64;
  a.q_units = (a.Hq + kQHeads - 1) / kQHeads;
  divisor(a.q_units, &a.q_mul, &a.q_shift);
  divisor(a.Hkv, &a.kv_mul, &a.kv_shift);
  if ((int64_t)a.M * (a.Hq > a.Hkv ? a.Hq : a.Hkv) > 0x7FFFFFFF) return FRT_ERR_UNSUPPORTED;
  a.warps_q = ((int64_t)a.M * a.q_units + per - 1) / per;
  a.warps_kv = ((int64_t)a.M * a.Hkv + per - 1) / per;
  const int64_t blocks = (a.warps_q + 2 * a.warps_kv + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return FRT_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(kThreads);
  switch (P) {
    case 1: return launch(write_kernel<DT, 1>, grid, block, 0, stream, a);
    case 2: return launch(write_kernel<DT, 2>, grid, block, 0, stream, a);
    case 4: return launch(write_kernel<DT, 4>, grid, block, 0, stream, a);
    case 8: return launch(write_kernel<DT, 8>, grid, block, 0, stream, a);
    default: return launch(write_kernel<DT, 16>, grid, block, 0, stream, a);
  }
}

// Reader: bound by the 4 B an element pair it writes.  A thread takes kReadUnits
// units of 8 codes (4 bytes to one 16-byte store) of K and of V, their loads
// issued together: 16384 slots of 8 heads of 128 in 17.0 us, 5.05 TB/s (26 us
// with a unit of one tensor to a thread).
constexpr int kReadUnits = 2;
template <int DT>
__global__ void __launch_bounds__(kThreads) read_kernel(const uint32_t* k_codes, const uint8_t* k_sf,
                                                        const uint32_t* v_codes, const uint8_t* v_sf,
                                                        const float* kv_scales, const int32_t* slots, uint4* k_out,
                                                        uint4* v_out, int32_t* status, int n, int Hkv, int L,
                                                        int capacity, uint32_t u_mul, int u_shift) {
  const float gs[2] = {__ldg(kv_scales), __ldg(kv_scales + 1)};
  pdl_enter();
  const int U = 2 * L * Hkv;  // 8-element units of a slot
  const int64_t at0 = (int64_t)blockIdx.x * (kThreads * kReadUnits) + threadIdx.x;
  const int64_t total = (int64_t)n * U;
  int slot[kReadUnits], u[kReadUnits];
#pragma unroll
  for (int j = 0; j < kReadUnits; ++j) {
    const int64_t at = at0 + j * kThreads;
    const int64_t i = total <= 0x7FFFFFFF ? (int64_t)divide((int)at, u_mul, u_shift) : at / U;
    u[j] = (int)(at - i * U);
    slot[j] = -1;
    if (at < total && FRT_IDX_OK(i, n)) {
      slot[j] = slots != nullptr ? __ldg(slots + i) : (int)i;
      if (slot[j] < 0 || slot[j] >= capacity) {
        if (status != nullptr && u[j] == 0) atomicOr(status, 1);
        slot[j] = -1;
      }
    }
  }
  uint32_t w[kReadUnits][2], f[kReadUnits][2];
#pragma unroll
  for (int j = 0; j < kReadUnits; ++j) {
    const int64_t c = (int64_t)slot[j] * U + u[j];
    const int64_t s = ((int64_t)(slot[j] >> 2) * (U >> 1) + (u[j] >> 1)) * 4 + (slot[j] & 3);
    const bool on = slot[j] >= 0 && FRT_IDX_OK(c, (int64_t)capacity * U) &&
                    FRT_IDX_OK(s, (int64_t)((capacity + 3) >> 2) * (U >> 1) * 4);
    w[j][0] = on ? __ldg(k_codes + c) : 0;
    w[j][1] = on ? __ldg(v_codes + c) : 0;
    f[j][0] = on ? __ldg(k_sf + s) : 0;
    f[j][1] = on ? __ldg(v_sf + s) : 0;
  }
#pragma unroll
  for (int j = 0; j < kReadUnits; ++j) {
    const int64_t at = at0 + j * kThreads;
    if (slot[j] < 0 || !FRT_IDX_OK(at, total)) continue;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t sf = e4m3_to_both(f[j][t]);
      uint32_t h[4], o[4];
      e2m1x8_to_half2(w[j][t], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // code * sf is exact in binary16
        const float2 v = __fmul2_rn(Pack16<FRT_F16>::to_float2(hmul2(h[e], sf)), make_float2(gs[t], gs[t]));
        o[e] = Pack16<DT>::from_float2(v.x, v.y);
      }
      (t == 0 ? k_out : v_out)[at] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

constexpr int kMaxHeads = 1 << 20;  // (head indices times hd stay within 32 bits)

bool cache_ok(const void* k_codes, const void* k_sf, const void* v_codes, const void* v_sf, const void* kv_scales) {
  for (const void* p : {k_codes, k_sf, v_codes, v_sf})
    if (p == nullptr || !aligned(p, 16)) return false;
  return kv_scales != nullptr && aligned(kv_scales, 4);
}

}  // namespace
}  // namespace frt

using namespace frt;

extern "C" frt_status frt_qkv_norm_rope_nvfp4_kvcache(const void* qkv, const void* q_norm_w, const void* k_norm_w,
                                                      const float* cos_tab, const float* sin_tab,
                                                      const int32_t* positions, const int32_t* slots, void* q_out,
                                                      uint8_t* k_codes, uint8_t* k_sf, uint8_t* v_codes,
                                                      uint8_t* v_sf, const float* kv_scales, int32_t* status, int M,
                                                      int Hq, int Hkv, int hd, int max_pos, int capacity, float eps,
                                                      frt_dtype dt, cudaStream_t stream) {
  if (M < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || hd <= 0 || hd % 16 != 0 || max_pos <= 0 || capacity <= 0 ||
      !valid_dtype(dt))
    return FRT_ERR_INVALID_ARG;
  if (hd > 256 || Hq > kMaxHeads) return FRT_ERR_UNSUPPORTED;
  if (M == 0) return FRT_OK;
  for (const void* p : {qkv, (const void*)cos_tab, (const void*)sin_tab, (const void*)q_out})
    if (p == nullptr || !aligned(p, 16)) return FRT_ERR_INVALID_ARG;
  for (const void* p : {q_norm_w, k_norm_w})
    if (!aligned(p, 16)) return FRT_ERR_INVALID_ARG;
  if (positions == nullptr || !aligned(positions, 4) || !aligned(slots, 4) || !aligned(status, 4) ||
      !cache_ok(k_codes, k_sf, v_codes, v_sf, kv_scales))
    return FRT_ERR_INVALID_ARG;
  WriteArgs a = {};
  a.qkv = static_cast<const uint4*>(qkv);
  a.q_norm_w = static_cast<const uint4*>(q_norm_w);
  a.k_norm_w = static_cast<const uint4*>(k_norm_w);
  a.cos_tab = reinterpret_cast<const float4*>(cos_tab);
  a.sin_tab = reinterpret_cast<const float4*>(sin_tab);
  a.positions = positions;
  a.slots = slots;
  a.q_out = static_cast<uint4*>(q_out);
  a.codes[0] = reinterpret_cast<uint32_t*>(k_codes);
  a.codes[1] = reinterpret_cast<uint32_t*>(v_codes);
  a.sf[0] = k_sf;
  a.sf[1] = v_sf;
  a.kv_scales = kv_scales;
  a.status = status;
  a.M = M;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.L = hd / 16;
  a.max_pos = max_pos;
  a.capacity = capacity;
  a.eps = eps;
  return dt == FRT_F16 ? launch_write<FRT_F16>(a, stream) : launch_write<FRT_BF16>(a, stream);
}

extern "C" frt_status frt_nvfp4_kvcache_read(const uint8_t* k_codes, const uint8_t* k_sf, const uint8_t* v_codes,
                                             const uint8_t* v_sf, const float* kv_scales, const int32_t* slots,
                                             void* k_out, void* v_out, int32_t* status, int n, int Hkv, int hd,
                                             int capacity, frt_dtype dt, cudaStream_t stream) {
  if (n < 0 || Hkv <= 0 || hd <= 0 || hd % 16 != 0 || capacity <= 0 || !valid_dtype(dt)) return FRT_ERR_INVALID_ARG;
  if (hd > 256 || Hkv > kMaxHeads) return FRT_ERR_UNSUPPORTED;
  if (n == 0) return FRT_OK;
  if (!cache_ok(k_codes, k_sf, v_codes, v_sf, kv_scales) || k_out == nullptr || v_out == nullptr ||
      !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 4) || !aligned(status, 4))
    return FRT_ERR_INVALID_ARG;
  const int64_t blocks = ((int64_t)n * Hkv * (hd / 8) + kThreads * kReadUnits - 1) / (kThreads * kReadUnits);
  if (blocks > 0x7FFFFFFF) return FRT_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(kThreads);
  uint32_t u_mul;
  int u_shift;
  divisor(Hkv * (hd / 8), &u_mul, &u_shift);
  return launch(dt == FRT_F16 ? read_kernel<FRT_F16> : read_kernel<FRT_BF16>, grid, block, 0, stream,
                reinterpret_cast<const uint32_t*>(k_codes), k_sf, reinterpret_cast<const uint32_t*>(v_codes), v_sf,
                kv_scales, slots, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), status, n, Hkv, hd / 16,
                capacity, u_mul, u_shift);
}
