// Softmax attention over an NVFP4 KV cache: one pass over the keys with a
// running maximum and sum, the keys split over warps and CTAs.
//
// What bounds it: a decoding step reads each cached code and factor once
// (1.125 hd bytes a slot and KV head) and does 4 hd operations per query head
// on it.  One token over 131072 slots of 8 heads of 128: 151 MB, 23 us at the
// copy rate; the kernel takes 40 us (3.8 TB/s; 43 with the one that joins its
// parts), of which the loads alone take 31 and the arithmetic alone 35: 650 instructions a tile of 32 slots and head,
// 256 of them the codes' conversion (a cvt and a multiply per two elements),
// 34 products; the integer pipe is at 49 %, issue slots at 55 %, no pipe full.
// Short calls are bound by the chain of dependent loads, about 3 us.
//
// Mapping.  A warp takes tiles of 32 slots of one KV head and computes with
// the keys on the 16-row side of mma.m16n8k16, 8 NT query rows on the other:
//   S^T = K Q^T,  O^T = V^T P^T.
// The order of dimensions inside a product is free, so each lane (g = lane / 4,
// t = lane % 4) loads long runs: of K the slots 4g .. 4g+3 at dimensions
// 16 J t .. 16 J (t+1) - 1 (J = HD / 64), of V the slots 8t .. 8t+7 at
// dimensions 8 J g .. 8 J (g+1) - 1.  One 32-bit word of the cache's factors
// holds a block's factors of four neighbouring slots: those of a lane's K rows,
// and with a second word the pairs (8t + i, 8t + 4 + i) that V needs.  V's
// operand wants two slots in one register: lo = (a & 0x0F..) | (b << 4 &
// 0xF0..) and the same for the high nibbles puts two slots' codes of one
// dimension into a byte before the conversion, half an instruction a
// conversion.  The weights go from S^T's layout (slot by row) to P^T's (slot by
// pairs of rows) with one 8x8 transpose for 8 slots.
//
// Weights: p = 2^(s - m + 11) in fp32, rounded to binary16; m is the row's
// maximum when it was last renewed, which happens when a score passes m by more
// than 4, so 2^11 <= p <= 2^15 for the largest and weights down to 2^-25 of it
// are normal numbers.  The sum is taken of the rounded weights (a row of ones
// beside V).  bf16 queries enter as binary16 times a power of two per row.
#include <algorithm>
#include <cmath>

#include "attn_nvfp4.cuh"

namespace frt {
namespace {

constexpr int kTile = 32;  // slots
using Args = AttnArgs;

__device__ __forceinline__ uint32_t select_bits(uint32_t mask, uint32_t a, uint32_t b) {
  return (a & mask) | (b & ~mask);
}

// Warps of a CTA: eight where registers let two such CTAs share an SM.
__host__ __device__ constexpr int attn_warps(int hd_build, int nt) { return nt == 1 && hd_build == 128 ? 8 : 4; }

// BYTES to shared memory, or zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool on) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(on ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// HD: head dimension of the build (a multiple of 64, at least hd); EXACT: hd ==
// HD; NT: query rows / 8.
//
// A warp's tiles come through its own ring of kStages tiles in shared memory
// (K codes, V codes, their factors), kStages - 1 of them on their way: 9 KB a
// warp at HD 128, what the HBM latency asks for, and none of it in registers
// (loads into registers half a tile ahead left 2.9 of 7 clocks an instruction
// waiting for memory, the ring 0.4).  Measured: 3 CTAs of 8 warps with 2 stages
// 50.8 us for the long call, 5 of 4 warps 45.2, this 43.
// Rows are stored so that the lanes' reads are free of bank conflicts: K's
// slots 4g + i at (i, g), V's 8t + i at (i, t) with the upper 16 slots' 32-byte
// halves swapped.
template <int HD, bool EXACT, int NT>
struct Attn {
  static constexpr int J = HD / 64;
  static constexpr int R = 8 * NT;
  static constexpr int W = attn_warps(HD, NT);
  static constexpr int kThreads = 32 * W;
  static constexpr int kSteps = HD / 16;
  static constexpr int kVs = J == 3 ? 3 : (J + 1) / 2;  // factor words a lane and quad of V
  static constexpr int kStages = HD == 256 ? 2 : 3;
  static constexpr int kRow = HD / 2;          // bytes of a slot's codes
  static constexpr int kSfRow = HD / 4;        // bytes of a quad's factors
  static constexpr int kV = kTile * kRow, kKSf = 2 * kV, kVSf = kKSf + 8 * kSfRow, kStage = kVSf + 8 * kSfRow;
  static constexpr int kMinCtas =
      W == 8 ? 2 : HD / 64 * NT <= 2 ? 4 : HD / 64 * NT <= 4 && HD <= 128 ? 3 : 2;
  static constexpr int kOStride = HD + 4;
  static constexpr size_t kRing = (size_t)W * kStages * kStage;
  static constexpr size_t kMerge = (size_t)W * R * kOStride * 4;
  static constexpr size_t kQ = kRing > kMerge ? kRing : kMerge;  // the merged parts lie over the ring
  static constexpr size_t kSmall = kQ + (size_t)kSteps * NT * 32 * 8;
  static constexpr size_t kSmem = kSmall + R * 4 + 2 * W * R * 4 + R * 8 + 8 * R * 4;

  struct KFrag {
    uint32_t c[4][2 * J];
    uint32_t sf[J];
  };
  struct VFrag {
    uint32_t c[2][4][J];
    uint32_t sf[2][kVs];
  };

  static __device__ __forceinline__ int k_at(int row) { return ((row & 3) * 8 + (row >> 2)) * kRow; }
  static __device__ __forceinline__ int v_at(int row) { return kV + ((row & 7) * 4 + (row >> 3)) * kRow; }
  static __device__ __forceinline__ int v_swap(int row) { return J == 2 ? (row >> 4 & 1) * 32 : 0; }

  // Where a lane copies from: its pieces of the slot of its row within a quad.
  struct Source {
    const uint8_t* k;
    const uint8_t* sf;  // of K for the lanes below kHalf, of V above (HD 256: of K)
    int64_t to_v, to_v_sf;
    int row_bytes, sf_row;
  };
  static constexpr int kPieces = kRow / 16, kSfPieces = kSfRow / 16, kHalf = 8 * kSfPieces;
  static __device__ __forceinline__ Source source(const Args& a, int kvh, int lane) {
    Source s;
    const int nblk = a.hd >> 4;
    s.row_bytes = a.Hkv * (a.hd >> 1);
    s.sf_row = a.Hkv * nblk;
    s.k = a.k_codes + kvh * (a.hd >> 1);
    s.sf = a.k_sf + kvh * nblk * 4;
    s.to_v = a.v_codes - a.k_codes;
    s.to_v_sf = a.v_sf - a.k_sf;
    if (EXACT && 32 % kPieces == 0) {
      s.k += (lane / kPieces & 3) * s.row_bytes + lane % kPieces * 16;
      s.sf += lane % kSfPieces * 16;
      if (lane >= kHalf) s.sf += s.to_v_sf;
    }
    return s;
  }

  // Starts the copies of a tile: `slot` is the first slot of the lane's quad g
  // (-1: not there), `left` the positions from the tile's first to the end.
  static __device__ __forceinline__ void fetch(const Args& a, const Source& src, int kvh, int slot, int left, int lane,
                                               uint32_t to) {
    const int64_t code_bytes = (int64_t)a.capacity * src.row_bytes;
    const int64_t sf_bytes = (int64_t)((a.capacity + 3) >> 2) * src.sf_row * 4;
    // the usual tile: every slot is there, no copy needs a condition
    if (EXACT && 32 % kPieces == 0 && left >= kTile && !__any_sync(0xFFFFFFFFu, slot < 0)) {
      const uint32_t to_k = to + k_at(lane / kPieces) + lane % kPieces * 16;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = 32 / kPieces * i + lane / kPieces;
        const int quad = __shfl_sync(0xFFFFFFFFu, slot, row & ~3);  // lane 4 (row / 4)
        const uint8_t* k = src.k + (int64_t)quad * src.row_bytes;
        const uint8_t* v = k + src.to_v;
        // rows a multiple of 4 on are that many quads on in K's order
        if (32 / kPieces % 4 == 0)
          copy_async<16>(to_k + 32 / kPieces / 4 * i * kRow, k, FRT_SPAN_OK(k - a.k_codes, 16, code_bytes));
        else
          copy_async<16>(to + k_at(row) + lane % kPieces * 16, k, FRT_SPAN_OK(k - a.k_codes, 16, code_bytes));
        copy_async<16>(to + v_at(row) + (lane % kPieces * 16 ^ v_swap(row)), v,
                       FRT_SPAN_OK(v - a.v_codes, 16, code_bytes));
      }
#pragma unroll
      for (int i = 0; i < (2 * kHalf + 31) / 32; ++i) {
        const int q = (32 * i + lane) % kHalf / kSfPieces;
        const int quad = __shfl_sync(0xFFFFFFFFu, slot, 4 * q);
        const uint8_t* f = src.sf + (int64_t)quad * src.sf_row + (i > 0 ? src.to_v_sf : 0);
        const bool v_side = i > 0 || lane >= kHalf;
        if (2 * kHalf % 32 == 0 || lane < 2 * kHalf)
          copy_async<16>(to + (v_side ? kVSf : kKSf) + q * kSfRow + lane % kSfPieces * 16, f,
                         FRT_SPAN_OK(f - (v_side ? a.v_sf : a.k_sf), 16, sf_bytes));
      }
      return;
    }
    const int nblk = a.hd >> 4;
    const int row_bytes = src.row_bytes, sf_row = src.sf_row;
    const uint8_t* k = a.k_codes + kvh * (a.hd >> 1);
    const uint8_t* v = a.v_codes + kvh * (a.hd >> 1);
    const uint8_t* k_sf = a.k_sf + kvh * nblk * 4;
    const uint8_t* v_sf = a.v_sf + kvh * nblk * 4;
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = (32 * i + lane) / kPieces, piece = (32 * i + lane) % kPieces * 16;
        const int quad = __shfl_sync(0xFFFFFFFFu, slot, row & ~3);  // lane 4 (row / 4)
        bool on = quad >= 0 && row < left;
        const int64_t at = (int64_t)(on ? quad + (row & 3) : 0) * row_bytes + piece;
        on = on && FRT_SPAN_OK(k + at - a.k_codes, 16, code_bytes);
        copy_async<16>(to + k_at(row) + piece, k + at, on);
        copy_async<16>(to + v_at(row) + (piece ^ v_swap(row)), v + at, on);
      }
#pragma unroll
      for (int i = 0; i < (2 * kHalf + 31) / 32; ++i) {
        const int id = 32 * i + lane, q = id % kHalf / kSfPieces, piece = id % kSfPieces * 16;
        const int quad = __shfl_sync(0xFFFFFFFFu, slot, 4 * q);
        const uint8_t* from = (id < kHalf ? k_sf : v_sf) + (int64_t)max(quad, 0) * sf_row + piece;
        const bool on = quad >= 0 && FRT_SPAN_OK(from - (id < kHalf ? a.k_sf : a.v_sf), 16, sf_bytes);
        if (2 * kHalf % 32 == 0 || id < 2 * kHalf)
          copy_async<16>(to + (id < kHalf ? kKSf : kVSf) + q * kSfRow + piece, from, on);
      }
    } else {  // rows of any multiple of 8 bytes: a lane a row
      const int quad = __shfl_sync(0xFFFFFFFFu, slot, lane & ~3);
      bool on = quad >= 0 && lane < left;
      const int64_t at = (int64_t)(on ? quad + (lane & 3) : 0) * row_bytes;
      on = on && FRT_SPAN_OK(k + at - a.k_codes, a.hd >> 1, code_bytes);
      for (int c = 0; c < nblk; ++c) {
        copy_async<8>(to + k_at(lane) + 8 * c, k + at + 8 * c, on);
        copy_async<8>(to + v_at(lane) + (8 * c ^ v_swap(lane)), v + at + 8 * c, on);
      }
      for (int c = lane & 3; c < nblk; c += 4) {
        const int64_t s = (int64_t)max(slot, 0) * sf_row + 4 * c;
        const bool there = slot >= 0 && FRT_SPAN_OK(k_sf + s - a.k_sf, 4, sf_bytes);
        copy_async<4>(to + kKSf + (lane >> 2) * kSfRow + 4 * c, k_sf + s, there);
        copy_async<4>(to + kVSf + (lane >> 2) * kSfRow + 4 * c, v_sf + s, there);
      }
    }
  }

  static __device__ __forceinline__ void read_k(const unsigned char* stage, int g, int t, KFrag& f) {
    const unsigned char* p = stage + g * kRow + 8 * J * t;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const unsigned char* q = p + i * 8 * kRow + 8 * j;
        if (J % 2 == 0) {
          if (j % 2 == 0) {
            const uint4 v = *reinterpret_cast<const uint4*>(q);
            f.c[i][2 * j] = v.x;
            f.c[i][2 * j + 1] = v.y;
            f.c[i][(2 * j + 2) % (2 * J)] = v.z;
            f.c[i][(2 * j + 3) % (2 * J)] = v.w;
          }
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(q);
          f.c[i][2 * j] = v.x;
          f.c[i][2 * j + 1] = v.y;
        }
      }
#pragma unroll
    for (int j = 0; j < J; ++j)
      f.sf[j] = *reinterpret_cast<const uint32_t*>(stage + kKSf + g * kSfRow + 4 * (J * t + j));
  }
  static __device__ __forceinline__ void read_v(const unsigned char* stage, int g, int t, VFrag& f) {
    const unsigned char* p = stage + kV + t * kRow + (4 * J * g ^ (J == 2 ? (t >> 1) * 32 : 0));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* q = p + (4 * h + i) * 4 * kRow;
        if (J == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(q);
          f.c[h][i][0] = v.x;
          f.c[h][i][1 % J] = v.y;
          f.c[h][i][2 % J] = v.z;
          f.c[h][i][3 % J] = v.w;
        } else if (J == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(q);
          f.c[h][i][0] = v.x;
          f.c[h][i][1 % J] = v.y;
        } else {
#pragma unroll
          for (int j = 0; j < J; ++j) f.c[h][i][j] = *reinterpret_cast<const uint32_t*>(q + 4 * j);
        }
      }
  }
  static __device__ __forceinline__ void read_v_sf(const unsigned char* stage, int g, int t, VFrag& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kVs; ++j) {
        const int blk = (g * J + (J == 3 ? j : 2 * j)) >> 1;
        f.sf[h][j] = *reinterpret_cast<const uint32_t*>(stage + kVSf + (2 * t + h) * kSfRow + 4 * blk);
      }
  }
};

template <int HD, bool EXACT, int NT>
__global__ void __launch_bounds__(Attn<HD, EXACT, NT>::kThreads, Attn<HD, EXACT, NT>::kMinCtas)
    attn_kernel(const Args a) {
  using A = Attn<HD, EXACT, NT>;
  constexpr int J = A::J, R = A::R, kWarps = A::W, kThreads = A::kThreads, kStages = A::kStages;
  extern __shared__ __align__(16) unsigned char smem[];
  uint2* q_frag = reinterpret_cast<uint2*>(smem + A::kQ);
  float* merge_o = reinterpret_cast<float*>(smem);
  float* q_scale = reinterpret_cast<float*>(smem + A::kSmall);
  float* merge_m = q_scale + R;
  float* merge_l = merge_m + kWarps * R;
  float2* cta_ml = reinterpret_cast<float2*>(merge_l + kWarps * R);
  float* factor = reinterpret_cast<float*>(cta_ml + R);  // [8][R]

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int b = blockIdx.y;
  const Place place = place_of(a);
  const int kvh = place.kvh, rt = place.rt, chunk = place.chunk;

  pdl_enter();
  const Seq seq = sequence(a, b);
  const RowRange rows = row_range<R>(a, seq, rt * R, kvh);
  if (rows.bad && a.status != nullptr) atomicOr(a.status, 1);
  const int tiles = rows.tiles(kTile);
  const int2 part = tiles_of(a, chunk, tiles);
  const int tile0 = part.x, tile1 = part.y;
  if (!rows.any || (!a.cluster && chunk > 0 && tile0 >= tiles)) return;  // no rows, or no work
  const QueryRow mine = query_row(a, seq, rt * R + lane, kvh);  // (lanes below R)

  const float gs_k = __ldg(a.kv_scales), gs_v = __ldg(a.kv_scales + 1);

  // first loads, on their way while the queries are laid out
  unsigned char* ring = smem + warp * kStages * A::kStage;
  const uint32_t ring_at = smem_addr(ring);
  const typename A::Source source = A::source(a, kvh, lane);
  int tile = tile0 + warp;
  auto position = [&](int tl) { return rows.first() + tl * kTile + 4 * g; };
  auto slot_of = [&](int tl) { return tl < tile1 ? quad_slot(a, b, position(tl), rows) : -1; };
  auto fetch = [&](int tl, int slot, int stage) {
    if (tl < tile1)
      A::fetch(a, source, kvh, slot, rows.all_hi - (rows.first() + tl * kTile), lane, ring_at + stage * A::kStage);
    copy_async_commit();
  };
  if (!EXACT) {  // factors of blocks behind hd stay 0
    for (int i = lane; i < kStages * 4 * HD / 4; i += 32) {
      const int stage = i / HD, w = i % HD;
      *reinterpret_cast<uint32_t*>(ring + stage * A::kStage + A::kKSf + 4 * w) = 0;
    }
    __syncwarp();
  }
  int slots[kStages];  // of this tile's quad g and the following tiles'
#pragma unroll
  for (int k = 0; k < kStages; ++k) slots[k] = slot_of(tile + k * kWarps);
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(tile + k * kWarps, slots[k], k);

  // queries: a warp a row, in the order that the lanes read them
  // (a negative scale changes their sign)
  const float q_c = a.scale_log2 * gs_k;
  const uint32_t flip = q_c < 0.0f ? 0x80008000u : 0u;
  constexpr int kEach = R / kWarps;  // (a power of two)
  uint4 raw[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = warp + kWarps * i;
    const int tok = __shfl_sync(0xFFFFFFFFu, mine.tok, r), head = __shfl_sync(0xFFFFFFFFu, mine.head, r);
    const int64_t at = ((int64_t)tok * a.Hq + head) * (a.hd / 8) + lane;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (tok >= 0 && lane < a.hd / 8 && FRT_IDX_OK(at, (int64_t)a.M * a.Hq * (a.hd / 8)))
      raw[i] = ld_plain(static_cast<const uint4*>(a.q) + at);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = warp + kWarps * i;
    float s = 1.0f;
    if (a.dt == FRT_BF16) {
      float2 v[4];
      unpack_pairs<FRT_BF16, 4>(&raw[i].x, v);
      const float amax = fmaxf(absmax4(v[0].x, v[0].y, v[1].x, v[1].y), absmax4(v[2].x, v[2].y, v[3].x, v[3].y));
      s = pow2_to_half_range(warp_max_abs(amax));
      mul_pairs<4>(v, s);
      pack_pairs<FRT_F16, 4>(v, &raw[i].x);
    }
    raw[i] = make_uint4(raw[i].x ^ flip, raw[i].y ^ flip, raw[i].z ^ flip, raw[i].w ^ flip);
    if (lane < HD / 8) {
      const int blk = lane >> 1;
      const int step = (blk % J) * 4 + (lane & 1) * 2;
      uint2* dst = q_frag + ((step * NT + (r >> 3)) * 32 + (r & 7) * 4 + blk / J);
      dst[0] = make_uint2(raw[i].x, raw[i].y);
      dst[NT * 32] = make_uint2(raw[i].z, raw[i].w);
    }
    // (never 0, which would make a masked score NaN)
    if (lane == 0) q_scale[r] = fmaxf(fabsf(q_c) / s, 0x1p-120f);
  }
  __syncthreads();

  const float kInf = __int_as_float(0x7F800000);
  float c[NT][2], m[NT][2], shift[NT][2];
  int lo[NT][2], hi[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      c[n][e] = q_scale[r];
      m[n][e] = -kInf;
      shift[n][e] = 11.0f;
      lo[n][e] = __shfl_sync(0xFFFFFFFFu, mine.lo, r);
      hi[n][e] = __shfl_sync(0xFFFFFFFFu, mine.hi, r);
    }
  float o[NT][HD / 16][4], l[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
    l[n][0] = l[n][1] = l[n][2] = l[n][3] = 0.0f;
  }

  // tiles full0 .. full1 - 1 are seen whole by every row
  const int full0 = (max(rows.full_lo - rows.first(), 0) + kTile - 1) / kTile;
  const int full1 = max(rows.full_hi - rows.first(), 0) / kTile;
  int stage = 0;
  for (; tile < tile1; tile += kWarps) {
    copy_async_wait<kStages - 2>();
    __syncwarp();  // this tile is there for all lanes, and the one before has been read by all
    fetch(tile + (kStages - 1) * kWarps, slots[kStages - 1], stage == 0 ? kStages - 1 : stage - 1);
    const int slot = slots[0];
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) slots[k] = slots[k + 1];
    slots[kStages - 1] = slot_of(tile + kStages * kWarps);
    const unsigned char* here = ring + stage * A::kStage;
    stage = stage == kStages - 1 ? 0 : stage + 1;
    typename A::KFrag kf;
    typename A::VFrag vf;
    A::read_k(here, g, t, kf);
    A::read_v_sf(here, g, t, vf);
    // ---- S^T = K Q^T
    float s[NT][8];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[n][e] = 0.0f;
#pragma unroll
    for (int jb = 0; jb < J; ++jb) {
      uint32_t sc[4];
      const uint32_t sf = kf.sf[jb];
      e4m3x4_to_half2(__byte_perm(sf, 0, 0x1100), sc);
      e4m3x4_to_half2(__byte_perm(sf, 0, 0x3322), sc + 2);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t h[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e2m1x8_to_half2(kf.c[i][2 * jb + w], h[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[i][e] = hmul2(h[i][e], sc[i]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a0[4] = {h[0][2 * j], h[1][2 * j], h[0][2 * j + 1], h[1][2 * j + 1]};
          const uint32_t a1[4] = {h[2][2 * j], h[3][2 * j], h[2][2 * j + 1], h[3][2 * j + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 qb = q_frag[((jb * 4 + w * 2 + j) * NT + n) * 32 + lane];
            mma_16816(s[n], a0, qb.x, qb.y);
            mma_16816(s[n] + 4, a1, qb.x, qb.y);
          }
        }
      }
    }

    // ---- masks.  A NaN factor of V turns the weights of its slot NaN (for
    // the rows that see it) and counts as zero itself, so that it cannot reach
    // other rows.
    uint32_t odd = slot < 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < A::kVs; ++j) odd |= nan_factors(vf.sf[h][j]);
    if (__any_sync(0xFFFFFFFFu, odd != 0) || tile < full0 || tile >= full1) {
      uint32_t nan_slots = 0;  // bit 8t + 4h + i
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t mark = 0;
#pragma unroll
        for (int j = 0; j < A::kVs; ++j) {
          const uint32_t nb = nan_factors(vf.sf[h][j]);
          mark |= nb;
          vf.sf[h][j] &= ~((nb >> 7) * 0xFFu);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((mark >> (8 * i + 7)) & 1) nan_slots |= 1u << (8 * t + 4 * h + i);
      }
      nan_slots = __reduce_or_sync(0xFFFFFFFFu, nan_slots);
      const int pos = position(tile);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if ((nan_slots >> (4 * g + i)) & 1) s[n][2 * i + e] = __int_as_float(0x7FC00000);
            if (slot < 0 || pos + i < lo[n][e] || pos + i >= hi[n][e]) s[n][2 * i + e] = -kInf;
          }
    }

    // ---- running maximum, renewed when a score passes it by more than 4
    bool above = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float top = fmaxf(fmaxf(s[n][e], s[n][2 + e]), fmaxf(s[n][4 + e], s[n][6 + e]));
        above |= fmaf(top, c[n][e], -4.0f) > m[n][e];
      }
    if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(s[n][e], s[n][2 + e]), fmaxf(s[n][4 + e], s[n][6 + e]));
#pragma unroll
          for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          top *= c[n][e];
          if (top > m[n][e]) {
            const float f = ex2_approx(m[n][e] - top);
            m[n][e] = top;
            shift[n][e] = 11.0f - top;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
              o[n][i][e] *= f;
              o[n][i][2 + e] *= f;
            }
            l[n][e] *= f;
            l[n][2 + e] *= f;
          }
        }
    }

    // ---- weights, and their move to P^T's layout
    uint32_t p[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[n][i] = transpose_8x8(
            Pack16<FRT_F16>::from_float2(ex2_approx(fmaf(s[n][2 * i], c[n][0], shift[n][0])),
                                         ex2_approx(fmaf(s[n][2 * i + 1], c[n][1], shift[n][1]))));
      const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
      mma_16816(l[n], ones, p[n][0], p[n][1]);
      mma_16816(l[n], ones, p[n][2], p[n][3]);
    }

    // ---- O^T += V^T P^T
    A::read_v(here, g, t, vf);
    uint32_t sc[4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int js = J == 3 ? j : j / 2;
      if (J == 3 || (j & 1) == 0) {
        e4m3x4_to_half2(__byte_perm(vf.sf[0][js], vf.sf[1][js], 0x5140), sc);
        e4m3x4_to_half2(__byte_perm(vf.sf[0][js], vf.sf[1][js], 0x7362), sc + 2);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // slot pairs 2k, 2k + 1
        uint32_t low[2][4], high[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t va = vf.c[0][2 * k + i][j], vb = vf.c[1][2 * k + i][j];
          e2m1x8_to_half2(select_bits(0x0F0F0F0Fu, va, vb << 4), low[i]);
          e2m1x8_to_half2(select_bits(0x0F0F0F0Fu, va >> 4, vb), high[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            low[i][e] = hmul2(low[i][e], sc[2 * k + i]);
            high[i][e] = hmul2(high[i][e], sc[2 * k + i]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t av[4] = {low[0][e], high[0][e], low[1][e], high[1][e]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816(o[n][4 * j + e], av, p[n][2 * k], p[n][2 * k + 1]);
        }
      }
    }
  }
  copy_async_wait<0>();

  // ---- the warps' parts joined
  if (g == 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) merge_m[warp * R + 8 * n + 2 * t + e] = m[n][e];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      float top = merge_m[r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, merge_m[w * R + r]);
      const float f = m[n][e] == -kInf ? 0.0f : ex2_approx(m[n][e] - top);
      float* row = merge_o + (size_t)(warp * R + r) * A::kOStride + g * 8 * J;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
        *reinterpret_cast<float2*>(row + 2 * i) = make_float2(o[n][i][e] * f, o[n][i][2 + e] * f);
      if (g == 0) merge_l[warp * R + r] = l[n][e] * f;
    }
  __syncthreads();
  const bool whole = !a.cluster && tiles <= a.chunk_tiles;  // this CTA saw all of the keys
  constexpr int kQuads = HD / 4;
  auto out_row = [&](int r) {  // row r of this CTA in out, or -1
    const int rr = rt * R + r, tok = fast_div(rr, a.group_mul, a.group_shift);
    return tok < seq.n ? (int64_t)(seq.t0 + tok) * a.Hq + kvh * a.group + (rr - tok * a.group) : (int64_t)-1;
  };
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    float top = merge_m[r], sum = merge_l[r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      top = fmaxf(top, merge_m[w * R + r]);
      sum += merge_l[w * R + r];
    }
    cta_ml[r] = make_float2(top, sum);
    const int64_t row = out_row(r);
    factor[r] = !whole ? 1.0f : sum == 0.0f ? 0.0f : gs_v / sum;
    if (!a.cluster && row >= 0) {
      if (chunk == 0) store_chunks(a, row, tiles);
      const int64_t at = (int64_t)chunk * a.M * a.Hq + row;
      if (!whole && FRT_IDX_OK(at, (int64_t)a.M * a.Hq * a.chunks)) a.part_ml[at] = make_float2(top, sum);
    }
  }
  if (!a.cluster) __syncthreads();
#pragma unroll 4
  for (int j = 0; j < R * kQuads / kThreads; ++j) {
    const int i = j * kThreads + threadIdx.x, r = i / kQuads, d = i % kQuads * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(merge_o + (w * R + r) * A::kOStride + d);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    if (a.cluster) {  // into the place of the first warp's part, which this thread alone reads
      *reinterpret_cast<float4*>(merge_o + r * A::kOStride + d) = v;
    } else {
      const int64_t row = out_row(r);
      if (row < 0 || d >= a.hd) continue;
      if (whole)
        store_out4(a, row * a.hd + d, v, factor[r]);
      else
        store_part4(a, chunk, row * a.hd + d, v);
    }
  }
  if (!a.cluster) return;
  cluster_sync();
  if (threadIdx.x < R) cluster_factors(a, smem_addr(cta_ml + threadIdx.x), gs_v, factor + threadIdx.x, R);
  __syncthreads();
#pragma unroll 1
  for (int i = chunk * kThreads + threadIdx.x; i < R * kQuads; i += a.chunks * kThreads) {
    const int r = i / kQuads, d = i % kQuads * 4;
    const int64_t row = out_row(r);
    if (row < 0 || d >= a.hd) continue;
    store_out4(a, row * a.hd + d,
               join_cluster4(a, smem_addr(merge_o + r * A::kOStride + d), chunk, factor + r, R), 1.0f);
  }
  cluster_sync();  // the parts are read
}

// The chunks' parts of a query row joined, in a fixed order.  TOGETHER: warps of
// a CTA that share a row (8: one row, many chunks; 1: a row a warp, few).  The
// loads depend on one another as little as can be: the chunk count and the
// chunks' maxima are fetched together.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
template <int TOGETHER>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Args a) {
  __shared__ float4 sums[TOGETHER > 1 ? kJoinWarps : 1][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % TOGETHER;
  const int b = blockIdx.y;
  const int x = blockIdx.x * (kJoinWarps / TOGETHER) + warp / TOGETHER;
  const int kvh = x % a.Hkv, r = x / a.Hkv;
  pdl_enter();
  const Seq seq = sequence(a, b);
  const int i0 = fast_div(r, a.group_mul, a.group_shift);
  if (i0 >= seq.n) return;
  const int64_t n_rows = (int64_t)a.M * a.Hq;
  const int64_t row = (int64_t)(seq.t0 + i0) * a.Hq + kvh * a.group + (r - i0 * a.group);
  const float kInf = __int_as_float(0x7F800000);
  if (!FRT_IDX_OK(row, n_rows)) return;
  const float gs_v = __ldg(a.kv_scales + 1);
  const int n = a.part_n[row];
  float2 ml = make_float2(-kInf, 0.0f);  // of chunk `lane`; entries behind the count mean nothing
  if (lane < a.chunks && FRT_IDX_OK(lane * n_rows + row, n_rows * a.chunks)) ml = a.part_ml[lane * n_rows + row];
  if (n <= 1) return;
  if (lane >= n) ml = make_float2(-kInf, 0.0f);
  float top = ml.x;
  for (int i = 32 + lane; i < n; i += 32)
    if (FRT_IDX_OK(i * n_rows + row, n_rows * a.chunks)) top = fmaxf(top, a.part_ml[i * n_rows + row].x);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  float f = ml.x == -kInf ? 0.0f : ex2_approx(ml.x - top);
  float sum = ml.y * f;
  float4 v[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  for (int base = 0; base < n; base += 32) {
    if (base > 0) {
      ml = make_float2(-kInf, 0.0f);
      if (base + lane < n && FRT_IDX_OK((base + lane) * n_rows + row, n_rows * a.chunks))
        ml = a.part_ml[(base + lane) * n_rows + row];
      f = ml.x == -kInf ? 0.0f : ex2_approx(ml.x - top);
      sum += ml.y * f;
    }
    const int count = min(32, n - base);
#pragma unroll 4
    for (int i = part; i < count; i += TOGETHER) {
      const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
      const int64_t at0 = ((base + i) * n_rows + row) * a.hd;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = 128 * h + 4 * lane;
        if (d >= a.hd || !FRT_SPAN_OK(at0 + d, 4, n_rows * a.chunks * a.hd)) continue;
        const float4 u = *reinterpret_cast<const float4*>(a.part_o + at0 + d);
        v[h].x = fmaf(u.x, fi, v[h].x);
        v[h].y = fmaf(u.y, fi, v[h].y);
        v[h].z = fmaf(u.z, fi, v[h].z);
        v[h].w = fmaf(u.w, fi, v[h].w);
      }
    }
  }
  sum = group_sum<32>(sum);
  if (TOGETHER > 1) {
    sums[warp][lane] = v[0];
    sums[warp][32 + lane] = v[1];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < TOGETHER; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 u = sums[warp + w][32 * h + lane];
        v[h].x += u.x;
        v[h].y += u.y;
        v[h].z += u.z;
        v[h].w += u.w;
      }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (128 * h + 4 * lane < a.hd) store_out4(a, row * a.hd + 128 * h + 4 * lane, v[h], sum == 0.0f ? 0.0f : gs_v / sum);
}

// How a call is cut: the rows of a CTA (8 nt, or the tile kernel's), and the
// keys into chunks.
struct Plan {
  int nt;  // 0: the tile kernel
  int row_tiles, chunks, chunk_tiles, cluster, keys;
};
// What the sizes but max_kv_len say of a kernel (nt as in Plan).
struct Cut {
  int keys;              // positions of a tile
  int64_t row_tiles, ctas;
  int64_t least;         // a CTA's smallest share: a tile for every warp
  int per_sm;            // CTAs
  int64_t at_once;       // on the GPU
  int64_t in_cluster;    // CTAs that a cluster may have without a second wave
  int64_t most;          // chunks of a row tile, where there are more
};
Cut cut_of(int nt, int64_t rows, int n_seqs, int Hkv, int hd) {
  Cut c;
  const int build = hd <= 64 ? 64 : hd <= 128 ? 128 : hd <= 192 ? 192 : 256;
  const int tile_rows = nt == 0 ? kTileRows : 8 * nt;
  c.keys = nt == 0 ? tile_keys(hd) : kTile;
  c.row_tiles = (rows + tile_rows - 1) / tile_rows;
  // (below 2^63 for sizes that the call takes; more than a grid holds is as good as that)
  c.ctas = std::min(c.row_tiles * Hkv * n_seqs, (int64_t)1 << 40);
  c.least = nt == 0 ? 1 : attn_warps(build, nt);
  c.per_sm = nt == 0 ? (hd > 192 ? 1 : 2) : 16 / attn_warps(build, nt);
  c.at_once = (int64_t)kSMs * c.per_sm;
  c.in_cluster = 1;
  while (c.in_cluster < 8 && c.ctas * c.in_cluster * 2 <= c.at_once) c.in_cluster *= 2;
  // sequences whose lengths differ get twice as many CTAs as run at once
  c.most = c.at_once * (n_seqs > 1 ? 2 : 1) / c.ctas;
  return c;
}
int64_t tiles_in(const Cut& c, int64_t max_kv_len) { return max_kv_len > 0 ? (max_kv_len + c.keys - 1) / c.keys : 1; }
// More chunks than a cluster has CTAs cost a second kernel and a way through
// memory, about as long as kJoinRounds tiles of a warp (or CTA) take.  (By sizes
// alone: the caller asks for the workspace before the call, and perhaps without a
// GPU.)
constexpr int64_t kJoinRounds = 8;
// Tiles of a chunk where a second kernel joins them, else 0.
int64_t joined_tiles(const Cut& c, int64_t tiles) {
  if (c.in_cluster == 1) return 0;
  int64_t per = (tiles + c.most - 1) / c.most;
  per = (per + c.least - 1) / c.least * c.least;
  return tiles / (c.in_cluster * c.least) > per / c.least + kJoinRounds ? per : 0;
}
// The most chunks that any call of up to so many tiles is joined from.  (A chunk
// has `least` tiles or more, whole multiples of them, so the count itself falls
// and rises with the length.)
int64_t joined_chunks(const Cut& c, int64_t tiles) {
  if (c.in_cluster == 1 || tiles / (c.in_cluster * c.least) <= 1 + kJoinRounds) return 0;
  return std::min(c.most, (tiles + c.least - 1) / c.least);
}
// The tile kernel takes calls with at least kManyRows rows to a sequence and KV
// head and kManyPairs (row, key) pairs times hd / 128: a call of it costs about
// 10 us and does 1 M such pairs in a microsecond, the kernel for few rows 5 us
// and 0.27 M.
constexpr int64_t kManyRows = 48, kManyPairs = 2500000;
double pairs_a_key(int64_t rows, int n_seqs, int Hkv, int hd) { return (double)rows * Hkv * n_seqs * hd / 128; }
int few_rows_nt(int64_t rows, int n_seqs, int Hkv, int hd) {
  // 32 rows to a CTA only where 16 would fill the GPU already
  const bool small = (double)((rows + 15) / 16) * Hkv * n_seqs * 8 < kSMs * 3;
  return rows <= 8 ? 1 : rows <= 16 || hd > 128 || small ? 2 : 4;
}
Plan make_plan(int n_seqs, int Hq, int Hkv, int hd, int max_q_len, int max_kv_len) {
  Plan p;
  const int64_t rows = (int64_t)max_q_len * (Hq / Hkv);
  const bool many = rows >= kManyRows && pairs_a_key(rows, n_seqs, Hkv, hd) * max_kv_len >= kManyPairs;
  p.nt = many ? 0 : few_rows_nt(rows, n_seqs, Hkv, hd);
  const Cut cut = cut_of(p.nt, rows, n_seqs, Hkv, hd);
  const int64_t tiles = tiles_in(cut, max_kv_len), ctas = cut.ctas, least = cut.least;
  const int per_sm = cut.per_sm;
  p.keys = cut.keys;
  p.row_tiles = (int)(cut.row_tiles > 0x7FFFFFFF ? 0x7FFFFFFF : cut.row_tiles);
  p.cluster = 0;
  p.chunks = 1;
  p.chunk_tiles = (int)tiles;
  if (const int64_t per = joined_tiles(cut, tiles)) {
    p.chunk_tiles = (int)per;
    p.chunks = (int)((tiles + per - 1) / per);
    return p;
  }
  // The keys among the CTAs of a cluster: the cheapest of 1, 2, 4 and 8, in turns
  // of a CTA (a tile for each warp) on a full SM.  A CTA costs about 2.5 besides
  // its turns (measured: 5.5 to 7 us beside turns of 2.4 at hd 128, 4.3 beside 1.6
  // at hd 64), CTAs beyond those that run at once come one wave after the other,
  // a GPU that is not full is up to 0.6 faster, and the last wave ends unevenly.
  // 33 sequences of 1500 keys and 8 heads take 22, 29, 41 and 64 us in 1, 2, 4
  // and 8 parts, 64 of 8000 144, 139, 169 and 228.
  double best = 0;
  for (int c = 1; c <= 8 && (c == 1 || tiles > c / 2 * least); c *= 2) {
    const double waves = (double)ctas / cluster_room(per_sm, c);
    const double turns = (double)((tiles + c * least - 1) / (c * least));
    const double cost = 2.5 * std::max(1.0, waves) + turns * std::max(0.6, waves) + (waves > 1 ? 0.3 * turns : 0.0);
    if (c > 1 && cost >= best) continue;
    best = cost;
    p.chunks = c;
    p.cluster = c > 1;
  }
  return p;
}

// floor(p / d) = (p + umulhi(p, mul)) >> shift with 2^shift >= d, mul = floor(2^32
// (2^shift - d) / d) + 1, for every 0 <= p < 2^31.
void divisor(int d, uint32_t* mul, int* shift) {
  *shift = 0;
  while ((1LL << *shift) < d) ++*shift;
  *mul = (uint32_t)((((1ULL << *shift) - d) << 32) / d + 1);
}

frt_status check_sizes(int M, int n_seqs, int Hq, int Hkv, int hd, int max_q_len, int max_kv_len) {
  if (M < 0 || n_seqs <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || hd <= 0 || hd % 16 != 0 || max_q_len <= 0 ||
      max_kv_len < 0)
    return FRT_ERR_INVALID_ARG;
  return hd > 256 || Hq > 1 << 20 || n_seqs > 65535 || max_kv_len > 0x7FFFFF00 ? FRT_ERR_UNSUPPORTED : FRT_OK;
}

size_t workspace_bytes_of(int M, int Hq, int hd, int64_t chunks) {
  return (size_t)M * Hq * (chunks * (8 + 4 * (size_t)hd) + 4);
}

template <int HD, bool EXACT, int NT>
frt_status launch_attn(const Args& a, cudaStream_t stream) {
  using A = Attn<HD, EXACT, NT>;
  static SmemOptIn opted;
  const frt_status st = opt_in_smem(attn_kernel<HD, EXACT, NT>, A::kSmem, opted);
  if (st != FRT_OK) return st;
  const dim3 grid((unsigned)(a.Hkv * a.row_tiles * a.chunks), a.n_seqs), block(A::kThreads);
  if (a.cluster) return launch_cluster(attn_kernel<HD, EXACT, NT>, grid, block, A::kSmem, stream, a.chunks, a);
  return launch(attn_kernel<HD, EXACT, NT>, grid, block, A::kSmem, stream, a);
}
template <int HD, int NT>
frt_status launch_exact(const Args& a, cudaStream_t stream) {
  return a.hd == HD ? launch_attn<HD, true, NT>(a, stream) : launch_attn<HD, false, NT>(a, stream);
}
template <int NT>
frt_status launch_hd(const Args& a, cudaStream_t stream) {
  if (a.hd <= 64) return launch_exact<64, NT>(a, stream);
  if constexpr (NT <= 2) {
    if (a.hd > 192) return launch_exact<256, NT>(a, stream);
    if (a.hd > 128) return launch_exact<192, NT>(a, stream);
  }
  return launch_exact<128, NT>(a, stream);
}

}  // namespace
}  // namespace frt

using namespace frt;

extern "C" size_t frt_attn_nvfp4_workspace_bytes(int M, int n_seqs, int Hq, int Hkv, int hd, int max_q_len,
                                                 int max_kv_len) {
  if (check_sizes(M, n_seqs, Hq, Hkv, hd, max_q_len, max_kv_len) != FRT_OK) return 0;
  // what the longest call that the kernel for few rows takes may want, and, if
  // some are the tile kernel's, the longest of all
  const int64_t rows = (int64_t)max_q_len * (Hq / Hkv);
  const double pairs = pairs_a_key(rows, n_seqs, Hkv, hd);
  int64_t few_len = max_kv_len, chunks = 0;
  if (rows >= kManyRows && pairs * max_kv_len >= kManyPairs) {
    few_len = std::min(few_len, (int64_t)(kManyPairs / pairs) + 1);
    const Cut cut = cut_of(0, rows, n_seqs, Hkv, hd);
    chunks = joined_chunks(cut, tiles_in(cut, max_kv_len));
  }
  const Cut cut = cut_of(few_rows_nt(rows, n_seqs, Hkv, hd), rows, n_seqs, Hkv, hd);
  chunks = std::max(chunks, joined_chunks(cut, tiles_in(cut, few_len)));
  return chunks == 0 ? 0 : workspace_bytes_of(M, Hq, hd, chunks);
}

extern "C" frt_status frt_attn_nvfp4_kvcache(const void* q, const uint8_t* k_codes, const uint8_t* k_sf,
                                             const uint8_t* v_codes, const uint8_t* v_sf, const float* kv_scales,
                                             const int32_t* kv_len, const int32_t* q_indptr,
                                             const int32_t* page_table, void* out, void* workspace,
                                             size_t workspace_bytes, int32_t* status, int M, int n_seqs, int Hq,
                                             int Hkv, int hd, int capacity, int page_size, int max_pages,
                                             int max_q_len, int max_kv_len, int window, float softmax_scale,
                                             frt_dtype dt, cudaStream_t stream) {
  const frt_status sizes = check_sizes(M, n_seqs, Hq, Hkv, hd, max_q_len, max_kv_len);
  if (sizes == FRT_ERR_INVALID_ARG || capacity <= 0 || !std::isfinite(softmax_scale) || !valid_dtype(dt))
    return FRT_ERR_INVALID_ARG;
  if (page_table != nullptr && (page_size <= 0 || page_size % 4 != 0 || max_pages < 0)) return FRT_ERR_INVALID_ARG;
  if (q_indptr == nullptr && n_seqs != 1) return FRT_ERR_INVALID_ARG;
  if (sizes != FRT_OK) return sizes;
  if (M == 0) return FRT_OK;
  for (const void* p : {q, (const void*)k_codes, (const void*)k_sf, (const void*)v_codes, (const void*)v_sf,
                        (const void*)out})
    if (p == nullptr || !aligned(p, 16)) return FRT_ERR_INVALID_ARG;
  if (kv_scales == nullptr || !aligned(kv_scales, 4) || kv_len == nullptr || !aligned(kv_len, 4) ||
      !aligned(q_indptr, 4) || !aligned(page_table, 4) || !aligned(status, 4))
    return FRT_ERR_INVALID_ARG;
  const Plan p = make_plan(n_seqs, Hq, Hkv, hd, max_q_len, max_kv_len);
  const bool joined = p.chunks > 1 && !p.cluster;  // by a second kernel
  if (joined && (workspace == nullptr || !aligned(workspace, 16) ||
                 workspace_bytes < workspace_bytes_of(M, Hq, hd, p.chunks)))
    return FRT_ERR_INVALID_ARG;
  Args a = {};
  a.q = q;
  a.k_codes = k_codes;
  a.k_sf = k_sf;
  a.v_codes = v_codes;
  a.v_sf = v_sf;
  a.kv_scales = kv_scales;
  a.kv_len = kv_len;
  a.q_indptr = q_indptr;
  a.page_table = page_table;
  a.out = out;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)p.chunks * M * Hq * hd);
  a.part_n = reinterpret_cast<int32_t*>(a.part_ml + (size_t)p.chunks * M * Hq);
  a.status = status;
  a.M = M;
  a.n_seqs = n_seqs;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.hd = hd;
  a.group = Hq / Hkv;
  a.capacity = capacity;
  a.max_q_len = max_q_len;
  a.max_len = max_kv_len < capacity ? max_kv_len : capacity;
  if (page_table != nullptr) {
    const int64_t holds = (int64_t)max_pages * page_size;
    a.max_len = (int)(holds < max_kv_len ? holds : max_kv_len);
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.n_pages = capacity / page_size;
    divisor(page_size, &a.page_mul, &a.page_shift);
  }
  divisor(a.group, &a.group_mul, &a.group_shift);
  a.window = window;
  a.row_tiles = p.row_tiles;
  a.chunks = p.chunks;
  a.chunk_tiles = p.chunk_tiles;
  a.cluster = p.cluster;
  a.scale_log2 = softmax_scale * kLog2e;
  a.dt = dt;
  const int rows = p.nt == 0 ? kTileRows : 8 * p.nt;
  if ((int64_t)Hkv * p.row_tiles * (p.chunks > rows ? p.chunks : rows) > 0x7FFFFFFF) return FRT_ERR_UNSUPPORTED;
  const frt_status st = p.nt == 0   ? launch_attn_tiles(a, stream)
                        : p.nt == 1 ? launch_hd<1>(a, stream)
                        : p.nt == 2 ? launch_hd<2>(a, stream)
                                    : launch_hd<4>(a, stream);
  if (st != FRT_OK || !joined) return st;
  // rows of a sequence and KV head: no more than max_q_len tokens'
  const int64_t warps = (int64_t)max_q_len * a.group * Hkv;
  const bool many = p.chunks > 8;
  const int64_t gx = many ? warps : (warps + kJoinWarps - 1) / kJoinWarps;
  if (gx > 0x7FFFFFFF) return FRT_ERR_UNSUPPORTED;
  return launch(many ? join_kernel<kJoinWarps> : join_kernel<1>, dim3((unsigned)gx, n_seqs), dim3(kJoinThreads), 0,
                stream, a);
}
