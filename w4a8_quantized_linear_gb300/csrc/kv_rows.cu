// kv_rows.cu -- attention over the paged, quantized cache for few query rows
// per key/value head (new tokens x grouped heads <= 32): decoding one token,
// and short chains or trees.
//
// Mathematics, for a row i (one new token and query head) and position j:
//   x_ij = scale log2(e) sk_j (q_i . ck_j) + log2 sv_j,   p'_ij = 2^(x_ij - m_i),
//   o_i  = sum_j p'_ij cv_j / sum_j p'_ij / sv_j,
// the softmax-weighted sum of the values sv_j cv_j with the value's scale moved
// into the exponent.  So the largest p' is near 1 whatever the scales are, and
// p' goes to the tensor core as fp16 against integer codes, which are exact in
// fp16; no scale is ever rounded to 16 bits.  m_i is raised only when some x
// exceeds it by 8 (p' stays below 2^14 with the shift of 6; fp16 goes to 2^16),
// so the outputs are rarely rescaled.  Scales below 2^-90 count as 2^-90: a
// value's error is then at most 127 * 2^-90.  A scale of 0 marks a position
// that is not there (a page out of range is filled with zeros).  A row of zeros
// (scale 1) counts as one of scale 2^-60, so that its weight, which nothing is
// multiplied by, does not set m_i.
//
// q . ck on the fp16 pipe: a code plus 128 (INT4: plus 8), as the bits of an
// fp16 subnormal, is (code + 128) 2^-24 exactly, one mask per two codes; the
// accumulator starts at -128 sum_d q_d 2^-24, which takes the offset out again.
// What is added up is at most 255 sum_d |q_d| (INT4: 15), not bounded by the
// result: for a q of one sign and D = 128 about 50 times the size of a typical
// q . ck.  The error is fp32's rounding of that in D / 16 + 1 steps, at most 2^-23
// each: 5e-5 of a typical score of such a q at worst, more of one that cancels.
// Odd INT4 codes are taken four bits up, 16 times as large, against q / 16.  q is
// first scaled by a power of two so that it fits fp16 (bf16 reaches further).  For
// p' . cv the offset would not stay small (it grows with the sum of the
// weights while the values average out), so the value codes are centred, exactly.
//
// Layout: tokens are the tensor core's M (16), rows its N (8), so few rows
// waste little and each code is converted once for all rows:
//   S^T[16 tokens][8 rows] = K[16][D] Q^T,   O^T[16 dims][8 rows] += V^T P^T.
// The order of dims within both products is free, so each lane takes whole
// 16-byte chunks of a cached row and q is laid out to match.
//
// Bound: HBM (each code is read once) for INT8; for INT4 the issue of the ~265
// instructions per 16 positions, a third of them masks.  Each warp keeps its
// own ring of stages of 16 or 32 positions, filled by 16-byte asynchronous
// copies; there is no barrier in the loop.  The positions of all requests and
// heads form one axis of tiles that is cut evenly over the resident CTAs, on the
// device (only it knows the lengths): a request is cut where the share of a CTA
// ends, its parts are joined by a second small kernel that is launched as a
// programmatic dependent.  The shares depend on the lengths alone, so the same
// inputs give the same bits.
// Measured (32 / 8 heads of 128, one token): 64 requests of 2048 .. 8192
// positions INT8 114 us (0.90 of the copy rate), INT4 81 us (0.66), 16 rows
// (4 tokens) 134 / 124 us, 32 rows 224 / 221 us; one request of 131071 INT8
// 58 us (0.70), INT4 43 us; of 333 10 us.  Three CTAs per SM: four, at 128
// registers, spill (INT4 86 -> 92 us when it was tried).  A warp's outputs are joined through
// shared memory laid out so that a warp touches 64 words in a row; with rows of
// D values there it was 106 us instead of 86.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"
#include "kv_parts.cuh"

namespace cider {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// NB: blocks of 8 rows.
template <int D, int BITS, int NB>
struct RowsCfg {
  static constexpr int kGroups = NB > 2 ? 1 : 2;            // groups of 16 positions per stage
  static constexpr int kSub = 16 * kGroups;                 // positions per stage of a warp
  static constexpr int kTile = kSub * kWarps;               // positions per tile of the axis
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kSide = kSub * kRowBytes;            // codes of K (or V) of a stage
  static constexpr int kStage = 2 * kSide + 2 * kSub * 4;   // and their scales
  static constexpr int kRows = 8 * NB;
  static constexpr int kSteps = D / 16;                     // k-steps of q . ck, m-blocks of V^T
  static constexpr bool kQInRegs = NB == 1;
  static constexpr int kQBytes = kQInRegs ? 0 : NB * kSteps * 32 * 8;
  static constexpr int kOutBytes = kRows * D * 4;
  static constexpr int kStatBytes = kWarps * kRows * 8;
  static constexpr int kMaskBytes = kRows * 8;
  static constexpr int kScaleBytes = kWarps * kSub * 16;
  static constexpr int kRest = kQBytes + kOutBytes + kStatBytes + kMaskBytes + kScaleBytes;
  static constexpr int kCtas = NB == 1 ? 3 : 2;   // per SM
  // as many stages as the resident CTAs' shared memory holds, at most 6
  static constexpr int kFit = (227 * 1024 / kCtas - 1024 - kRest) / (kWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kRing = kStage * kStages;
  static constexpr int kSmem = kWarps * kRing + kRest;
  static_assert(kStages >= 2, "a stage is loaded while another is computed");
};

// d = a b + c, and the same with c = d.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, float c0, float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes from src + SRC to dst + DST; bytes 0: zeros.
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0+%3], [%1+%4], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "n"(DST), "n"(SRC)
               : "memory");
}
// BYTES (4, 8 or 16) of a cached row from shared memory.
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
// Where byte `o` of a stage's keys (values) is put: 16-byte chunks exchanged
// within 128-byte lines so that the fragment loads below touch each bank once.
// For the lanes' fixed pattern of rows and chunks the exchange is one xor that
// is worked out once: every later address is that base plus a constant.
template <int RB>
__device__ __forceinline__ uint32_t swz_k(uint32_t o) {
  if constexpr (RB == 128) return o ^ ((o >> 7 & 1) << 6);
  return o;
}
template <int RB>
__device__ __forceinline__ uint32_t swz_v(uint32_t o) {
  if constexpr (RB == 128) return o ^ ((o >> 8 & 3) << 5);
  if constexpr (RB == 64) return o ^ ((o >> 7 & 3) << 5);
  return o ^ ((o >> 7 & 1) << 5);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) {
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ __half2 bits_h2(uint32_t u) {
  __half2 h;
  memcpy(&h, &u, 4);
  return h;
}

// Centred fp16 pairs (token a, token b), times 2^-9, of the dims in the words
// wa, wb: four INT8 codes or eight INT4 codes each, in order.  A code plus 128
// (plus 8) as an fp16 subnormal is (code + 128) 2^-24; one fp16 FMA lifts it by
// 2^15 and takes 128 2^-9 off, exactly (INT4 codes four bits up: 2^11).  Each
// mask is then a single-constant operation: with the codes put under the
// exponent of 1024 instead, a third of this loop was moves of constants.
// (x & MASK) ^ flip in one operation.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t flip) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "n"(MASK), "r"(flip));
  return r;
}
// A constant that is kept in a register: as a literal, beside the mask's, each
// use of it would be a move and an operation.
__device__ __forceinline__ uint32_t in_register(uint32_t c) {
  asm volatile("" : "+r"(c));
  return c;
}
template <int BITS>
__device__ __forceinline__ void value_pairs(uint32_t wa, uint32_t wb, uint32_t flip_lo, uint32_t flip_hi,
                                            uint32_t* out) {
  const __half2 lift = bits_h2(0x78007800u);      // 2^15
  const __half2 lift_hi = bits_h2(0x68006800u);   // 2^11
  const __half2 off = bits_h2(BITS == 8 ? 0xB400B400u : 0xA400A400u);   // -128 2^-9, -8 2^-9
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t x = __byte_perm(wa, wb, half == 0 ? 0x5410u : 0x7632u);
    const uint32_t y = x >> 8;
    if constexpr (BITS == 8) {
      out[2 * half] = h2_bits(__hfma2(bits_h2(pick<0x00FF00FFu>(x, flip_hi)), lift, off));
      out[2 * half + 1] = h2_bits(__hfma2(bits_h2(pick<0x00FF00FFu>(y, flip_hi)), lift, off));
    } else {
      out[4 * half] = h2_bits(__hfma2(bits_h2(pick<0x000F000Fu>(x, flip_lo)), lift, off));
      out[4 * half + 1] = h2_bits(__hfma2(bits_h2(pick<0x00F000F0u>(x, flip_hi)), lift_hi, off));
      out[4 * half + 2] = h2_bits(__hfma2(bits_h2(pick<0x000F000Fu>(y, flip_lo)), lift, off));
      out[4 * half + 3] = h2_bits(__hfma2(bits_h2(pick<0x00F000F0u>(y, flip_hi)), lift_hi, off));
    }
  }
}

// This lane's D / 4 values of a row of q, in the order of the key fragments:
// INT8 the 16-byte chunks t, t + 4 of the cached row (16 dims each), INT4 a
// quarter of the row.
template <int D, int BITS>
__device__ __forceinline__ void query_load(const uint16_t* q, bool have, int t, uint4 (&w)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 4; i += 8) {
    const int d = BITS == 8 ? (t + 4 * (i / 16)) * 16 + i % 16 : t * (D / 4) + i;
    w[i / 8] = have ? *reinterpret_cast<const uint4*>(q + d) : make_uint4(0, 0, 0, 0);
  }
}
template <int D>
__device__ __forceinline__ void query_values(bool bf16, const uint4 (&w)[D / 32], float (&f)[D / 4]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float e[8];
    if (bf16) widen8<__nv_bfloat16>(w[i], e); else widen8<__half>(w[i], e);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[8 * i + j] = e[j];
  }
}

// Those values times `up` as fp16 pairs per k-step, and the row's sum (over its four lanes).
template <int D, int BITS>
__device__ __forceinline__ float query_frags(const float (&f)[D / 4], float up,
                                             uint32_t (&frag)[D / 16][2]) {
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    __half2 lo, hi;
    if constexpr (BITS == 8) {
      const float* p = f + 4 * s;
      lo = __floats2half2_rn(p[0] * up, p[2] * up);
      hi = __floats2half2_rn(p[1] * up, p[3] * up);
    } else {
      const float* p = f + 8 * (s >> 1) + 2 * (s & 1);
      lo = __floats2half2_rn(p[0] * up, p[4] * up);
      hi = __floats2half2_rn(p[1] * up * 0.0625f, p[5] * up * 0.0625f);
    }
    const float2 x = __half22float2(lo), y = __half22float2(hi);
    sum += (x.x + x.y) + (BITS == 8 ? 1.0f : 16.0f) * (y.x + y.y);
    frag[s][0] = h2_bits(lo);
    frag[s][1] = h2_bits(hi);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  return sum;
}

template <int D, int BITS, int NB>
__global__ void __launch_bounds__(kThreads, RowsCfg<D, BITS, NB>::kCtas)
    rows_kernel(AttendArgs a, PartsArgs parts, bool bf16) {
  using C = RowsCfg<D, BITS, NB>;
  constexpr int RB = C::kRowBytes;
  constexpr int G = C::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t* const ring = smem + warp * C::kRing;
  // copies: chunks lane, lane + 32, ...; 32 chunks further are 4, 8 or 16 rows
  const uint32_t copy_k = smem_u32(ring) + swz_k<RB>(lane * 16);
  const uint32_t copy_v = smem_u32(ring) + C::kSide + swz_v<RB>(lane * 16);
  const uint32_t copy_s = smem_u32(ring) + 2 * C::kSide + (lane >> 2 & 1) * C::kSub * 4 + (lane & 3) * 16;
  const float* const scale_src = (lane < 4 ? a.cache.k_scale : a.cache.v_scale) + (lane & 3) * 4;
  // fragments: keys of row g, chunk t; values of rows 2 t and 2 t + 1, D / 8 dims from D / 8 g
  constexpr int kChunk = RB / 4 < 16 ? RB / 4 : 16;   // bytes of one load of a key
  constexpr int kBytes = RB / 8;                      // of a value row per lane
  const uint32_t frag_k = swz_k<RB>(g * RB + t * kChunk);
  const uint32_t frag_v0 = C::kSide + swz_v<RB>(2 * t * RB + g * kBytes);
  const uint32_t frag_v1 = C::kSide + swz_v<RB>((2 * t + 1) * RB + g * kBytes);
  uint8_t* rest = smem + kWarps * C::kRing;
  float4* scale_smem = reinterpret_cast<float4*>(rest) + warp * C::kSub;
  uint2* q_smem = reinterpret_cast<uint2*>(rest + C::kScaleBytes);
  float* out_smem = reinterpret_cast<float*>(rest + C::kScaleBytes + C::kQBytes);
  float2* stat_smem = reinterpret_cast<float2*>(rest + C::kScaleBytes + C::kQBytes + C::kOutBytes);
  uint64_t* mask_smem = reinterpret_cast<uint64_t*>(rest + C::kScaleBytes + C::kQBytes +
                                                    C::kOutBytes + C::kStatBytes);
  const int group = a.q_heads / a.cache.heads;
  // two's complement to offset codes, of nibbles in place and four bits up (or bytes)
  const uint32_t flip_lo = in_register(0x00080008u), flip_hi = in_register(0x00800080u);

  Axis axis;
  axis.begin(a, C::kTile, lane, C::kRows);
  bool more = axis.more();
  if (threadIdx.x == 0) parts.announce(axis);

  // copies of the piece whose loads are in flight
  int subs = 0;                 // stages of this warp in the piece
  int first_pos = 0;            // position of its first stage; kTile further each
  int last_pos = 0;             // the piece's positions end here
  int rows32 = -1, next32 = -1;   // lane l: the cache row / 16 of 16 positions, -1 without a page
  int load_slot = 0;            // byte offset of the slot that the next copy fills
  const int32_t* table = nullptr;
  const int page16 = a.cache.page_shift - 4;
  // the row of the i-th 16 positions of this warp (G to a stage)
  auto load_rows16 = [&](int i) -> int {
    const int pos = first_pos + (i / G) * C::kTile + (i % G) * 16;
    if (i >= subs * G || pos >= last_pos) return -1;
    const int32_t id = table[pos >> a.cache.page_shift];
    if (id < 0 || id >= a.cache.pages) {
      atomicOr(a.err, kDevErrIndex);
      return -1;
    }
    return ((id * a.cache.heads + axis.unit) << page16) + ((pos >> 4) & ((1 << page16) - 1));
  };
  // a page holds at least 16 positions, and 16 positions of a stage lie in one;
  // row numbers are loaded 32 at a time, 16 copies before their first use
  auto copy = [&](int s) {   // stage s of this warp into the next slot
    if (s < subs) {
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const int i = s * G + u;
        if ((i & 15) == 0 && u == 0) {
          if ((i & 31) == 0 && i > 0) rows32 = next32;
          if ((i & 31) == 16) next32 = load_rows16(i + 16 + lane);
        }
        const int row = __shfl_sync(0xffffffffu, rows32, i & 31);
        const int bytes = row >= 0 ? 16 : 0;
        const int64_t at = max(row, 0);
        const uint8_t* k = a.cache.k + at * (16 * RB) + lane * 16;
        const uint8_t* v = a.cache.v + at * (16 * RB) + lane * 16;
        const uint32_t dk = copy_k + load_slot, dv = copy_v + load_slot;
        if constexpr (RB == 128) {
          cp_async16<0, 0>(dk + u * 2048, k, bytes);
          cp_async16<512, 512>(dk + u * 2048, k, bytes);
          cp_async16<1024, 1024>(dk + u * 2048, k, bytes);
          cp_async16<1536, 1536>(dk + u * 2048, k, bytes);
          // 4 rows further the values' exchange has its upper bit turned round
          cp_async16<0, 0>(dv + u * 2048, v, bytes);
          cp_async16<512, 512>((dv ^ 64) + u * 2048, v, bytes);
          cp_async16<1024, 1024>(dv + u * 2048, v, bytes);
          cp_async16<1536, 1536>((dv ^ 64) + u * 2048, v, bytes);
        } else if constexpr (RB == 64) {
          cp_async16<0, 0>(dk + u * 1024, k, bytes);
          cp_async16<512, 512>(dk + u * 1024, k, bytes);
          cp_async16<0, 0>(dv + u * 1024, v, bytes);
          cp_async16<512, 512>(dv + u * 1024, v, bytes);
        } else {
          cp_async16<0, 0>(dk + u * 512, k, bytes);
          cp_async16<0, 0>(dv + u * 512, v, bytes);
        }
        if (lane < 8) cp_async16<0, 0>(copy_s + load_slot + u * 64, scale_src + at * 16, bytes);
      }
      load_slot = load_slot + C::kStage == C::kRing ? 0 : load_slot + C::kStage;
    }
    cp_async_commit();
  };
  auto q_row = [&](int r, bool have) {
    const int node = have ? r / group : 0;
    return static_cast<const uint16_t*>(a.q) + (axis.req.first + node) * a.q_stride +
           static_cast<int64_t>(axis.unit * group + (have ? r - node * group : 0)) * D;
  };
  uint4 q_raw[NB == 1 ? D / 32 : 1];   // a single block of rows is loaded ahead too
  auto start = [&]() {   // the loads of the axis' current piece
    const int64_t begin = axis.piece_begin * C::kTile + warp * C::kSub;
    const int64_t end = min(axis.piece_end * C::kTile, axis.req.length);
    subs = begin < end ? static_cast<int>((end - begin + C::kTile - 1) / C::kTile) : 0;
    first_pos = static_cast<int>(begin);
    last_pos = static_cast<int>(end);
    table = a.table + axis.b * a.table_width;
    load_slot = 0;
    rows32 = load_rows16(lane);
    if constexpr (NB == 1) query_load<D, BITS>(q_row(g, g < axis.req.nodes * group), g < axis.req.nodes * group, t, q_raw);
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) copy(s);
  };
  if (more) start();

  while (more) {
    // ------------------------------------------------------ the piece's rows
    const Request req = axis.req;
    const int context = static_cast<int>(req.context);
    const int rows = req.nodes * group;
    const int my_subs = subs;
    int pos = first_pos;
    uint32_t qf[C::kQInRegs ? C::kSteps : 1][2];
    float start_s[NB][2];
    if (threadIdx.x < C::kRows) {
      const int node = threadIdx.x / group;
      uint64_t m = 0;
      if (threadIdx.x < rows)
        m = a.tree ? static_cast<uint64_t>(a.tree[req.first + node]) : ~0ull >> (63 - node);
      mask_smem[threadIdx.x] = m;
    }
    // one power of two for all rows puts the largest value in [2^13, 2^14): what
    // a smaller one loses is at most 2^-39 of it, absolutely (half of fp16's
    // smallest step; 2^-35 for q / 16 of INT4's odd codes)
    float top = 0.0f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g;
      uint4 w[D / 32];
      float f[D / 4];
      if constexpr (NB == 1) {
        query_values<D>(bf16, q_raw, f);
      } else {
        query_load<D, BITS>(q_row(r, r < rows), r < rows, t, w);
        query_values<D>(bf16, w, f);
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(f[i]));
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    int lift = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
    lift = top == 0.0f ? 0 : max(-126, min(lift, 126));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + lift) << 23);
    // 2^24 of the subnormals, and the scaling of q, taken out again
    const float mul = a.scale * 1.44269504f * 16777216.0f *
                      __uint_as_float(static_cast<uint32_t>(127 - lift) << 23);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g;
      uint4 w[D / 32];
      float f[D / 4];
      if constexpr (NB == 1) {
        query_values<D>(bf16, q_raw, f);
      } else {
        query_load<D, BITS>(q_row(r, r < rows), r < rows, t, w);
        query_values<D>(bf16, w, f);
      }
      uint32_t frag[C::kSteps][2];
      const float sum = query_frags<D, BITS>(f, up, frag);
      const float off = -(BITS == 8 ? 128.0f : 8.0f) * 0x1p-24f * sum;
#pragma unroll
      for (int e = 0; e < 2; ++e) start_s[nb][e] = __shfl_sync(0xffffffffu, off, (2 * t + e) * 4);
      if constexpr (C::kQInRegs) {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
          qf[s][0] = frag[s][0];
          qf[s][1] = frag[s][1];
        }
      } else if (nb % kWarps == warp) {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s)
          q_smem[(nb * C::kSteps + s) * 32 + lane] = make_uint2(frag[s][0], frag[s][1]);
      }
    }
    __syncthreads();

    float o[NB][C::kSteps][4];
    float l[NB][2], mu[NB][2], limit[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nb][s][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nb][e] = 0.0f;
        mu[nb][e] = 0.0f;
        limit[nb][e] = -INFINITY;
      }
    }

    const uint8_t* st = ring;
    for (int s = 0; s < my_subs; ++s, pos += C::kTile) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      copy(s + C::kStages - 1);
      // each position's scales once: sk, log2 sv, 1 / sv
      if (C::kSub == 32 || lane < C::kSub) {
        const float sk = reinterpret_cast<const float*>(st + 2 * C::kSide)[lane];
        const float sv = reinterpret_cast<const float*>(st + 2 * C::kSide)[C::kSub + lane];
        float kept = sv > 0.0f && sv < 0x1p-90f ? 0x1p-90f : sv;
        if (sv == 1.0f) {   // rarely any other than a row of zeros
          uint32_t any = 0;
#pragma unroll 1
          for (int i = 0; i < RB; i += 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(st + C::kSide + swz_v<RB>(lane * RB + i));
            any |= w.x | w.y | w.z | w.w;
          }
          if (any == 0) kept = kZeroRowScale;
        }
        scale_smem[lane] = make_float4(sk * mul, log2_approx(kept),
                                       kept > 0.0f && kept < INFINITY ? rcp_approx(kept) : 0.0f, 0.0f);
      }
      // -------------------------------------------------- S^T = K Q^T
      float x[NB][G][4];
#pragma unroll
      for (int c = 0; c < RB / 4 / kChunk; ++c) {
        uint32_t w[G][2][kChunk / 4];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            // INT8, D 128: the second 64 bytes of a row are the exchange's own bit
            load_words<kChunk>(st + (c == 0 ? frag_k : frag_k ^ 64) + (u * 16 + 8 * h) * RB, w[u][h]);
#pragma unroll
        for (int i = 0; i < kChunk / 4; ++i) {
          constexpr int kPerWord = BITS == 8 ? 1 : 2;   // k-steps
#pragma unroll
          for (int e = 0; e < kPerWord; ++e) {
            const int step = (c * (kChunk / 4) + i) * kPerWord + e;
            uint32_t f[G][4];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if constexpr (BITS == 8) {
                  const uint32_t v = w[u][h][i] ^ 0x80808080u;
                  f[u][h] = v & 0x00FF00FFu;
                  f[u][h + 2] = __byte_perm(v, 0u, 0x4341u);
                } else {
                  const uint32_t v = e ? w[u][h][i] >> 8 : w[u][h][i];
                  f[u][h] = pick<0x000F000Fu>(v, flip_lo);
                  f[u][h + 2] = pick<0x00F000F0u>(v, flip_hi);
                }
              }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              uint2 b;
              if constexpr (C::kQInRegs)
                b = make_uint2(qf[step][0], qf[step][1]);
              else
                b = q_smem[(nb * C::kSteps + step) * 32 + lane];
#pragma unroll
              for (int u = 0; u < G; ++u) {
                if (step == 0)
                  mma_f16(x[nb][u], f[u], b.x, b.y, start_s[nb][0], start_s[nb][1]);
                else
                  mma_f16(x[nb][u], f[u], b.x, b.y);
              }
            }
          }
        }
      }
      // -------------------------------------------------- scales and masks
      uint32_t v0[4][kBytes / 4];   // the first values, on their way meanwhile
#pragma unroll
      for (int r = 0; r < 4; ++r)
        load_words<kBytes>(st + (r & 1 ? frag_v1 : frag_v0) + 8 * (r >> 1) * RB, v0[r]);
      __syncwarp();
      float inv[G][2];
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = scale_smem[u * 16 + 8 * h + g];
          inv[u][h] = v.z;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              x[nb][u][2 * h + e] = fmaf(x[nb][u][2 * h + e], v.x, v.y);
        }
      if (context - pos < C::kSub) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t m = mask_smem[nb * 8 + 2 * t + e];
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int ahead = pos - context + u * 16 + 8 * h + g;
                const bool seen = ahead < 0 || (ahead < req.nodes && (m >> ahead & 1));
                if (!seen) x[nb][u][2 * h + e] = -INFINITY;
              }
          }
      }
      // -------------------------------------------------- raise the maximum
      bool raise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) raise |= x[nb][u][e] > limit[nb][e & 1];
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float high = fmaxf(x[nb][0][e], x[nb][0][e + 2]);
            if constexpr (G == 2) high = fmaxf(high, fmaxf(x[nb][G - 1][e], x[nb][G - 1][e + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
            if (high > limit[nb][e]) {
              // p' is 2^6 for the largest
              const float now = high - 6.0f;
              const float f = limit[nb][e] == -INFINITY ? 0.0f : exp2_approx(mu[nb][e] - now);
              mu[nb][e] = now;
              limit[nb][e] = high + 8.0f;
              l[nb][e] *= f;
#pragma unroll
              for (int b = 0; b < C::kSteps; ++b) {
                o[nb][b][e] *= f;
                o[nb][b][e + 2] *= f;
              }
            }
          }
      }
      // -------------------------------------------------- P^T
      uint32_t p[NB][G][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < G; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[nb][u][e] = exp2_approx(x[nb][u][e] - mu[nb][e & 1]);
            l[nb][e & 1] = fmaf(x[nb][u][e], inv[u][e >> 1], l[nb][e & 1]);
          }
          p[nb][u][0] = transpose8x8(h2_bits(__floats2half2_rn(x[nb][u][0], x[nb][u][1])));
          p[nb][u][1] = transpose8x8(h2_bits(__floats2half2_rn(x[nb][u][2], x[nb][u][3])));
        }
      // -------------------------------------------------- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < G; ++u) {
        uint32_t w[4][kBytes / 4];
        if (u == 0) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) w[r][i] = v0[r][i];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            load_words<kBytes>(st + (r & 1 ? frag_v1 : frag_v0) + (u * 16 + 8 * (r >> 1)) * RB, w[r]);
        }
        constexpr int kCodes = BITS == 8 ? 4 : 8;   // per word
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
          uint32_t lo[kCodes], hi[kCodes];
          value_pairs<BITS>(w[0][i], w[1][i], flip_lo, flip_hi, lo);
          value_pairs<BITS>(w[2][i], w[3][i], flip_lo, flip_hi, hi);
#pragma unroll
          for (int j = 0; j < kCodes / 2; ++j) {
            const uint32_t f[4] = {lo[2 * j], lo[2 * j + 1], hi[2 * j], hi[2 * j + 1]};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_f16(o[nb][i * (kCodes / 2) + j], f, p[nb][u][0], p[nb][u][1]);
          }
        }
      }
      st = st + C::kStage == ring + C::kRing ? ring : st + C::kStage;
    }

    // the next piece's loads overlap the join of this one
    const bool whole = axis.whole();
    const int slot = axis.slot();
    const int unit = axis.unit;
    __syncwarp();
    more = axis.next(a, C::kTile, C::kRows);
    if (more) start(); else pdl_launch_dependents();

    // -------------------------------------------- join the warps' parts
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
        if (g == 0)
          stat_smem[warp * C::kRows + nb * 8 + 2 * t + e] =
              make_float2(limit[nb][e] == -INFINITY ? -INFINITY : mu[nb][e], l[nb][e]);
      }
    __syncthreads();
    float f[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nb * 8 + 2 * t + e;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat_smem[w * C::kRows + r].x);
        const float mine = stat_smem[warp * C::kRows + r].x;
        f[nb][e] = mine == -INFINITY ? 0.0f : exp2f(mine - top) * 512.0f;   // and the codes' 2^9
      }
    // the warps add their outputs one after another, always in this order; an
    // element lies at [2 b + e / 2][g][row] so that a warp touches 64 words in a row
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int b = 0; b < C::kSteps; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // O^T element: dim (D / 8) g + 2 b + h, rows 2 t and 2 t + 1
              float2* dst = reinterpret_cast<float2*>(out_smem + nb * 8 * D + (2 * b + h) * 64 + g * 8 + 2 * t);
              float2 v = make_float2(o[nb][b][2 * h] * f[nb][0], o[nb][b][2 * h + 1] * f[nb][1]);
              if (w > 0) {
                const float2 old = *dst;
                v.x += old.x;
                v.y += old.y;
              }
              *dst = v;
            }
      }
      __syncthreads();
    }
    // normalised to the output, or as a part
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat_smem[w * C::kRows + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 s = stat_smem[w * C::kRows + r];
        sum += s.x == -INFINITY ? 0.0f : s.y * exp2f(s.x - top);
      }
      const float* src = out_smem + (r >> 3) * 8 * D + d % (D / 8) * 64 + d / (D / 8) * 8 + (r & 7);
      const float4 v = make_float4(src[0], src[64], src[128], src[192]);
      if (whole) {
        const int node = r / group;
        store_out4(a.out, bf16,
                   ((req.first + node) * a.q_heads + unit * group + r - node * group) * D + d, v,
                   sum > 0.0f ? 1.0f / sum : 0.0f);
      } else {
        parts.store(slot, r, D, d, v, top, sum);
      }
    }
    __syncthreads();   // out_smem, stat_smem and mask_smem are written again
  }
}

template <int D, int BITS, int NB>
cudaError_t launch_rows(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  using C = RowsCfg<D, BITS, NB>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(rows_kernel<D, BITS, NB>),
                                          C::kSmem, done);
  if (e != cudaSuccess) return e;
  const int ctas = C::kCtas * num_sms;
  PartsArgs parts;
  ScratchSource scratch = ScratchSource::pooled(st);
  e = parts.allocate(scratch, ctas, C::kRows, D);
  if (e != cudaSuccess) return e;
  rows_kernel<D, BITS, NB><<<ctas, kThreads, C::kSmem, st>>>(a, parts, bf16);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join(a, parts, ctas, std::min(C::kRows, a.max_nodes * (a.q_heads / a.cache.heads)),
                     bf16, st);
}

template <int D, int BITS>
cudaError_t by_rows(const AttendArgs& a, bool bf16, int rows, int num_sms, cudaStream_t st) {
  if (rows <= 8) return launch_rows<D, BITS, 1>(a, bf16, num_sms, st);
  if (rows <= 16) return launch_rows<D, BITS, 2>(a, bf16, num_sms, st);
  if (rows <= 24) return launch_rows<D, BITS, 3>(a, bf16, num_sms, st);
  return launch_rows<D, BITS, 4>(a, bf16, num_sms, st);
}

}  // namespace

cudaError_t launch_attend_rows(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  const int rows = a.max_nodes * (a.q_heads / a.cache.heads);
  if (a.cache.head_dim == 128)
    return a.cache.bits == 8 ? by_rows<128, 8>(a, bf16, rows, num_sms, st)
                             : by_rows<128, 4>(a, bf16, rows, num_sms, st);
  return a.cache.bits == 8 ? by_rows<64, 8>(a, bf16, rows, num_sms, st)
                           : by_rows<64, 4>(a, bf16, rows, num_sms, st);
}

}  // namespace cider
