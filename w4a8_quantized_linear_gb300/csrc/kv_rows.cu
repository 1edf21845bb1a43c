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
// that is not there (a page out of range is filled with zeros).
//
// q . ck on the fp16 pipe: a code plus 128 (INT4: plus 8), as the bits of an
// fp16 subnormal, is (code + 128) 2^-24 exactly, one mask per two codes; the
// accumulator starts at -128 sum_d q_d 2^-24, which takes the offset out again
// (magnitudes stay within 4x of the result's, in fp32).  Odd INT4 codes are
// taken four bits up, 16 times as large, against q / 16.  q is first scaled by
// a power of two per row so that it fits fp16 (bf16 reaches further).  For
// p' . cv the offset would not stay small (it grows with the sum of the
// weights while the values average out), so the value codes are centred: two
// tokens' codes of one dimension are put in the mantissas of 1024 and the
// offset subtracted, exactly.
//
// Layout: tokens are the tensor core's M (16), rows its N (8), so few rows
// waste little and each code is converted once for all rows:
//   S^T[16 tokens][8 rows] = K[16][D] Q^T,   O^T[16 dims][8 rows] += V^T P^T.
// The order of dims within both products is free, so each lane takes whole
// 16-byte chunks of a cached row and q is laid out to match.
//
// Bound: HBM (each code is read once; ~0.75 + 1.5 instructions a code).  Each
// warp keeps its own ring of 16-position stages, filled by 16-byte asynchronous
// copies; there is no barrier in the loop.  The positions of all requests and
// heads form one axis of 64-position tiles that is cut evenly over the resident
// CTAs, on the device (only it knows the lengths): a request is cut where the
// share of a CTA ends, its parts are joined by a second small kernel that is
// launched as a programmatic dependent.  The shares depend on the lengths
// alone, so the same inputs give the same bits.
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
constexpr int kSub = 16;               // positions per stage of a warp
constexpr int kTile = kSub * kWarps;   // positions per tile of the axis

template <int D, int BITS, int NB>
struct RowsCfg {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kSide = kSub * kRowBytes;            // codes of K (or V) of a stage
  static constexpr int kStage = 2 * kSide + 2 * kSub * 4;   // and their scales
  static constexpr int kStages = kRowBytes == 128 ? 4 : kRowBytes == 64 ? 6 : 8;
  static constexpr int kRing = kStage * kStages;
  static constexpr int kRows = 8 * NB;
  static constexpr int kSteps = D / 16;                     // k-steps of q . ck, m-blocks of V^T
  static constexpr int kQBytes = NB > 2 ? NB * kSteps * 32 * 8 : 0;
  static constexpr int kOutBytes = kRows * D * 4;
  static constexpr int kStatBytes = kWarps * kRows * 8;
  static constexpr int kMaskBytes = kRows * 8;
  static constexpr int kSmem = kWarps * kRing + kQBytes + kOutBytes + kStatBytes + kMaskBytes;
  static constexpr int kCtas = NB > 2 ? 2 : 3;              // per SM
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Where byte `o` of a stage's keys (values) is put: 16-byte chunks exchanged
// within 128-byte lines so that the fragment loads below touch each bank once.
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

// Centred fp16 pairs (token a, token b) of the dims in the words wa, wb: four
// INT8 codes or eight INT4 codes each, in order.
template <int BITS>
__device__ __forceinline__ void value_pairs(uint32_t wa, uint32_t wb, uint32_t* out) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t x = __byte_perm(wa, wb, half == 0 ? 0x5410u : 0x7632u);
    if constexpr (BITS == 8) {
      const __half2 bias = bits_h2(0x64806480u);   // 1152
      const uint32_t y = x >> 8;
      out[2 * half] = h2_bits(__hsub2(bits_h2((x & 0x00FF00FFu) ^ 0x64806480u), bias));
      out[2 * half + 1] = h2_bits(__hsub2(bits_h2((y & 0x00FF00FFu) ^ 0x64806480u), bias));
    } else {
      const __half2 bias_lo = bits_h2(0x64086408u);       // 1032
      const __half2 sixteenth = bits_h2(0x2C002C00u);
      const __half2 bias_hi = bits_h2(0xD480D480u);       // -72
      const uint32_t y = x >> 8;
      out[4 * half] = h2_bits(__hsub2(bits_h2((x & 0x000F000Fu) ^ 0x64086408u), bias_lo));
      out[4 * half + 1] = h2_bits(__hfma2(bits_h2((x & 0x00F000F0u) ^ 0x64806480u), sixteenth, bias_hi));
      out[4 * half + 2] = h2_bits(__hsub2(bits_h2((y & 0x000F000Fu) ^ 0x64086408u), bias_lo));
      out[4 * half + 3] = h2_bits(__hfma2(bits_h2((y & 0x00F000F0u) ^ 0x64806480u), sixteenth, bias_hi));
    }
  }
}

// One row of q for this lane: fp16 pairs in the order of the key fragments,
// the sum of all its values (over the row's four lanes) and 2^-k of its scaling.
template <int D, int BITS>
__device__ __forceinline__ void query_row(const AttendArgs& a, bool bf16, const uint16_t* q, bool have,
                                          int t, uint32_t (&frag)[D / 16][2], float& sum, float& unscale) {
  constexpr int kPer = D / 4;   // values per lane
  float f[kPer];
  // a lane's values: INT8 16-byte chunks t, t + 4 of the cached row (16 dims
  // each); INT4 a quarter of the row
#pragma unroll
  for (int i = 0; i < kPer; i += 8) {
    const int d = BITS == 8 ? (t + 4 * (i / 16)) * 16 + i % 16 : t * kPer + i;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (have) w = *reinterpret_cast<const uint4*>(q + d);
    float e[8];
    if (bf16) widen8<__nv_bfloat16>(w, e); else widen8<__half>(w, e);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i + j] = e[j];
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(f[i]));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // the largest value to [2^13, 2^14)
  int k = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
  k = top == 0.0f ? 0 : max(-126, min(k, 126));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  unscale = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  sum = 0.0f;
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
}

template <int D, int BITS, int NB>
__global__ void __launch_bounds__(kThreads, RowsCfg<D, BITS, NB>::kCtas)
    rows_kernel(AttendArgs a, PartsArgs parts, bool bf16) {
  using C = RowsCfg<D, BITS, NB>;
  constexpr int RB = C::kRowBytes;
  constexpr bool kQInRegs = NB <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  uint2* q_smem = reinterpret_cast<uint2*>(smem + kWarps * C::kRing);
  float* out_smem = reinterpret_cast<float*>(smem + kWarps * C::kRing + C::kQBytes);
  float2* stat_smem = reinterpret_cast<float2*>(smem + kWarps * C::kRing + C::kQBytes + C::kOutBytes);
  uint64_t* mask_smem = reinterpret_cast<uint64_t*>(smem + kWarps * C::kRing + C::kQBytes +
                                                    C::kOutBytes + C::kStatBytes);
  const int group = a.q_heads / a.cache.heads;

  Axis axis;
  axis.begin(a, kTile, lane, 1);
  bool more = axis.more();
  if (threadIdx.x == 0) parts.announce(axis);

  // copies of the piece whose loads are in flight
  int subs = 0;               // stages of this warp in the piece
  int32_t ids = -1;           // lane l: the page of stage l, l + 32, ... of this warp
  int ids_base = 0;
  int64_t first_sub = 0;
  const int32_t* table = nullptr;
  int head = 0;
  auto load_ids = [&](int base) {
    ids_base = base;
    const int s = base + lane;
    ids = -1;
    if (s < subs) {
      const int64_t pos = (first_sub + static_cast<int64_t>(s) * kWarps) * kSub;
      const int32_t id = table[pos >> a.cache.page_shift];
      if (id >= 0 && id < a.cache.pages) ids = id; else atomicOr(a.err, kDevErrIndex);
    }
  };
  auto copy = [&](int s) {   // stage s of this warp into its slot
    if (s < subs) {
      if (s >= ids_base + 32) load_ids(ids_base + 32);
      const int32_t id = __shfl_sync(0xffffffffu, ids, s - ids_base);
      const int64_t pos = (first_sub + static_cast<int64_t>(s) * kWarps) * kSub;
      const int64_t row = a.cache.row(id < 0 ? 0 : id, head,
                                      static_cast<int>(pos & ((1 << a.cache.page_shift) - 1)));
      const uint32_t dst = ring + (s % C::kStages) * C::kStage;
      const uint8_t* k = a.cache.k + row * RB;
      const uint8_t* v = a.cache.v + row * RB;
#pragma unroll
      for (int c = lane; c < C::kSide / 16; c += 32) {
        cp_async16(dst + swz_k<RB>(c * 16), k + c * 16, id >= 0);
        cp_async16(dst + C::kSide + swz_v<RB>(c * 16), v + c * 16, id >= 0);
      }
      if (lane < 8) {
        const float* s4 = (lane < 4 ? a.cache.k_scale : a.cache.v_scale) + row + (lane & 3) * 4;
        cp_async16(dst + 2 * C::kSide + lane * 16, s4, id >= 0);
      }
    }
    cp_async_commit();
  };
  auto start = [&]() {   // the loads of the axis' current piece
    const int64_t tiles = axis.piece_end - axis.piece_begin;
    const int64_t length = axis.req.length;
    first_sub = axis.piece_begin * kWarps + warp;
    const int64_t all = (length + kSub - 1) / kSub;
    const int64_t end = min((axis.piece_begin + tiles) * kWarps, all);
    subs = first_sub < end ? static_cast<int>((end - first_sub + kWarps - 1) / kWarps) : 0;
    table = a.table + axis.b * a.table_width;
    head = axis.unit;
    load_ids(0);
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) copy(s);
  };
  if (more) start();

  while (more) {
    // ------------------------------------------------------ the piece's rows
    const Request req = axis.req;
    const int64_t context = req.context, length = req.length;
    const int rows = req.nodes * group;
    const int my_subs = subs;
    const int64_t my_first = first_sub;
    uint32_t qf[kQInRegs ? NB : 1][C::kSteps][2];
    float start_s[NB][2], mul[NB][2];
    if (threadIdx.x < C::kRows) {
      const int node = threadIdx.x / group;
      uint64_t m = 0;
      if (threadIdx.x < rows)
        m = a.tree ? static_cast<uint64_t>(a.tree[req.first + node]) : ~0ull >> (63 - node);
      mask_smem[threadIdx.x] = m;
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + g;
      const bool have = r < rows;
      const int node = have ? r / group : 0;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (req.first + node) * a.q_stride +
                          static_cast<int64_t>(axis.unit * group + (have ? r - node * group : 0)) * D;
      float sum, unscale;
      uint32_t frag[C::kSteps][2];
      query_row<D, BITS>(a, bf16, q, have, t, frag, sum, unscale);
      // 2^24 of the subnormals; 24 - k stays an exponent: k >= -100 but for
      // rows that reach past 2^113, where the product overflows anyway
      const float m = a.scale * 1.44269504f * 16777216.0f * unscale;
      const float off = -(BITS == 8 ? 128.0f : 8.0f) * 0x1p-24f * sum;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mul[nb][e] = __shfl_sync(0xffffffffu, m, (2 * t + e) * 4);
        start_s[nb][e] = __shfl_sync(0xffffffffu, off, (2 * t + e) * 4);
      }
      if constexpr (kQInRegs) {
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
          qf[nb][s][0] = frag[s][0];
          qf[nb][s][1] = frag[s][1];
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

    for (int s = 0; s < my_subs; ++s) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      copy(s + C::kStages - 1);
      const uint32_t st = ring + (s % C::kStages) * C::kStage;
      // -------------------------------------------------- S^T = K Q^T
      float x[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nb][e] = start_s[nb][e & 1];
      constexpr int kChunk = RB / 4 < 16 ? RB / 4 : 16;   // bytes of one load
#pragma unroll
      for (int c = 0; c < RB / 4 / kChunk; ++c) {
        uint32_t wa[4], wb[4];
        const uint32_t oa = g * RB + (t + 4 * c) * kChunk, ob = oa + 8 * RB;
        if constexpr (kChunk == 16) {
          const uint4 u = lds128(st + swz_k<RB>(oa)), v = lds128(st + swz_k<RB>(ob));
          wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
          wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
        } else {
          const uint2 u = lds64(st + oa), v = lds64(st + ob);
          wa[0] = u.x; wa[1] = u.y;
          wb[0] = v.x; wb[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < kChunk / 4; ++i) {
          constexpr int kPerWord = BITS == 8 ? 1 : 2;   // k-steps
#pragma unroll
          for (int e = 0; e < kPerWord; ++e) {
            uint32_t f[4];
            if constexpr (BITS == 8) {
              const uint32_t u = wa[i] ^ 0x80808080u, v = wb[i] ^ 0x80808080u;
              f[0] = u & 0x00FF00FFu;
              f[1] = v & 0x00FF00FFu;
              f[2] = __byte_perm(u, 0u, 0x4341u);
              f[3] = __byte_perm(v, 0u, 0x4341u);
            } else {
              const uint32_t u = e ? wa[i] >> 8 : wa[i], v = e ? wb[i] >> 8 : wb[i];
              f[0] = (u & 0x000F000Fu) ^ 0x00080008u;
              f[1] = (v & 0x000F000Fu) ^ 0x00080008u;
              f[2] = (u & 0x00F000F0u) ^ 0x00800080u;
              f[3] = (v & 0x00F000F0u) ^ 0x00800080u;
            }
            const int step = (c * (kChunk / 4) + i) * kPerWord + e;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if constexpr (kQInRegs) {
                mma_f16(x[nb], f, qf[nb][step][0], qf[nb][step][1]);
              } else {
                const uint2 b = q_smem[(nb * C::kSteps + step) * 32 + lane];
                mma_f16(x[nb], f, b.x, b.y);
              }
            }
          }
        }
      }
      // -------------------------------------------------- scales and masks
      float sk[2], lg[2], inv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sk[e] = __uint_as_float(lds32(st + 2 * C::kSide + (g + 8 * e) * 4));
        const float sv = __uint_as_float(lds32(st + 2 * C::kSide + 64 + (g + 8 * e) * 4));
        const float kept = sv > 0.0f && sv < 0x1p-90f ? 0x1p-90f : sv;
        lg[e] = __log2f(kept);
        inv[e] = kept > 0.0f && kept < INFINITY ? __frcp_rn(kept) : 0.0f;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nb][e] = fmaf(x[nb][e] * mul[nb][e & 1], sk[e >> 1], lg[e >> 1]);
      const int64_t pos = (my_first + static_cast<int64_t>(s) * kWarps) * kSub;
      if (pos + kSub > context) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t ahead = pos + g + 8 * (e >> 1) - context;
            const uint64_t m = mask_smem[nb * 8 + 2 * t + (e & 1)];
            const bool seen = ahead < 0 || (ahead < req.nodes && (m >> ahead & 1));
            if (!seen) x[nb][e] = -INFINITY;
          }
      }
      // -------------------------------------------------- raise the maximum
      bool raise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) raise |= x[nb][e] > limit[nb][e & 1];
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(x[nb][e], x[nb][e + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (top > limit[nb][e]) {
              // p' near 2^6 for the largest
              const float now = top - 6.0f;
              const float f = limit[nb][e] == -INFINITY ? 0.0f : exp2f(mu[nb][e] - now);
              mu[nb][e] = now;
              limit[nb][e] = top + 8.0f;
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
      uint32_t p[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[nb][e] = exp2_approx(x[nb][e] - mu[nb][e & 1]);
          l[nb][e & 1] = fmaf(x[nb][e], inv[e >> 1], l[nb][e & 1]);
        }
        p[nb][0] = transpose8x8(h2_bits(__floats2half2_rn(x[nb][0], x[nb][1])));
        p[nb][1] = transpose8x8(h2_bits(__floats2half2_rn(x[nb][2], x[nb][3])));
      }
      // -------------------------------------------------- O^T += V^T P^T
      constexpr int kBytes = RB / 8;   // of a row per lane
      const uint32_t sv0 = st + C::kSide;
      uint32_t w[4][kBytes / 4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t o0 = (2 * t + (r & 1) + 8 * (r >> 1)) * RB + g * kBytes;
        if constexpr (kBytes == 16) {
          const uint4 u = lds128(sv0 + swz_v<RB>(o0));
          w[r][0] = u.x; w[r][1] = u.y; w[r][2] = u.z; w[r][3] = u.w;
        } else if constexpr (kBytes == 8) {
          const uint2 u = lds64(sv0 + swz_v<RB>(o0));
          w[r][0] = u.x; w[r][1] = u.y;
        } else {
          w[r][0] = lds32(sv0 + swz_v<RB>(o0));
        }
      }
      constexpr int kCodes = BITS == 8 ? 4 : 8;   // per word
#pragma unroll
      for (int i = 0; i < kBytes / 4; ++i) {
        uint32_t lo[kCodes], hi[kCodes];
        value_pairs<BITS>(w[0][i], w[1][i], lo);
        value_pairs<BITS>(w[2][i], w[3][i], hi);
#pragma unroll
        for (int j = 0; j < kCodes / 2; ++j) {
          const uint32_t f[4] = {lo[2 * j], lo[2 * j + 1], hi[2 * j], hi[2 * j + 1]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma_f16(o[nb][i * (kCodes / 2) + j], f, p[nb][0], p[nb][1]);
        }
      }
    }

    // the next piece's loads overlap the join of this one
    const bool whole = axis.whole();
    const int slot = axis.slot();
    const int unit = axis.unit;
    __syncwarp();
    more = axis.next(a, kTile, lane, 1);
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
        f[nb][e] = mine == -INFINITY ? 0.0f : exp2f(mine - top);
      }
    // the warps add their outputs one after another, always in this order
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int b = 0; b < C::kSteps; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // O^T element: dim (D / 8) g + 2 b + e / 2, row 2 t + e % 2
              float* dst = out_smem + (nb * 8 + 2 * t + (e & 1)) * D + g * (D / 8) + 2 * b + (e >> 1);
              const float v = o[nb][b][e] * f[nb][e & 1];
              *dst = w == 0 ? v : *dst + v;
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
      const float4 v = *reinterpret_cast<const float4*>(out_smem + r * D + d);
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
  static_assert(C::kCtas * (C::kSmem + 1024) <= 228 * 1024, "shared memory of the resident CTAs");
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
  return launch_join(a, parts, ctas, std::min(C::kRows, a.max_nodes * (a.q_heads / a.cache.heads)), 1,
                     bf16, st);
}

template <int D, int BITS>
cudaError_t by_rows(const AttendArgs& a, bool bf16, int rows, int num_sms, cudaStream_t st) {
  if (rows <= 8) return launch_rows<D, BITS, 1>(a, bf16, num_sms, st);
  if (rows <= 16) return launch_rows<D, BITS, 2>(a, bf16, num_sms, st);
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
