// fp4_common.cuh -- what the kernels of microscaled 4-bit floating point share:
// the matrix as the host passes it, the block-scaled tcgen05 product and the
// copies of its scales into tensor memory, the activations.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cider_device.cuh"
#include "cider_internal.h"

namespace cider {

constexpr int kFpTileRows = 128;    // rows of a tile of block scales
constexpr int kFpTileBytes = 512;   // a tile: 128 rows x 4 blocks
constexpr int kFpStageK = 256;      // K of a pipeline stage: rows of 128 bytes, one swizzle span
constexpr int kFpStepK = 64;        // K of one MMA
constexpr int kFpSteps = kFpStageK / kFpStepK;
constexpr uint64_t kFpWaitNs = 2000000000ull;

// Tiles of block scales along K, and those of a stage (BS 16: one a step; 32: one for two steps).
__host__ __device__ constexpr int fp4_tiles(int64_t K, int block) {
  return static_cast<int>((K / block + 3) / 4);
}
template <int BS>
struct FpBlock {
  static constexpr int kTiles = kFpStageK / (4 * BS);         // scale tiles of a stage
  static constexpr int kBytes = kTiles * kFpTileBytes;        // of 128 rows
  static constexpr int kCols = kTiles * 4;                    // tensor-memory columns of 128 rows
};

// One side of a gated product's activation: t(g) of g * sigmoid(t(g)).
enum FpAct : int { kActSilu = 0, kActGelu = 1 };

#ifdef __CUDACC__
// 16 * 8 bytes at a time: the scales of 32 rows x 4 blocks of 4 groups of rows,
// copied to 4 columns of each of the four lane quarters.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 32;   // 8 rows x 16 bytes between groups of 8 rows
  d |= static_cast<uint64_t>(1u) << 46;          // descriptor version for tcgen05; no swizzle
  return d;
}
// The copy and the MMAs that follow it from the same thread run in the order they are issued in.
template <int CG>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands, both K-major, K = 64;
// scales E4M3 (BS 16) or E8M0 (BS 32), of which `id` 0 or 2 names the two bytes of a step.
template <int BS>
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, int id) {
  return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | ((BS == 32 ? 1u : 0u) << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(id) << 29);
}

// D (+)= (A * its scales) (B * its scales)^T, 64 of K.
template <int CG, int BS>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
#define CIDER_FP4_MMA(CGS, VEC)                                                                   \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred p;\n\t"                                                                   \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                \
      "tcgen05.mma.cta_group::" CGS ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                         \
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                            \
      : "memory")
  if constexpr (CG == 1 && BS == 16) CIDER_FP4_MMA("1", "4X");
  if constexpr (CG == 1 && BS == 32) CIDER_FP4_MMA("1", "2X");
  if constexpr (CG == 2 && BS == 16) CIDER_FP4_MMA("2", "4X");
  if constexpr (CG == 2 && BS == 32) CIDER_FP4_MMA("2", "2X");
#undef CIDER_FP4_MMA
}

// act(g) * u with act(g) = g / (1 + e^-t): t = g (SiLU), or t = 2 sqrt(2 / pi) (g + 0.044715 g^3),
// for which g / (1 + e^-t) = g (1 + tanh(t / 2)) / 2 (GELU).  2^x and the reciprocal are the
// hardware's approximations (2 ulp each), far below the 16-bit result's half step, as long as the
// reciprocal is a normal number: below t = -87 act(g), less than 2e-35, counts as zero, whatever u is.
// (Giving e^(t / 2) to each factor there costs five operations an output, 2 us in 34 for 1334 tokens
// through a block of 6144 x 2048; one test for 64 outputs and a second form of them 4 us and more.)
__device__ __forceinline__ float gated(float g, float u, int act) {
  const float t = act == kActSilu ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}
// ------------------------------------------------------------ quantization of 16 values
// Two fp32 numbers, low and high half, and their packed arithmetic (each rounded as alone).
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Sixteen values as they were loaded.
template <typename T>
struct Sixteen {
  static constexpr int kWords = 4 * sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  // FRESH: the launch just before, with whose end this kernel overlaps, may have written them.
  template <bool FRESH = false>
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint32_t* at = reinterpret_cast<const uint32_t*>(p) + 4 * i;
      const uint4 u = FRESH ? ld_global_v4(at) : ld_stream_v4(at);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
  // The largest |x| as the bits of an fp32 number: these are ordered like |x|, infinity and NaN above
  // all numbers.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      if constexpr (__is_same(T, __nv_bfloat16)) return m << 16;
      return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
  }
  // Values 2 i and 2 i + 1 in fp32.
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 4) return pack2(w[2 * i], w[2 * i + 1]);
    if constexpr (__is_same(T, __nv_bfloat16)) return pack2(w[i] << 16, w[i] & 0xFFFF0000u);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    return pack2(__float_as_uint(f.x), __float_as_uint(f.y));
  }
};

// Eight quotients -> their E2M1 codes (nearest, ties to even, at most 6), the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t* q) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .f32 l, h;\n\t"
      "mov.b64 {l, h}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 a, h, l;\n\t"
      "mov.b64 {l, h}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b, h, l;\n\t"
      "mov.b64 {l, h}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, h, l;\n\t"
      "mov.b64 {l, h}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 d, h, l;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "l"(q[0]), "l"(q[1]), "l"(q[2]), "l"(q[3]));
  return r;
}
// The smallest k with a <= m * 2^k for a finite a > 0 given by its bits and m = f 2^w, f given as the
// bits behind its leading one (a subnormal a counts as the least normal number or less).
__device__ __forceinline__ int power_for(uint32_t a, uint32_t f_bits, int w) {
  return static_cast<int>(a >> 23) - 127 - w + ((a & 0x7FFFFFu) > f_bits ? 1 : 0);
}
__device__ __forceinline__ bool not_finite(uint32_t a) { return a >= 0x7F800000u; }
// 2^k, k of -127 .. 127.
__device__ __forceinline__ float pow2(int k) {
  return k == -127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}
// The exponent of a row's scale from the bits of its maximum: at least -126, 0 for zeros.
__device__ __forceinline__ int row_power(uint32_t a) {
  return a == 0u ? 0 : max(power_for(a, 0x280000u, 11), -126);   // 2688 = 1.3125 * 2^11
}
// The row's scale: NaN where a value is not finite.
__device__ __forceinline__ float row_scale(uint32_t a) {
  return not_finite(a) ? __uint_as_float(0x7FC00000u) : pow2(row_power(a));
}

// The exponent of the scale of 32 values, from the bits of their finite maximum.
__device__ __forceinline__ int block_power(uint32_t top) {
  return top != 0u ? max(power_for(top, 0x400000u, 2), -127) : 0;   // 6 = 1.5 * 2^2
}
// Where the scale of block j of row r lies.
__device__ __forceinline__ int64_t scale_at(int64_t r, int j, int tiles) {
  return ((r >> 7) * tiles + (j >> 2)) * kFpTileBytes + 16 * (r & 31) + 4 * ((r >> 5) & 3) + (j & 3);
}

// 16 values, their block's maximum (block 32: of both halves) and the inverse of the row's scale (a
// power of two; 1 for block 32) -> two words of codes, the scale byte.
// Quotients are correctly rounded: by a power of two exact, by b a product with the reciprocal and
// Markstein's correction (as in div_rn_by).
template <typename T, int BS>
__device__ __forceinline__ uint32_t encode16(const Sixteen<T>& v, uint32_t top, float inv_row, uint32_t (&c)[2]) {
  uint64_t q[8];
  c[0] = c[1] = 0u;
  if constexpr (BS == 32) {
    if (not_finite(top)) return 0xFFu;
    const int e = block_power(top);
    const uint64_t inv = both(pow2(-e));
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = mul2(v.pair(i), inv);
    c[0] = e2m1x8(q);
    c[1] = e2m1x8(q + 4);
    return static_cast<uint32_t>(e + 127);
  } else {
    // a quotient so small that the correction underflows is a scale of 0 either way
    const float t = div_rn_by(__uint_as_float(top) * inv_row, 6.0f, 1.0f / 6.0f);
    const uint32_t byte = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    if (byte == 0u) return 0u;
    const float b = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
    const float r = __frcp_rn(b);
    // the quotients' negatives: so a zero keeps its sign through the correction
    if (inv_row > 0x1p-100f && inv_row < 0x1p100f) {
      // the row's scale goes into b and its reciprocal: the same quotients in one step less
      const uint64_t bb = both(b * __uint_as_float(0x7F000000u - __float_as_uint(inv_row))), rr = both(-r * inv_row);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t x = v.pair(i), q0 = mul2(x, rr);
        q[i] = fma2(fma2(q0, bb, x), rr, q0);
      }
    } else {
      const uint64_t inv = both(inv_row), bb = both(b), rr = both(-r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t x = mul2(v.pair(i), inv), q0 = mul2(x, rr);
        q[i] = fma2(fma2(q0, bb, x), rr, q0);
      }
    }
    c[0] = e2m1x8(q) ^ 0x88888888u;
    c[1] = e2m1x8(q + 4) ^ 0x88888888u;
    return byte;
  }
}
#endif

// A quantized matrix, as the host passes it on.
struct FpMat {
  const uint8_t* codes = nullptr;
  const uint8_t* scales = nullptr;
  const float* row = nullptr;
  int64_t rows = 0;
};

// fp4.cu.  x of dtype (cider_dtype_t), x_stride elements between rows.  pad: the scales of the rows
// behind the last one in its tile are written too, as zeros (a product does not need them: they
// reach only outputs that it does not store).  release: as in quant.cu.
cudaError_t launch_quantize_fp4(const void* x, int dtype, int64_t x_stride, int64_t rows, int64_t K,
                                int block, uint8_t* codes, uint8_t* scales, float* row, bool pad,
                                int num_sms, cudaStream_t st, bool release);
cudaError_t launch_dequantize_fp4(const FpMat& q, int64_t K, int block, void* x, int dtype,
                                  int num_sms, cudaStream_t st);

// One product: y = x w^T, or with `up` h = act(x w^T) (x up^T).
struct FpProduct {
  FpMat x, w, up;
  const void* wide_x = nullptr;   // x in 16 bits, for the kernel that quantizes it itself
  int64_t x_stride = 0;
  bool x_bf16 = false;
  int64_t M = 0, N = 0, K = 0;
  int block = 0;
  bool is_gated = false;
  int act = kActSilu;
  void* y = nullptr;
  bool y_bf16 = false;
  // gated, block 32, N % 32 == 0: the rounded outputs are quantized again, to here in place of y
  uint8_t *q_codes = nullptr, *q_scales = nullptr;
  bool after_launch = false;   // the launch just before is this call's own: overlap with its end
  int num_sms = 0;
  cudaStream_t st = nullptr;
};
// fp4_rows.cu: 128 rows of weights against up to 128 tokens, K split over a cluster.
cudaError_t launch_fp4_rows(const FpProduct& p);
// Whether it can quantize x itself (wide_x): few tokens, a part of K that fits beside the weights.
bool fp4_rows_quantizes_itself(const FpProduct& p);
// fp4_pair.cu: 256 tokens x 256 weight rows on a CTA pair.
cudaError_t launch_fp4_pair(const FpProduct& p);

}  // namespace cider
