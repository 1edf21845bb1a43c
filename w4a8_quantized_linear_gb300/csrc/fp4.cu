// fp4.cu -- microscaled 4-bit floating point: quantization of a matrix and back.
//
// A row is cut into blocks of 32 values with an E8M0 scale (a power of two), or
// of 16 values with an E4M3 scale and one fp32 scale (a power of two) for the row:
//   block 32: s = the smallest 2^e with max|x| <= 6 s;  code = E2M1(x / s)
//   block 16: r = the smallest 2^k with max|row| <= 6 * 448 r;
//             b = E4M3(max|x| / r / 6);  code = E2M1(x / r / b), 0 where b is 0
// All roundings are to the nearest, ties to even; quotients are taken in fp32.
// Divisions by powers of two are exact, so block 32 rounds once and block 16
// rounds the scale's quotient, the scale, a value's quotient and the value.
//
// A thread holds 16 values: 8 bytes of codes, one E4M3 scale or (two threads)
// one E8M0 scale.  Memory bounds it: 2 or 4 bytes read and 1/2 + 1/16 written a
// value; each row is read once, the row's maximum is exchanged through shared
// memory while the values stay in registers.
#include <math.h>

#include "fp4_common.cuh"

namespace cider {
namespace {

constexpr int kRowK = 16384;   // longest row whose values stay in registers: 1024 threads x 16

struct QuantArgs {
  const void* x;
  int64_t x_stride;
  int64_t rows;     // of x
  int64_t padded;   // rows whose scales are written: zeros behind the last row of x
  int K, tiles;     // scale tiles along K
  uint8_t* codes;
  uint8_t* scales;
  float* row;
};

// Where the scale of block j of row r lies.
__device__ __forceinline__ int64_t scale_at(int64_t r, int j, int tiles) {
  return ((r >> 7) * tiles + (j >> 2)) * kFpTileBytes + 16 * (r & 31) + 4 * ((r >> 5) & 3) + (j & 3);
}

// Four neighbouring blocks' bytes, one word of a tile: gathered over the lanes that hold them.
template <int BS>
__device__ __forceinline__ void store_scales(const QuantArgs& p, int64_t r, int first, uint32_t byte, int lane) {
  constexpr int kStep = BS / 16;   // lanes of a block
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, byte, (lane & ~(4 * kStep - 1)) + i * kStep) << (8 * i);
  if ((lane & (4 * kStep - 1)) == 0) {
    const int j = first / BS;      // `first`: the lane's first value of the row
    if (r < p.padded && j < 4 * p.tiles) *reinterpret_cast<uint32_t*>(p.scales + scale_at(r, j, p.tiles)) = word;
  }
}

// `warps` warps take a row (K <= 512 warps), blockDim / (32 warps) rows a CTA.
template <typename T, int BS>
__global__ void quantize_fp4_kernel(const QuantArgs p, int warps, bool release) {
  __shared__ float part[32];
  if (release) pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / warps, w = warp - sub * warps;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / (32 * warps)) + sub;
  const int k = (w * 32 + lane) * 16;
  const bool have = r < p.rows && k < p.K;   // K % 32 == 0: a thread's 16 values are all in or all out
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (have) load16(static_cast<const T*>(p.x) + r * p.x_stride + k, v);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max_abs_nan(top, v[i]);
  float inv_row = 1.0f;
  bool bad = false;
  if constexpr (BS == 32) {
    top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  } else {
    float most = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_abs_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (warps > 1) {
      if (lane == 0) part[warp] = most;
      __syncthreads();
      for (int i = 0; i < warps; ++i) most = max_abs_nan(most, part[sub * warps + i]);
    }
    bad = not_finite(most);
    const int e = row_power(most);
    inv_row = pow2(-e);
    if (w == 0 && lane == 0 && r < p.rows) p.row[r] = bad ? __uint_as_float(0x7FC00000u) : pow2(e);
  }
  uint32_t c[2] = {0u, 0u}, byte = 0u;
  if (have && !bad) byte = encode16<BS>(v, top, inv_row, c);
  if (have) *reinterpret_cast<uint2*>(p.codes + r * (p.K >> 1) + (k >> 1)) = make_uint2(c[0], c[1]);
  store_scales<BS>(p, r, k, byte, lane);
}

// Rows of any length: one CTA a row, which is read twice for the row's scale.
template <typename T, int BS>
__global__ void __launch_bounds__(1024) quantize_fp4_long_kernel(const QuantArgs p, bool release) {
  __shared__ float part[32];
  if (release) pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
  const bool row_here = r < p.rows;
  float inv_row = 1.0f;
  bool bad = false;
  if constexpr (BS == 16) {
    float most = 0.0f;
    if (row_here)
      for (int k = threadIdx.x * 16; k < p.K; k += 1024 * 16) {
        float v[16];
        load16(x + k, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) most = max_abs_nan(most, v[i]);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_abs_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) part[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int i = 0; i < 32; ++i) most = max_abs_nan(most, part[i]);
    bad = not_finite(most);
    const int e = row_power(most);
    inv_row = pow2(-e);
    if (threadIdx.x == 0 && row_here) p.row[r] = bad ? __uint_as_float(0x7FC00000u) : pow2(e);
  }
  // whole warps together: the scales' bytes are gathered over the lanes
  const int span = 4 * BS * p.tiles;
  for (int k0 = (threadIdx.x & ~31) * 16; k0 < span; k0 += 1024 * 16) {
    const int k = k0 + lane * 16;
    const bool have = row_here && k < p.K;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (have) load16(x + k, v);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max_abs_nan(top, v[i]);
    if constexpr (BS == 32) top = max_abs_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    uint32_t c[2] = {0u, 0u}, byte = 0u;
    if (have && !bad) byte = encode16<BS>(v, top, inv_row, c);
    if (have) *reinterpret_cast<uint2*>(p.codes + r * (p.K >> 1) + (k >> 1)) = make_uint2(c[0], c[1]);
    store_scales<BS>(p, r, k, byte, lane);
  }
}

template <typename T, int BS>
cudaError_t launch_quantize(const QuantArgs& p, cudaStream_t st, bool release) {
  if (p.K > kRowK) {
    quantize_fp4_long_kernel<T, BS><<<static_cast<unsigned>(p.padded), 1024, 0, st>>>(p, release);
    return cudaGetLastError();
  }
  const int warps = (p.K + 511) / 512;
  const int per = warps >= 8 ? 1 : 8 / warps;
  quantize_fp4_kernel<T, BS><<<static_cast<unsigned>((p.padded + per - 1) / per), 32 * warps * per, 0, st>>>(p, warps, release);
  return cudaGetLastError();
}

template <int BS>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (BS == 32) return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : pow2(static_cast<int>(byte) - 127);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// The value of a code: 0, 1/2, 1, 3/2, 2, 3, 4, 6, twice each in four bits.
__device__ __forceinline__ float e2m1(uint32_t c) {
  const float m = static_cast<float>((0xC8643210u >> (4 * (c & 7u))) & 15u) * 0.5f;
  return c & 8u ? -m : m;
}

template <typename T, int BS>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             const float* row, int64_t rows, int K, int tiles, T* x) {
  const int per_row = K / 16;
  const int64_t n = rows * per_row, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
    const int64_t r = i / per_row;
    const int k = static_cast<int>(i - r * per_row) * 16;
    const uint2 c = *reinterpret_cast<const uint2*>(codes + r * (K >> 1) + (k >> 1));
    const float b = scale_value<BS>(scales[scale_at(r, k / BS, tiles)]);
    const float s = row ? row[r] : 1.0f;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = e2m1(((j < 8 ? c.x : c.y) >> (4 * (j & 7))) & 15u) * b * s;
    T* d = x + r * K + k;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(d)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      constexpr bool kBf = __is_same(T, __nv_bfloat16);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<uint4*>(d)[j] =
            make_uint4(y_bits2<kBf>(v[8 * j], v[8 * j + 1]), y_bits2<kBf>(v[8 * j + 2], v[8 * j + 3]),
                       y_bits2<kBf>(v[8 * j + 4], v[8 * j + 5]), y_bits2<kBf>(v[8 * j + 6], v[8 * j + 7]));
    }
  }
}

template <typename T, int BS>
cudaError_t launch_dequantize(const FpMat& q, int64_t K, T* x, cudaStream_t st) {
  const int64_t n = q.rows * (K / 16);
  const int64_t grid = (n + 255) / 256;
  dequantize_fp4_kernel<T, BS><<<static_cast<unsigned>(grid < 1 << 20 ? grid : 1 << 20), 256, 0, st>>>(
      q.codes, q.scales, q.row, q.rows, static_cast<int>(K), fp4_tiles(K, BS), x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, int dtype, int64_t x_stride, int64_t rows, int64_t K,
                                int block, uint8_t* codes, uint8_t* scales, float* row, bool pad,
                                cudaStream_t st, bool release) {
  const int64_t padded = pad ? (rows + kFpTileRows - 1) / kFpTileRows * kFpTileRows : rows;
  const QuantArgs p{x, x_stride, rows, padded, static_cast<int>(K), fp4_tiles(K, block), codes, scales, row};
  if (block == 16)
    return dtype == CIDER_F16    ? launch_quantize<__half, 16>(p, st, release)
           : dtype == CIDER_BF16 ? launch_quantize<__nv_bfloat16, 16>(p, st, release)
                                 : launch_quantize<float, 16>(p, st, release);
  return dtype == CIDER_F16    ? launch_quantize<__half, 32>(p, st, release)
         : dtype == CIDER_BF16 ? launch_quantize<__nv_bfloat16, 32>(p, st, release)
                               : launch_quantize<float, 32>(p, st, release);
}

cudaError_t launch_dequantize_fp4(const FpMat& q, int64_t K, int block, void* x, int dtype,
                                  cudaStream_t st) {
  if (block == 16)
    return dtype == CIDER_F16    ? launch_dequantize<__half, 16>(q, K, static_cast<__half*>(x), st)
           : dtype == CIDER_BF16 ? launch_dequantize<__nv_bfloat16, 16>(q, K, static_cast<__nv_bfloat16*>(x), st)
                                 : launch_dequantize<float, 16>(q, K, static_cast<float*>(x), st);
  return dtype == CIDER_F16    ? launch_dequantize<__half, 32>(q, K, static_cast<__half*>(x), st)
         : dtype == CIDER_BF16 ? launch_dequantize<__nv_bfloat16, 32>(q, K, static_cast<__nv_bfloat16*>(x), st)
                               : launch_dequantize<float, 32>(q, K, static_cast<float*>(x), st);
}

}  // namespace cider
