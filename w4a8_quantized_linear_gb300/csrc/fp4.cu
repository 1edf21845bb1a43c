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
// A thread holds one unit of 16 values, or two: 8 bytes of codes, one E4M3 scale or (two threads)
// one E8M0 scale.  Memory bounds it: 2 or 4 bytes read and 1/2 + 1/16 written a
// value; each row is read once, the row's maximum is exchanged through shared
// memory while the values stay in registers.
#include <math.h>

#include "fp4_common.cuh"

namespace cider {
namespace {

constexpr int kRowK = 32768;   // longest row whose values stay in registers: 1024 threads x 32
// Threads an SM that quantize_fp4_kernel is compiled and launched for (48 or 40 registers a thread; 64 for two units).
template <int BS, int U>
constexpr int kResident = U == 2 ? 1024 : BS == 16 ? 1280 : 1536;

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

// Four neighbouring blocks' bytes, one word of a tile: gathered over the lanes that hold them.  `at`: the
// row's place in its first tile, or null; `first`: the lane's first value of the row.
template <int BS>
__device__ __forceinline__ void store_scales(uint8_t* at, int tiles, int first, uint32_t byte, int lane) {
  constexpr int kStep = BS / 16;   // lanes of a block
  uint32_t word = byte << (8 * (lane / kStep & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, kStep);
  word |= __shfl_xor_sync(0xffffffffu, word, 2 * kStep);
  const int tile = first / (4 * BS);
  if (at && (lane & (4 * kStep - 1)) == 0 && tile < tiles) *reinterpret_cast<uint32_t*>(at + tile * kFpTileBytes) = word;
}
__device__ __forceinline__ uint8_t* scale_row(const QuantArgs& p, int64_t r) {
  return r < p.padded ? p.scales + scale_at(r, 0, p.tiles) : nullptr;
}

// `warps` warps take a row (K <= 512 U warps), blockDim / (32 warps) rows a CTA at a time.  (The next
// rows' values asked for before these are encoded: 8.3 us for 7.4, in registers that other CTAs use better.)
template <typename T, int BS, int U>
__global__ void __launch_bounds__(U == 1 ? 256 : 1024, U == 1 ? kResident<BS, U> / 256 : 1)
quantize_fp4_kernel(const QuantArgs p, int warps, bool release) {
  __shared__ uint32_t part[2][32];
  if (release) pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / warps, w = warp - sub * warps;
  const int per = blockDim.x / (32 * warps);
  const int k = (w * 32 + lane) * 16, across = warps * 512;   // a thread's 16 values: k + u across
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t r = static_cast<int64_t>(blockIdx.x) * per + sub;
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride + k;
  const int64_t x_step = step * p.x_stride;
  uint8_t* codes = p.codes + r * (p.K >> 1) + (k >> 1);
  const int64_t codes_step = step * (p.K >> 1);
  // every thread of the CTA makes the same turns
  for (int64_t turn = static_cast<int64_t>(blockIdx.x) * per, n = 0; turn < p.padded; turn += step, r += step, ++n) {
    bool have[U];
    Sixteen<T> v[U];
    uint32_t top[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      have[u] = k + u * across < p.K && r < p.rows;   // K % 32 == 0: 16 values are all in or all out
      if (have[u])
        v[u].load(x + u * across);
      else
        v[u].clear();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = v[u].top();
    x += x_step;
    float inv_row = 1.0f;
    bool bad = false;
    if constexpr (BS == 32) {
#pragma unroll
      for (int u = 0; u < U; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
    } else {
      uint32_t most = top[0];
#pragma unroll
      for (int u = 1; u < U; ++u) most = max(most, top[u]);
      most = __reduce_max_sync(0xffffffffu, most);
      if (warps > 1) {
        if (lane == 0) part[n & 1][warp] = most;
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, lane < warps ? part[n & 1][sub * warps + lane] : 0u);
      }
      bad = not_finite(most);
      inv_row = pow2(-row_power(most));
      if (w == 0 && lane == 0 && r < p.rows) p.row[r] = row_scale(most);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t c[2] = {0u, 0u}, byte = 0u;
      if (have[u] && !bad) byte = encode16<T, BS>(v[u], top[u], inv_row, c);
      if (have[u]) *reinterpret_cast<uint2*>(codes + u * (across >> 1)) = make_uint2(c[0], c[1]);
      store_scales<BS>(scale_row(p, r), p.tiles, k + u * across, byte, lane);
    }
    codes += codes_step;
  }
}

// Rows of any length: one CTA a row, which is read twice for the row's scale.
template <typename T, int BS>
__global__ void __launch_bounds__(1024) quantize_fp4_long_kernel(const QuantArgs p, bool release) {
  __shared__ uint32_t part[32];
  if (release) pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
  const bool row_here = r < p.rows;
  float inv_row = 1.0f;
  bool bad = false;
  if constexpr (BS == 16) {
    uint32_t most = 0u;
    if (row_here)
      for (int k = threadIdx.x * 16; k < p.K; k += 1024 * 16) {
        Sixteen<T> v;
        v.load(x + k);
        most = max(most, v.top());
      }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) part[threadIdx.x >> 5] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, part[lane]);
    bad = not_finite(most);
    inv_row = pow2(-row_power(most));
    if (threadIdx.x == 0 && row_here) p.row[r] = row_scale(most);
  }
  // whole warps together: the scales' bytes are gathered over the lanes
  const int span = 4 * BS * p.tiles;
  for (int k0 = (threadIdx.x & ~31) * 16; k0 < span; k0 += 1024 * 16) {
    const int k = k0 + lane * 16;
    const bool have = row_here && k < p.K;
    Sixteen<T> v;
    v.clear();
    if (have) v.load(x + k);
    uint32_t top = v.top();
    if constexpr (BS == 32) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    uint32_t c[2] = {0u, 0u}, byte = 0u;
    if (have && !bad) byte = encode16<T, BS>(v, top, inv_row, c);
    if (have) *reinterpret_cast<uint2*>(p.codes + r * (p.K >> 1) + (k >> 1)) = make_uint2(c[0], c[1]);
    store_scales<BS>(scale_row(p, r), p.tiles, k, byte, lane);
  }
}

template <typename T, int BS, int U>
cudaError_t launch_rows(const QuantArgs& p, int num_sms, cudaStream_t st, bool release) {
  const int warps = (p.K + 512 * U - 1) / (512 * U);
  const int per = warps >= 8 ? 1 : 8 / warps, threads = 32 * warps * per;
  // As many CTAs as run at once.  4096 x 4096 bf16, block 32: 7.8 us, a CTA a row 10.1; 10240 x 2560 fp32 19.4, 27.0;
  // equal rows in fewer CTAs 8.7 and 20.9.
  const int64_t groups = (p.padded + per - 1) / per, most = static_cast<int64_t>(num_sms) * (kResident<BS, U> / threads);
  quantize_fp4_kernel<T, BS, U><<<static_cast<unsigned>(groups < most ? groups : most), threads, 0, st>>>(p, warps, release);
  return cudaGetLastError();
}

template <typename T, int BS>
cudaError_t launch_quantize(const QuantArgs& p, int num_sms, cudaStream_t st, bool release) {
  if (p.K > kRowK) {
    quantize_fp4_long_kernel<T, BS><<<static_cast<unsigned>(p.padded), 1024, 0, st>>>(p, release);
    return cudaGetLastError();
  }
  // Long rows: two units a thread keep two CTAs or more on an SM, and half as many warps meet for a row's maximum.
  // bf16, block 16, one unit against two: 4096 x 4096 11.1 us, 10.0; 8192 x 12288 94, 57 (block 32: 48, 38); but fp16
  // 4096 x 2560 7.6, 8.1.  Few rows, fp16, block 16: 64 x 4096 2.0, 2.2 (from 150 rows on no worse), 64 x 8192 2.4, 2.3,
  // 64 x 12288 2.9, 2.7; block 32 1.7, 1.8 and 2.05, 1.9 and 2.4, 2.1.
  return p.K >= 4096 ? launch_rows<T, BS, 2>(p, num_sms, st, release) : launch_rows<T, BS, 1>(p, num_sms, st, release);
}

template <int BS>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (BS == 32) return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : pow2(static_cast<int>(byte) - 127);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// Two codes of a byte -> their values in fp32.
__device__ __forceinline__ float2 e2m1_pair(uint32_t word, int byte) {
  uint32_t h;
  switch (byte) {   // unrolled: one instruction each
    case 0: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(word)); break;
    case 1: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(word)); break;
    case 2: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h) : "r"(word)); break;
    default: asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(h) : "r"(word)); break;
  }
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A thread reads 8 bytes of codes and writes 16 values, 32 bytes at a time; rows by the CTA's second index.
// (Eight values a thread for fp32, so that a warp's store covers whole lines: 22.2 us for 10240 x 2560, not 20.1.)
template <typename T, int BS>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                             const float* row, int64_t rows, int K, int tiles,
                                                             bool wide, T* x) {
  const int per_row = K >> 4;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; r < rows;
       r += static_cast<int64_t>(gridDim.x) * blockDim.y) {
    const float s = row ? __ldg(row + r) : 1.0f;
    for (int i = threadIdx.x; i < per_row; i += blockDim.x) {
      const int k = i * 16;
      const uint2 c = *reinterpret_cast<const uint2*>(codes + r * (K >> 1) + (k >> 1));
      const float b = scale_value<BS>(scales[scale_at(r, k / BS, tiles)]);
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = e2m1_pair(j < 4 ? c.x : c.y, j & 3);
        v[2 * j] = f.x * b * s;
        v[2 * j + 1] = f.y * b * s;
      }
      constexpr int kWords = 4 * sizeof(T);
      uint32_t o[kWords];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = y_bits2<__is_same(T, __nv_bfloat16)>(v[2 * j], v[2 * j + 1]);
      }
      uint32_t* d = reinterpret_cast<uint32_t*>(x + r * K + k);
      if (wide) {   // 32-byte boundaries: whole sectors
#pragma unroll
        for (int j = 0; j < kWords / 8; ++j) st_global_v8(d + 8 * j, o + 8 * j);
      } else {
#pragma unroll
        for (int j = 0; j < kWords / 4; ++j)
          reinterpret_cast<uint4*>(d)[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      }
    }
  }
}

template <typename T, int BS>
cudaError_t launch_dequantize(const FpMat& q, int64_t K, T* x, int num_sms, cudaStream_t st) {
  // threads along a row, 16 values each: equal turns of whole warps, or a power of two that covers it
  const unsigned units = static_cast<unsigned>(K / 16), turns = (units + 255) / 256;
  unsigned tx = 1;
  while (tx < 32 && tx < units) tx *= 2;
  if (units > 32) tx = ((units + turns - 1) / turns + 31) / 32 * 32;
  const dim3 block(tx, 256 / tx);
  const int64_t groups = (q.rows + block.y - 1) / block.y, most = static_cast<int64_t>(num_sms) * 16;
  dequantize_fp4_kernel<T, BS><<<static_cast<unsigned>(groups < most ? groups : most), block, 0, st>>>(
      q.codes, q.scales, q.row, q.rows, static_cast<int>(K), fp4_tiles(K, BS),
      reinterpret_cast<uintptr_t>(x) % 32 == 0, x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, int dtype, int64_t x_stride, int64_t rows, int64_t K,
                                int block, uint8_t* codes, uint8_t* scales, float* row, bool pad,
                                int num_sms, cudaStream_t st, bool release) {
  const int64_t padded = pad ? (rows + kFpTileRows - 1) / kFpTileRows * kFpTileRows : rows;
  const QuantArgs p{x, x_stride, rows, padded, static_cast<int>(K), fp4_tiles(K, block), codes, scales, row};
  if (block == 16)
    return dtype == CIDER_F16    ? launch_quantize<__half, 16>(p, num_sms, st, release)
           : dtype == CIDER_BF16 ? launch_quantize<__nv_bfloat16, 16>(p, num_sms, st, release)
                                 : launch_quantize<float, 16>(p, num_sms, st, release);
  return dtype == CIDER_F16    ? launch_quantize<__half, 32>(p, num_sms, st, release)
         : dtype == CIDER_BF16 ? launch_quantize<__nv_bfloat16, 32>(p, num_sms, st, release)
                               : launch_quantize<float, 32>(p, num_sms, st, release);
}

cudaError_t launch_dequantize_fp4(const FpMat& q, int64_t K, int block, void* x, int dtype,
                                  int num_sms, cudaStream_t st) {
  if (block == 16)
    return dtype == CIDER_F16    ? launch_dequantize<__half, 16>(q, K, static_cast<__half*>(x), num_sms, st)
           : dtype == CIDER_BF16 ? launch_dequantize<__nv_bfloat16, 16>(q, K, static_cast<__nv_bfloat16*>(x), num_sms, st)
                                 : launch_dequantize<float, 16>(q, K, static_cast<float*>(x), num_sms, st);
  return dtype == CIDER_F16    ? launch_dequantize<__half, 32>(q, K, static_cast<__half*>(x), num_sms, st)
         : dtype == CIDER_BF16 ? launch_dequantize<__nv_bfloat16, 32>(q, K, static_cast<__nv_bfloat16*>(x), num_sms, st)
                               : launch_dequantize<float, 32>(q, K, static_cast<float*>(x), num_sms, st);
}

}  // namespace cider
