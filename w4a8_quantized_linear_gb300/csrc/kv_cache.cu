// kv_cache.cu -- the paged, quantized key/value cache: rows are quantized as
// they are written, read back as fp16 / bf16, and moved up behind the context
// after a tree of drafted tokens was verified.
//
// Mathematics, per token and key/value head (a row x of D values):
//   amax = max |x|,  s = RN32(amax / q) with q = 127 (INT8) or 7 (INT4),
//   s = 1 for a zero row,  code = rint(RN32(x / s)), ties to even;
// the value a row stands for is code * s.  Rounding RN32(x / s) is monotonic
// and |x| <= amax, so |code| <= q without a clamp for finite rows (s rounded
// down by at most 2^-10 of itself, for bf16 subnormals, still gives at most
// 127.13 and 7.01); the division path clamps all the same.
//
// What bounds these kernels is HBM traffic: every input byte is read once and
// every output byte written once, eight values (16 bytes of fp16 / bf16) per
// thread and access, key and value side by side so that each thread has two
// independent loads in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"

namespace cider {
namespace {

constexpr int kRowThreads = 256;

// ------------------------------------------------------------------ append
// Eight values of a row -> their codes as bytes (INT8: 8 bytes) or packed
// nibbles (INT4: 4 bytes in lo).  FAST: r = RN(1/s) and Markstein's corrected
// quotient; it needs s normal and far from the ends of the exponent range.
template <int BITS, bool FAST>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float r) {
  constexpr float kTop = BITS == 8 ? 127.0f : 7.0f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q;
    if constexpr (FAST) {
      q = div_rn_by(f[i], s, r);
    } else {
      q = fminf(fmaxf(__fdiv_rn(f[i], s), -kTop), kTop);
    }
    // 1.5 * 2^23 puts the nearest whole number (ties to even) in the low
    // mantissa bits, in two's complement
    c[i] = __float_as_uint(__fadd_rn(q, 12582912.0f));
  }
  if constexpr (BITS == 8) {
    const uint32_t a = __byte_perm(c[0], c[1], 0x0040u), b = __byte_perm(c[2], c[3], 0x0040u);
    const uint32_t d = __byte_perm(c[4], c[5], 0x0040u), e = __byte_perm(c[6], c[7], 0x0040u);
    return make_uint2(__byte_perm(a, b, 0x5410u), __byte_perm(d, e, 0x5410u));
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (c[i] & 0xFu) << (4 * i);
    return make_uint2(w, 0u);
  }
}

template <typename T, int D, int BITS>
__device__ __forceinline__ void append_row(const uint4& in, uint8_t* codes, float* scale, int lane,
                                           bool write) {
  constexpr int kLanes = D / 8;
  float f[8];
  widen8<T>(in, f);
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  constexpr float kTop = BITS == 8 ? 127.0f : 7.0f;
  const float s = a > 0.0f ? __fdiv_rn(a, kTop) : 1.0f;
  // fp16 scales are always in this range; bf16 ones reach 2^-140
  const bool fast = s > 1e-30f && s < 1e30f;
  const uint2 c = fast ? encode8<BITS, true>(f, s, __frcp_rn(s)) : encode8<BITS, false>(f, s, 0.0f);
  if (!write) return;
  if constexpr (BITS == 8)
    *reinterpret_cast<uint2*>(codes + lane * 8) = c;
  else
    *reinterpret_cast<uint32_t*>(codes + lane * 4) = c.x;
  if (lane == 0) *scale = s;
}

// D / 8 neighbouring threads hold one (token, head) row of K and of V.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kRowThreads)
    kv_append_kernel(KvCache cache, const T* __restrict__ k, int64_t k_stride,
                     const T* __restrict__ v, int64_t v_stride, const int64_t* __restrict__ slots,
                     uint32_t rows, int* err) {
  constexpr int kLanes = D / 8;
  const uint32_t row = (blockIdx.x * kRowThreads + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  const bool have = row < rows;
  const uint32_t token = have ? row / static_cast<uint32_t>(cache.heads) : 0;
  const uint32_t head = have ? row - token * cache.heads : 0;
  uint4 kin = make_uint4(0, 0, 0, 0), vin = make_uint4(0, 0, 0, 0);
  int64_t slot = -1;
  if (have) {
    kin = ld_stream_v4(k + static_cast<int64_t>(token) * k_stride + head * D + lane * 8);
    vin = ld_stream_v4(v + static_cast<int64_t>(token) * v_stride + head * D + lane * 8);
    slot = slots[token];
  }
  const bool inside = slot >= 0 && slot < cache.pages << cache.page_shift;
  if (slot >= 0 && !inside && lane == 0) atomicOr(err, kDevErrIndex);
  const int64_t at =
      inside ? cache.row(slot >> cache.page_shift, head,
                         static_cast<int>(slot & ((1 << cache.page_shift) - 1)))
             : 0;
  constexpr int kRowBytes = D * BITS / 8;
  append_row<T, D, BITS>(kin, cache.k + at * kRowBytes, cache.k_scale + at, lane, inside);
  append_row<T, D, BITS>(vin, cache.v + at * kRowBytes, cache.v_scale + at, lane, inside);
}

// -------------------------------------------------------------------- read
template <typename T, int BITS>
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
  uint4 out;
  uint32_t* o = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int lo, hi;
    if constexpr (BITS == 8) {
      const uint32_t w = j < 2 ? c.x : c.y;
      lo = static_cast<int8_t>(w >> (16 * (j & 1)));
      hi = static_cast<int8_t>(w >> (16 * (j & 1) + 8));
    } else {
      lo = static_cast<int>(c.x << (28 - 8 * j)) >> 28;
      hi = static_cast<int>(c.x << (24 - 8 * j)) >> 28;
    }
    // the value is the fp32 product, rounded once to the output type
    o[j] = y_bits2<std::is_same<T, __nv_bfloat16>::value>(__fmul_rn(static_cast<float>(lo), s),
                                                         __fmul_rn(static_cast<float>(hi), s));
  }
  return out;
}

// A CTA reads `tile` tokens (at most 32) of one layer, all heads.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kRowThreads)
    kv_read_kernel(KvCache cache, const int32_t* __restrict__ table, int64_t table_width,
                   const int32_t* __restrict__ starts, const int32_t* __restrict__ offsets,
                   int requests, int64_t tokens, int tile, T* __restrict__ k, T* __restrict__ v,
                   int* err) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRowThreads / kLanes;
  constexpr int kRowBytes = D * BITS / 8;
  __shared__ int64_t place[32];   // row of the cache for head 0, or -1
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile;
  const int here = static_cast<int>(min(static_cast<int64_t>(tile), tokens - t0));
  if (threadIdx.x < here) {
    const int64_t i = t0 + threadIdx.x;
    const int b = find_request(offsets, requests, i);
    int64_t at = -1;
    if (b >= 0) {
      const int64_t pos = static_cast<int64_t>(starts[b]) + i - offsets[b];
      const int64_t slot_page = pos >> cache.page_shift;
      int64_t page = -1;
      if (pos >= 0 && slot_page < table_width) page = table[b * table_width + slot_page];
      if (page >= 0 && page < cache.pages)
        at = cache.row(page, 0, static_cast<int>(pos & ((1 << cache.page_shift) - 1)));
    }
    if (at < 0) atomicOr(err, kDevErrIndex);
    place[threadIdx.x] = at;
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  const int64_t layer_rows = cache.layer_rows();
  const uint8_t* ck = cache.k + blockIdx.y * layer_rows * kRowBytes;
  const uint8_t* cv = cache.v + blockIdx.y * layer_rows * kRowBytes;
  const float* sk = cache.k_scale + blockIdx.y * layer_rows;
  const float* sv = cache.v_scale + blockIdx.y * layer_rows;
  const int64_t out0 = (static_cast<int64_t>(blockIdx.y) * tokens + t0) * cache.heads;
  const int rows = here * cache.heads;
#pragma unroll 2
  for (int r = threadIdx.x / kLanes; r < rows; r += kGroups) {
    const int token = r / cache.heads, head = r - token * cache.heads;
    const int64_t at = place[token];
    uint4 ok = make_uint4(0, 0, 0, 0), ov = ok;
    if (at >= 0) {
      const int64_t row = at + (static_cast<int64_t>(head) << cache.page_shift);
      uint2 a, b;
      if constexpr (BITS == 8) {
        a = *reinterpret_cast<const uint2*>(ck + row * kRowBytes + lane * 8);
        b = *reinterpret_cast<const uint2*>(cv + row * kRowBytes + lane * 8);
      } else {
        a = make_uint2(*reinterpret_cast<const uint32_t*>(ck + row * kRowBytes + lane * 4), 0u);
        b = make_uint2(*reinterpret_cast<const uint32_t*>(cv + row * kRowBytes + lane * 4), 0u);
      }
      ok = decode8<T, BITS>(a, sk[row]);
      ov = decode8<T, BITS>(b, sv[row]);
    }
    const int64_t o = (out0 + r) * D + lane * 8;
    *reinterpret_cast<uint4*>(k + o) = ok;
    *reinterpret_cast<uint4*>(v + o) = ov;
  }
}

// ----------------------------------------------------------------- compact
// One CTA per (layer, request, head): row start + path[i] moves to start + i.
// Every row is read before any is written, so a path may overlap its target.
constexpr int kCompactThreads = 128;

__global__ void __launch_bounds__(kCompactThreads)
    kv_compact_kernel(KvCache cache, int row_bytes, const int32_t* __restrict__ table,
                      int64_t table_width, const int32_t* __restrict__ starts,
                      const int32_t* __restrict__ path, int path_width,
                      const int32_t* __restrict__ kept, int* err) {
  __shared__ int64_t from[kMaxNodes], to[kMaxNodes];   // cache rows of this head, -1: nothing moves
  const int b = blockIdx.x, head = blockIdx.y;
  const int64_t layer = blockIdx.z;
  const int n = kept[b];
  if (n <= 0) return;
  const bool bad_count = n > path_width;
  const int count = bad_count ? 0 : n;
  if (bad_count && threadIdx.x == 0) atomicOr(err, kDevErrIndex);
  if (threadIdx.x < count) {
    const int i = threadIdx.x;
    const int src = path[static_cast<int64_t>(b) * path_width + i];
    const int64_t f = src < 0 ? -1 : static_cast<int64_t>(starts[b]) + src;
    const int64_t t = static_cast<int64_t>(starts[b]) + i;
    const int64_t rf = cache_row_of(cache, table, table_width, b, f, head);
    const int64_t rt = cache_row_of(cache, table, table_width, b, t, head);
    const bool ok = rf >= 0 && rt >= 0;
    if (!ok) atomicOr(err, kDevErrIndex);
    const bool moves = ok && rf != rt;
    from[i] = moves ? rf + layer * cache.layer_rows() : -1;
    to[i] = moves ? rt + layer * cache.layer_rows() : -1;
  }
  __syncthreads();
  // 64 rows x 128 bytes x (K, V) = 16 KiB at most: 8 chunks of 16 bytes a thread
  const int chunks = row_bytes / 16;
  constexpr int kMost = 2 * kMaxNodes * 8 / kCompactThreads;
  uint4 hold[kMost];
  float hs = 0.0f;
  const int total = 2 * count * chunks;
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int c = j * kCompactThreads + threadIdx.x;
    if (c < total) {
      const int i = c / (2 * chunks), rest = c % (2 * chunks);
      if (from[i] >= 0) {
        const uint8_t* base = rest < chunks ? cache.k : cache.v;
        hold[j] = *reinterpret_cast<const uint4*>(base + from[i] * row_bytes + (rest % chunks) * 16);
      }
    }
  }
  if (threadIdx.x < 2 * count && from[threadIdx.x >> 1] >= 0)
    hs = (threadIdx.x & 1 ? cache.v_scale : cache.k_scale)[from[threadIdx.x >> 1]];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    const int c = j * kCompactThreads + threadIdx.x;
    if (c < total) {
      const int i = c / (2 * chunks), rest = c % (2 * chunks);
      if (to[i] >= 0) {
        uint8_t* base = rest < chunks ? cache.k : cache.v;
        *reinterpret_cast<uint4*>(base + to[i] * row_bytes + (rest % chunks) * 16) = hold[j];
      }
    }
  }
  if (threadIdx.x < 2 * count && to[threadIdx.x >> 1] >= 0)
    (threadIdx.x & 1 ? cache.v_scale : cache.k_scale)[to[threadIdx.x >> 1]] = hs;
}

// Calls f(T*, head_dim constant, bits constant) for the run-time choice.
template <typename T, typename F>
cudaError_t by_format(const KvCache& c, F&& f) {
  if (c.head_dim == 64)
    return c.bits == 8 ? f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{})
                       : f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  return c.bits == 8 ? f(std::integral_constant<int, 128>{}, std::integral_constant<int, 8>{})
                     : f(std::integral_constant<int, 128>{}, std::integral_constant<int, 4>{});
}

template <typename T>
cudaError_t append_typed(const KvCache& c, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, const int64_t* slots, int64_t tokens, int* err,
                         cudaStream_t st) {
  const uint32_t rows = static_cast<uint32_t>(tokens * c.heads);
  return by_format<T>(c, [&](auto d, auto bits) {
    constexpr int kPerCta = kRowThreads / (decltype(d)::value / 8);
    kv_append_kernel<T, decltype(d)::value, decltype(bits)::value>
        <<<(rows + kPerCta - 1) / kPerCta, kRowThreads, 0, st>>>(
            c, static_cast<const T*>(k), k_stride, static_cast<const T*>(v), v_stride, slots, rows,
            err);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t read_typed(const KvCache& c, int64_t layers, const int32_t* table, int64_t table_width,
                       const int32_t* starts, const int32_t* offsets, int requests, int64_t tokens,
                       void* k, void* v, int* err, int num_sms, cudaStream_t st) {
  // enough CTAs to fill the GPU while there are tokens for it
  int64_t tile = tokens * layers / (8 * num_sms);
  tile = tile < 1 ? 1 : tile > 32 ? 32 : tile;
  const dim3 grid(static_cast<unsigned>((tokens + tile - 1) / tile), static_cast<unsigned>(layers));
  return by_format<T>(c, [&](auto d, auto bits) {
    kv_read_kernel<T, decltype(d)::value, decltype(bits)::value><<<grid, kRowThreads, 0, st>>>(
        c, table, table_width, starts, offsets, requests, tokens, static_cast<int>(tile),
        static_cast<T*>(k), static_cast<T*>(v), err);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv_append(const KvCache& c, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, bool bf16, const int64_t* slots, int64_t tokens,
                             int* err, cudaStream_t st) {
  return bf16 ? append_typed<__nv_bfloat16>(c, k, k_stride, v, v_stride, slots, tokens, err, st)
              : append_typed<__half>(c, k, k_stride, v, v_stride, slots, tokens, err, st);
}

cudaError_t launch_kv_read(const KvCache& c, int64_t layers, const int32_t* table,
                           int64_t table_width, const int32_t* starts, const int32_t* offsets,
                           int requests, int64_t tokens, void* k, void* v, bool bf16, int* err,
                           int num_sms, cudaStream_t st) {
  return bf16 ? read_typed<__nv_bfloat16>(c, layers, table, table_width, starts, offsets, requests,
                                          tokens, k, v, err, num_sms, st)
              : read_typed<__half>(c, layers, table, table_width, starts, offsets, requests, tokens,
                                   k, v, err, num_sms, st);
}

cudaError_t launch_kv_compact(const KvCache& c, int64_t layers, const int32_t* table,
                              int64_t table_width, const int32_t* starts, const int32_t* path,
                              int path_width, const int32_t* kept, int requests, int* err,
                              cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(requests), static_cast<unsigned>(c.heads),
                  static_cast<unsigned>(layers));
  kv_compact_kernel<<<grid, kCompactThreads, 0, st>>>(c, c.head_dim * c.bits / 8, table, table_width,
                                                      starts, path, path_width, kept, err);
  return cudaGetLastError();
}

}  // namespace cider
