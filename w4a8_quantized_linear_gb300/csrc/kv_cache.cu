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
// thread and access, several independent loads in flight per thread.  Issue
// slots come second: at 4 instructions a clock the append has ~11 a value, so
// the maximum is taken on packed pairs, the scale and the quotients by
// corrected reciprocals, and the codes come out of float additions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"

namespace cider {
namespace {

constexpr int kRowThreads = 256;

// ------------------------------------------------------------------ append
// Eight rounded quotients plus 1.5 * 2^23 (the nearest whole number, ties to
// even, in the low mantissa bits; INT8 in two's complement, INT4 with 8 more, an
// even offset that leaves the ties as they are) -> codes as bytes (INT8: 8
// bytes) or packed nibbles (INT4: 4 bytes in x).
template <int BITS>
__device__ __forceinline__ uint2 pack8(const uint32_t (&c)[8]) {
  if constexpr (BITS == 8) {
    const uint32_t a = __byte_perm(c[0], c[1], 0x0040u), b = __byte_perm(c[2], c[3], 0x0040u);
    const uint32_t d = __byte_perm(c[4], c[5], 0x0040u), e = __byte_perm(c[6], c[7], 0x0040u);
    return make_uint2(__byte_perm(a, b, 0x5410u), __byte_perm(d, e, 0x5410u));
  } else {
    // sum of c_i 16^i: the nibbles side by side above the sum of the constant
    // float bits, which is taken off; then plus 8 -> two's complement
    uint32_t w = c[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) w = w * 16u + c[i];
    return make_uint2((w - 0x4B400000u * 0x11111111u) ^ 0x88888888u, 0u);
  }
}
template <int BITS>
__device__ __forceinline__ float code_base() {
  return BITS == 8 ? 12582912.0f : 12582920.0f;
}

// A row whose scale is near an end of the exponent range: plain divisions.
template <int BITS>
__device__ __noinline__ uint2 encode8_divide(const float* f, float s) {
  constexpr float kTop = BITS == 8 ? 127.0f : 7.0f;
  uint32_t c[8];
  for (int i = 0; i < 8; ++i)
    c[i] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fdiv_rn(f[i], s), -kTop), kTop), code_base<BITS>()));
  return pack8<BITS>(c);
}

// Eight packed 16-bit values -> fp32; bf16 values are the upper halves.
template <typename T>
__device__ __forceinline__ void spread8(const uint4& in, float (&f)[8]) {
  if constexpr (std::is_same<T, __half>::value) {
    widen8<T>(in, f);
  } else {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// The larger of two packed pairs without signs.
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  P x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}

// Eight values of a row (with those of its D / 8 - 1 neighbours) -> their codes
// and the row's scale.  Quotients by r = RN(1/s) and Markstein's correction,
// the scale by the constant's reciprocal likewise; they hold while nothing
// underflows on the way (fp16 always; bf16 maxima reach 2^-133): else `plain`
// is set and s is the row's maximum.  r: one Newton step from the approximate reciprocal rounds correctly
// but for an all-ones mantissa of s, which no s = RN(a / 127) or RN(a / 7) of
// an 8- or 11-bit a has (a / 127 would have to be within 2^-23 of a power of 2).
template <typename T, int D, int BITS>
__device__ __forceinline__ uint2 encode_row(const uint4& in, float& s, bool& plain) {
  constexpr int kLanes = D / 8;
  constexpr float kTop = BITS == 8 ? 127.0f : 7.0f;
  uint32_t m = max2<T>(max2<T>(in.x & 0x7FFF7FFFu, in.y & 0x7FFF7FFFu),
                       max2<T>(in.z & 0x7FFF7FFFu, in.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max2<T>(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max2<T>(m, __byte_perm(m, m, 0x1032u));
  float f[8];
  spread8<T>(make_uint4(m, m, m, m), f);
  const float a = f[0];
  plain = !(a > 1e-28f && a < 1e32f) && a != 0.0f;
  s = a == 0.0f ? 1.0f : plain ? a : div_rn_by(a, kTop, 1.0f / kTop);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = __fmaf_rn(r, __fmaf_rn(-s, r, 1.0f), r);
  spread8<T>(in, f);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(__fadd_rn(div_rn_by(f[i], s, r), code_base<BITS>()));
  return pack8<BITS>(c);
}

// D / 8 neighbouring threads hold one (token, head) row of K and of V.  Blocks
// of all heads of the same tokens run together.  (Two tokens per thread left
// room for a third of the warps: 32768 tokens INT4, with the read back, 90 us instead of 75.)
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kRowThreads, 8)
    kv_append_kernel(KvCache cache, const T* __restrict__ k, int64_t k_stride,
                     const T* __restrict__ v, int64_t v_stride, const int64_t* __restrict__ slots,
                     int tokens, int64_t capacity, int* err) {
  constexpr int kLanes = D / 8, kGroups = kRowThreads / kLanes, kRowBytes = D * BITS / 8;
  constexpr float kTop = BITS == 8 ? 127.0f : 7.0f;
  const int lane = threadIdx.x % kLanes, head = blockIdx.x;
  const int64_t token = (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * kGroups + threadIdx.x / kLanes;
  uint4 in[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  int64_t slot = -1;
  if (token < tokens) {
    in[0] = ld_stream_v4(k + token * k_stride + head * D + lane * 8);
    in[1] = ld_stream_v4(v + token * v_stride + head * D + lane * 8);
    slot = slots[token];
  }
  const bool inside = slot >= 0 && slot < capacity;
  if (slot >= 0 && !inside && lane == 0) atomicOr(err, kDevErrIndex);
  // 16-row blocks of a layer fit 32 bits
  const int page = static_cast<int>(slot >> cache.page_shift);
  const int at = static_cast<int>(slot) & ((1 << cache.page_shift) - 1);
  const int block = ((page * cache.heads + head) << (cache.page_shift - 4)) + (at >> 4);
  const int64_t row = static_cast<int64_t>(block) * 16 + (at & 15);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float s;
    bool plain;
    uint2 code = encode_row<T, D, BITS>(in[i], s, plain);
    if (plain) {   // the same for all threads of a row: s is still the row's maximum
      float f[8];
      spread8<T>(in[i], f);
      s = __fdiv_rn(s, kTop);
      code = encode8_divide<BITS>(f, s);
    }
    if (inside) {
      uint8_t* c = (i == 0 ? cache.k : cache.v) + row * kRowBytes + lane * BITS;
      if constexpr (BITS == 8)
        *reinterpret_cast<uint2*>(c) = code;
      else
        *reinterpret_cast<uint32_t*>(c) = code.x;
      if (lane == 0) (i == 0 ? cache.k_scale : cache.v_scale)[row] = s;
    }
  }
}

// -------------------------------------------------------------------- read
// Eight codes times s: each an exact float (its byte in the mantissa of 2^23,
// the offset subtracted; a conversion instruction runs at a quarter of the
// rate), the fp32 product rounded once to the output type.
template <typename T, int BITS>
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
  uint32_t even, odd;   // INT8: codes 0..3, 4..7 plus 128; INT4: even, odd ones plus 8
  if constexpr (BITS == 8) {
    even = c.x ^ 0x80808080u;
    odd = c.y ^ 0x80808080u;
  } else {
    const uint32_t u = c.x ^ 0x88888888u;
    even = u & 0x0F0F0F0Fu;
    odd = u >> 4 & 0x0F0F0F0Fu;
  }
  constexpr float kOff = 8388608.0f + (BITS == 8 ? 128.0f : 8.0f);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __byte_perm(even, 0x4B000000u, 0x7440u | i), b = __byte_perm(odd, 0x4B000000u, 0x7440u | i);
    f[BITS == 8 ? i : 2 * i] = __fmul_rn(__uint_as_float(a) - kOff, s);
    f[BITS == 8 ? i + 4 : 2 * i + 1] = __fmul_rn(__uint_as_float(b) - kOff, s);
  }
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  return make_uint4(y_bits2<kBf16>(f[0], f[1]), y_bits2<kBf16>(f[2], f[3]), y_bits2<kBf16>(f[4], f[5]),
                    y_bits2<kBf16>(f[6], f[7]));
}

// A CTA reads `tile` tokens (at most 32) of one layer, all heads.  (Four rows
// per thread on their way at once took 133 us instead of 120 at 131072 tokens INT4.)
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kRowThreads, 8)
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
    if (b >= 0) at = cache_row_of(cache, table, table_width, b, static_cast<int64_t>(starts[b]) + i - offsets[b], 0);
    if (at < 0) atomicOr(err, kDevErrIndex);
    place[threadIdx.x] = at;
  }
  __syncthreads();
  const int lane = threadIdx.x % kLanes;
  const int64_t layer_rows = cache.layer_rows();
  const uint8_t* ck = cache.k + blockIdx.y * layer_rows * kRowBytes + lane * BITS;
  const uint8_t* cv = cache.v + blockIdx.y * layer_rows * kRowBytes + lane * BITS;
  const float* sk = cache.k_scale + blockIdx.y * layer_rows;
  const float* sv = cache.v_scale + blockIdx.y * layer_rows;
  const int64_t out0 = (static_cast<int64_t>(blockIdx.y) * tokens + t0) * cache.heads * D + lane * 8;
  T* const ko = k + out0;
  T* const vo = v + out0;
  const int rows = here * cache.heads;
  // the rows of this group: one division, then steps with a carry
  int r = threadIdx.x / kLanes;
  int token = r / cache.heads, head = r - token * cache.heads;
  const int step_token = kGroups / cache.heads, step_head = kGroups - step_token * cache.heads;
#pragma unroll 2
  for (; r < rows; r += kGroups) {
    const int64_t at = place[token];
    uint2 a = make_uint2(0, 0), b = a;   // without a page: zeros
    float s = 0.0f, t = 0.0f;
    if (at >= 0) {
      const int64_t row = at + (static_cast<int64_t>(head) << cache.page_shift);
      if constexpr (BITS == 8) {
        a = *reinterpret_cast<const uint2*>(ck + row * kRowBytes);
        b = *reinterpret_cast<const uint2*>(cv + row * kRowBytes);
      } else {
        a.x = *reinterpret_cast<const uint32_t*>(ck + row * kRowBytes);
        b.x = *reinterpret_cast<const uint32_t*>(cv + row * kRowBytes);
      }
      s = sk[row];
      t = sv[row];
    }
    *reinterpret_cast<uint4*>(ko + static_cast<int64_t>(r) * D) = decode8<T, BITS>(a, s);
    *reinterpret_cast<uint4*>(vo + static_cast<int64_t>(r) * D) = decode8<T, BITS>(b, t);
    token += step_token;
    head += step_head;
    if (head >= cache.heads) {
      head -= cache.heads;
      ++token;
    }
  }
}

// ----------------------------------------------------------------- compact
// Row start + path[i] moves to start + i, in every layer and head.  A thread
// moves one 16-byte column of a (layer, head)'s rows (or its scales): the
// columns do not depend on one another, so no barrier is needed, and the rows
// are looked up once per CTA for all its columns.  (One CTA per layer, request
// and head, with a barrier between reading and writing, spent its time on the
// look-ups: 30 us for 26 MB.)  While the path only goes forward, as accepted
// paths do, no target is a later source, and a thread moves 8 rows at a time;
// else it reads all rows (64 at most, in local memory) before it writes.
constexpr int kCompactThreads = 256;
constexpr int kMoveAtOnce = 8;

template <typename V>
__device__ __forceinline__ void move_column(char* base, int64_t pitch, const int64_t* from, const int64_t* to,
                                            int count, bool forward) {
  if (forward) {
    for (int i = 0; i < count; i += kMoveAtOnce) {
      V hold[kMoveAtOnce];
#pragma unroll
      for (int j = 0; j < kMoveAtOnce; ++j)
        if (i + j < count && from[i + j] >= 0) hold[j] = *reinterpret_cast<const V*>(base + from[i + j] * pitch);
#pragma unroll
      for (int j = 0; j < kMoveAtOnce; ++j)
        if (i + j < count && from[i + j] >= 0) *reinterpret_cast<V*>(base + to[i + j] * pitch) = hold[j];
    }
  } else {
    V hold[kMaxNodes];
    for (int i = 0; i < count; ++i)
      if (from[i] >= 0) hold[i] = *reinterpret_cast<const V*>(base + from[i] * pitch);
    for (int i = 0; i < count; ++i)
      if (from[i] >= 0) *reinterpret_cast<V*>(base + to[i] * pitch) = hold[i];
  }
}

__global__ void __launch_bounds__(kCompactThreads)
    kv_compact_kernel(KvCache cache, int row_bytes, int units, const int32_t* __restrict__ table,
                      int64_t table_width, const int32_t* __restrict__ starts,
                      const int32_t* __restrict__ path, int path_width,
                      const int32_t* __restrict__ kept, int* err) {
  __shared__ int64_t from[kMaxNodes], to[kMaxNodes];   // rows of layer 0, head 0; -1: nothing moves
  const int b = blockIdx.y;
  const int n = kept[b];
  if (n == 0) return;
  if (n < 0 || n > path_width) {
    if (threadIdx.x == 0) atomicOr(err, kDevErrIndex);
    return;
  }
  bool forward = true;
  if (threadIdx.x < n) {
    const int i = threadIdx.x;
    const int32_t* p = path + static_cast<int64_t>(b) * path_width + i;
    const int src = p[0];
    forward = src >= i && (i == 0 || p[-1] < src);
    const int64_t start = starts[b];
    const int64_t rf = src < 0 ? -1 : cache_row_of(cache, table, table_width, b, start + src, 0);
    const int64_t rt = cache_row_of(cache, table, table_width, b, start + i, 0);
    const bool ok = rf >= 0 && rt >= 0;
    if (!ok) atomicOr(err, kDevErrIndex);
    from[i] = ok && rf != rt ? rf : -1;
    to[i] = rt;
  }
  forward = __syncthreads_and(forward);
  const int chunks = row_bytes / 16;   // of 16 bytes in a row
  const int64_t columns = static_cast<int64_t>(units) * 2 * chunks, all = columns + 2 * units;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kCompactThreads + threadIdx.x;
  if (id >= all) return;
  const bool scales = id >= columns;
  const int64_t rest = scales ? id - columns : id;
  const int width = scales ? 2 : 2 * chunks;
  const int unit = static_cast<int>(rest / width), column = static_cast<int>(rest - static_cast<int64_t>(unit) * width);
  const int layer = unit / cache.heads, head = unit - layer * cache.heads;
  const int64_t row0 = layer * cache.layer_rows() + (static_cast<int64_t>(head) << cache.page_shift);
  if (scales) {
    char* base = reinterpret_cast<char*>((column ? cache.v_scale : cache.k_scale) + row0);
    move_column<float>(base, 4, from, to, n, forward);
  } else {
    char* base = reinterpret_cast<char*>((column < chunks ? cache.k : cache.v) + row0 * row_bytes) +
                 (column < chunks ? column : column - chunks) * 16;
    move_column<uint4>(base, row_bytes, from, to, n, forward);
  }
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
  return by_format<T>(c, [&](auto d, auto bits) {
    constexpr int kPerCta = kRowThreads / (decltype(d)::value / 8);
    const int64_t blocks = (tokens + kPerCta - 1) / kPerCta;
    const int64_t y = std::min<int64_t>(blocks, 32768);
    const dim3 grid(static_cast<unsigned>(c.heads), static_cast<unsigned>(y),
                    static_cast<unsigned>((blocks + y - 1) / y));
    kv_append_kernel<T, decltype(d)::value, decltype(bits)::value><<<grid, kRowThreads, 0, st>>>(
        c, static_cast<const T*>(k), k_stride, static_cast<const T*>(v), v_stride, slots,
        static_cast<int>(tokens), c.pages << c.page_shift, err);
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
  const int row_bytes = c.head_dim * c.bits / 8;
  const int64_t units = layers * c.heads;
  const int64_t ctas = (units * (2 * (row_bytes / 16) + 2) + kCompactThreads - 1) / kCompactThreads;
  // requests in runs that the grid's second dimension holds
  for (int b = 0; b < requests; b += 65535) {
    const int n = std::min(requests - b, 65535);
    kv_compact_kernel<<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(n)), kCompactThreads, 0, st>>>(
        c, row_bytes, static_cast<int>(units), table + b * table_width, table_width, starts + b,
        path + static_cast<int64_t>(b) * path_width, path_width, kept + b, err);
  }
  return cudaGetLastError();
}

}  // namespace cider
