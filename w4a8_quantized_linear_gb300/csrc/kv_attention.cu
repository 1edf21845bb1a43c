// kv_attention.cu -- attention of a request's new tokens (one token, a chain
// or a tree of drafted tokens) over its paged, quantized key/value cache.
//
// Mathematics, for a new token t of request b and query head h (key/value
// head h / group):
//   S_j = scale * sk_j * (q . ck_j),   p_j = exp(S_j - max S),
//   o = sum_j p_j sv_j cv_j / sum_j p_j
// over the positions j that t sees: the context (all but the request's last T
// positions) and, of those last T, the ones whose bit is set in t's mask.  A
// token that sees nothing gets zeros.  ck, cv are the codes, sk, sv the scales.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"
#include "kv_parts.cuh"

namespace cider {
namespace {

constexpr int kPlainWarps = 4;

// Value `lane * PER + e` of a row of codes.
template <int D, int BITS>
__device__ __forceinline__ void row_values(const uint8_t* row, int lane, float (&f)[D / 32]) {
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    const int d = lane * (D / 32) + e;
    if constexpr (BITS == 8) {
      f[e] = static_cast<float>(static_cast<int8_t>(row[d]));
    } else {
      const int w = row[d / 2];
      f[e] = static_cast<float>(static_cast<int>(static_cast<unsigned>(w) << (28 - 4 * (d & 1))) >> 28);
    }
  }
}

// One CTA per (row of q, query head); its warps take positions in turn, each
// with its own running maximum, sum and output, joined at the end.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(32 * kPlainWarps) attend_kernel(AttendArgs a) {
  constexpr int kPer = D / 32;
  constexpr int kRowBytes = D * BITS / 8;
  __shared__ float sm[kPlainWarps], sl[kPlainWarps], so[kPlainWarps][D];
  const int64_t i = blockIdx.x;
  const int hq = blockIdx.y, head = hq / (a.q_heads / a.cache.heads);
  const int b = find_request(a.offsets, a.requests, i);
  if (b < 0) return;
  const Request r = request_of(a, b);
  if (r.nodes == 0) return;
  const int t = static_cast<int>(i - r.first);
  const uint64_t mask = a.tree ? static_cast<uint64_t>(a.tree[i]) : (~0ull >> (63 - t));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(a.q) + i * a.q_stride + static_cast<int64_t>(hq) * D;
  float qf[kPer], o[kPer], f[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    qf[e] = static_cast<float>(q[lane * kPer + e]);
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = warp; j < r.length; j += kPlainWarps) {
    const int64_t ahead = j - r.context;
    if (ahead >= 0 && !(mask >> ahead & 1)) continue;
    const int64_t at = cache_row_of(a.cache, a.table, a.table_width, b, j, head);
    if (at < 0) {
      if (lane == 0) atomicOr(a.err, kDevErrIndex);
      continue;
    }
    row_values<D, BITS>(a.cache.k + at * kRowBytes, lane, f);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s += qf[e] * f[e];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale * a.cache.k_scale[at];
    const float top = fmaxf(m, s);
    const float keep = __expf(m - top), p = __expf(s - top);
    m = top;
    l = l * keep + p;
    row_values<D, BITS>(a.cache.v + at * kRowBytes, lane, f);
    const float pv = p * a.cache.v_scale[at];
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + pv * f[e];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kPlainWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kPlainWarps; ++w) sum += top == -INFINITY ? 0.0f : sl[w] * __expf(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += 32 * kPlainWarps) {
    float x = 0.0f;
    for (int w = 0; w < kPlainWarps; ++w)
      x += top == -INFINITY ? 0.0f : so[w][d] * __expf(sm[w] - top);
    static_cast<T*>(a.out)[(i * a.q_heads + hq) * D + d] = static_cast<T>(sum > 0.0f ? x / sum : 0.0f);
  }
}

// Share c begins within a unit and the share before it began the unit: adds the
// unit's parts in the order of the shares and writes its rows.  One CTA of D
// threads per (share, row).  The shares' ends follow from the axis' length, so
// the parts' statistics are loaded side by side; walking from share to share
// cost a memory round trip each (18 us for 57 parts).
__global__ void join_kernel(AttendArgs a, PartsArgs parts, int blocks, bool bf16) {
  extern __shared__ float2 weight[];   // per part: its factor
  __shared__ float2 red[4];
  pdl_wait();
  const int c = blockIdx.x, row = blockIdx.y, d = threadIdx.x, dim = blockDim.x;
  if (c == 0) return;
  const PartsArgs::Info i = parts.info[c];
  // the share before holds the unit's first tile unless it begins within it too
  if (i.begin < 0 || parts.info[c - 1].begin == i.begin) return;
  const Request r = request_of(a, i.b, false);
  const int group = a.q_heads / a.cache.heads;
  const int head = i.unit / blocks, block = i.unit - head * blocks;
  const int at = block * parts.rows + row;
  if (at >= r.nodes * group) return;
  // parts: the last slot of the share before, then the first slot of every share that begins before the unit's end
  const int ctas = static_cast<int>(min(i.total, static_cast<int64_t>(gridDim.x)));
  int last = static_cast<int>(min(static_cast<int64_t>(ctas - 1), (i.end * ctas - 1) / i.total));
  while (last + 1 < ctas && i.total * (last + 1) / ctas < i.end) ++last;
  while (last > c && i.total * last / ctas >= i.end) --last;
  const int n = last - c + 2;
  auto stat_of = [&](int j) { return (2 * static_cast<int64_t>(c - 1 + j) + (j == 0 ? 1 : 0)) * parts.rows + row; };
  float top = -INFINITY, sum = 0.0f;
  for (int j = d; j < n; j += dim) {
    weight[j] = parts.stat[stat_of(j)];
    top = fmaxf(top, weight[j].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((d & 31) == 0) red[d >> 5].x = top;
  __syncthreads();
  for (int w = 0; w < dim / 32; ++w) top = fmaxf(top, red[w].x);
  for (int j = d; j < n; j += dim) {
    const float f = weight[j].x == -INFINITY ? 0.0f : exp2f(weight[j].x - top);
    sum += weight[j].y * f;
    weight[j].x = f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((d & 31) == 0) red[d >> 5].y = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < dim / 32; ++w) sum += red[w].y;
  float o = 0.0f;
#pragma unroll 8
  for (int j = 0; j < n; ++j) o += parts.out[stat_of(j) * dim + d] * weight[j].x;
  const float v = sum > 0.0f ? o / sum : 0.0f;
  const int node = at / group;
  const int64_t dst = ((r.first + node) * a.q_heads + head * group + at - node * group) * dim + d;
  static_cast<uint16_t*>(a.out)[dst] = bf16 ? y_bits<true>(v) : y_bits<false>(v);
}

}  // namespace

cudaError_t launch_join(const AttendArgs& a, const PartsArgs& parts, int ctas, int rows, int blocks,
                        bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(rows));
  cfg.blockDim = dim3(static_cast<unsigned>(a.cache.head_dim));
  cfg.dynamicSmemBytes = static_cast<size_t>(ctas + 1) * sizeof(float2);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, a, parts, blocks, bf16);
}

cudaError_t launch_attend(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  if (a.max_nodes * (a.q_heads / a.cache.heads) <= 32)
    return launch_attend_rows(a, bf16, num_sms, st);
  const dim3 grid(static_cast<unsigned>(a.rows), static_cast<unsigned>(a.q_heads));
  const bool wide = a.cache.head_dim == 128, b8 = a.cache.bits == 8;
  auto go = [&](auto t) {
    using T = decltype(t);
    if (wide && b8) attend_kernel<T, 128, 8><<<grid, 32 * kPlainWarps, 0, st>>>(a);
    else if (wide) attend_kernel<T, 128, 4><<<grid, 32 * kPlainWarps, 0, st>>>(a);
    else if (b8) attend_kernel<T, 64, 8><<<grid, 32 * kPlainWarps, 0, st>>>(a);
    else attend_kernel<T, 64, 4><<<grid, 32 * kPlainWarps, 0, st>>>(a);
  };
  if (bf16) go(__nv_bfloat16()); else go(__half());
  return cudaGetLastError();
}

}  // namespace cider
