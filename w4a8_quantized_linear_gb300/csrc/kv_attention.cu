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

// Share c begins within a unit and the share before it began the unit: adds the
// unit's parts in the order of the shares and writes its rows.  One CTA of D
// threads per (share, row).  The shares' ends follow from the axis' length, so
// the parts' statistics are loaded side by side; walking from share to share
// cost a memory round trip each (18 us for 57 parts).
__global__ void join_kernel(AttendArgs a, PartsArgs parts, bool bf16) {
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
  const int blocks = Axis::blocks_of(a, r, parts.rows);
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

cudaError_t launch_join(const AttendArgs& a, const PartsArgs& parts, int ctas, int rows, bool bf16,
                        cudaStream_t st) {
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
  return cudaLaunchKernelEx(&cfg, join_kernel, a, parts, bf16);
}

cudaError_t launch_attend(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  return a.max_nodes * (a.q_heads / a.cache.heads) <= 16 ? launch_attend_rows(a, bf16, num_sms, st)
                                                         : launch_attend_tree(a, bf16, num_sms, st);
}

}  // namespace cider
