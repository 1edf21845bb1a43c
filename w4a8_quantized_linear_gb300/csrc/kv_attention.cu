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

// Zeros for the rows of the output that no request owns, before the first offset
// and past the last, and their report.  The first launch of the call does not
// touch them, and what ran before it is over: nothing is waited for.
__device__ __forceinline__ void zero_unowned(const AttendArgs& a) {
  const int64_t before = max(static_cast<int64_t>(a.offsets[0]), int64_t{0});
  const int64_t past = max(static_cast<int64_t>(a.offsets[a.requests]), int64_t{0});
  if (before == 0 && past >= a.rows) return;
  if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, kDevErrIndex);
  const int64_t chunks = static_cast<int64_t>(a.q_heads) * a.cache.head_dim / 8;   // 16 bytes each, of a row
  uint4* const out = static_cast<uint4*>(a.out);
  const int64_t first = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x;
  for (int64_t i = first; i < min(before, a.rows) * chunks; i += step) out[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = past * chunks + first; i < a.rows * chunks; i += step) out[i] = make_uint4(0, 0, 0, 0);
}

// Share c begins within a unit and the share before it began the unit: adds the
// unit's parts in the order of the shares and writes its rows.  One CTA per
// (share, kJoinRows rows), a warp per row.  The shares' ends follow from the
// axis' length, so the parts' statistics are loaded side by side; walking from
// share to share cost a memory round trip each (18 us for 57 parts), and a CTA
// per row repeated the 64-bit divisions too often (38 us for 152 x 128 rows).
constexpr int kJoinRows = 4, kJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(AttendArgs a, PartsArgs parts, bool bf16) {
  extern __shared__ float weights[];   // per warp and part: its factor
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (c == 0) {   // no share lies before this one: its CTAs see to the rows without a request
    zero_unowned(a);
    return;
  }
  pdl_wait();
  const PartsArgs::Info i = parts.info[c];
  const int64_t before = parts.info[c - 1].begin;
  // the share before holds the unit's first tile unless it begins within it too
  if (i.begin < 0 || before == i.begin) return;
  const int group = a.q_heads / a.cache.heads;
  const int blocks = Axis::blocks_of(a, i.nodes, parts.rows);
  const int head = i.unit / blocks, block = i.unit - head * blocks;
  const int rows = min(parts.rows, i.nodes * group - block * parts.rows);
  const int first_row = blockIdx.y * kJoinRows;
  if (first_row >= rows) return;
  // parts: the last slot of the share before, then the first slot of every share that begins before the unit's end
  const int ctas = static_cast<int>(min(i.total, static_cast<int64_t>(gridDim.x)));
  int last = static_cast<int>(min(static_cast<int64_t>(ctas - 1), (i.end * ctas - 1) / i.total));
  while (last + 1 < ctas && i.total * (last + 1) / ctas < i.end) ++last;
  while (last > c && i.total * last / ctas >= i.end) --last;
  const int n = last - c + 2;
  float* weight = weights + warp * (static_cast<int>(gridDim.x) + 1);
  const int64_t slot0 = 2 * static_cast<int64_t>(c - 1);   // part j: slot0 + 2 j, and one more for j = 0
  for (int row = first_row + warp; row < min(rows, first_row + kJoinRows); row += kJoinWarps) {
    float top = -INFINITY, sum = 0.0f;
    for (int j = lane; j < n; j += 32) {
      const float2 s = parts.stat[(slot0 + 2 * j + (j == 0 ? 1 : 0)) * parts.rows + row];
      weight[j] = s.x;
      top = fmaxf(top, s.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int j = lane; j < n; j += 32) {
      const float f = weight[j] == -INFINITY ? 0.0f : exp2f(weight[j] - top);
      sum += parts.stat[(slot0 + 2 * j + (j == 0 ? 1 : 0)) * parts.rows + row].y * f;
      weight[j] = f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    constexpr int kPer = D / 32;
    float v[kPer] = {};
#pragma unroll 16
    for (int j = 0; j < n; ++j) {
      const float* src = parts.out + ((slot0 + 2 * j + (j == 0 ? 1 : 0)) * parts.rows + row) * D + lane * kPer;
      const float f = weight[j];
      if constexpr (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] += x.x * f; v[1] += x.y * f; v[2] += x.z * f; v[3] += x.w * f;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] += x.x * f; v[1] += x.y * f;
      }
    }
    const int at = block * parts.rows + row, node = at / group;
    const int64_t dst = ((i.first + node) * a.q_heads + head * group + at - node * group) * D + lane * kPer;
    const float scale = sum > 0.0f ? 1.0f / sum : 0.0f;
    if constexpr (kPer == 4) {
      store_out4(a.out, bf16, dst, make_float4(v[0], v[1], v[2], v[3]), scale);
    } else {
      const uint32_t u = bf16 ? y_bits2<true>(v[0] * scale, v[1] * scale) : y_bits2<false>(v[0] * scale, v[1] * scale);
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + dst) = u;
    }
    __syncwarp();   // the weights are written again
  }
}

}  // namespace

cudaError_t launch_join(const AttendArgs& a, const PartsArgs& parts, int ctas, int rows, bool bf16,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = static_cast<size_t>(ctas + 1) * kJoinWarps * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.cache.head_dim == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128>, a, parts, bf16)
                                 : cudaLaunchKernelEx(&cfg, join_kernel<64>, a, parts, bf16);
}

// By the query rows of a key/value head (new tokens x grouped heads).  At 32
// requests of 4096 .. 16384 positions the many-row kernel takes the same time
// for 1 to 128 rows, the other one grows with them: up to 32 rows (64 requests
// of up to 8192, INT8: 224 us against 304) it is ahead.
constexpr int kFewRows = 32;

cudaError_t launch_attend(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  return a.max_nodes * (a.q_heads / a.cache.heads) <= kFewRows ? launch_attend_rows(a, bf16, num_sms, st)
                                                               : launch_attend_tree(a, bf16, num_sms, st);
}

}  // namespace cider
