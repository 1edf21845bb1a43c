// verify.cu -- verification of drafted tokens against the target model's
// probabilities, from random numbers that the caller gives.
//
// Mathematics.  A request's nodes form a tree; node 0 is the last token that
// is certain.  With p = softmax(logits of the current node / temperature), the
// current node's children are asked in increasing order.
//   Drafts drawn from a distribution q without replacement: with the residual
//   r (first p, mass Z = 1) and the rest of q (mass Q = 1), a child with token
//   x is accepted if u q(x) Z < r(x) Q; otherwise r <- max(r / Z - q / Q, 0),
//   Z <- sum r (r and Z stay when nothing is left), Q <- Q - q(x), q(x) <- 0.
//   Certain drafts (no q): accepted if u Z < r(x); otherwise Z <- Z - r(x),
//   r(x) <- 0.
// An accepted child becomes the current node.  When no child is accepted, or
// there is none, the next token is argmax_x r(x) / e(x) with e the caller's
// exponential noise (a draw from r / Z), ties to the lowest index.
// Temperature 0: a child is accepted if its token is the logits' first
// maximum, which is also the next token.
//
// Only the nodes on the accepted path are read.  Sums and softmax statistics
// are fp32, in an order that depends on the sizes alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"

namespace cider {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

struct VerifyArgs {
  const void* logits;
  int64_t logits_stride;
  const int32_t *tokens, *parents, *offsets;
  int requests;
  int64_t nodes;
  int vocab, max_nodes;
  const float *uniforms, *noise, *draft, *temperature;
  int32_t *count, *path, *next;
  int* err;
};

__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A float's order as an unsigned number, above the index's reversed order:
// the largest packed value is the largest float, at its lowest index.
__device__ __forceinline__ uint64_t pack_best(float v, uint32_t i) {
  uint32_t b = __float_as_uint(v);
  b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return static_cast<uint64_t>(b) << 32 | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ uint32_t best_index(uint64_t p) {
  return 0xFFFFFFFFu - static_cast<uint32_t>(p);
}

// One rejected child of the current node.
struct Rejected {
  float inv_mass, inv_drawn;   // 1 / Z and 1 / Q when it was asked
  int32_t token;
  int32_t keeps;               // nothing was left: r stayed as it was
};

struct Shared {
  float fsum[kVerifyWarps];
  uint64_t best[kVerifyWarps];
  Rejected rejected[kMaxNodes];
};

__device__ __forceinline__ float block_sum(float v, Shared& sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.fsum[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kVerifyWarps; ++i) s += sh.fsum[i];
  return s;
}

__device__ __forceinline__ uint64_t block_best(uint64_t v, Shared& sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.best[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t s = sh.best[0];
#pragma unroll
  for (int i = 1; i < kVerifyWarps; ++i) s = sh.best[i] > s ? sh.best[i] : s;
  return s;
}

// r(x) after the node's rejected children so far; q: the drafter's row's value at x.
__device__ __forceinline__ float residual(float p, float q, int x, bool sampled,
                                          const Rejected* rejected, int n) {
  float r = p;
  for (int j = 0; j < n; ++j) {
    const Rejected& e = rejected[j];
    if (sampled) {
      if (!e.keeps) r = fmaxf(r * e.inv_mass - q * e.inv_drawn, 0.0f);
      if (x == e.token) q = 0.0f;
    } else if (x == e.token) {
      r = 0.0f;
    }
  }
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(VerifyArgs a) {
  __shared__ Shared sh;
  const int b = blockIdx.x;
  const int64_t first = a.offsets[b];
  const int64_t end = a.offsets[b + 1];
  const bool bad = first < 0 || end > a.nodes || end - first > a.max_nodes || end < first;
  const int size = bad ? 0 : static_cast<int>(end - first);
  if (bad && threadIdx.x == 0) atomicOr(a.err, kDevErrIndex);
  for (int i = threadIdx.x; i < a.max_nodes; i += kVerifyThreads)
    a.path[static_cast<int64_t>(b) * a.max_nodes + i] = size > 0 && i == 0 ? 0 : -1;
  if (size == 0) {
    if (threadIdx.x == 0) {
      a.count[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  const float temperature = a.temperature ? a.temperature[b] : 1.0f;
  const bool greedy = !(temperature > 0.0f);
  const float inv_t = greedy ? 1.0f : 1.0f / temperature;
  const float* noise = a.noise + static_cast<int64_t>(b) * a.vocab;
  int now = 0, count = 1;
  for (;;) {
    const T* row = static_cast<const T*>(a.logits) + (first + now) * a.logits_stride;
    const float* q = a.draft ? a.draft + (first + now) * a.vocab : nullptr;
    uint64_t best = 0;
    for (int x = threadIdx.x; x < a.vocab; x += kVerifyThreads) {
      const uint64_t p = pack_best(as_float(row[x]), x);
      best = p > best ? p : best;
    }
    const int hot = static_cast<int>(best_index(block_best(best, sh)));
    const float top = as_float(row[hot]);
    float sum = 0.0f;
    if (!greedy) {
      for (int x = threadIdx.x; x < a.vocab; x += kVerifyThreads)
        sum += __expf((as_float(row[x]) - top) * inv_t);
      sum = block_sum(sum, sh);
    }
    // a row of -inf alone is no distribution: nothing is accepted
    const float inv_sum = top == -INFINITY ? 0.0f : 1.0f / sum;
    auto prob = [&](int x) {
      const float l = as_float(row[x]);
      return l == -INFINITY ? 0.0f : __expf((l - top) * inv_t) * inv_sum;
    };
    float mass = 1.0f, drawn = 1.0f;
    int rejected = 0, accepted = -1;
    for (int i = now + 1; i < size; ++i) {
      if (a.parents[first + i] != now) continue;
      const int x = a.tokens[first + i];
      if (x < 0 || x >= a.vocab) {
        if (threadIdx.x == 0) atomicOr(a.err, kDevErrIndex);
        continue;
      }
      if (greedy) {
        if (x == hot) {
          accepted = i;
          break;
        }
        continue;
      }
      const float u = a.uniforms[first + i];
      float qx = q ? q[x] : 1.0f;
      const float r = residual(prob(x), qx, x, q != nullptr, sh.rejected, rejected);
      if (!q) {
        if (u * mass < r) {
          accepted = i;
          break;
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.rejected[rejected] = Rejected{0.0f, 0.0f, x, 0};
        __syncthreads();
        ++rejected;
        mass -= r;
        continue;
      }
      for (int j = 0; j < rejected; ++j)
        if (sh.rejected[j].token == x) qx = 0.0f;
      if (u * qx * mass < r * drawn) {
        accepted = i;
        break;
      }
      __syncthreads();
      if (threadIdx.x == 0) sh.rejected[rejected] = Rejected{1.0f / mass, 1.0f / drawn, x, 0};
      __syncthreads();
      ++rejected;
      float rest = 0.0f;
      for (int y = threadIdx.x; y < a.vocab; y += kVerifyThreads)
        rest += residual(prob(y), q[y], y, true, sh.rejected, rejected);
      rest = block_sum(rest, sh);
      drawn -= qx;
      if (rest == 0.0f) {
        if (threadIdx.x == 0) sh.rejected[rejected - 1].keeps = 1;
        __syncthreads();
      } else {
        mass = rest;
      }
    }
    if (accepted >= 0) {
      if (threadIdx.x == 0) a.path[static_cast<int64_t>(b) * a.max_nodes + count] = accepted;
      ++count;
      now = accepted;
      continue;
    }
    int next = hot;
    if (!greedy) {
      best = 0;
      for (int x = threadIdx.x; x < a.vocab; x += kVerifyThreads) {
        const float r = residual(prob(x), q ? q[x] : 0.0f, x, q != nullptr, sh.rejected, rejected);
        const uint64_t p = pack_best(__fdiv_rn(r, noise[x]), x);
        best = p > best ? p : best;
      }
      next = static_cast<int>(best_index(block_best(best, sh)));
    }
    if (threadIdx.x == 0) {
      a.count[b] = count;
      a.next[b] = next;
    }
    return;
  }
}

}  // namespace

cudaError_t launch_verify(const void* logits, int64_t logits_stride, bool bf16,
                          const int32_t* tokens, const int32_t* parents, const int32_t* offsets,
                          int requests, int64_t nodes, int vocab, int max_nodes,
                          const float* uniforms, const float* noise, const float* draft,
                          const float* temperature, int32_t* count, int32_t* path, int32_t* next,
                          int* err, int num_sms, cudaStream_t st) {
  (void)num_sms;
  const VerifyArgs a{logits, logits_stride, tokens, parents, offsets, requests, nodes,
                     vocab,  max_nodes,     uniforms, noise, draft,   temperature, count,
                     path,   next,          err};
  if (bf16)
    verify_kernel<__nv_bfloat16><<<requests, kVerifyThreads, 0, st>>>(a);
  else
    verify_kernel<__half><<<requests, kVerifyThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace cider
