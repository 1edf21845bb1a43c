// verify.cu -- verification of drafted tokens against the target model's
// probabilities, from random numbers that the caller gives.
//
// Mathematics.  A request's nodes form a tree; node 0 is the last token that
// is certain.  With p = softmax(logits of the current node / temperature), the
// current node's children are asked in increasing order.
//   Drafts drawn from a distribution q without replacement: with the residual
//   r (first p, mass Z = 1) and the rest of q (mass Q = 1), a child with token
//   x is accepted if u q(x) / Q Z < r(x); otherwise r <- max(r / Z - q / Q, 0),
//   Z <- sum r (r and Z stay when nothing is left), q(x) <- 0, Q <- sum q.
//   Q is added up anew each time: as 1 - q(x1) - q(x2) - ... it would be rounding
//   noise, of either sign, once a peaked drafter's first tokens are refused.
//   Nothing is left of a sum below 2^-126 (its reciprocal may overflow).  With
//   nothing left of q no later child can have been drawn: all are refused.
//   Certain drafts (no q): accepted if u Z < r(x); otherwise Z <- Z - r(x),
//   r(x) <- 0.
// An accepted child becomes the current node.  When no child is accepted, or
// there is none, the next token is argmax_x r(x) / e(x) with e the caller's
// exponential noise (a draw from r / Z), ties to the lowest index.
// Temperature 0: a child is accepted if its token is the logits' first
// maximum, which is also the next token.
//
// Only the nodes on the accepted path are read: its rows of logits once from
// HBM (again from L2 where a residual or the draw needs them), and the noise of
// the one draw.  The walk is serial, so what bounds it is latency: a cluster of
// up to 8 CTAs shares a request's vocabulary, each visited node costs one pass
// over a CTA's share (softmax maximum and sum in one pass, 8 x 16 bytes per
// lane in flight; ~3500 cycles for 16000 tokens, most of it the loads' latency)
// and one exchange between the CTAs through distributed shared memory (~2000
// cycles with the wait for the slowest warp; 3000 by cluster barriers); the
// noise, and the row of the child that is asked first, are prefetched to L2
// meanwhile.  Every wait for another CTA has a limit; the CTA agrees on its
// outcome by one barrier (0.3 .. 0.6 us a call).  Measured: 48 trees of 16 .. 32
// nodes over 128000 tokens 29 us (the longest path has 8 nodes; logits in L2), two
// chains of 4 drafts over 32003 tokens 18 us.
// Every CTA adds the shares' results in the order of their ranks, so all take the
// same decisions and the same inputs give the same path.  Sums and softmax
// statistics are fp32.
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

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kBlock = 256;     // tokens that a warp takes at once: 8 per lane
constexpr int kAtOnce = 8;      // blocks in flight
constexpr int kMaxCluster = 8;

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
  uint64_t wait_ns;   // limit of a wait for the other ranks
  int silent;         // this rank sends nothing (-1: all send); for tests of that limit
};

__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A float's order as an unsigned number, above the index's reversed order:
// the largest packed value is the largest float, at its lowest index.  -0 is +0.
__device__ __forceinline__ uint64_t pack_best(float v, uint32_t i) {
  uint32_t b = __float_as_uint(v + 0.0f);
  b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return static_cast<uint64_t>(b) << 32 | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ uint32_t best_index(uint64_t p) {
  return 0xFFFFFFFFu - static_cast<uint32_t>(p);
}

// One rejected child of the current node.
struct Rejected {
  float inv_mass, inv_rest;    // 1 / Z and 1 / Q when it was asked
  int32_t token;
  int32_t keeps;               // nothing was left: r stayed as it was
};

// What a thread, a warp or a CTA found in its share: sum counts from top.  Of a
// pair of plain sums, `top` is the second one.
struct Found {
  float top, sum;
  uint64_t best;
};
constexpr float kLeast = 0x1p-126f;   // nothing is left of a smaller sum

struct Shared {
  Found warp[2][kVerifyWarps];   // by exchange
  Found cta[2][kMaxCluster];
  uint64_t bar[2];               // the ranks' results of an exchange have arrived
  uint32_t abort;
  Rejected rejected[kMaxNodes];
  int32_t parent[kMaxNodes], token[kMaxNodes];
  float uniform[kMaxNodes];
  float logit[kMaxNodes], drafted[kMaxNodes];   // of the current node's children's tokens
};

// 16 bytes to another CTA's shared memory, counted on its mbarrier when they
// are there.  (A cluster barrier with its release costs ~1500 cycles on GB300,
// an exchange by it took 3000.)
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(addr),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
      : "memory");
}

// The largest top, the sums from it added in a fixed tree, and the largest
// best, over N lanes (a power of two).  c: the softmax's factor.  SUMS: two plain
// sums instead, in the same tree.
template <int N, bool SUMS>
__device__ __forceinline__ Found join_lanes(Found v, float c) {
  if constexpr (SUMS) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
      v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
      v.top += __shfl_xor_sync(0xffffffffu, v.top, o);
    }
    return v;
  }
  float top = v.top;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  v.sum *= top == -INFINITY ? 1.0f : exp2_approx((v.top - top) * c);
  v.top = top;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    v.sum += __shfl_xor_sync(0xffffffffu, v.sum, o);
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v.best, o);
    v.best = w > v.best ? w : v.best;
  }
  return v;
}

// The cluster's result from each thread's, into v: all threads of all its CTAs
// get the same, by the same additions.  Every second exchange uses the same
// buffers: a rank sends for the one after the next only when it has this CTA's
// results of the next, which are sent when all threads here have read the
// present ones.  False, for all threads of a CTA alike, when the wait for the
// other ranks gave up: v is then worth nothing, and the CTA has to leave
// (nothing more may be expected of a barrier whose phase is open, and threads
// that went on with different results could wait at different barriers).
template <bool SUMS>
__device__ __forceinline__ bool exchange(Found& v, float c, Shared& sh, int ranks, int rank, uint32_t& count,
                                         const VerifyArgs& a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t parity = count & 1, phase = count >> 1 & 1;
  v = join_lanes<32, SUMS>(v, c);
  if (lane == 0) sh.warp[parity][warp] = v;
  __syncthreads();
  v = join_lanes<kVerifyWarps, SUMS>(sh.warp[parity][lane % kVerifyWarps], c);
  if (ranks > 1) {
    volatile uint32_t* abort_flag = &sh.abort;
    const uint32_t bar = smem_u32(&sh.bar[parity]);
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, ranks * 16u);
    if (threadIdx.x < ranks && rank != a.silent)
      st_async_v4(mapa_shared(smem_u32(&sh.cta[parity][rank]), threadIdx.x), __float_as_uint(v.top),
                  __float_as_uint(v.sum), static_cast<uint32_t>(v.best), static_cast<uint32_t>(v.best >> 32),
                  mapa_shared(bar, threadIdx.x));
    const bool here = mbar_wait_bounded(bar, phase, abort_flag, a.err, a.wait_ns);
    if (!__syncthreads_and(here)) return false;
    v = Found{SUMS ? 0.0f : sh.cta[parity][0].top, 0.0f, 0};   // of a rank that is not there
    if ((lane & (kMaxCluster - 1)) < ranks) v = sh.cta[parity][lane & (kMaxCluster - 1)];
    v = join_lanes<kMaxCluster, SUMS>(v, c);
  }
  ++count;
  return true;
}

// r(x) of sampled drafts after the node's rejected children so far; q: the
// drafter's row's value at x, afterwards what is left of it.
__device__ __forceinline__ float residual(float r, float& q, int x, const Rejected* rejected, int n) {
  for (int j = 0; j < n; ++j) {
    const Rejected& e = rejected[j];
    if (!e.keeps) r = fmaxf(r * e.inv_mass - q * e.inv_rest, 0.0f);
    if (x == e.token) q = 0.0f;
  }
  return r;
}

// Every row begins on 16 bytes and holds whole groups of 8: a lane takes 8
// neighbouring tokens; else it takes every 32nd of the warp's block.
template <bool VEC>
__device__ __forceinline__ int token_of(int block, int lane, int j) {
  return block * kBlock + (VEC ? lane * 8 + j : j * 32 + lane);
}
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int block, int lane, int vocab, float (&f)[8]) {
  if constexpr (VEC) {
    const int x = token_of<true>(block, lane, 0);
    if (x < vocab) {
      if constexpr (sizeof(T) == 2) {
        widen8<T>(*reinterpret_cast<const uint4*>(row + x), f);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(row + x), b = *reinterpret_cast<const float4*>(row + x + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = token_of<false>(block, lane, j);
      if constexpr (sizeof(T) == 2)
        f[j] = x < vocab ? as_float(row[x]) : -INFINITY;
      else
        f[j] = x < vocab ? row[x] : -INFINITY;
    }
  }
}

// The same as packed 16-bit values; tokens past the end are -inf.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_raw(const T* row, int block, int lane, int vocab) {
  constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0xFC00u : 0xFF80u;
  uint4 r = make_uint4(kInf << 16 | kInf, kInf << 16 | kInf, kInf << 16 | kInf, kInf << 16 | kInf);
  if constexpr (VEC) {
    const int x = token_of<true>(block, lane, 0);
    if (x < vocab) r = *reinterpret_cast<const uint4*>(row + x);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = token_of<false>(block, lane, 2 * j), y = token_of<false>(block, lane, 2 * j + 1);
      w[j] = (x < vocab ? p[x] : kInf) | static_cast<uint32_t>(y < vocab ? p[y] : kInf) << 16;
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hmax2(x, y);
    memcpy(&a, &x, 4);
  } else {
    __nv_bfloat162 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hmax2(x, y);
    memcpy(&a, &x, 4);
  }
  return a;
}

__device__ __forceinline__ void prefetch_range(const void* begin, const void* end) {
  const uintptr_t a = (reinterpret_cast<uintptr_t>(begin) + 15) & ~uintptr_t{15};
  const uintptr_t b = reinterpret_cast<uintptr_t>(end) & ~uintptr_t{15};
  const uint64_t most = 1u << 20;
  if (b > a)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a),
                 "r"(static_cast<uint32_t>(b - a < most ? b - a : most))
                 : "memory");
}

// DRAFT: the drafts were drawn from `draft`; else they are certain.  (As a choice
// at run time the sums of q's rest, which certain drafts do not need, cost them
// spills: 48 trees 34 us instead of 29.)
template <typename T, bool VEC, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(VerifyArgs a, int ranks) {
  __shared__ __align__(16) Shared sh;
  const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = a.offsets[b];
  const int64_t end = a.offsets[b + 1];
  const bool bad = first < 0 || end > a.nodes || end - first > a.max_nodes || end < first;
  const int size = bad ? 0 : static_cast<int>(end - first);
  if (bad && rank == 0 && threadIdx.x == 0) atomicOr(a.err, kDevErrIndex);
  if (rank == 0)
    for (int i = threadIdx.x; i < a.max_nodes; i += kVerifyThreads)
      a.path[static_cast<int64_t>(b) * a.max_nodes + i] = size > 0 && i == 0 ? 0 : -1;
  if (size == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      a.count[b] = 0;
      a.next[b] = -1;
    }
    return;   // all CTAs of the cluster do
  }
  if (threadIdx.x < size) {
    sh.parent[threadIdx.x] = a.parents[first + threadIdx.x];
    sh.token[threadIdx.x] = a.tokens[first + threadIdx.x];
    sh.uniform[threadIdx.x] = a.uniforms[first + threadIdx.x];
  }
  if (threadIdx.x == 0) {
    sh.abort = 0;
    mbar_init(smem_u32(&sh.bar[0]), 1);
    mbar_init(smem_u32(&sh.bar[1]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  // the other CTAs' barriers must be there before they are sent anything
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  bool started = ranks == 1;
  const int blocks = (a.vocab + kBlock - 1) / kBlock;
  const int begin_block = static_cast<int>(static_cast<int64_t>(blocks) * rank / ranks);
  const int end_block = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / ranks);
  const int x0 = begin_block * kBlock, x1 = min(end_block * kBlock, a.vocab);
  const float temperature = a.temperature ? a.temperature[b] : 1.0f;
  const bool greedy = !(temperature > 0.0f);
  const float c = greedy ? 1.0f : 1.44269504f / temperature;   // softmax in powers of two
  const float* noise = a.noise + static_cast<int64_t>(b) * a.vocab;
  const T* logits = static_cast<const T*>(a.logits);
  if (threadIdx.x == 0 && !greedy && x0 < x1) prefetch_range(noise + x0, noise + x1);
  int now = 0, count = 1;
  uint32_t exchanges = 0;
  bool lost = false;   // a wait for the other ranks gave up
  for (;;) {
    const T* row = logits + (first + now) * a.logits_stride;
    const float* q = DRAFT ? a.draft + (first + now) * a.vocab : nullptr;
    // the children, in a word; what is asked of them below is fetched meanwhile
    uint64_t children;
    {
      const int i0 = now + 1 + lane, i1 = i0 + 32;
      const uint32_t lo = __ballot_sync(0xffffffffu, i0 < size && sh.parent[min(i0, kMaxNodes - 1)] == now);
      const uint32_t hi = __ballot_sync(0xffffffffu, i1 < size && sh.parent[min(i1, kMaxNodes - 1)] == now);
      children = static_cast<uint64_t>(hi) << 32 | lo;   // bit i: node now + 1 + i
    }
    if (children && threadIdx.x == 0 && x0 < x1) {
      const T* next = logits + (first + now + __ffsll(static_cast<long long>(children))) * a.logits_stride;
      prefetch_range(next + x0, next + x1);
    }
    if (threadIdx.x > now && threadIdx.x < size && sh.parent[threadIdx.x] == now) {
      const int x = sh.token[threadIdx.x];
      if (x >= 0 && x < a.vocab) {
        sh.logit[threadIdx.x] = as_float(row[x]);
        if (DRAFT) sh.drafted[threadIdx.x] = q[x];
      }
    }
    // ------------------------------------------------ maximum and sum, one pass
    Found v{-INFINITY, 0.0f, 0};
    for (int k = begin_block + warp; k < end_block; k += kVerifyWarps * kAtOnce) {
      uint4 raw[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)   // past the share: past the vocabulary
        raw[u] = load_raw<T, VEC>(row, k + u * kVerifyWarps, lane, k + u * kVerifyWarps < end_block ? a.vocab : 0);
      uint32_t high = raw[0].x;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        high = max2<T>(max2<T>(high, max2<T>(raw[u].x, raw[u].y)), max2<T>(raw[u].z, raw[u].w));
      float f[8];
      widen8<T>(make_uint4(high, high, high, high), f);
      const float top = fmaxf(v.top, fmaxf(f[0], f[1]));
      if (greedy) {
        if (top > v.top) {   // a later token with the same value is not the first maximum
#pragma unroll
          for (int u = kAtOnce - 1; u >= 0; --u) {
            widen8<T>(raw[u], f);
#pragma unroll
            for (int j = 7; j >= 0; --j)
              if (f[j] == top) v.best = pack_best(top, token_of<VEC>(k + u * kVerifyWarps, lane, j));
          }
        }
      } else {
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = v.sum * exp2_approx((v.top - base) * c);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          if (u > 0 && k + u * kVerifyWarps >= end_block) break;
          widen8<T>(raw[u], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += exp2_approx((f[j] - base) * c);
        }
        v.sum = sum;
      }
      v.top = top;
    }
    if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    started = true;
    lost = !exchange<false>(v, c, sh, ranks, rank, exchanges, a);
    if (lost) break;
    // an all -inf row has no maximum of its own: its first token stands for it
    const int hot = v.best ? static_cast<int>(best_index(v.best)) : 0;
    const float top = v.top;
    // a row of -inf alone is no distribution: nothing is accepted
    const float inv_sum = top == -INFINITY ? 0.0f : 1.0f / v.sum;
    auto prob = [&](float l) { return l == -INFINITY ? 0.0f : exp2_approx((l - top) * c) * inv_sum; };
    float mass = 1.0f, q_rest = 1.0f;   // Z and Q
    int rejected = 0, accepted = -1;
    uint64_t refused = 0;   // certain drafts: the rejected children, by node
    while (children) {
      const int i = now + __ffsll(static_cast<long long>(children));
      children &= children - 1;
      const int x = sh.token[i];
      if (x < 0 || x >= a.vocab) {
        if (threadIdx.x == 0 && rank == 0) atomicOr(a.err, kDevErrIndex);
        continue;
      }
      if (greedy) {
        if (x == hot) {
          accepted = i;
          break;
        }
        continue;
      }
      if (DRAFT && q_rest < kLeast) continue;
      const float u = sh.uniform[i];
      float qx = DRAFT ? sh.drafted[i] : 1.0f;
      float r = prob(sh.logit[i]);
      if (!DRAFT) {
        for (uint64_t m = refused; m; m &= m - 1)
          if (sh.token[__ffsll(static_cast<long long>(m)) - 1] == x) r = 0.0f;
        if (u * mass < r) {
          accepted = i;
          break;
        }
        refused |= uint64_t{1} << i;
        mass -= r;
        continue;
      }
      r = residual(r, qx, x, sh.rejected, rejected);
      const float inv_rest = 1.0f / q_rest;
      if (u * (qx * inv_rest) * mass < r) {
        accepted = i;
        break;
      }
      __syncthreads();
      if (threadIdx.x == 0) sh.rejected[rejected] = Rejected{1.0f / mass, inv_rest, x, 0};
      __syncthreads();
      ++rejected;
      Found rest{0.0f, 0.0f, 0};   // sums: of r, and of q in `top`
      for (int k = begin_block + warp; k < end_block; k += kVerifyWarps) {
        float f[8], g[8];
        load8<T, VEC>(row, k, lane, a.vocab, f);
        load8<float, VEC>(q, k, lane, a.vocab, g);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (token_of<VEC>(k, lane, j) < a.vocab) {
            rest.sum += residual(prob(f[j]), g[j], token_of<VEC>(k, lane, j), sh.rejected, rejected);
            rest.top += g[j];
          }
      }
      lost = !exchange<true>(rest, 0.0f, sh, ranks, rank, exchanges, a);
      if (lost) break;
      q_rest = rest.top;
      if (rest.sum < kLeast) {
        if (threadIdx.x == 0) sh.rejected[rejected - 1].keeps = 1;
        __syncthreads();
      } else {
        mass = rest.sum;
      }
    }
    if (lost) break;
    if (accepted >= 0) {
      if (rank == 0 && threadIdx.x == 0) a.path[static_cast<int64_t>(b) * a.max_nodes + count] = accepted;
      ++count;
      now = accepted;
      continue;
    }
    int next = hot;
    if (!greedy) {
      // the largest r / e at its lowest token; r's factor 1 / sum is left out
      // where nothing is subtracted from it
      const float base = top == -INFINITY ? 0.0f : top;
      float high = -1.0f;
      int at = 0;
      for (int k = begin_block + warp; k < end_block; k += kVerifyWarps * 2) {
        float f[2][8], e[2][8], g[2][8];
        uint64_t here[2] = {0, 0};   // rejected certain drafts among the block's tokens
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (k + u * kVerifyWarps < end_block) {
            load8<T, VEC>(row, k + u * kVerifyWarps, lane, a.vocab, f[u]);
            load8<float, VEC>(noise, k + u * kVerifyWarps, lane, a.vocab, e[u]);
            if (DRAFT) load8<float, VEC>(q, k + u * kVerifyWarps, lane, a.vocab, g[u]);
          }
        for (uint64_t m = refused; m; m &= m - 1) {
          const int i = __ffsll(static_cast<long long>(m)) - 1;
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (sh.token[i] / kBlock == k + u * kVerifyWarps) here[u] |= uint64_t{1} << i;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (k + u * kVerifyWarps >= end_block) continue;
          for (uint64_t m = here[u]; m; m &= m - 1) {
            const int x = sh.token[__ffsll(static_cast<long long>(m)) - 1];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (token_of<VEC>(k + u * kVerifyWarps, lane, j) == x) f[u][j] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int x = token_of<VEC>(k + u * kVerifyWarps, lane, j);
            float r = exp2_approx((f[u][j] - base) * c);
            if (DRAFT) r = residual(r * inv_sum, g[u][j], x, sh.rejected, rejected);
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(e[u][j]));
            const float key = x < a.vocab ? r * inv : -1.0f;
            if (key > high) {
              high = key;
              at = x;
            }
          }
        }
      }
      Found drawn_token{0.0f, 0.0f, high < 0.0f ? 0 : pack_best(high, at)};
      lost = !exchange<false>(drawn_token, 0.0f, sh, ranks, rank, exchanges, a);
      if (lost) break;
      next = static_cast<int>(best_index(drawn_token.best));
    }
    if (rank == 0 && threadIdx.x == 0) {
      a.count[b] = count;
      a.next[b] = next;
    }
    break;
  }
  if (lost) {
    // no walk to speak of: as a request without nodes
    if (rank == 0) {
      for (int i = threadIdx.x; i < a.max_nodes; i += kVerifyThreads)
        a.path[static_cast<int64_t>(b) * a.max_nodes + i] = -1;
      if (threadIdx.x == 0) {
        a.count[b] = 0;
        a.next[b] = -1;
      }
    }
    // The others may still send to this CTA: until they have given up too or
    // are through (each of their waits has its limit), and for as long as what
    // they sent last is on its way, microseconds.
    cluster_sync_all();
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000u) __nanosleep(1000);
  }
}

template <typename T, bool VEC, bool DRAFT>
cudaError_t launch_as(const VerifyArgs& a, int num_sms, cudaStream_t st) {
  // two CTAs fit an SM: as many per request as fit at once, and have a block of
  // tokens for each of their warps
  int ranks = kMaxCluster;
  while (ranks > 1 && (static_cast<int64_t>(a.requests) * ranks > 2 * num_sms ||
                       (a.vocab + kBlock - 1) / kBlock < ranks * kVerifyWarps / 2))
    ranks /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.requests) * ranks);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC, DRAFT>, a, ranks);
}
template <typename T, bool VEC>
cudaError_t launch_typed(const VerifyArgs& a, int num_sms, cudaStream_t st) {
  return a.draft ? launch_as<T, VEC, true>(a, num_sms, st) : launch_as<T, VEC, false>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_verify(const void* logits, int64_t logits_stride, bool bf16,
                          const int32_t* tokens, const int32_t* parents, const int32_t* offsets,
                          int requests, int64_t nodes, int vocab, int max_nodes,
                          const float* uniforms, const float* noise, const float* draft,
                          const float* temperature, int32_t* count, int32_t* path, int32_t* next,
                          int* err, int num_sms, cudaStream_t st, uint64_t wait_ns, int silent) {
  const VerifyArgs a{logits, logits_stride, tokens, parents, offsets, requests, nodes,
                     vocab,  max_nodes,     uniforms, noise, draft,   temperature, count,
                     path,   next,          err,      wait_ns, silent};
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = vocab % 8 == 0 && logits_stride % 8 == 0 && on16(logits) && on16(noise) && on16(draft);
  if (bf16)
    return vec ? launch_typed<__nv_bfloat16, true>(a, num_sms, st) : launch_typed<__nv_bfloat16, false>(a, num_sms, st);
  return vec ? launch_typed<__half, true>(a, num_sms, st) : launch_typed<__half, false>(a, num_sms, st);
}

}  // namespace cider
