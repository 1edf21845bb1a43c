// fp4_rows.cu -- products of microscaled 4-bit matrices for few tokens:
// y[m, n] = sum_k x[m, k] w[n, k], both E2M1 with block scales, on the
// block-scaled tensor cores.
//
// 128 rows of weights are the MMA's M, up to 128 tokens its N, so one token
// wastes tensor-core rows (which are free here) and no bytes: the weights are
// read once, straight from HBM into shared memory by TMA, and nothing converts
// them.  K is split over a cluster of CTAs, which add up their partial sums
// through distributed shared memory in the order of their ranks: no scratch in
// global memory, no second launch, the same bits each time.
//
// FUSE: up to 16 tokens whose rows this kernel quantizes itself, each CTA the
// part of K that it multiplies (block size 16 takes the row's maximum from the
// whole row, which every CTA reads), into the operand's place in shared memory:
// a decoding step's linear is one launch and needs no scratch.  Block size 16
// keeps all of x in registers, 16384 values at most: one token to K = 16384,
// four to 4096; block size 32 parts of 32768 values.
//
// Warp 0 copies (weights' stages before x is there: they do not depend on it),
// warp 1 issues scale copies and MMAs, the others quantize; warps 2..5 drain the
// accumulators, all warps add up and store.
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "fp4_common.cuh"

namespace cider {
namespace {

constexpr int kRMaxStages = 12;
constexpr int kROperand = 128 * 128;   // bytes of 128 rows of a stage's codes
constexpr int kRBars = 2 * kRMaxStages + 2;
constexpr int kRTail = kRBars * 8 + 16 + 2 * 16 * 4;   // barriers, flags, the fused rows' maxima and scales
constexpr int kRTokens = 16;                           // of the fused form
constexpr int kRQuantWarps = 8;
constexpr int kRThreads = 64 + 32 * kRQuantWarps;
constexpr int kRBatch = 4;
constexpr int kRMaxFusedStages = 16;                   // of a CTA's part of K, held whole

struct RowsArgs {
  int M, N, K;
  int tn;            // tokens of a tile: 16, 32, 64 or 128
  int m_tiles;       // token tiles (one, unless tn is 64 or 128)
  int splits;        // CTAs of a cluster
  int nkb;           // stages of K in all
  int nsteps;        // MMAs of K in all
  int stages;        // ring slots
  int stage_bytes, tok_offset, sfw_offset, sfu_offset, sft_offset;   // within a stage
  int x_offset, xs_offset;   // FUSE: all of the part's codes, and scales, of x
  int tail;          // barriers and what follows
  int sc_tiles;      // tiles of scales along K
  uint32_t tmem_cols;
  const uint8_t *scw, *scu, *scx;   // block scales
  const float *sx, *sw, *su;
  const void* x;     // FUSE
  int64_t x_stride;
  int x_bf16;
  void* y;
  int y_bf16, act;
  uint8_t *q_codes, *q_scales;      // or null
  int q_tiles;                      // tiles of scales along the outputs
  int* err;
};

// The part of the rows of x that this CTA multiplies, quantized into shared memory.  A thread asks for
// four units of 16 values before it works on the first; block size 16, which needs the rows' maxima,
// keeps all of x in registers until it has them.  `meet` is called when the first values are on their way:
// shared memory is not used before it.
template <typename T, int BS, typename F>
__device__ __forceinline__ void quantize_part(const RowsArgs& p, uint8_t* codes, uint8_t* scales, uint32_t* most,
                                              float* row, int kb0, int kb1, int thread, F&& meet) {
  constexpr int kThreads = 32 * kRQuantWarps, kBatch = kRBatch;
  const T* x = static_cast<const T*>(p.x);
  const int k0 = kb0 * kFpStageK;
  // 16 values' codes and (one of the threads that hold a block) their block's scale
  auto put = [&](int r, int k, const uint32_t (&c)[2], uint32_t byte, bool first) {
    const int kk = k & (kFpStageK - 1), kb = (k - k0) / kFpStageK;
    // 128-byte rows, their 16-byte pieces swizzled within groups of 8 rows
    uint8_t* at = codes + kb * (kRTokens * 128) + (r >> 3) * 1024 + (r & 7) * 128 + (((kk >> 5) ^ (r & 7)) << 4) +
                  ((kk >> 1) & 8);
    *reinterpret_cast<uint2*>(at) = make_uint2(c[0], c[1]);
    // tiles half as far apart as they are long: rows 16 .. 31 are not there
    if (first)
      scales[(kb * FpBlock<BS>::kTiles + kk / (4 * BS)) * (kFpTileBytes / 2) + 16 * r + (kk / BS & 3)] =
          static_cast<uint8_t>(byte);
  };
  if constexpr (BS == 16) {
    const int per = p.K >> 4, units = p.M * per;   // at most kBatch * kThreads
    const uint32_t magic = 0xFFFFFFFFu / per + 1u;   // u / per = the high half of u magic: u per < 2^32, per >= 2
    Sixteen<T> v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int u = j * kThreads + thread, r = __umulhi(u, magic);
      v[j].clear();
      if (u < units) v[j].template load<true>(x + r * p.x_stride + (u - r * per) * 16);
    }
    meet();
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (j * kThreads >= units) break;
      const int u = min(j * kThreads + thread, units - 1), r = __umulhi(u, magic);
      uint32_t top = v[j].top();
      if (__all_sync(0xffffffffu, r == __shfl_sync(0xffffffffu, r, 0))) {
        top = __reduce_max_sync(0xffffffffu, top);
        if ((thread & 31) == 0) atomicMax(most + r, top);
      } else {
        atomicMax(most + r, top);
      }
    }
    named_barrier_sync(1, kThreads);
    if (thread < p.M) row[thread] = row_scale(most[thread]);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int u = j * kThreads + thread, r = __umulhi(u, magic), k = (u - r * per) * 16;
      if (u >= units || k < k0 || k >= kb1 * kFpStageK) continue;
      uint32_t c[2] = {0u, 0u}, byte = 0u;
      if (!not_finite(most[r])) byte = encode16<T, BS>(v[j], v[j].top(), pow2(-row_power(most[r])), c);
      put(r, k, c, byte, true);
    }
    // zeros up to a whole step of 64
    if (kb1 == p.nkb && (p.K & 32) != 0 && thread < 2 * p.M) {
      const uint32_t c[2] = {0u, 0u};
      put(thread >> 1, p.K + 16 * (thread & 1), c, 0u, true);
    }
  } else {
    // whole steps of 64: zeros behind the end of the row
    const int k1 = min(kb1 * kFpStageK, p.nsteps * kFpStepK);
    const int per = (k1 - k0) >> 4, units = p.M * per;   // a multiple of 4: a block's two threads stay together
    const uint32_t magic = 0xFFFFFFFFu / per + 1u;
    for (int u0 = 0; u0 < units; u0 += kBatch * kThreads) {
      Sixteen<T> v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int u = u0 + j * kThreads + thread, r = __umulhi(u, magic), k = k0 + 16 * (u - r * per);
        v[j].clear();
        if (u < units && k < p.K) v[j].template load<true>(x + r * p.x_stride + k);
      }
      if (u0 == 0) meet();
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int u = u0 + j * kThreads + thread, r = __umulhi(u, magic), k = k0 + 16 * (u - r * per);
        uint32_t top = v[j].top();
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        uint32_t c[2] = {0u, 0u};
        const uint32_t byte = encode16<T, BS>(v[j], top, 1.0f, c);
        if (u < units) put(r, k, c, byte, (u & 1) == 0);
      }
    }
  }
}

// Four rounded outputs from n on of token m, of a block of the quantized matrix that eight neighbouring
// threads hold.
__device__ __forceinline__ void store_quantized(const RowsArgs& p, int64_t m, int n, uint2 w, int lane) {
  const uint32_t group = 0xFFu << (lane & 24);
  const uint32_t both_tops = max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu);
  uint32_t top = max(both_tops & 0xFFFFu, both_tops >> 16);
#pragma unroll
  for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(group, top, o));
  float f[4];
  if (p.y_bf16) {
    top <<= 16;
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xFFFF0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xFFFF0000u);
  } else {
    top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&w.x)),
                 hi = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    f[0] = lo.x;
    f[1] = lo.y;
    f[2] = hi.x;
    f[3] = hi.y;
  }
  const bool bad = not_finite(top);
  const int e = bad ? 0 : block_power(top);
  const float inv = pow2(-e);
  const uint64_t q[4] = {pack2(__float_as_uint(f[0] * inv), __float_as_uint(f[1] * inv)),
                         pack2(__float_as_uint(f[2] * inv), __float_as_uint(f[3] * inv)), 0ull, 0ull};
  *reinterpret_cast<uint16_t*>(p.q_codes + m * (p.N >> 1) + (n >> 1)) =
      bad ? uint16_t{0} : static_cast<uint16_t>(e2m1x8(q));
  if ((lane & 7) == 0) {
    uint8_t* at = p.q_scales + scale_at(m, n >> 5, p.q_tiles);
    *at = bad ? uint8_t{0xFF} : static_cast<uint8_t>(e + 127);
    // the other block of a step of 64 that the row ends in
    if (n + 32 == p.N && (p.N & 32) != 0) at[1] = 0;
  }
}

template <bool GATED, int BS, bool FUSE>
__global__ void __launch_bounds__(kRThreads, 2)
    fp4_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_u,
                    const __grid_constant__ CUtensorMap tm_x, const RowsArgs p) {
  using B = FpBlock<BS>;
  constexpr int kThreads = kRThreads;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + p.tail;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kRMaxStages + s); };
  const uint32_t acc_bar = bars + 8u * (2 * kRMaxStages);
  const uint32_t x_bar = bars + 8u * (2 * kRMaxStages + 1);
  const uint32_t tmem_slot = bars + 8u * kRBars;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + p.tail + 8 * kRBars + 4);
  uint32_t* most = reinterpret_cast<uint32_t*>(gbase + p.tail + 8 * kRBars + 16);
  float* row = reinterpret_cast<float*>(most + kRTokens);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the rank in the cluster; of blockIdx, so that the compiler knows it to be the same for all threads
  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int unit = blockIdx.x / p.splits;
  const int mt = unit % p.m_tiles, nt = unit / p.m_tiles;
  const int m0 = mt * p.tn;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * p.nkb / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.nkb / p.splits);

  // bytes of scales that a stage has (the last one may have fewer tiles)
  auto scale_bytes = [&](int kb) { return min(B::kTiles, p.sc_tiles - kb * B::kTiles) * kFpTileBytes; };
  auto weights = [&](int kb, int s) {
    const uint32_t at = base + s * p.stage_bytes, sb = scale_bytes(kb);
    const int64_t from = (static_cast<int64_t>(nt) * p.sc_tiles + kb * B::kTiles) * kFpTileBytes;
    mbar_arrive_expect_tx(full_bar(s), (GATED ? 2u : 1u) * (kROperand + sb) + (FUSE ? 0u : p.tn * 128u + sb));
    tma_load_2d(at, &tm_w, full_bar(s), kb * 128, nt * 128);
    if (GATED) tma_load_2d(at + kROperand, &tm_u, full_bar(s), kb * 128, nt * 128);
    bulk_load(at + p.sfw_offset, p.scw + from, sb, full_bar(s));
    if (GATED) bulk_load(at + p.sfu_offset, p.scu + from, sb, full_bar(s));
  };
  const int ahead = min(kb1 - kb0, p.stages);   // stages whose slots nothing has used before
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(full_bar(s), 1);
        mbar_init(empty_bar(s), 1);
      }
      mbar_init(acc_bar, 1);
      mbar_init(x_bar, kRQuantWarps);
      *abort_flag = 0u;
      fence_mbar_init();
    }
    __syncwarp();
    named_barrier_arrive(2, kThreads);   // this warp needs nothing of what the others set up
    if (elect_one())
      for (int i = 0; i < ahead; ++i) weights(kb0 + i, i);
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  // barriers initialised, tensor memory held
  auto meet = [&] {
    tc_fence_before();
    named_barrier_sync(2, kThreads);
    tc_fence_after();
  };
  if (FUSE && warp >= 2) {
    // ------------------------------------------------------------ quantization of x
    const int thread = threadIdx.x - 64;
    if (thread < kRTokens) most[thread] = 0u;
    pdl_wait();   // x may be what the launch just before wrote
    if (p.x_bf16)
      quantize_part<__nv_bfloat16, BS>(p, gbase + p.x_offset, gbase + p.xs_offset, most, row, kb0, kb1, thread, meet);
    else
      quantize_part<__half, BS>(p, gbase + p.x_offset, gbase + p.xs_offset, most, row, kb0, kb1, thread, meet);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(x_bar);
  } else if (warp >= 1) {
    meet();
  }
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + p.tail + 8 * kRBars);
  const int acc_cols = GATED ? 2 * p.tn : p.tn;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (elect_one()) {
      auto tokens = [&](int kb, int s) {
        const uint32_t at = base + s * p.stage_bytes, sb = scale_bytes(kb);
        tma_load_2d(at + p.tok_offset, &tm_x, full_bar(s), kb * 128, m0);
        bulk_load(at + p.sft_offset,
                  p.scx + (static_cast<int64_t>(m0 >> 7) * p.sc_tiles + kb * B::kTiles) * kFpTileBytes, sb, full_bar(s));
      };
      if (!FUSE) {
        pdl_wait();
        for (int i = 0; i < ahead; ++i) tokens(kb0 + i, i);
      }
      int i = ahead;
      for (; kb0 + i < kb1; ++i) {
        const int s = i % p.stages;
        if (!mbar_wait_bounded(empty_bar(s), ((i / p.stages) & 1) ^ 1u, abort_flag, p.err, kFpWaitNs)) break;
        weights(kb0 + i, s);
        if (!FUSE) tokens(kb0 + i, s);
      }
      // what was issued has landed before the CTA leaves, also after a wait that gave up
      volatile uint32_t keep_waiting = 0u;
      for (int j = max(0, i - p.stages); j < i; ++j)
        mbar_wait_bounded(full_bar(j % p.stages), (j / p.stages) & 1, &keep_waiting, p.err, kFpWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const uint32_t sfw = tmem + acc_cols, sfu = sfw + B::kCols, sft = sfw + (GATED ? 2 : 1) * B::kCols;
    const uint32_t sfm = sft + ((m0 >> 5) & 3);   // 64 tokens may start in the middle of a tile of scales
    if (elect_one()) {   // one lane runs the whole loop
      int s = 0, i = 0;
      uint32_t phase = 0;
      bool go = !FUSE || mbar_wait_bounded(x_bar, 0, abort_flag, p.err, kFpWaitNs);
      // a stage: its scales, then `steps` MMAs (a weight tile's each)
      auto stage = [&](auto full, int steps, bool first) {
        if (!mbar_wait_bounded(full_bar(s), phase, abort_flag, p.err, kFpWaitNs)) {
          go = false;
          return;
        }
        tc_fence_after();
        const uint32_t at = base + s * p.stage_bytes;
        const uint64_t dw = smem_desc_scales(at + p.sfw_offset), du = smem_desc_scales(at + p.sfu_offset);
        // FUSE: tiles of scales half as far apart as they are long
        constexpr int kPitch = FUSE ? kFpTileBytes / 2 : kFpTileBytes;
        const uint64_t dt = smem_desc_scales(FUSE ? base + p.xs_offset + i * B::kTiles * kPitch : at + p.sft_offset);
#pragma unroll
        for (int a = 0; a < B::kTiles; ++a) {
          tc_cp_scales<1>(sfw + 4 * a, dw + a * (kFpTileBytes >> 4));
          if (GATED) tc_cp_scales<1>(sfu + 4 * a, du + a * (kFpTileBytes >> 4));
          tc_cp_scales<1>(sft + 4 * a, dt + a * (kPitch >> 4));
        }
        const uint64_t wd = smem_desc_k_sw128(at), ud = smem_desc_k_sw128(at + kROperand),
                       td = smem_desc_k_sw128(FUSE ? base + p.x_offset + i * (kRTokens * 128) : at + p.tok_offset);
#pragma unroll
        for (int j = 0; j < kFpSteps; ++j) {
          if (!decltype(full)::value && j >= steps) break;
          const int a = BS == 16 ? j : j >> 1, id = BS == 16 ? 0 : 2 * (j & 1);
          const uint32_t idesc = idesc_fp4<BS>(128, FUSE ? kRTokens : p.tn, id), acc = first && j == 0 ? 0u : 1u;
          tc_mma_fp4<1, BS>(tmem, wd + 2 * j, td + 2 * j, idesc, sfw + 4 * a, sfm + 4 * a, acc);
          if (GATED) tc_mma_fp4<1, BS>(tmem + p.tn, ud + 2 * j, td + 2 * j, idesc, sfu + 4 * a, sfm + 4 * a, acc);
        }
        tc_commit(empty_bar(s));
        ++i;
        if (++s == p.stages) {
          s = 0;
          phase ^= 1u;
        }
      };
      // a test per MMA would cost more than its issue: only the last stage, when it is not full, has them
      const int full_end = min(kb1, p.nsteps / kFpSteps);
      for (int kb = kb0; kb < full_end && go; ++kb) stage(std::true_type{}, kFpSteps, kb == kb0);
      if (full_end < kb1 && go) stage(std::false_type{}, p.nsteps - full_end * kFpSteps, full_end == kb0);
      tc_commit(acc_bar);
    }
    __syncwarp();
  }
  // ---------------------------------------------------------------- sums
  // Every MMA that was issued has run (also after a wait that gave up); then the ring is free and
  // takes the partial sums [accumulator column][weight row].
  const int mv = min(p.tn, p.M - m0);
  float* part = reinterpret_cast<float*>(gbase);
  // four weight rows of a token at a time, the same four for a thread; the cluster's CTAs take equal shares
  // in blocks of 32 outputs (eight threads)
  const int u0 = 8 * (rank * mv * 4 / p.splits), u1 = 8 * ((rank + 1) * mv * 4 / p.splits);
  const int row0 = nt * 128 + 4 * ((u0 + static_cast<int>(threadIdx.x)) & 31);
  float sw[4], su[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sw[i] = p.sw && row0 < p.N ? __ldg(p.sw + row0 + i) : 1.0f;
    su[i] = GATED && p.su && row0 < p.N ? __ldg(p.su + row0 + i) : 1.0f;
  }
  pdl_wait();
  __syncthreads();   // the copies have landed: an abort leaves none in flight
  bool ok;
  {
    volatile uint32_t keep_waiting = 0u;
    ok = mbar_wait_bounded(acc_bar, 0, &keep_waiting, p.err, kFpWaitNs);
  }
  ok = __syncthreads_and(ok && *abort_flag == 0u);
  if (ok && warp >= 2 && warp < 6) {
    tc_fence_after();
    const int q = warp & 3, n = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    for (int c = 0; c < acc_cols; c += 32) {
      // columns of tokens behind the last one are not needed
      if (p.tn >= 32 && (c & (p.tn - 1)) >= mv) continue;
      uint32_t v[32];
      tmem_ld32(tmem + lane_base + c, v);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < acc_cols) part[(c + i) * 128 + n] = __uint_as_float(v[i]);
    }
    tc_fence_before();
  }
  if (p.splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  // U tokens' and kAsk ranks' partial sums are asked for before the first is added
  auto finish = [&](auto tokens, auto ranks) {
    constexpr int U = decltype(tokens)::value, kAsk = decltype(ranks)::value, kSides = GATED ? 2 : 1;
    for (int u = u0 + static_cast<int>(threadIdx.x); u < u1; u += U * kThreads) {
      float a[U][4 * kSides], sx[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int t = (u + k * kThreads) >> 5;
        const bool have = u + k * kThreads < u1;
        sx[k] = FUSE ? (BS == 16 && have ? row[t] : 1.0f) : p.sx && have ? ld_global_f32(p.sx + m0 + t) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4 * kSides; ++i) a[k][i] = 0.0f;
      }
#pragma unroll
      for (int r0 = 0; r0 < 8; r0 += kAsk) {
        if (r0 >= p.splits) break;
        float4 f[U][kAsk][kSides];
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int r = 0; r < kAsk; ++r)
            if (r0 + r < p.splits && u + k * kThreads < u1) {
#pragma unroll
              for (int h = 0; h < kSides; ++h) {
                const int at = (h * p.tn + ((u + k * kThreads) >> 5)) * 128 + 4 * (u & 31);
                f[k][r][h] = p.splits > 1 ? ld_cluster_v4(mapa_shared(base + 4u * at, r0 + r))
                                          : *reinterpret_cast<const float4*>(part + at);
              }
            }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int r = 0; r < kAsk; ++r)
            if (r0 + r < p.splits && u + k * kThreads < u1) {
#pragma unroll
              for (int h = 0; h < kSides; ++h) {
                a[k][4 * h] += f[k][r][h].x;
                a[k][4 * h + 1] += f[k][r][h].y;
                a[k][4 * h + 2] += f[k][r][h].z;
                a[k][4 * h + 3] += f[k][r][h].w;
              }
            }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (u + k * kThreads >= u1) break;
        const int t = (u + k * kThreads) >> 5;
        float out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          out[i] = a[k][i] * sx[k] * sw[i];
          if constexpr (GATED) out[i] = gated(out[i], a[k][4 + i] * sx[k] * su[i], p.act);
        }
        uint2 w;
        if (p.y_bf16) {
          w = make_uint2(y_bits2<true>(out[0], out[1]), y_bits2<true>(out[2], out[3]));
        } else {
          w = make_uint2(y_bits2<false>(out[0], out[1]), y_bits2<false>(out[2], out[3]));
        }
        if (GATED && BS == 32 && p.q_codes)
          store_quantized(p, m0 + t, row0, w, lane);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + static_cast<int64_t>(m0 + t) * p.N + row0) = w;
      }
    }
  };
  if (ok && row0 < p.N) {   // N % 8 == 0: four weight rows are all in or all out
    if (p.splits <= 2)
      finish(std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
    else
      finish(std::integral_constant<int, 1>{}, std::integral_constant<int, GATED ? 4 : 8>{});
  }
  __syncwarp();
  // the partial sums stay until every CTA has read them (what was stored need not be seen by then)
  if (p.splits > 1) cluster_sync_relaxed();
}

template <bool GATED, int BS, bool FUSE>
cudaError_t launch(const FpProduct& p, RowsArgs& a, int smem, int tiles) {
  CUtensorMap mw, mu, mx;
  auto codes = [&](CUtensorMap* m, const FpMat& q, int rows) {
    return make_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, p.K / 2, q.rows, p.K / 2, 128, rows,
                              CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!codes(&mw, p.w, 128)) return cudaErrorInvalidValue;
  mu = mx = mw;
  if ((GATED && !codes(&mu, p.up, 128)) || (!FUSE && !codes(&mx, p.x, a.tn))) return cudaErrorInvalidValue;
  auto kern = fp4_rows_kernel<GATED, BS, FUSE>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), 232448, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits), 1, 1);
  cfg.blockDim = dim3(kRThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = p.st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (a.splits > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = a.splits;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (p.after_launch) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, mw, mu, mx, a);
}

// The launch's sizes; false: a part of K that the fused form does not hold.
bool plan(const FpProduct& p, bool fuse, RowsArgs& a, int* smem_out, int* tiles_out) {
  const int sides = p.is_gated ? 2 : 1;
  const int per_tiles = kFpStageK / (4 * p.block), bytes = per_tiles * kFpTileBytes, cols_side = per_tiles * 4;
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.K = static_cast<int>(p.K);
  // up to 64 tokens in one tile; more by 64 where that leaves two CTAs' worth of SMs to each tile, else by 128
  const int n_tiles = static_cast<int>((p.N + 127) / 128);
  a.tn = 16;
  while (a.tn < 64 && a.tn < p.M) a.tn *= 2;
  if (p.M > 64 && (p.M + 63) / 64 * n_tiles > p.num_sms / 2) a.tn = 128;
  a.m_tiles = static_cast<int>((p.M + a.tn - 1) / a.tn);
  a.nkb = static_cast<int>((p.K + kFpStageK - 1) / kFpStageK);
  a.nsteps = static_cast<int>((p.K + kFpStepK - 1) / kFpStepK);
  a.sc_tiles = fp4_tiles(p.K, p.block);
  a.tok_offset = sides * kROperand;
  a.sfw_offset = a.tok_offset + (fuse ? 0 : a.tn * 128);
  a.sfu_offset = a.sfw_offset + bytes;
  a.sft_offset = a.sfw_offset + sides * bytes;
  a.stage_bytes = (a.sft_offset + (fuse ? 0 : bytes) + 1023) / 1024 * 1024;
  const int cols = sides * a.tn + (sides + 1) * cols_side;   // at most 176
  a.tmem_cols = 64;
  while (static_cast<int>(a.tmem_cols) < cols) a.tmem_cols *= 2;
  // As many CTAs as SMs, or a few more, K split in a power of two.  Measured (two more splits, a CTA
  // or two on each SM): one token through 4096 x 4096, 32 tiles in 4 parts 5.7 us, in 8 parts 7.4; 16
  // through 2560 x 10240, 20 tiles in 8 parts 10.6, in 4 parts 11.8; 128 through 10240 x 2560, 80 tiles
  // in 2 parts 12.9, whole 14.3.  Other numbers of parts lose 5 us to the placing of their clusters.
  // Clusters of 4 and of 8 do not reach every SM (144 and 120 of 152 with a CTA on each).  Where there are
  // more CTAs than that they share SMs in pairs: they hold at most half of the tensor memory, and their shared
  // memory allows two and no third.  All others have an SM to themselves.  So no CTA of a cluster waits for
  // tensor memory that another cluster's holds.
  const int tiles = a.m_tiles * n_tiles;
  a.splits = 1;
  while (a.splits < 8 && a.nkb >= a.splits * 4 && tiles * a.splits * 2 <= p.num_sms + p.num_sms / 16) a.splits *= 2;
  const bool two = tiles * a.splits > (a.splits == 8   ? p.num_sms * 3 / 4
                                       : a.splits == 4 ? p.num_sms * 15 / 16
                                                       : p.num_sms);
  const int budget = two ? 110 * 1024 : 224 * 1024;
  const int mine = (a.nkb + a.splits - 1) / a.splits;   // stages of a CTA, at most
  int held = 0;
  if (fuse) {
    if (p.M > kRTokens || mine > kRMaxFusedStages) return false;
    // All of x in the threads' registers (block size 16), or a part that is soon done: 16 tokens' parts of
    // 1280 values cost 3 us more than rows that are quantized already, of 4096 values 5 us; a launch of its
    // own 1 us, and the caller 6 us of host time.
    const int64_t values = p.block == 16 ? p.M * p.K : p.M * mine * kFpStageK;
    if (values > (p.block == 16 ? 16 * kRBatch * 32 * kRQuantWarps : 32768)) return false;
    // the last tile of scales is read to its end, half a tile behind the next one's start
    held = mine * (kRTokens * 128) + (mine * per_tiles + 1) * (kFpTileBytes / 2);
    held = (held + 1023) / 1024 * 1024;
  }
  a.stages = (budget - held) / a.stage_bytes;
  if (a.stages > kRMaxStages) a.stages = kRMaxStages;
  a.x_offset = a.stages * a.stage_bytes;
  a.xs_offset = a.x_offset + mine * (kRTokens * 128);
  a.tail = a.x_offset + held;
  int smem = a.tail + kRTail + 1024;
  if (two && smem < 79 * 1024) smem = 79 * 1024;
  a.scw = p.w.scales;
  a.scu = p.up.scales;
  a.scx = p.x.scales;
  a.sx = p.x.row;
  a.sw = p.w.row;
  a.su = p.up.row;
  a.x = p.wide_x;
  a.x_stride = p.x_stride;
  a.x_bf16 = p.x_bf16;
  a.y = p.y;
  a.y_bf16 = p.y_bf16;
  a.act = p.act;
  a.q_codes = p.q_codes;
  a.q_scales = p.q_scales;
  a.q_tiles = fp4_tiles(p.N, 32);
  *smem_out = smem;
  *tiles_out = tiles;
  return true;
}

}  // namespace

bool fp4_rows_quantizes_itself(const FpProduct& p) {
  RowsArgs a{};
  int smem, tiles;
  return plan(p, true, a, &smem, &tiles);
}

cudaError_t launch_fp4_rows(const FpProduct& p) {
  RowsArgs a{};
  int smem = 0, tiles = 0;
  const bool fuse = p.wide_x != nullptr;
  if (!plan(p, fuse, a, &smem, &tiles)) return cudaErrorInvalidValue;
  const cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  auto go = [&](auto gated_, auto block) {
    constexpr bool G = decltype(gated_)::value;
    constexpr int BS = decltype(block)::value;
    return fuse ? launch<G, BS, true>(p, a, smem, tiles) : launch<G, BS, false>(p, a, smem, tiles);
  };
  using B16 = std::integral_constant<int, 16>;
  using B32 = std::integral_constant<int, 32>;
  if (p.is_gated) return p.block == 16 ? go(std::true_type{}, B16{}) : go(std::true_type{}, B32{});
  return p.block == 16 ? go(std::false_type{}, B16{}) : go(std::false_type{}, B32{});
}

}  // namespace cider
