// fp4_rows.cu -- products of microscaled 4-bit matrices for few tokens:
// y[m, n] = sum_k x[m, k] w[n, k], both E2M1 with block scales, on the
// block-scaled tensor cores.
//
// 128 rows of weights are the MMA's M, up to 256 tokens its N, so one token
// wastes tensor-core rows (which are free here) and no bytes: the weights are
// read once, straight from HBM into shared memory by TMA, and nothing converts
// them.  K is split over a cluster of CTAs, which add up their partial sums
// through distributed shared memory in the order of their ranks: no scratch in
// global memory, no second launch, the same bits each time.
//
// Warp 0 copies (weights' stages before the quantization of x has ended: they
// do not depend on it), warp 1 issues scale copies and MMAs, warps 2..5 drain
// the accumulators; all warps add up and store.
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "fp4_common.cuh"

namespace cider {
namespace {

constexpr int kRThreads = 192;
constexpr int kRMaxStages = 12;
constexpr int kROperand = 128 * 128;   // bytes of 128 rows of a stage's codes
constexpr int kRBars = 2 * kRMaxStages + 1;
constexpr int kRTail = kRBars * 8 + 16;

struct RowsArgs {
  int M, N;
  int tn;            // tokens of a tile: 16, 32, 64, 128 or 256
  int m_tiles;       // token tiles (one, unless tn is 128 or 256)
  int splits;        // CTAs of a cluster
  int nkb;           // stages of K in all
  int nsteps;        // MMAs of K in all
  int stages;        // ring slots
  int stage_bytes, tok_offset, sfw_offset, sfu_offset, sft_offset;   // within a stage
  int tok_tiles;     // 128-row tiles of the tokens' scales in a stage: 1 or 2
  uint32_t tmem_cols;
  const float *sx, *sw, *su;
  void* y;
  int y_bf16, act;
  int* err;
};

template <bool GATED, int BS>
__global__ void __launch_bounds__(kRThreads, 1)
    fp4_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_u,
                    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_sw,
                    const __grid_constant__ CUtensorMap tm_su, const __grid_constant__ CUtensorMap tm_sx,
                    const RowsArgs p) {
  using B = FpBlock<BS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int ring = p.stages * p.stage_bytes;
  const uint32_t bars = base + ring;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kRMaxStages + s); };
  const uint32_t acc_bar = bars + 8u * (2 * kRMaxStages);
  const uint32_t tmem_slot = bars + 8u * kRBars;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + ring + 8 * kRBars + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the rank in the cluster; of blockIdx, so that the compiler knows it to be the same for all threads
  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int unit = blockIdx.x / p.splits;
  const int mt = unit % p.m_tiles, nt = unit / p.m_tiles;
  const int m0 = mt * p.tn;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * p.nkb / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.nkb / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + ring + 8 * kRBars);
  const int acc_cols = GATED ? 2 * p.tn : p.tn;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      const uint32_t bytes = (GATED ? 2u : 1u) * (kROperand + B::kBytes) + p.tn * 128 + p.tok_tiles * B::kBytes;
      auto weights = [&](int kb, int s) {
        const uint32_t at = base + s * p.stage_bytes;
        mbar_arrive_expect_tx(full_bar(s), bytes);
        tma_load_2d(at, &tm_w, full_bar(s), kb * 128, nt * 128);
        tma_load_2d(at + p.sfw_offset, &tm_sw, full_bar(s), kb * (B::kBytes / 8), nt);
        if (GATED) {
          tma_load_2d(at + kROperand, &tm_u, full_bar(s), kb * 128, nt * 128);
          tma_load_2d(at + p.sfu_offset, &tm_su, full_bar(s), kb * (B::kBytes / 8), nt);
        }
      };
      auto tokens = [&](int kb, int s) {
        const uint32_t at = base + s * p.stage_bytes;
        tma_load_2d(at + p.tok_offset, &tm_x, full_bar(s), kb * 128, m0);
        for (int t = 0; t < p.tok_tiles; ++t)
          tma_load_2d(at + p.sft_offset + t * B::kBytes, &tm_sx, full_bar(s), kb * (B::kBytes / 8), (m0 >> 7) + t);
      };
      const int ahead = min(kb1 - kb0, p.stages);
      for (int i = 0; i < ahead; ++i) weights(kb0 + i, i);
      pdl_wait();
      for (int i = 0; i < ahead; ++i) tokens(kb0 + i, i);
      int i = ahead;
      for (; kb0 + i < kb1; ++i) {
        const int s = i % p.stages;
        if (!mbar_wait_bounded(empty_bar(s), ((i / p.stages) & 1) ^ 1u, abort_flag, p.err, kFpWaitNs)) break;
        weights(kb0 + i, s);
        tokens(kb0 + i, s);
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
    const uint32_t tcols = 4 * p.tok_tiles;   // columns of the tokens' scales of one tile of K
    if (elect_one()) {   // one lane runs the whole loop
      int s = 0;
      uint32_t phase = 0;
      bool go = true;
      // a stage: its scales, then `steps` MMAs (a weight tile's each)
      auto stage = [&](auto full, int steps, bool first) {
        if (!mbar_wait_bounded(full_bar(s), phase, abort_flag, p.err, kFpWaitNs)) {
          go = false;
          return;
        }
        tc_fence_after();
        const uint32_t at = base + s * p.stage_bytes;
        const uint64_t dw = smem_desc_scales(at + p.sfw_offset), du = smem_desc_scales(at + p.sfu_offset),
                       dt = smem_desc_scales(at + p.sft_offset);
#pragma unroll
        for (int a = 0; a < B::kTiles; ++a) {
          tc_cp_scales<1>(sfw + 4 * a, dw + a * (kFpTileBytes >> 4));
          if (GATED) tc_cp_scales<1>(sfu + 4 * a, du + a * (kFpTileBytes >> 4));
          tc_cp_scales<1>(sft + tcols * a, dt + a * (kFpTileBytes >> 4));
        }
        if (p.tok_tiles == 2)
#pragma unroll
          for (int a = 0; a < B::kTiles; ++a)
            tc_cp_scales<1>(sft + tcols * a + 4, dt + ((B::kBytes + a * kFpTileBytes) >> 4));
        const uint64_t wd = smem_desc_k_sw128(at), ud = smem_desc_k_sw128(at + kROperand),
                       td = smem_desc_k_sw128(at + p.tok_offset);
#pragma unroll
        for (int j = 0; j < kFpSteps; ++j) {
          if (!decltype(full)::value && j >= steps) break;
          const int a = BS == 16 ? j : j >> 1, id = BS == 16 ? 0 : 2 * (j & 1);
          const uint32_t idesc = idesc_fp4<BS>(128, p.tn, id), acc = first && j == 0 ? 0u : 1u;
          tc_mma_fp4<1, BS>(tmem, wd + 2 * j, td + 2 * j, idesc, sfw + 4 * a, sft + tcols * a, acc);
          if (GATED) tc_mma_fp4<1, BS>(tmem + p.tn, ud + 2 * j, td + 2 * j, idesc, sfu + 4 * a, sft + tcols * a, acc);
        }
        tc_commit(empty_bar(s));
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
  pdl_wait();
  __syncthreads();   // the copies have landed: an abort leaves none in flight
  bool ok;
  {
    volatile uint32_t keep_waiting = 0u;
    ok = mbar_wait_bounded(acc_bar, 0, &keep_waiting, p.err, kFpWaitNs);
  }
  ok = __syncthreads_and(ok && *abort_flag == 0u);
  if (ok && warp >= 2) {
    tc_fence_after();
    const int q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    for (int c = 0; c < acc_cols; c += 32) {
      // columns of tokens behind the last one are not needed
      if (p.tn >= 32 && (c & (p.tn - 1)) >= mv) continue;
      uint32_t v[32];
      tmem_ld32(tmem + lane_base + c, v);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < acc_cols) part[(c + i) * 128 + row] = __uint_as_float(v[i]);
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
  if (ok) {
    // four weight rows of a token at a time; the cluster's CTAs take equal shares
    const int units = mv * 32;
    const int u0 = static_cast<int>(static_cast<int64_t>(rank) * units / p.splits);
    const int u1 = static_cast<int>(static_cast<int64_t>(rank + 1) * units / p.splits);
    for (int u = u0 + static_cast<int>(threadIdx.x); u < u1; u += kRThreads) {
      const int t = u >> 5, n = nt * 128 + 4 * (u & 31);
      if (n >= p.N) continue;   // N % 8 == 0: four rows are all in or all out
      float a[GATED ? 8 : 4];
#pragma unroll
      for (int i = 0; i < (GATED ? 8 : 4); ++i) a[i] = 0.0f;
      for (int r = 0; r < p.splits; ++r) {
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
          const uint32_t local = base + static_cast<uint32_t>(((h * p.tn + t) * 128 + 4 * (u & 31)) * 4);
          float4 f;
          asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                       : "r"(mapa_shared(local, p.splits > 1 ? r : 0))
                       : "memory");
          a[4 * h] += f.x;
          a[4 * h + 1] += f.y;
          a[4 * h + 2] += f.z;
          a[4 * h + 3] += f.w;
        }
      }
      const float sx = p.sx ? __ldg(p.sx + m0 + t) : 1.0f;
      float out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = a[i] * sx * (p.sw ? __ldg(p.sw + n + i) : 1.0f);
        if (GATED) out[i] = gated(out[i], a[(GATED ? 4 : 0) + i] * sx * (p.su ? __ldg(p.su + n + i) : 1.0f), p.act);
      }
      uint2 w;
      if (p.y_bf16) {
        w = make_uint2(y_bits2<true>(out[0], out[1]), y_bits2<true>(out[2], out[3]));
      } else {
        w = make_uint2(y_bits2<false>(out[0], out[1]), y_bits2<false>(out[2], out[3]));
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + static_cast<int64_t>(m0 + t) * p.N + n) = w;
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();   // the partial sums stay until every CTA has read them
}

template <bool GATED, int BS>
cudaError_t launch(const FpProduct& p) {
  using B = FpBlock<BS>;
  RowsArgs a{};
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  const int most = GATED ? 128 : 256;
  a.tn = 16;
  while (a.tn < most && a.tn < p.M) a.tn *= 2;
  a.m_tiles = static_cast<int>((p.M + a.tn - 1) / a.tn);
  a.nkb = static_cast<int>((p.K + kFpStageK - 1) / kFpStageK);
  a.nsteps = static_cast<int>((p.K + kFpStepK - 1) / kFpStepK);
  a.tok_tiles = a.tn > 128 ? 2 : 1;
  a.tok_offset = (GATED ? 2 : 1) * kROperand;
  a.sfw_offset = a.tok_offset + a.tn * 128;
  a.sfu_offset = a.sfw_offset + B::kBytes;
  a.sft_offset = a.sfw_offset + (GATED ? 2 : 1) * B::kBytes;
  a.stage_bytes = (a.sft_offset + a.tok_tiles * B::kBytes + 1023) / 1024 * 1024;
  const int acc = (GATED ? 2 : 1) * a.tn;
  const int cols = acc + ((GATED ? 2 : 1) + a.tok_tiles) * B::kCols;
  a.tmem_cols = 64;
  while (static_cast<int>(a.tmem_cols) < cols) a.tmem_cols *= 2;
  // CTAs that hold at most half of the tensor memory share an SM in pairs (their shared memory
  // allows two and no third), the others have one to themselves: no CTA of a cluster waits for
  // tensor memory that another cluster's holds.
  const bool two = a.tmem_cols <= 256;
  const int budget = two ? 110 * 1024 : 224 * 1024;
  const int tiles = a.m_tiles * static_cast<int>((p.N + 127) / 128);
  a.splits = 1;
  while (a.splits < 8 && tiles * a.splits * 2 <= p.num_sms * (two ? 2 : 1) && a.nkb >= a.splits * 2) a.splits *= 2;
  a.stages = budget / a.stage_bytes;
  if (a.stages > kRMaxStages) a.stages = kRMaxStages;
  int smem = a.stages * a.stage_bytes + kRTail + 1024;
  if (two && smem < 79 * 1024) smem = 79 * 1024;
  a.sx = p.x.row;
  a.sw = p.w.row;
  a.su = p.up.row;
  a.y = p.y;
  a.y_bf16 = p.y_bf16;
  a.act = p.act;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;

  CUtensorMap mw, mu, mx, msw, msu, msx;
  auto codes = [&](CUtensorMap* m, const FpMat& q, int rows) {
    return make_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, p.K / 2, q.rows, p.K / 2, 128, rows,
                              CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto scales = [&](CUtensorMap* m, const FpMat& q) {
    const uint64_t words = static_cast<uint64_t>(fp4_tiles(p.K, BS)) * (kFpTileBytes / 8);
    return make_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_INT64, q.scales, words, (q.rows + 127) / 128, words * 8,
                              B::kBytes / 8, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  const FpMat& up = GATED ? p.up : p.w;
  if (!codes(&mw, p.w, 128) || !codes(&mu, up, 128) || !codes(&mx, p.x, a.tn) || !scales(&msw, p.w) ||
      !scales(&msu, up) || !scales(&msx, p.x))
    return cudaErrorInvalidValue;

  auto kern = fp4_rows_kernel<GATED, BS>;
  static std::atomic<uint64_t> done{0};
  e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), 232448, done);
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
  return cudaLaunchKernelEx(&cfg, kern, mw, mu, mx, msw, msu, msx, a);
}

}  // namespace

cudaError_t launch_fp4_rows(const FpProduct& p) {
  if (p.is_gated) return p.block == 16 ? launch<true, 16>(p) : launch<true, 32>(p);
  return p.block == 16 ? launch<false, 16>(p) : launch<false, 32>(p);
}

}  // namespace cider
