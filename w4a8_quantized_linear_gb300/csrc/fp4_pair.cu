// fp4_pair.cu -- products of microscaled 4-bit matrices for many tokens:
// y[m, n] = sum_k x[m, k] w[n, k] on CTA pairs, tcgen05.mma.cta_group::2,
// kind::mxf4nvf4 with block scales; gated: h = act(x w^T) (x up^T) in one pass.
//
// A pair computes 256 tokens x 256 weight rows: CTA r holds tokens [128 r, ..)
// of the tile (A) and weight rows [128 r, ..) (half of B), each CTA's tensor
// memory its own 128 tokens x all 256 weight rows.  At 4 bits an MMA reads its
// operands from shared memory as fast as it multiplies only when a pair shares
// them: 8 KB per SM in the 128 cycles of 128 x 256 x 64 products, where an SM
// alone would take in 12.  The accumulators of two tiles share 24 or 48 columns,
// because the scales need some too; the next tile starts once these are drained,
// ~800 cycles behind the last one's end.  (Tiles of 192 weight rows, with nothing
// shared, cost more in all: the issue of their MMAs is as long.)  Gated, the
// even CTA's half of B is 128 rows of w, the odd one's the same rows of `up`:
// columns j and 128 + j of an accumulator are the two sides of one output.
//
// The scales of a stage go by TMA into shared memory (their tiles of 128 rows x
// 4 blocks are contiguous) and by tcgen05.cp into tensor memory, both in the
// MMAs' own order.
//
// Roles (one CTA per SM, persistent over tiles): warp 0 copies, warp 1 issues
// (even CTA only), warps 2..5 drain, scale, round, and store by TMA (or quantize
// what they rounded and store codes and scales).
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "fp4_common.cuh"

namespace cider {
namespace {

constexpr int kFThreads = 192;
constexpr int kFOperand = 128 * 128;             // bytes of a stage's codes of 128 tokens
constexpr int kFOut = 4 * 4096;                  // 4 warps x 32 rows x 128 bytes
constexpr int kFTmemCols = 512;

template <int BS>
struct FCfg {
  using B = FpBlock<BS>;
  static constexpr int kSfx = 2 * kFOperand;                   // tokens' scales
  static constexpr int kSfw = kSfx + B::kBytes;                // the weights', two tiles
  static constexpr int kStage = kSfw + 2 * B::kBytes;          // bytes that a CTA loads a stage
  static constexpr int kStages = (232448 - 1024 - 512 - kFOut - 2 * 256 * 4) / kStage;
  static constexpr int kOut = kStages * kStage;
  static constexpr int kRowScale = kOut + kFOut;               // 2 tiles x 256 fp32
  static constexpr int kBars = kRowScale + 2 * 256 * 4;
  static constexpr int kNumBars = 2 * kStages + 4;
  static constexpr int kSmem = kBars + kNumBars * 8 + 16 + 1024;
  // tensor memory: an accumulator, another one that shares its last columns, the scales
  static constexpr int kColX = kFTmemCols - 3 * B::kCols;
  static constexpr int kColW = kColX + B::kCols;
  static constexpr int kAcc1 = kColX - 256;
  static_assert(kStage % 1024 == 0, "stages must keep 1024-byte alignment for the swizzle");
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(256 - kAcc1 <= 64, "the shared columns are among those that are drained first");
};

struct FPairArgs {
  int M, N;
  int m_tiles, tiles;
  int nkb, nsteps;
  const float *sx, *sw, *su;
  int y_bf16, act;
  uint8_t *q_codes, *q_scales;   // or null
  int q_tiles;                   // tiles of scales along the outputs
  int* err;
};

// 32 rounded outputs from n on of token m, as a block of the quantized matrix.
template <typename T>
__device__ __forceinline__ uint32_t encode_block(const uint32_t* h, uint32_t (&c)[4]) {
  Sixteen<T> a, b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a.w[i] = h[i];
    b.w[i] = h[8 + i];
  }
  const uint32_t top = max(a.top(), b.top());
  uint32_t lo[2], hi[2];
  const uint32_t byte = encode16<T, 32>(a, top, 1.0f, lo);
  encode16<T, 32>(b, top, 1.0f, hi);
  c[0] = lo[0];
  c[1] = lo[1];
  c[2] = hi[0];
  c[3] = hi[1];
  return byte;
}
__device__ __forceinline__ void store_block(const FPairArgs& p, int m, int n, const uint32_t* h) {
  uint32_t c[4];
  const uint32_t byte = p.y_bf16 ? encode_block<__nv_bfloat16>(h, c) : encode_block<__half>(h, c);
  *reinterpret_cast<uint4*>(p.q_codes + static_cast<int64_t>(m) * (p.N >> 1) + (n >> 1)) =
      make_uint4(c[0], c[1], c[2], c[3]);
  uint8_t* at = p.q_scales + scale_at(m, n >> 5, p.q_tiles);
  *at = static_cast<uint8_t>(byte);
  // the other block of a step of 64 that the row ends in
  if (n + 32 == p.N && (p.N & 32) != 0) at[1] = 0;
}

template <bool GATED, int BS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_u, const __grid_constant__ CUtensorMap tm_sx,
                    const __grid_constant__ CUtensorMap tm_sw, const __grid_constant__ CUtensorMap tm_su,
                    const __grid_constant__ CUtensorMap tm_y, const FPairArgs p) {
  using C = FCfg<BS>;
  using B = FpBlock<BS>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::kBars;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  const uint32_t accf_bar0 = bars + 8u * (2 * S);       // x 2, one per accumulator
  const uint32_t acce_bar = bars + 8u * (2 * S + 2);    // drained, as far as the next tile needs it
  const uint32_t done_bar = bars + 8u * (2 * S + 3);
  const uint32_t tmem_slot = bars + 8u * C::kNumBars;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + C::kBars + 8 * C::kNumBars + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;   // of the pair; known to be the same for all threads
  const int cid = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accf_bar0, 1);
    mbar_init(accf_bar0 + 8, 1);
    mbar_init(acce_bar, 8);   // 4 warps x 2 CTAs
    mbar_init(done_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kFTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // the CTA holds all columns

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const uint32_t full0 = mapa_shared(full_bar(0), 0);
    int s = 0, it = 0;
    uint32_t phase = 1;
    bool go = true;
    auto weights = [&](int nt, int kb, int slot) {
      if (rank == 0) mbar_arrive_expect_tx(full_bar(slot), 2 * C::kStage);
      const uint32_t at = base + slot * C::kStage, bar = full0 + 8u * slot;
      const int sk = kb * (B::kBytes / 8);
      if (GATED) {
        if (rank == 0)
          tma_load_2d_pair(at + kFOperand, &tm_w, bar, kb * 128, nt * 128);
        else
          tma_load_2d_pair(at + kFOperand, &tm_u, bar, kb * 128, nt * 128);
        tma_load_2d_pair(at + C::kSfw, &tm_sw, bar, sk, nt);
        tma_load_2d_pair(at + C::kSfw + B::kBytes, &tm_su, bar, sk, nt);
      } else {
        tma_load_2d_pair(at + kFOperand, &tm_w, bar, kb * 128, nt * 256 + rank * 128);
        tma_load_2d_pair(at + C::kSfw, &tm_sw, bar, sk, nt * 2);
        tma_load_2d_pair(at + C::kSfw + B::kBytes, &tm_sw, bar, sk, nt * 2 + 1);
      }
    };
    auto tokens = [&](int mt, int kb, int slot) {
      const uint32_t at = base + slot * C::kStage, bar = full0 + 8u * slot;
      tma_load_2d_pair(at, &tm_x, bar, kb * 128, mt * 256 + rank * 128);
      tma_load_2d_pair(at + C::kSfx, &tm_sx, bar, kb * (B::kBytes / 8), mt * 2 + rank);
    };
    // the first tile's first weights do not depend on the launch before, which makes x
    const int ahead = min(S, p.nkb);
    if (elect_one())
      for (int kb = 0; kb < ahead; ++kb) weights(cid / p.m_tiles, kb, kb);
    pdl_wait();
    for (int tile = cid; tile < p.tiles && go; tile += pairs) {
      const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
      for (int kb = 0; kb < p.nkb; ++kb, ++it) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(s), phase, abort_flag, p.err, kFpWaitNs))) {
          go = false;
          break;
        }
        if (elect_one()) {
          if (it >= ahead) weights(nt, kb, s);
          tokens(mt, kb, s);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // both CTAs' copies have landed before either leaves, also after a wait that gave up
    if (rank == 0) {
      volatile uint32_t keep_waiting = 0u;
      for (int j = max(0, it - S); j < it; ++j)
        mbar_wait_bounded(full_bar(j % S), (j / S) & 1, &keep_waiting, p.err, kFpWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    // One elected lane runs the whole loop: a vote and an election per stage would cost it 150 cycles
    // of a stage's 512.
    if (rank == 0 && elect_one()) {
      int n = 0, s = 0;
      uint32_t phase = 0;
      bool go = true;
      for (int tile = cid; tile < p.tiles && go; tile += pairs, ++n) {
        const uint32_t d = tmem + ((n & 1) ? C::kAcc1 : 0);
        // a stage: its scales, then `steps` MMAs
        auto stage = [&](auto full, int steps, bool first) {
          if (!mbar_wait_bounded(full_bar(s), phase, abort_flag, p.err, kFpWaitNs)) {
            go = false;
            return;
          }
          tc_fence_after();
          const uint32_t at = base + s * C::kStage;
          const uint64_t dx = smem_desc_scales(at + C::kSfx), dw = smem_desc_scales(at + C::kSfw);
#pragma unroll
          for (int a = 0; a < B::kTiles; ++a) {
            tc_cp_scales<2>(tmem + C::kColX + 4 * a, dx + a * (kFpTileBytes >> 4));
            tc_cp_scales<2>(tmem + C::kColW + 8 * a, dw + a * (kFpTileBytes >> 4));
            tc_cp_scales<2>(tmem + C::kColW + 8 * a + 4, dw + ((B::kBytes + a * kFpTileBytes) >> 4));
          }
          // the tile before has given up the columns that its accumulator shares with this one's (and,
          // earlier, everything of the tile before that)
          if (first && n > 0) {
            if (!mbar_wait_bounded(acce_bar, (n - 1) & 1, abort_flag, p.err, kFpWaitNs)) {
              go = false;
              return;
            }
            tc_fence_after();
          }
          const uint64_t ad = smem_desc_k_sw128(at), bd = smem_desc_k_sw128(at + kFOperand);
#pragma unroll
          for (int j = 0; j < kFpSteps; ++j) {
            if (!decltype(full)::value && j >= steps) break;
            const int a = BS == 16 ? j : j >> 1, id = BS == 16 ? 0 : 2 * (j & 1);
            tc_mma_fp4<2, BS>(d, ad + 2 * j, bd + 2 * j, idesc_fp4<BS>(256, 256, id), tmem + C::kColX + 4 * a,
                              tmem + C::kColW + 8 * a, first && j == 0 ? 0u : 1u);
          }
          tc_commit_pair_mc(empty_bar(s), 0x3);
          if (++s == S) {
            s = 0;
            phase ^= 1u;
          }
        };
        // a test per MMA would cost more than its issue: only the last stage, when it is not full, has them
        const int full_stages = p.nsteps / kFpSteps;
        for (int kb = 0; kb < full_stages && go; ++kb) stage(std::true_type{}, kFpSteps, kb == 0);
        if (full_stages < p.nkb && go) stage(std::false_type{}, p.nsteps - full_stages * kFpSteps, full_stages == 0);
        if (go) tc_commit_pair_mc(accf_bar0 + 8u * (n & 1), 0x3);
      }
      tc_commit_pair_mc(done_bar, 0x3);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = q * 32 + lane, e = threadIdx.x - 64;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t acce0 = mapa_shared(acce_bar, 0);
    float* scale = reinterpret_cast<float*>(gbase + C::kRowScale);
    constexpr int kCols = GATED ? 128 : 256;   // outputs of a token in a tile
    int n = 0;
    bool ok = true;
    pdl_wait();   // row scales of x come from the launch before
    for (int tile = cid; tile < p.tiles; tile += pairs, ++n) {
      const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
      const int m0 = mt * 256 + static_cast<int>(rank) * 128, m = m0 + row, n0 = nt * kCols;
      const float sx = p.sx && m < p.M ? ld_global_f32(p.sx + m) : 1.0f;
      float* w = scale + (n & 1) * 256;
      // weight rows' scales of the tile, in the order of the accumulator's columns
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* src = GATED && h == 1 ? p.su : p.sw;
        const int c = n0 + e + (GATED ? 0 : 128 * h);
        w[128 * h + e] = src && c < p.N ? __ldg(src + c) : 1.0f;
      }
      // warps whose waits gave up and warps whose did not leave together
      if (!named_barrier_and(1, 128, ok)) break;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_bounded(accf_bar0 + 8u * (n & 1), (n >> 1) & 1, abort_flag, p.err, kFpWaitNs));
      if (!ok) continue;
      tc_fence_after();
      const uint32_t d = tmem + lane_base + ((n & 1) ? C::kAcc1 : 0);
      // 64 outputs a turn, first those whose columns the next tile's accumulator shares: the last ones
      // of the first accumulator, the first ones of the second
#pragma unroll 1
      for (int i = 0; i < kCols / 64; ++i) {
        const int c = 64 * ((n & 1) ? i : kCols / 64 - 1 - i);
        uint32_t v[64], u[GATED ? 64 : 1];
        tmem_ld32(d + c, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld32(d + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        if constexpr (GATED) {
          tmem_ld32(d + 128 + c, *reinterpret_cast<uint32_t(*)[32]>(u));
          tmem_ld32(d + 160 + c, *reinterpret_cast<uint32_t(*)[32]>(u + 32));
        }
        tmem_wait_ld();
        if (i == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(acce0);
        }
        uint32_t h[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 s = *reinterpret_cast<const float2*>(w + c + 2 * j);
          float a = __uint_as_float(v[2 * j]) * sx * s.x, b = __uint_as_float(v[2 * j + 1]) * sx * s.y;
          if constexpr (GATED) {
            const float2 t = *reinterpret_cast<const float2*>(w + 128 + c + 2 * j);
            a = gated(a, __uint_as_float(u[2 * j]) * sx * t.x, p.act);
            b = gated(b, __uint_as_float(u[2 * j + 1]) * sx * t.y, p.act);
          }
          h[j] = p.y_bf16 ? y_bits2<true>(a, b) : y_bits2<false>(a, b);
        }
        if constexpr (GATED && BS == 32) {
          if (p.q_codes) {
            // a thread's outputs are two blocks of the quantized matrix
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (m < p.M && n0 + c + 32 * k < p.N) store_block(p, m, n0 + c + 32 * k, h + 16 * k);
            continue;
          }
        }
        // the last turn's store has read the buffer
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        const uint32_t out = base + C::kOut + q * 4096;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t x[4] = {h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]};
          st_shared_v4(out + lane * 128 + ((j ^ (lane & 7)) << 4), x);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (m0 + q * 32 < p.M && n0 + c < p.N) tma_store_2d(&tm_y, out, n0 + c, m0 + q * 32);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  // The odd CTA's warp 1 has nothing to do until here: it begins to wait when the last tile has been drained,
  // not with the call, which may take longer than a wait does.
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    // no MMA is in flight when the pair frees its tensor memory, also after a wait that gave up
    if (lane == 0) {
      volatile uint32_t keep_waiting = 0u;
      mbar_wait_bounded(done_bar, 0, &keep_waiting, p.err, kFpWaitNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kFTmemCols);
  }
}

template <bool GATED, int BS>
cudaError_t launch(const FpProduct& p) {
  using C = FCfg<BS>;
  using B = FpBlock<BS>;
  auto kern = fp4_pair_kernel<GATED, BS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::kSmem, done);
  if (e != cudaSuccess) return e;
  FPairArgs a{};
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.m_tiles = static_cast<int>((p.M + 255) / 256);
  const int64_t tiles = a.m_tiles * (GATED ? (p.N + 127) / 128 : (p.N + 255) / 256);
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  a.tiles = static_cast<int>(tiles);
  a.nkb = static_cast<int>((p.K + kFpStageK - 1) / kFpStageK);
  a.nsteps = static_cast<int>((p.K + kFpStepK - 1) / kFpStepK);
  a.sx = p.x.row;
  a.sw = p.w.row;
  a.su = p.up.row;
  a.y_bf16 = p.y_bf16;
  a.act = p.act;
  a.q_codes = p.q_codes;
  a.q_scales = p.q_scales;
  a.q_tiles = fp4_tiles(p.N, 32);
  e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  CUtensorMap mx, mw, mu, msx, msw, msu, my;
  auto codes = [&](CUtensorMap* m, const FpMat& q) {
    return make_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, p.K / 2, q.rows, p.K / 2, 128, 128,
                              CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto scales = [&](CUtensorMap* m, const FpMat& q) {
    const uint64_t words = static_cast<uint64_t>(fp4_tiles(p.K, BS)) * (kFpTileBytes / 8);
    return make_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_INT64, q.scales, words, (q.rows + 127) / 128, words * 8,
                              B::kBytes / 8, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  const FpMat& up = GATED ? p.up : p.w;
  if (!codes(&mx, p.x) || !codes(&mw, p.w) || !codes(&mu, up) || !scales(&msx, p.x) || !scales(&msw, p.w) ||
      !scales(&msu, up))
    return cudaErrorInvalidValue;
  my = mx;
  if (!p.q_codes &&
      !make_tensor_map_2d(&my, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.y, p.N, p.M, p.N * 2, 64, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kFThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  // pairs that the device holds at once (an odd number of SMs in a part of it leaves one alone)
  static std::atomic<int> held[64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = dev < 64 ? held[dev].load(std::memory_order_relaxed) : 0;
  if (most <= 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_sms & ~1), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&most, reinterpret_cast<const void*>(kern), &cfg) != cudaSuccess || most <= 0) {
      (void)cudaGetLastError();
      most = p.num_sms / 2;
    }
    if (dev < 64) held[dev].store(most, std::memory_order_relaxed);
  }
  const int pairs = a.tiles < most ? a.tiles : most;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.stream = p.st;
  cudaLaunchAttribute attr[1];
  if (p.after_launch) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, mx, mw, mu, msx, msw, msu, my, a);
}

}  // namespace

cudaError_t launch_fp4_pair(const FpProduct& p) {
  if (p.is_gated) return p.block == 16 ? launch<true, 16>(p) : launch<true, 32>(p);
  return p.block == 16 ? launch<false, 16>(p) : launch<false, 32>(p);
}

}  // namespace cider
