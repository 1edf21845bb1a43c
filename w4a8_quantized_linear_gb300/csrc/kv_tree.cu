// kv_tree.cu -- attention over the paged, quantized cache for many query rows
// per key/value head (trees of drafted tokens x grouped heads): 128 rows and
// 128 positions at a time on the tensor core.
//
// Mathematics as in kv_rows.cu: x_ij = scale log2(e) sk_j (q_i . ck_j) + log2
// sv_j, p'_ij = 2^(x_ij - m_i), o_i = sum p' cv / sum p' / sv.  The codes become
// exact fp16 values once per tile, for all rows; q is fp16 (bf16 rows are
// scaled by one power of two first), p' is rounded to fp16, sums are fp32.
//
// Per tile: S = Q K^T with Q in tensor memory and K's tile in shared memory,
// p' back into the tensor memory of its own S, O += P V with V's tile as it
// lies ([position][dim], the operand's "MN-major" form).  Tensor memory: two S
// tiles (one is computed while the other is in softmax), O, Q: 448 columns.
// Both operands from shared memory would need the SM's whole shared-memory
// bandwidth; with Q and P in tensor memory it is half.
//
// Bound: HBM for INT8 up to 128 rows in theory (a tile is 33 KiB: ~1400 cycles
// of an SM's share of HBM against 1024 of tensor work); in practice the softmax
// of a tile (~1600 cycles with four warps per scheduler, ~6 a warp's
// instruction) and the steps around it (waits, agreement, P's store, the issue
// of eight MMAs at ~110 cycles each) follow one another, ~3700 cycles a tile: the
// tensor pipe is active 26 % of the time.  The softmax warps' 80 registers do not
// hold a tile's scores and weights beside the rest: 396 .. 420 bytes are spilled.
// 32 requests of 4096 .. 16384 positions, 16 .. 32 new tokens, 32 / 8 heads of
// 128, INT8: 289 us (2.5 TB/s of codes, 488 TFLOP/s), whatever the number of
// rows up to 128.  Measured and not kept: two groups of softmax warps on
// alternate tiles, each with an S and an O of its own and Q in shared memory
// (316 us: two warps per scheduler at a time leave the latencies open), the same
// with one warp per quarter and tile (392 us), eight softmax warps of 64
// positions each (318 us).
//
// Roles (896 threads, one CTA per SM, persistent over its share of the axis):
//   warps 0, 1    one thread each issues the MMAs of S and of O
//   warps 2, 3    load the codes as they are cached, keys and values, by bulk
//                 copies of a page's part of a tile (each takes a lane ~80
//                 cycles to issue, one lane after another), into a ring in
//                 shared memory
//   warps 4-11    converters: codes to fp16 tiles in shared memory; each
//                 position's sk, log2 sv, 1 / sv.  (Loading the codes themselves,
//                 to registers or by asynchronous copies, was what held a tile
//                 up: 5000 and 3300 cycles.)
//   warps 12-27   softmax: four warps per quarter of the rows, 32 positions of
//                 the tile each.  S is read in the layout that gives a thread 4
//                 rows x 2 neighbouring positions, so that a position's scales
//                 are loaded once for 4 rows.  m_i is only raised when a p'
//                 passes 2^14: the four warps of a quarter agree on that with
//                 one reducing barrier per tile.  They also put Q's tile into
//                 tensor memory and take O's out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "cider_device.cuh"
#include "cider_internal.h"
#include "kv_common.cuh"
#include "kv_parts.cuh"

namespace cider {
namespace {

constexpr int kTileRows = 128;    // query rows of a unit
constexpr int kTilePos = 128;     // positions of a tile
constexpr int kThreads = 896;
constexpr int kConvWarp0 = 4, kConvWarps = 8;
constexpr int kSoftWarp0 = 12, kSoftWarps = 16;
constexpr int kParts = 4;         // of a tile's positions (and of O's columns): one softmax warp each per quarter
constexpr int kRegsMisc = 64, kRegsConv = 56, kRegsSoft = 80, kRegsLaunch = 72;
constexpr int kRegsNeeded = 128 * kRegsMisc + 256 * kRegsConv + 512 * kRegsSoft;
static_assert(kRegsNeeded <= kThreads * kRegsLaunch, "register split exceeds the launch's registers");
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColAll = 512;
constexpr float kNone = -3.0e38f;   // m of a row that has seen nothing: any x is far above it

template <int D, int BITS>
struct TreeCfg {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks of a row
  static constexpr int kCodes = 128 / BITS;                  // codes of a chunk
  static constexpr int kUnits = kCodes / 8;                  // 16-byte fp16 units of a chunk
  static constexpr int kRowsPer = 512 / kRowBytes;           // rows of one warp load
  static constexpr int kLoads = kTilePos / (kConvWarps * kRowsPer);   // per thread, K or V
  static constexpr int kSub = 16384;                         // [128][64] fp16, 128-byte swizzle
  static constexpr int kSide = kSub * (D / 64);              // a K or V tile
  static constexpr int kScaleOffset = 4 * kSide;             // two stages of K, V
  static constexpr int kScaleStage = 64 * 16 + 64 * 8;       // per pair of positions: sk sk lg lg, inv inv
  static constexpr int kStatOffset = kScaleOffset + 4 * kScaleStage;
  static constexpr int kStatBytes = kParts * kTileRows * 8;  // per part and row: two floats
  static constexpr int kMaskOffset = kStatOffset + kStatBytes;
  // Codes as they are cached, on their way to the converters: a K or a V tile
  // per slot, and the scales of a tile's positions.
  static constexpr int kRingOffset = kMaskOffset + kTileRows * 8;
  static constexpr int kRingSlot = kTilePos * kRowBytes;
  static constexpr int kScaleRing = 4 * 2 * kTilePos * 4;    // four tiles of sk, sv
  static constexpr int kFit = (226 * 1024 - kRingOffset - kScaleRing) / kRingSlot;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;         // at most: the scales' four tiles
  static constexpr int kScaleRingOffset = kRingOffset + kSlots * kRingSlot;
  static constexpr int kBarOffset = kScaleRingOffset + kScaleRing;
  static constexpr int kSmem = kBarOffset + 40 * 8 + 128 + 1024;
  // Order of the dims in the fp16 tiles: unit `lin` of a row (8 values) holds
  // codes (lin / kChunks) * 8 .. + 8 of chunk lin % kChunks, so that the lanes
  // that convert a row's chunks store to different banks.
  __host__ __device__ static constexpr int dim_of(int lin) {
    return lin % kChunks * kCodes + lin / kChunks * 8;
  }
};

// Barriers, by number.
enum Bar : int {
  kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPReady = 10, kQFull = 12,
  kOFull = 13, kOEmpty = 14, kDone = 15, kRawFull = 17, kRawEmpty = 25, kScFull = 33, kBars = 37
};

template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// A K-major / MN-major tile's descriptors, 128-byte swizzle.  MN-major (the
// values, [position][dim]): 64 dims are a row of 128 bytes, 8 positions 1024
// bytes (stride offset), the next 64 dims `kSub` further (leading offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t leading) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((leading >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kBMajorMn = 1u << 16;   // instruction descriptor: B is MN-major

// 16 lanes x 32 columns (fp32): register 4 i + 2 h + e of thread T is lane
// T / 4 + 8 h, column 8 i + 2 (T % 4) + e.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float (&r)[16]) {
  uint32_t u[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
// After tmem_wait_ld: nothing that reads these registers is moved above the wait.
template <int N>
__device__ __forceinline__ void loaded(float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// 16 lanes x 16 columns: register 2 i + h of thread T is lane T / 4 + 8 h, column 4 i + T % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// One lane per thread, N consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_ld_row(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_ld32(taddr, r);
  } else {
    static_assert(N == 16);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tmem_st_row(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_st32(taddr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  } else {
    static_assert(N == 8);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
  }
}
// Whether any thread of the `count` threads of barrier `id` has `v`.
__device__ __forceinline__ bool barrier_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Two fp32 operations at once.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void un2(const F2& x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(const F2& a, const F2& b, const F2& c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(const F2& a, const F2& b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(const F2& a, const F2& b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ __half2 as_h2(uint32_t u) {
  __half2 h;
  memcpy(&h, &u, 4);
  return h;
}

// Unit h of a 16-byte chunk as 8 fp16 values.  INT8: the codes in order.  INT4:
// code 2^-9, in the order 0 4 1 5 2 6 3 7 (code + 8 as a subnormal, lifted).
template <int BITS>
__device__ __forceinline__ uint4 convert_unit(const uint4& c, int h) {
  uint4 r;
  if constexpr (BITS == 8) {
    s8x4_to_h2x2(h == 0 ? c.x : c.z, r.x, r.y);
    s8x4_to_h2x2(h == 0 ? c.y : c.w, r.z, r.w);
  } else {
    const uint32_t x = (h == 0 ? c.x : h == 1 ? c.y : h == 2 ? c.z : c.w) ^ 0x88888888u;
    const uint32_t y = x >> 8;
    const __half2 lift = as_h2(0x78007800u), lift_hi = as_h2(0x68006800u), off = as_h2(0xA400A400u);
    auto f = [&](uint32_t u, __half2 m) {
      const __half2 v = __hfma2(as_h2(u), m, off);
      uint32_t w;
      memcpy(&w, &v, 4);
      return w;
    };
    r.x = f(x & 0x000F000Fu, lift);
    r.y = f(x & 0x00F000F0u, lift_hi);
    r.z = f(y & 0x000F000Fu, lift);
    r.w = f(y & 0x00F000F0u, lift_hi);
  }
  return r;
}

// The MMAs of a tile in stage ST: S = Q K^T, and O (+)= P V.
template <typename C, int ST>
__device__ __forceinline__ void issue_s(uint32_t sbase) {
  const uint64_t desc = smem_desc_k_sw128(sbase + ST * 2 * C::kSide);
#pragma unroll
  for (int s = 0; s < C::kSide / C::kSub * 4; ++s)
    tc_mma_ts(kColS + ST * 128, kColQ + s * 8, desc + ((s >> 2) * C::kSub + (s & 3) * 32 >> 4),
              idesc_f16_f32(128, 128), s > 0);
}
template <typename C, int D, int ST>
__device__ __forceinline__ void issue_o(uint32_t sbase, bool add) {
  const uint64_t desc = smem_desc_mn_sw128(sbase + ST * 2 * C::kSide + C::kSide, C::kSub);
#pragma unroll
  for (int s = 0; s < kTilePos / 16; ++s)   // P of each part lies at the beginning of its columns of S
    tc_mma_ts(kColO, kColS + ST * 128 + (s >> 1) * 32 + (s & 1) * 8, desc + (s * 2048 >> 4),
              idesc_f16_f32(128, D) | kBMajorMn, s > 0 ? 1u : add ? 1u : 0u);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(AttendArgs a, PartsArgs parts, bool bf16) {
  using C = TreeCfg<D, BITS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.q_heads / a.cache.heads;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kBarOffset + kBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOffset + kBars * 8 + 4);
  float* lift_max = reinterpret_cast<float*>(smem + C::kBarOffset + kBars * 8 + 16);   // 16 warps
  auto bar = [&](int i) { return sbase + C::kBarOffset + i * 8; };
  auto wait = [&](int i, uint32_t parity) {
    return mbar_sleep_bounded(bar(i), parity & 1, abort_flag, a.err, kWaitNs);
  };

  if (warp == 0) {
    if (lane == 0) {
      *abort_flag = 0;
      for (int s = 0; s < 2; ++s) {
        mbar_init(bar(kKFull + s), kConvWarps);
        mbar_init(bar(kKEmpty + s), 1);
        mbar_init(bar(kVFull + s), kConvWarps);
        mbar_init(bar(kVEmpty + s), 1);
        mbar_init(bar(kSFull + s), 1);
        mbar_init(bar(kPReady + s), kSoftWarps);
      }
      mbar_init(bar(kQFull), kSoftWarps);
      mbar_init(bar(kOFull), 1);
      mbar_init(bar(kOEmpty), kSoftWarps);
      mbar_init(bar(kDone), 1);
      mbar_init(bar(kDone + 1), 1);
      for (int s = 0; s < 4; ++s) mbar_init(bar(kScFull + s), 4);
      for (int s = 0; s < C::kSlots; ++s) {
        mbar_init(bar(kRawFull + s), 1);
        mbar_init(bar(kRawEmpty + s), kConvWarps);
      }
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), kColAll);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's: they begin at 0 (a constant for the MMAs' operands)
  constexpr uint32_t tmem = 0;

  // Every role walks the same pieces.  A wait that gives up raises the abort
  // flag.  Then no more MMAs or copies are issued, and the other roles run to
  // their ends without waiting (all their memory accesses stay in bounds), so
  // that no named barrier is left with a thread missing.
  if (warp < kConvWarp0) {
    regs_dec<kRegsMisc>();
    // Two issuers: an MMA takes a thread ~75 cycles and more to issue, sixteen a
    // tile are more than the tile's tensor time.  Whole-warp waits, one lane issues.
    if (warp == 0) {
      // S(n) = Q K(n)^T
      Axis axis;
      axis.begin(a, kTilePos, lane, kTileRows);
      if (lane == 0) parts.announce(axis);
      bool more = axis.more();
      uint32_t n = 0, piece = 0;
      bool ok = true;
      while (more) {
        const int tiles = static_cast<int>(axis.piece_end - axis.piece_begin);
        more = axis.next(a, kTilePos, kTileRows);
        ok = wait(kQFull, piece) && ok;
        for (int i = 0; i < tiles; ++i, ++n) {
          const uint32_t st = n & 1, ph = n >> 1;
          ok = wait(kKFull + st, ph) && ok;
          ok = wait(kVEmpty + st, ph + 1) && ok;   // P(n - 2), in the same columns, is read
          tc_fence_after();
          if (__all_sync(0xffffffffu, ok) && elect_one()) {
            // a constant stage keeps every operand a constant or uniform
            if (st == 0) issue_s<C, 0>(sbase); else issue_s<C, 1>(sbase);
            tc_commit(bar(kSFull + st));
            tc_commit(bar(kKEmpty + st));
          }
          __syncwarp();
        }
        ++piece;
      }
    } else if (warp == 1) {
      // O += P(n) V(n)
      Axis axis;
      axis.begin(a, kTilePos, lane, kTileRows);
      bool more = axis.more();
      uint32_t n = 0, piece = 0;
      bool ok = true;
      while (more) {
        const int tiles = static_cast<int>(axis.piece_end - axis.piece_begin);
        more = axis.next(a, kTilePos, kTileRows);
        ok = wait(kOEmpty, piece + 1) && ok;
        for (int i = 0; i < tiles; ++i, ++n) {
          const uint32_t st = n & 1, ph = n >> 1;
          ok = wait(kVFull + st, ph) && ok;
          ok = wait(kPReady + st, ph) && ok;
          tc_fence_after();
          if (__all_sync(0xffffffffu, ok) && elect_one()) {
            if (st == 0) issue_o<C, D, 0>(sbase, i > 0); else issue_o<C, D, 1>(sbase, i > 0);
            tc_commit(bar(kVEmpty + st));
            if (i == tiles - 1) tc_commit(bar(kOFull));
          }
          __syncwarp();
        }
        ++piece;
      }
    }
    else {
      // loads: warp 2 the keys and their scales, warp 3 the values and theirs, a
      // run of positions that lie in one page per lane
      const bool v = warp == 3;
      const uint8_t* const codes = v ? a.cache.v : a.cache.k;
      const float* const scale_src = v ? a.cache.v_scale : a.cache.k_scale;
      Axis axis;
      axis.begin(a, kTilePos, lane, kTileRows);
      bool more = axis.more();
      const int run_shift = min(a.cache.page_shift, 7);
      const int runs = kTilePos >> run_shift;                 // of a tile: 1, 2, 4 or 8
      const uint32_t run_bytes = static_cast<uint32_t>(C::kRowBytes) << run_shift;
      const uint32_t scale_bytes = 4u << run_shift;
      uint32_t side = v ? 1 : 0, slot = side, n = 0;          // slot = side mod kSlots
      while (more) {
        const int tiles = static_cast<int>(axis.piece_end - axis.piece_begin);
        const int first = static_cast<int>(axis.piece_begin) * runs;
        const int last = static_cast<int>(min(axis.piece_end * runs,
                                              (axis.req.length + (1 << run_shift) - 1) >> run_shift));
        const int head = axis.unit / Axis::blocks_of(a, axis.req, kTileRows);
        const int32_t* table = a.table + axis.b * a.table_width;
        // lane l: the page of run 32 i + l, -1 without one
        auto load_ids = [&](int base) -> int {
          const int at = first + base + lane;
          if (at >= last) return -1;
          const int32_t id = table[at >> (a.cache.page_shift - run_shift)];
          if (id >= 0 && id < a.cache.pages) return id;
          atomicOr(a.err, kDevErrIndex);
          return -1;
        };
        int ids = load_ids(0), next = load_ids(32);
        more = axis.next(a, kTilePos, kTileRows);
        for (int i = 0; i < tiles; ++i, ++n) {
          const int base = i * runs;
          if (i > 0 && (base & 31) == 0) {
            ids = next;
            next = load_ids(base + 32);
          }
          const int id = __shfl_sync(0xffffffffu, ids, (base & 31) + (lane & (runs - 1)));
          const uint32_t there = __popc(__ballot_sync(0xffffffffu, id >= 0) & ((1u << runs) - 1));
          // a page of 128 positions or fewer is one run
          const int64_t row = a.cache.row(max(id, 0), head, 0);
          const uint32_t scales = sbase + C::kScaleRingOffset + (n & 3) * 2 * kTilePos * 4 +
                                  (v ? kTilePos * 4 : 0) + lane * scale_bytes;
          // after a wait that gave up nothing more is loaded: a barrier that
          // expects bytes must not be arrived at twice in a phase
          if (!__all_sync(0xffffffffu, wait(kRawEmpty + slot, side / C::kSlots + 1))) {
            more = false;
            break;
          }
          // a position without a page counts as one with scales of 0
          if (id < 0 && lane < runs) {
            const uint32_t zero[4] = {0, 0, 0, 0};
            for (uint32_t j = 0; j < scale_bytes; j += 16) st_shared_v4(scales + j, zero);
            fence_proxy_async_smem();   // later tiles' copies write here too
          }
          __syncwarp();
          const uint32_t full = bar(kRawFull + slot);
          if (lane == 0) mbar_arrive_expect_tx(full, there * (run_bytes + scale_bytes));
          __syncwarp();
          if (id >= 0 && lane < runs) {
            bulk_load(sbase + C::kRingOffset + slot * C::kRingSlot + lane * run_bytes,
                      codes + row * C::kRowBytes, run_bytes, full);
            bulk_load(scales, scale_src + row, scale_bytes, full);
          }
          __syncwarp();
          side += 2;
          slot = slot + 2 >= C::kSlots ? slot + 2 - C::kSlots : slot + 2;
        }
      }
      // the converters wait for every copy before the CTA ends; after a wait that
      // gave up they may not have: what is in flight lands within microseconds
      if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000u) __nanosleep(1000);
      }
    }
    // no MMA may be in flight when the tensor memory is freed, also after an abort
    if (warp < 2) {
      if (elect_one()) {
        tc_commit(bar(kDone + warp));
        volatile uint32_t keep_waiting = 0u;
        mbar_wait_bounded(bar(kDone + warp), 0, &keep_waiting, a.err, kWaitNs);
      }
      __syncwarp();
    }
  } else if (warp < kSoftWarp0) {
    regs_dec<kRegsConv>();
    // ------------------------------------------------------------ converters
    const int cw = warp - kConvWarp0;
    int c, row;   // this lane's chunk, and its row among the rows of one load
    if constexpr (C::kChunks == 8) {
      c = lane & 7;
      row = lane >> 3;
    } else if constexpr (C::kChunks == 4) {
      c = lane & 3;
      row = (lane >> 3) + 4 * (lane >> 2 & 1);
    } else {
      c = lane & 1;
      row = (lane >> 3 & 1) + 2 * (lane >> 1 & 3) + 8 * (lane >> 4);
    }
    const int token0 = cw * C::kRowsPer + row;   // of load j: + j * kConvWarps * kRowsPer
    const int token_s = (cw & 3) * 32 + lane;    // warps 4-7: this lane's position's scales
    const float mul = a.scale * 1.44269504f * (BITS == 4 ? 512.0f : 1.0f);
    uint8_t* dst[C::kUnits];                     // of load 0: 1024 bytes further for 8 tokens
#pragma unroll
    for (int h = 0; h < C::kUnits; ++h) {
      const int lin = c + C::kChunks * h;
      dst[h] = smem + (lin >> 3) * C::kSub + token0 * 128 + (((lin & 7) ^ (token0 & 7)) << 4);
    }
    static_assert(kConvWarps * C::kRowsPer % 8 == 0, "the swizzle of a lane's rows is the same");
    const uint8_t* src0 = smem + C::kRingOffset + token0 * C::kRowBytes + c * 16;
    uint32_t side = 0, slot = 0;
    auto convert_side = [&](int to) {   // the next slot's tile to the stage at `to`
      wait(kRawFull + slot, side / C::kSlots);
      uint4 in[C::kLoads];
#pragma unroll
      for (int j = 0; j < C::kLoads; ++j)
        in[j] = *reinterpret_cast<const uint4*>(src0 + slot * C::kRingSlot + j * (kConvWarps * 512));
#pragma unroll
      for (int j = 0; j < C::kLoads; ++j)
#pragma unroll
        for (int h = 0; h < C::kUnits; ++h)
          *reinterpret_cast<uint4*>(dst[h] + to + j * (kConvWarps * C::kRowsPer * 128)) =
              convert_unit<BITS>(in[j], h);
    };
    auto release_side = [&]() {   // after the warp's loads of the slot
      if (lane == 0) mbar_arrive(bar(kRawEmpty + slot));
      ++side;
      slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    };

    Axis axis;
    axis.begin(a, kTilePos, lane, kTileRows);
    const int64_t all = axis.more() ? axis.end - axis.at : 0;   // tiles of the share
    for (uint32_t n = 0; n < all; ++n) {
      const uint32_t st = n & 1, ph = n >> 1;
      // K's stage is free: S(n - 2) is done, so O(n - 4) is, and the softmax is
      // past the scales of tile n - 4
      wait(kKEmpty + st, ph + 1);
      convert_side(st * 2 * C::kSide);
      if (cw < 4) {
        // the values' scales come with the next slot
        wait(kRawFull + (slot + 1 == C::kSlots ? 0 : slot + 1), (side + 1) / C::kSlots);
        const float* in = reinterpret_cast<const float*>(smem + C::kScaleRingOffset) + (n & 3) * 2 * kTilePos + token_s;
        const float sk = in[0], sv = in[kTilePos];
        float* f = reinterpret_cast<float*>(smem + C::kScaleOffset + (n & 3) * C::kScaleStage);
        const int pair = token_s >> 1, e = token_s & 1;
        float kept = sv > 0.0f && sv < 0x1p-90f ? 0x1p-90f : sv;
        if (sv == 1.0f) {   // a row of zeros does not set the maximum; the codes came with the scales
          const uint8_t* codes = smem + C::kRingOffset + (slot + 1 == C::kSlots ? 0 : slot + 1) * C::kRingSlot +
                                 token_s * C::kRowBytes;
          uint32_t any = 0;
#pragma unroll 1
          for (int i = 0; i < C::kRowBytes; i += 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(codes + i);
            any |= w.x | w.y | w.z | w.w;
          }
          if (any == 0) kept = kZeroRowScale;
        }
        float lg, inv;
        asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(kept));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(kept));
        f[pair * 4 + e] = sk * mul;
        f[pair * 4 + 2 + e] = lg;
        f[256 + pair * 2 + e] = kept > 0.0f && kept < INFINITY ? inv : 0.0f;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kScFull + (n & 3)));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull + st));
      release_side();
      wait(kVEmpty + st, ph + 1);
      convert_side(st * 2 * C::kSide + C::kSide);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kVFull + st));
      release_side();
    }
  } else {
    regs_inc<kRegsSoft>();
    // --------------------------------------------------------------- softmax
    const int sw = warp - kSoftWarp0, quarter = sw & 3, part = sw >> 2;
    const int g = lane >> 2, t = lane & 3;
    constexpr int kCols = D / kParts;   // of O (and dims of Q) per thread
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float2* stat = reinterpret_cast<float2*>(smem + C::kStatOffset);
    float2* my_stat = stat + part * kTileRows + quarter * 32;
    uint64_t* masks = reinterpret_cast<uint64_t*>(smem + C::kMaskOffset);
    const int quarter_bar = 1 + quarter;   // the four warps of a quarter

    Axis axis;
    axis.begin(a, kTilePos, lane, kTileRows);
    bool more = axis.more();
    uint32_t n = 0, piece = 0;
    // This thread's row of the axis' piece, and its dims of that row of q.
    int rows = 0, row = quarter * 32 + lane;
    int64_t out_at = 0;
    uint4 raw[kCols / 8];
    uint64_t mask = 0;
    auto load_q = [&]() {
      const int blocks = Axis::blocks_of(a, axis.req, kTileRows);
      const int head = axis.unit / blocks, block = axis.unit - head * blocks;
      rows = min(kTileRows, axis.req.nodes * group - block * kTileRows);
      const bool have = row < rows;
      const int at = block * kTileRows + row;
      const int node = have ? at / group : 0;
      const int hq = head * group + (have ? at - node * group : 0);
      out_at = ((axis.req.first + node) * a.q_heads + hq) * D;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (axis.req.first + node) * a.q_stride +
                          static_cast<int64_t>(hq) * D;
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i)
        raw[i] = have ? *reinterpret_cast<const uint4*>(q + C::dim_of(part * (kCols / 8) + i))
                      : make_uint4(0, 0, 0, 0);
      mask = 0;
      if (have && part == 0)
        mask = a.tree ? static_cast<uint64_t>(a.tree[axis.req.first + node]) : ~0ull >> (63 - node);
    };
    if (more) load_q();
    while (more) {
      // ------------------------------------------------------------- Q's tile
      const int nodes = axis.req.nodes, context = static_cast<int>(axis.req.context);
      const int tiles = static_cast<int>(axis.piece_end - axis.piece_begin);
      if (part == 0) masks[row] = mask;
      float lift = 1.0f, unlift = 1.0f;
      if (bf16) {
        // one power of two for all rows puts the largest value in [2^13, 2^14)
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          float f[8];
          widen8<__nv_bfloat16>(raw[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) lift_max[sw] = top;
        named_barrier_sync(5, 32 * kSoftWarps);
        top = lift_max[lane & 15];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        int k = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
        k = top == 0.0f ? 0 : max(-126, min(k, 126));
        lift = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        unlift = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      }
      {
        uint32_t u[kCols / 2];
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {
          uint4 w = raw[j];
          if (bf16) {
            float f[8];
            widen8<__nv_bfloat16>(w, f);
            w = make_uint4(pack_h2(f[0] * lift, f[1] * lift), pack_h2(f[2] * lift, f[3] * lift),
                           pack_h2(f[4] * lift, f[5] * lift), pack_h2(f[6] * lift, f[7] * lift));
          }
          if constexpr (BITS == 4)   // the order of the converted codes
            w = make_uint4(__byte_perm(w.x, w.z, 0x5410u), __byte_perm(w.x, w.z, 0x7632u),
                           __byte_perm(w.y, w.w, 0x5410u), __byte_perm(w.y, w.w, 0x7632u));
          u[4 * j] = w.x;
          u[4 * j + 1] = w.y;
          u[4 * j + 2] = w.z;
          u[4 * j + 3] = w.w;
        }
        tmem_st_row(lanes + kColQ + part * (kCols / 2), u);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
      wait(kQFull, piece);   // also: the masks are there
      const F2 unlift2 = f2(unlift, unlift);

      // ------------------------------------------------------ the piece's tiles
      const bool active = quarter * 32 < rows;   // some row of this warp exists
      float mu[4], l[4];   // rows g, g + 8, g + 16, g + 24 of the quarter
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        mu[r] = kNone;
        l[r] = 0.0f;
      }
      int pos = static_cast<int>(axis.piece_begin) * kTilePos + part * 32;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i, pos += kTilePos, ++n) {
        const uint32_t st = n & 1, ph = n >> 1;
        // not K's own barrier, which may be two tiles on by now: a waiter must
        // never be more than one phase behind.  The scales have four stages, and
        // none is written again before this warp's P of the tile that it holds
        wait(kScFull + (n & 3), n >> 2);
        wait(kSFull + st, ph);
        tc_fence_after();
        if (active) {
          const uint32_t s_at = lanes + kColS + st * 128 + part * 32;
          const uint8_t* sc = smem + C::kScaleOffset + (n & 3) * C::kScaleStage;
          uint32_t p[2][8];   // [hh][2 j + h]: 8-position groups j, rows g + 8 h + 16 hh
          float add[4];
          bool raised = false;
          for (;;) {
            // x of the 32 positions: [hh][4 j + 2 h + e]
            float x[2][16];
            tmem_ld_16x256b_x4(s_at, x[0]);
            tmem_ld_16x256b_x4(s_at + (16u << 16), x[1]);
            tmem_wait_ld();
            loaded(x[0]);
            loaded(x[1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 v = reinterpret_cast<const float4*>(sc)[part * 16 + 4 * j + t];
              const F2 sk2 = mul2(f2(v.x, v.y), unlift2), lg2 = f2(v.z, v.w);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float& x0 = x[r >> 1][4 * j + 2 * (r & 1)];
                float& x1 = x[r >> 1][4 * j + 2 * (r & 1) + 1];
                un2(fma2(f2(x0, x1), sk2, lg2), x0, x1);
              }
            }
            if (context - pos < 32) {
#pragma unroll 1
              for (int r = 0; r < 4; ++r) {
                const uint64_t m = masks[quarter * 32 + 8 * r + g];
                uint32_t seen = 0;   // bit 2 j + e
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int ahead = pos - context + 8 * j + 2 * t + e;
                    if (ahead < 0 || (ahead < nodes && (m >> ahead & 1))) seen |= 1u << (2 * j + e);
                  }
#pragma unroll
                for (int rr = 0; rr < 4; ++rr)
                  if (rr == r)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                      for (int e = 0; e < 2; ++e)
                        if (!(seen >> (2 * j + e) & 1)) x[rr >> 1][4 * j + 2 * (rr & 1) + e] = -INFINITY;
              }
            }
            __half2 high[4];
            F2 sum[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              high[r] = as_h2(0u);
              sum[r] = f2(0.0f, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 v = reinterpret_cast<const float2*>(sc + 1024)[part * 16 + 4 * j + t];
              const F2 inv2 = f2(v.x, v.y);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float d0, d1;
                un2(add2(f2(x[r >> 1][4 * j + 2 * (r & 1)], x[r >> 1][4 * j + 2 * (r & 1) + 1]),
                         f2(-mu[r], -mu[r])), d0, d1);
                const float p0 = exp2_approx(d0), p1 = exp2_approx(d1);
                sum[r] = fma2(f2(p0, p1), inv2, sum[r]);
                const uint32_t u = pack_h2(p0, p1);
                high[r] = __hmax2(high[r], as_h2(u));
                p[r >> 1][2 * j + (r & 1)] = u;
              }
            }
            bool over = false;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float s0, s1;
              un2(sum[r], s0, s1);
              add[r] = s0 + s1;
              over |= __half2float(__hmax(__low2half(high[r]), __high2half(high[r]))) > 16384.0f;
            }
            if (raised || !barrier_or(quarter_bar, 32 * kParts, over)) break;
            // some row's m is raised: its maximum over the tile, from all parts
            raised = true;
            float top[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              top[r] = -INFINITY;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                top[r] = fmaxf(top[r], fmaxf(x[r >> 1][4 * j + 2 * (r & 1)], x[r >> 1][4 * j + 2 * (r & 1) + 1]));
              top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
              top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
              if (t == 0) my_stat[8 * r + g].x = top[r];
            }
            named_barrier_sync(quarter_bar, 32 * kParts);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int w = 0; w < kParts; ++w)
                top[r] = fmaxf(top[r], stat[w * kTileRows + quarter * 32 + 8 * r + g].x);
              float f = 1.0f;
              if (top[r] > mu[r] + 14.0f) {
                const float now = top[r] - 6.0f;   // p' is 2^6 for the largest
                f = exp2_approx(mu[r] - now);
                l[r] *= f;
                mu[r] = now;
              }
              if (t == 0) my_stat[8 * r + g].y = f;
            }
            if (i > 0) {   // this warp's columns of O; the products so far are done
              wait(kVEmpty + ((n - 1) & 1), (n - 1) >> 1);
              tc_fence_after();
              __syncwarp();
              const float f = my_stat[lane].y;
              uint32_t o[kCols];
              tmem_ld_row(lanes + kColO + part * kCols, o);
              tmem_wait_ld();
              loaded(o);
#pragma unroll
              for (int j = 0; j < kCols; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_row(lanes + kColO + part * kCols, o);
            }
            // the others have read this warp's maxima before they are written again
            named_barrier_sync(quarter_bar, 32 * kParts);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) l[r] += add[r];
          // P over this part's own columns of S
          tmem_st_16x128b_x4(s_at, p[0]);
          tmem_st_16x128b_x4(s_at + (16u << 16), p[1]);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPReady + st));
      }

      // ------------------------------------------------------------ the output
      const bool whole = axis.whole();
      const int slot = axis.slot(), my_rows = rows;
      const int64_t my_out = out_at;
      more = axis.next(a, kTilePos, kTileRows);
      if (more) load_q();   // on its way during the output
      if (active) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
          l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
          if (t == 0) my_stat[8 * r + g] = make_float2(mu[r], l[r]);
        }
        named_barrier_sync(quarter_bar, 32 * kParts);
      }
      wait(kOFull, piece);
      tc_fence_after();
      if (active) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kParts; ++w) sum += stat[w * kTileRows + row].y;
        const float m = stat[row].x;
        const float top = m == kNone ? -INFINITY : m;
        const float codes = BITS == 4 ? 512.0f : 1.0f;
        const float f = whole ? (sum > 0.0f ? codes / sum : 0.0f) : codes;
        uint32_t o[kCols];
        tmem_ld_row(lanes + kColO + part * kCols, o);
        tmem_wait_ld();
        loaded(o);
        if (row < my_rows) {
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) {
            const int d = C::dim_of(part * (kCols / 8) + j);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)   // INT4 units hold the dims 0 4 1 5 2 6 3 7
              v[BITS == 4 ? (e & 1) * 4 + (e >> 1) : e] = __uint_as_float(o[8 * j + e]) * f;
            const float4 lo = make_float4(v[0], v[1], v[2], v[3]), hi = make_float4(v[4], v[5], v[6], v[7]);
            if (whole) {
              store_out4(a.out, bf16, my_out + d, lo, 1.0f);
              store_out4(a.out, bf16, my_out + d + 4, hi, 1.0f);
            } else {
              parts.store(slot, row, D, d, lo, top, sum);
              parts.store(slot, row, D, d + 4, hi, top, sum);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOEmpty));
      // every warp is past this piece's statistics and masks before they are written again
      named_barrier_sync(6, 32 * kSoftWarps);
      ++piece;
    }
  }
  __syncwarp();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kColAll);
  }
}

template <int D, int BITS>
cudaError_t launch_tree(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  using C = TreeCfg<D, BITS>;
  static_assert(C::kSmem <= 232448, "shared memory budget");
  const void* kern = reinterpret_cast<const void*>(tree_kernel<D, BITS>);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_max_dynamic_smem(kern, C::kSmem, done);
  if (e != cudaSuccess) return e;
  // the warpgroups' register increase draws on what the CTA was launched with
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    regs.store(attr.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  PartsArgs parts;
  ScratchSource scratch = ScratchSource::pooled(st);
  e = parts.allocate(scratch, num_sms, kTileRows, D);
  if (e != cudaSuccess) return e;
  tree_kernel<D, BITS><<<num_sms, kThreads, C::kSmem, st>>>(a, parts, bf16);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join(a, parts, num_sms, std::min(kTileRows, a.max_nodes * (a.q_heads / a.cache.heads)),
                     bf16, st);
}

}  // namespace

cudaError_t launch_attend_tree(const AttendArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  if (a.cache.head_dim == 128)
    return a.cache.bits == 8 ? launch_tree<128, 8>(a, bf16, num_sms, st)
                             : launch_tree<128, 4>(a, bf16, num_sms, st);
  return a.cache.bits == 8 ? launch_tree<64, 8>(a, bf16, num_sms, st)
                           : launch_tree<64, 4>(a, bf16, num_sms, st);
}

}  // namespace cider
