// kv_parts.cuh -- how the attention kernels share out their work, and how the
// parts of a request that was cut are joined.
//
// The axis: every (request, key/value head, block of query rows) is a unit of
// ceil(length / tile) tiles; the units of all requests lie one after another.
// CTA c of C <= N takes the tiles [N c / C, N (c + 1) / C) of the N: at most two of
// its pieces are parts of cut units, the first (continuing a unit) and the last.
// Each CTA finds its share from the lengths alone, so the host need not know
// them, and the same lengths are always cut in the same places.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cider_internal.h"
#include "kv_common.cuh"

namespace cider {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Axis {
  Request req;          // of request b
  int b, unit;          // unit: head * (the request's row blocks) + row block
  int64_t unit_begin;   // the unit's first tile on the axis
  int64_t unit_tiles;
  int64_t at, end;      // this CTA's current tile and the end of its share
  int64_t piece_begin, piece_end;   // tiles within the unit
  int64_t total;        // tiles of the axis
  bool continued;       // the unit began in an earlier share

  __device__ static int64_t tiles_of(const Request& r, int tile) {
    return r.nodes == 0 ? 0 : (r.length + tile - 1) / tile;
  }
  // Row blocks per head of a request.
  __device__ static int blocks_of(const AttendArgs& a, int nodes, int block_rows) {
    return (nodes * (a.q_heads / a.cache.heads) + block_rows - 1) / block_rows;
  }
  __device__ static int blocks_of(const AttendArgs& a, const Request& r, int block_rows) {
    return blocks_of(a, r.nodes, block_rows);
  }
  // Called by whole warps; block_rows: query rows of a unit at most.
  __device__ void begin(const AttendArgs& a, int tile, int lane, int block_rows) {
    total = 0;
    for (int b0 = 0; b0 < a.requests; b0 += 32) {
      const int i = b0 + lane;
      if (i < a.requests) {
        const Request r = request_of(a, i, blockIdx.x == 0);
        total += tiles_of(r, tile) * a.cache.heads * blocks_of(a, r, block_rows);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // with fewer tiles than CTAs the first ones take one tile each, so that no
    // empty share lies between two parts of a unit
    const int64_t ctas = min(total, static_cast<int64_t>(gridDim.x));
    const bool works = blockIdx.x < ctas;
    at = works ? total * blockIdx.x / ctas : 0;
    end = works ? total * (blockIdx.x + 1) / ctas : 0;
    if (!works) return;
    int64_t before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int i = b0 + lane;
      int64_t mine = 0;
      if (i < a.requests) {
        const Request r = request_of(a, i, false);
        mine = tiles_of(r, tile) * a.cache.heads * blocks_of(a, r, block_rows);
      }
      int64_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + sum > at);
      if (hit) {
        const int l = __ffs(hit) - 1;
        before += __shfl_sync(0xffffffffu, sum - mine, l);
        b = b0 + l;
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    req = request_of(a, b, false);
    unit_tiles = tiles_of(req, tile);
    unit = static_cast<int>((at - before) / unit_tiles);
    unit_begin = before + unit * unit_tiles;
    cut();
  }
  __device__ void cut() {
    continued = at > unit_begin;
    piece_begin = at - unit_begin;
    piece_end = min(unit_tiles, end - unit_begin);
  }
  __device__ bool more() const { return at < end; }
  __device__ bool whole() const { return piece_begin == 0 && piece_end == unit_tiles; }
  // Where a part goes: two slots per CTA.
  __device__ int slot() const { return 2 * blockIdx.x + (continued ? 0 : 1); }
  __device__ bool next(const AttendArgs& a, int tile, int block_rows) {
    at = unit_begin + piece_end;
    if (at >= end) return false;
    unit_begin += unit_tiles;
    if (++unit == a.cache.heads * blocks_of(a, req, block_rows)) {
      unit = 0;
      do {
        req = request_of(a, ++b, false);
        unit_tiles = tiles_of(req, tile);
      } while (unit_tiles == 0);
    }
    cut();
    return true;
  }
};

// Parts of cut units: unnormalised outputs, their maxima and sums.
struct PartsArgs {
  float* out;       // [2 ctas][rows][D]
  float2* stat;     // [2 ctas][rows]: maximum (log2), sum
  // Of a share that begins within a unit: the unit's first and end tile on the
  // axis, the axis' length, the unit, and its request's first row and number of
  // new tokens; else begin is -1.
  struct Info {
    int64_t begin, end, total, first;
    int unit, nodes;
  };
  Info* info;       // [ctas]
  int rows;

  cudaError_t allocate(ScratchSource& scratch, int ctas, int rows_, int d) {
    rows = rows_;
    const size_t o = static_cast<size_t>(2) * ctas * rows * d * 4;
    const size_t s = static_cast<size_t>(2) * ctas * rows * 8;
    void* p = nullptr;
    if (scratch.get(o + s + static_cast<size_t>(ctas) * sizeof(Info), &p) != CIDER_OK)
      return cudaErrorMemoryAllocation;
    out = static_cast<float*>(p);
    stat = reinterpret_cast<float2*>(static_cast<char*>(p) + o);
    info = reinterpret_cast<Info*>(static_cast<char*>(p) + o + s);
    return cudaSuccess;
  }
  __device__ void announce(const Axis& x) const {
    const bool mid = x.more() && x.continued;
    info[blockIdx.x] = mid ? Info{x.unit_begin, x.unit_begin + x.unit_tiles, x.total, x.req.first, x.unit,
                                  x.req.nodes}
                           : Info{-1, -1, 1, 0, 0, 0};
  }
  __device__ void store(int slot, int row, int d_all, int d, const float4& v, float top,
                        float sum) const {
    const int64_t r = static_cast<int64_t>(slot) * rows + row;
    *reinterpret_cast<float4*>(out + r * d_all + d) = v;
    if (d == 0) stat[r] = make_float2(top, sum);
  }
};

// Four outputs, each rounded once.
__device__ __forceinline__ void store_out4(void* out, bool bf16, int64_t at, const float4& v,
                                           float f) {
  uint2 u;
  if (bf16)
    u = make_uint2(y_bits2<true>(v.x * f, v.y * f), y_bits2<true>(v.z * f, v.w * f));
  else
    u = make_uint2(y_bits2<false>(v.x * f, v.y * f), y_bits2<false>(v.z * f, v.w * f));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = u;
}

// Joins the parts of every cut unit (kv_attention.cu).  rows: at most this many
// rows of a unit exist; its kernel is a programmatic dependent of the launch before.
cudaError_t launch_join(const AttendArgs& a, const PartsArgs& parts, int ctas, int rows, bool bf16,
                        cudaStream_t st);

}  // namespace cider
