// kv_common.cuh -- the paged, quantized key/value cache as the kernels see it.
//
// One layer's keys (and likewise values) are [pages][heads][page size][D]
// codes, INT8 or two INT4 per byte (element 2j in the low nibble), and
// [pages][heads][page size] fp32 scales.  A head's rows of one page lie next
// to each other: 16 tokens of 128 INT8 codes are one run of 2 KiB.  Row
// numbers and byte offsets are 64-bit: a cache may be larger than 2^32 bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace cider {

// A page, slot, offset or count outside of what the caller gave: the access
// is skipped and this bit of the device error word set.
constexpr int kDevErrIndex = 2;

// A value row of zeros has scale 1.  It adds nothing to an output however large
// its weight, so its scale must not set the maximum that the other weights are
// rounded against: the attention takes it as 2^-60, far below the scales of
// ordinary values (fp16's lie in 2^-31 .. 2^9) and far enough above fp32's least
// number that its weight still counts in the sum (down to 2^-63 of the others'
// for scales of 2^9).  Only rows of scale 1 are looked at.
constexpr float kZeroRowScale = 0x1p-60f;

constexpr int kMaxNodes = 64;   // new tokens of one request: a mask is 64 bits

struct KvCache {
  uint8_t* k;
  float* k_scale;
  uint8_t* v;
  float* v_scale;
  int64_t pages;
  int heads, page_shift, head_dim, bits;

  __host__ __device__ int64_t layer_rows() const { return (pages * heads) << page_shift; }
  __host__ __device__ int64_t row(int64_t page, int head, int at) const {
    return ((page * heads + head) << page_shift) + at;
  }
};

// The last request that begins at or before row i, or -1 when i belongs to none.
__device__ __forceinline__ int find_request(const int32_t* offsets, int requests, int64_t i) {
  int lo = 0, hi = requests;   // offsets[lo] <= i < offsets[hi], if they are in order
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= i) lo = mid; else hi = mid;
  }
  return offsets[lo] <= i && i < offsets[lo + 1] ? lo : -1;
}

// Row (within a layer) of request b's position `pos` for `head`, or -1 when
// the table has no such page.
__device__ __forceinline__ int64_t cache_row_of(const KvCache& c, const int32_t* table,
                                                int64_t table_width, int64_t b, int64_t pos,
                                                int head) {
  const int64_t i = pos >> c.page_shift;
  if (pos < 0 || i >= table_width) return -1;
  const int64_t page = table[b * table_width + i];
  if (page < 0 || page >= c.pages) return -1;
  return c.row(page, head, static_cast<int>(pos & ((1 << c.page_shift) - 1)));
}

// One attention call, as the C entry point receives it.
struct AttendArgs {
  KvCache cache;                 // of the layer
  const void* q;                 // [rows][q_heads][D], q_stride elements between rows
  int64_t q_stride, rows;
  int q_heads;
  const int32_t* table;          // [requests][table_width] page numbers
  int64_t table_width;
  const int32_t *lengths, *offsets;
  int requests, max_nodes;
  const int64_t* tree;           // [rows] masks, or null: every earlier token
  float scale;
  void* out;                     // [rows][q_heads][D]
  int* err;
};

// Request b's new tokens (rows first .. first + nodes) and positions.  Offsets
// and lengths that contradict each other or the call's sizes set the error
// bit; then nodes is 0.
struct Request {
  int64_t first, length, context;
  int nodes;
};
__device__ __forceinline__ Request request_of(const AttendArgs& a, int b, bool report = true) {
  Request r;
  r.first = a.offsets[b];
  const int64_t end = a.offsets[b + 1];
  r.length = a.lengths[b];
  const int64_t n = end - r.first;
  const bool bad = n != 0 && (r.first < 0 || n < 0 || end > a.rows || n > a.max_nodes ||
                              r.length < n || r.length > a.table_width << a.cache.page_shift);
  if (bad && report) atomicOr(a.err, kDevErrIndex);
  r.nodes = bad ? 0 : static_cast<int>(n);
  r.context = r.length - r.nodes;
  return r;
}

// Eight packed 16-bit values -> fp32, exactly.
template <typename T>
__device__ __forceinline__ void widen8(const uint4& in, float (&f)[8]) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 p;
    if constexpr (std::is_same<T, __half>::value) {
      __half2 h;
      memcpy(&h, &w[j], 4);
      p = __half22float2(h);
    } else {
      __nv_bfloat162 h;
      memcpy(&h, &w[j], 4);
      p = __bfloat1622float2(h);
    }
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
}

}  // namespace cider
