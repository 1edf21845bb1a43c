// fp4_api.cu -- C entry points of microscaled 4-bit floating point: argument
// checks in the order that include/cider.h states, the device check, scratch
// from the library's pool, then the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cider.h"
#include "cider_internal.h"
#include "fp4_common.cuh"

namespace {

constexpr int64_t kMaxDim = 2147483647;
constexpr int64_t kMaxK = 131072;
constexpr int64_t kMaxTiles = 1 << 30;   // output tiles of a product, CTAs of a quantization

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cider_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return CIDER_OK;
  cudaGetLastError();
  return CIDER_ERR_CUDA;
}

template <typename F>
cider_status_t guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return CIDER_ERR_CUDA;
  }
}

bool valid16(int dtype) { return dtype == CIDER_F16 || dtype == CIDER_BF16; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Sizes and pointers of a matrix with rows.
bool valid(const cider_fp4_t* q) {
  return q && q->codes && q->scales && q->rows >= 0 && q->rows <= kMaxDim && q->cols >= 32 &&
         q->cols <= kMaxK && q->cols % 32 == 0 && (q->block_size == 16 || q->block_size == 32);
}
bool well_aligned(const cider_fp4_t* q) {
  return aligned(q->codes, 16) && aligned(q->scales, 16) && aligned(q->row_scale, 4);
}
cider::FpMat mat(const cider_fp4_t* q) { return cider::FpMat{q->codes, q->scales, q->row_scale, q->rows}; }

// A row stride in elements: at least a row, whole 16-byte units.
bool valid_stride(int64_t stride, int64_t cols, int bytes) {
  return stride >= cols && stride % (16 / bytes) == 0 && stride <= (int64_t{1} << 40);
}

// Codes, block scales and row scales of `rows` x `cols` in scratch memory.
struct Held {
  size_t codes, scales, row;
  Held(int64_t rows, int64_t cols, int block)
      : codes(round256(static_cast<size_t>(rows) * cols / 2)),
        scales(static_cast<size_t>((rows + 127) / 128) * cider::fp4_tiles(cols, block) * cider::kFpTileBytes),
        row(block == 16 ? round256(static_cast<size_t>(rows) * 4) : 0) {}
  size_t bytes() const { return codes + scales + row; }
  cider::FpMat at(uint8_t* base, int64_t rows) const {
    return cider::FpMat{base, base + codes, row ? reinterpret_cast<const float*>(base + codes + scales) : nullptr, rows};
  }
};

// Few tokens: 128 rows of weights a CTA, K split.  Up to 64 tokens, or where its tiles of 64 (128, if not
// gated) tokens are at most half as many as the SMs.  Measured (us, that against pairs of 256 x 256), weights
// from memory: 64 tokens through 10240 x 2560 8.6, 9.3, gated 12288 x 4096 16.0, 19.0, gated 6144 x 2048 9.1,
// 9.5; 96 through 10240 x 2560 9.7, 9.5, gated 6144 x 2048 9.9, 9.8; 128 through 4096 x 4096 8.8, 10.9; 256
// through 1024 x 4096 6.8, 10.2, through 2560 x 10240 13.0, 17.7; 512 through 2048 x 6144 11.0, 13.0, gated
// 1024 x 1024 6.8, 7.2; 768 through 2048 x 6144 13.8, 12.9, gated 1024 x 1024 7.7, 7.2.
bool few_rows(const cider::FpProduct& p) {
  const int64_t rows = (p.N + 127) / 128, half = p.num_sms / 2;
  return p.M <= 64 || (p.M + 63) / 64 * rows <= half || (!p.is_gated && (p.M + 127) / 128 * rows <= half);
}

// Few enough that the product's kernel quantizes the rows itself, each CTA its part of K: one launch
// instead of two.  Not where y lies on x: CTAs that are done would write what others still read.  A null x
// or y is scratch of the call, which neither the caller's matrices nor other scratch overlap.
bool quantizes_itself(const cider::FpProduct& p, const void* x, const void* y) {
  if (!few_rows(p) || !cider::fp4_rows_quantizes_itself(p)) return false;
  if (!x || !y) return true;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  const uintptr_t xn = 2 * ((p.M - 1) * p.x_stride + p.K), yn = 2 * p.M * p.N;
  return !(x0 < y0 + yn && y0 < x0 + xn);
}

// A product of x in 16 bits: quantized by the product's kernel (`itself`: what quantizes_itself said when
// the scratch was sized), or into `held` (scratch) first.
cudaError_t product(cider::FpProduct& p, bool itself, const cider::FpMat& held) {
  if (p.wide_x) {
    if (itself) return cider::launch_fp4_rows(p);
    const cudaError_t e = cider::launch_quantize_fp4(
        p.wide_x, p.x_bf16 ? CIDER_BF16 : CIDER_F16, p.x_stride, p.M, p.K, p.block, const_cast<uint8_t*>(held.codes),
        const_cast<uint8_t*>(held.scales), const_cast<float*>(held.row), false, p.num_sms, p.st, true);
    if (e != cudaSuccess) return e;
    p.x = held;
    p.wide_x = nullptr;
    p.after_launch = true;
  }
  return few_rows(p) ? cider::launch_fp4_rows(p) : cider::launch_fp4_pair(p);
}

// One product's arguments, as the entry points receive them.
struct Call {
  const void* x = nullptr;   // or qx
  int x_dtype = CIDER_F16;
  int64_t x_stride = 0, M = 0;
  const cider_fp4_t* qx = nullptr;
  const cider_fp4_t *w = nullptr, *up = nullptr, *down = nullptr;
  bool gated = false;
  int act = 0;
  void* y = nullptr;
  int y_dtype = CIDER_F16;
  void* stream = nullptr;
};

cider_status_t check(const Call& c, int64_t M, int64_t N) {
  if (M < 0 || M > kMaxDim || !c.y || !valid(c.w) || N % 8 != 0) return CIDER_ERR_INVALID_ARGUMENT;
  const int64_t K = c.w->cols;
  const int block = c.w->block_size;
  if (c.gated) {
    if (!valid(c.up) || c.up->rows != c.w->rows || c.up->cols != K || c.up->block_size != block ||
        (c.act != CIDER_SILU && c.act != CIDER_GELU))
      return CIDER_ERR_INVALID_ARGUMENT;
  }
  if (c.down && (!valid(c.down) || c.down->cols != c.w->rows || c.down->block_size != block || c.w->rows % 32 != 0))
    return CIDER_ERR_INVALID_ARGUMENT;
  if (c.qx) {
    if (!valid(c.qx) || c.qx->cols != K || c.qx->block_size != block) return CIDER_ERR_INVALID_ARGUMENT;
  } else if (!c.x || !valid16(c.x_dtype) || !valid_stride(c.x_stride, K, 2)) {
    return CIDER_ERR_INVALID_ARGUMENT;
  }
  if (!valid16(c.y_dtype)) return CIDER_ERR_INVALID_ARGUMENT;
  if (((M + 127) / 128) * ((N + 127) / 128) > kMaxTiles) return CIDER_ERR_INVALID_ARGUMENT;
  if (c.down && ((M + 127) / 128) * ((c.w->rows + 127) / 128) > kMaxTiles) return CIDER_ERR_INVALID_ARGUMENT;
  if (!well_aligned(c.w) || (c.gated && !well_aligned(c.up)) || (c.down && !well_aligned(c.down)) ||
      (c.qx ? !well_aligned(c.qx) : !aligned(c.x, 16)) || !aligned(c.y, 16))
    return CIDER_ERR_MISALIGNED;
  return CIDER_OK;
}

cider_status_t run(const Call& c) {
  return guarded([&]() -> cider_status_t {
    const cider_fp4_t* last = c.down ? c.down : c.w;
    if (!last) return CIDER_ERR_INVALID_ARGUMENT;
    const int64_t M = c.qx ? c.qx->rows : c.M, N = last->rows;
    if (M == 0 || N == 0) return CIDER_OK;
    cider_status_t s = check(c, M, N);
    if (s != CIDER_OK) return s;
    int sms = 0;
    s = cider::check_device(nullptr, &sms);
    if (s != CIDER_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(c.stream);
    const int64_t K = c.w->cols, F = c.w->rows;
    const int block = c.w->block_size;
    cider::FpProduct p;
    p.w = mat(c.w);
    if (c.gated) p.up = mat(c.up);
    p.is_gated = c.gated;
    p.act = c.act;
    p.M = M;
    p.N = F;
    p.K = K;
    p.block = block;
    p.num_sms = sms;
    p.st = st;
    if (c.qx) p.x = mat(c.qx);
    p.wide_x = c.qx ? nullptr : c.x;
    p.x_stride = c.x_stride;
    p.x_bf16 = c.x_dtype == CIDER_BF16;
    p.y_bf16 = (c.down ? c.x_dtype : c.y_dtype) == CIDER_BF16;
    cider::FpProduct d;
    if (c.down) {
      d.w = mat(c.down);
      d.M = M;
      d.N = N;
      d.K = F;
      d.block = block;
      d.num_sms = sms;
      d.st = st;
      d.x_stride = F;
      d.x_bf16 = p.x_bf16;
      d.y = c.y;
      d.y_bf16 = c.y_dtype == CIDER_BF16;
    }
    // scratch: x's codes and scales; for a whole block the hidden values, their codes and scales.  Block
    // size 32: the first product writes the hidden values quantized.  Block size 16 needs their rows' maxima.
    const bool straight = c.down && block == 32;
    // Who quantizes is decided here alone: the launches below follow it.
    const bool first = p.wide_x && quantizes_itself(p, c.x, c.down ? nullptr : c.y),
               second = c.down && !straight && quantizes_itself(d, nullptr, c.y);
    const Held hx(p.wide_x && !first ? M : 0, K, block), hh(c.down && !second ? M : 0, c.down ? F : 32, block);
    const size_t wide = c.down && !straight ? round256(static_cast<size_t>(M) * F * 2) : 0;
    cider::ScratchSource scratch = cider::ScratchSource::pooled(st);
    uint8_t* base = nullptr;
    if (hx.bytes() + wide + hh.bytes() > 0) {
      void* ptr = nullptr;
      s = scratch.get(hx.bytes() + wide + hh.bytes(), &ptr);
      if (s != CIDER_OK) return s;
      base = static_cast<uint8_t*>(ptr);
    }
    const cider::FpMat hidden = hh.at(base + hx.bytes() + wide, M);
    p.y = c.down ? base + hx.bytes() : c.y;
    if (straight) {
      p.q_codes = const_cast<uint8_t*>(hidden.codes);
      p.q_scales = const_cast<uint8_t*>(hidden.scales);
    }
    const cudaError_t e = product(p, first, hx.at(base, M));
    if (e != cudaSuccess || !c.down) return cuda_status(e);
    // its weights do not depend on the launch before
    d.after_launch = true;
    if (straight)
      d.x = hidden;
    else
      d.wide_x = p.y;
    return cuda_status(product(d, second, hidden));
  });
}

}  // namespace

extern "C" {

cider_status_t cider_quantize_fp4(const void* x, int x_dtype, int64_t x_stride, const cider_fp4_t* q,
                                  void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!q) return CIDER_ERR_INVALID_ARGUMENT;
    if (q->rows == 0) return CIDER_OK;
    if (!valid(q) || !x || (!valid16(x_dtype) && x_dtype != CIDER_F32) ||
        (q->block_size == 16) != (q->row_scale != nullptr) || (q->rows + 127) / 128 * 128 > kMaxTiles ||
        !valid_stride(x_stride, q->cols, x_dtype == CIDER_F32 ? 4 : 2))
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !well_aligned(q)) return CIDER_ERR_MISALIGNED;
    int sms = 0;
    const cider_status_t s = cider::check_device(nullptr, &sms);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_quantize_fp4(x, x_dtype, x_stride, q->rows, q->cols, q->block_size, q->codes,
                                                  q->scales, q->row_scale, true, sms,
                                                  static_cast<cudaStream_t>(stream), false));
  });
}

cider_status_t cider_dequantize_fp4(const cider_fp4_t* q, void* x, int x_dtype, void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!q) return CIDER_ERR_INVALID_ARGUMENT;
    if (q->rows == 0) return CIDER_OK;
    if (!valid(q) || !x || (!valid16(x_dtype) && x_dtype != CIDER_F32)) return CIDER_ERR_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !well_aligned(q)) return CIDER_ERR_MISALIGNED;
    int sms = 0;
    const cider_status_t s = cider::check_device(nullptr, &sms);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_dequantize_fp4(mat(q), q->cols, q->block_size, x, x_dtype, sms,
                                                    static_cast<cudaStream_t>(stream)));
  });
}

cider_status_t cider_w4a4_linear(const void* x, int x_dtype, int64_t x_stride, int64_t M, const cider_fp4_t* w,
                                 void* y, int y_dtype, void* stream) {
  Call c;
  c.x = x;
  c.x_dtype = x_dtype;
  c.x_stride = x_stride;
  c.M = M;
  c.w = w;
  c.y = y;
  c.y_dtype = y_dtype;
  c.stream = stream;
  return run(c);
}

cider_status_t cider_w4a4_linear_prequant(const cider_fp4_t* x, const cider_fp4_t* w, void* y, int y_dtype,
                                          void* stream) {
  if (!x) return CIDER_ERR_INVALID_ARGUMENT;
  Call c;
  c.qx = x;
  c.w = w;
  c.y = y;
  c.y_dtype = y_dtype;
  c.stream = stream;
  return run(c);
}

cider_status_t cider_w4a4_gated_linear(const void* x, int x_dtype, int64_t x_stride, int64_t M,
                                       const cider_fp4_t* gate, const cider_fp4_t* up, int activation, void* h,
                                       int h_dtype, void* stream) {
  Call c;
  c.x = x;
  c.x_dtype = x_dtype;
  c.x_stride = x_stride;
  c.M = M;
  c.w = gate;
  c.up = up;
  c.gated = true;
  c.act = activation;
  c.y = h;
  c.y_dtype = h_dtype;
  c.stream = stream;
  return run(c);
}

cider_status_t cider_w4a4_gated_linear_prequant(const cider_fp4_t* x, const cider_fp4_t* gate,
                                                const cider_fp4_t* up, int activation, void* h, int h_dtype,
                                                void* stream) {
  if (!x) return CIDER_ERR_INVALID_ARGUMENT;
  Call c;
  c.qx = x;
  c.w = gate;
  c.up = up;
  c.gated = true;
  c.act = activation;
  c.y = h;
  c.y_dtype = h_dtype;
  c.stream = stream;
  return run(c);
}

cider_status_t cider_w4a4_feed_forward(const void* x, int x_dtype, int64_t x_stride, int64_t M,
                                       const cider_fp4_t* gate, const cider_fp4_t* up, const cider_fp4_t* down,
                                       int activation, void* y, int y_dtype, void* stream) {
  if (!down) return CIDER_ERR_INVALID_ARGUMENT;
  Call c;
  c.x = x;
  c.x_dtype = x_dtype;
  c.x_stride = x_stride;
  c.M = M;
  c.w = gate;
  c.up = up;
  c.down = down;
  c.gated = true;
  c.act = activation;
  c.y = y;
  c.y_dtype = y_dtype;
  c.stream = stream;
  return run(c);
}

}  // extern "C"
