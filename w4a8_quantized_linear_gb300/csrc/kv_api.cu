// kv_api.cu -- C entry points of the quantized key/value cache, the attention
// over it and the verification of drafted tokens: argument checks in the order
// that include/cider.h states, the device check, then one launch (two where
// attention joins parts).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cider.h"
#include "cider_internal.h"
#include "kv_common.cuh"

namespace {

constexpr int64_t kMaxDim = 2147483647;
constexpr int64_t kMaxGrid = 65535;   // blocks of a grid's second and third dimension

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

bool valid_dtype(int dtype) { return dtype == CIDER_F16 || dtype == CIDER_BF16; }

// Sizes and pointers of a cache that is not empty.
cider_status_t check_cache(const cider_kv_cache_t& c) {
  if (!c.k || !c.k_scale || !c.v || !c.v_scale) return CIDER_ERR_INVALID_ARGUMENT;
  if (c.layers < 0 || c.layers > kMaxGrid || c.pages < 0 || c.pages > kMaxDim || c.heads < 1 ||
      c.heads > kMaxGrid)
    return CIDER_ERR_INVALID_ARGUMENT;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    return CIDER_ERR_INVALID_ARGUMENT;
  // 16-row blocks of a layer are counted in 32 bits
  if (c.pages > kMaxDim / c.heads / (c.page_size / 16)) return CIDER_ERR_INVALID_ARGUMENT;
  if ((c.head_dim != 64 && c.head_dim != 128) || (c.bits != 8 && c.bits != 4))
    return CIDER_ERR_INVALID_ARGUMENT;
  return CIDER_OK;
}

bool cache_aligned(const cider_kv_cache_t& c) {
  return aligned(c.k, 16) && aligned(c.k_scale, 16) && aligned(c.v, 16) && aligned(c.v_scale, 16);
}

// One layer of the cache, as the kernels take it.
cider::KvCache layer_of(const cider_kv_cache_t& c, int64_t layer) {
  cider::KvCache k;
  k.pages = c.pages;
  k.heads = c.heads;
  k.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  k.head_dim = c.head_dim;
  k.bits = c.bits;
  const int64_t rows = layer * k.layer_rows(), bytes = rows * c.head_dim * c.bits / 8;
  k.k = static_cast<uint8_t*>(c.k) + bytes;
  k.v = static_cast<uint8_t*>(c.v) + bytes;
  k.k_scale = c.k_scale + rows;
  k.v_scale = c.v_scale + rows;
  return k;
}

// The device check and the error word of the current device.
cider_status_t device(int** err, int* num_sms) {
  const cider_status_t s = cider::check_device(nullptr, num_sms);
  if (s != CIDER_OK) return s;
  return cuda_status(cider::device_error_word(err));
}

// A verification whose waits between CTAs end after wait_ns; rank `silent` of
// each cluster sends nothing (-1: all send).
cider_status_t verify(const void* logits, int64_t logits_stride, int dtype,
                      const int32_t* tokens, const int32_t* parents,
                      const int32_t* offsets, int64_t requests, int64_t nodes,
                      int64_t vocab, int64_t max_nodes, const float* uniforms,
                      const float* noise, const float* draft,
                      const float* temperature, int32_t* count, int32_t* path,
                      int32_t* next, void* stream, uint64_t wait_ns, int silent) {
  return guarded([&]() -> cider_status_t {
    if (requests == 0) return CIDER_OK;
    // without a single node there is nothing behind the nodes' pointers
    if ((nodes != 0 && (!logits || !tokens || !parents || !uniforms)) || !offsets || !noise ||
        !count || !path || !next || !valid_dtype(dtype) || requests < 0 || requests > kMaxDim || nodes < 0 ||
        nodes > kMaxDim || vocab < 1 || vocab > kMaxDim || max_nodes < 1 ||
        max_nodes > cider::kMaxNodes || logits_stride < vocab)
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!aligned(logits, 2) || !aligned(tokens, 4) || !aligned(parents, 4) || !aligned(offsets, 4) ||
        !aligned(uniforms, 4) || !aligned(noise, 4) || !aligned(draft, 4) ||
        !aligned(temperature, 4) || !aligned(count, 4) || !aligned(path, 4) || !aligned(next, 4))
      return CIDER_ERR_MISALIGNED;
    int* err = nullptr;
    int sms = 0;
    cider_status_t s = device(&err, &sms);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_verify(
        logits, logits_stride, dtype == CIDER_BF16, tokens, parents, offsets,
        static_cast<int>(requests), nodes, static_cast<int>(vocab), static_cast<int>(max_nodes),
        uniforms, noise, draft, temperature, count, path, next, err, sms,
        static_cast<cudaStream_t>(stream), wait_ns, silent));
  });
}

}  // namespace

extern "C" {

cider_status_t cider_kv_append(const cider_kv_cache_t* cache, int64_t layer, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, int dtype,
                               const int64_t* slots, int64_t tokens, void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!cache) return CIDER_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || cache->pages == 0 || cache->layers == 0) return CIDER_OK;
    cider_status_t s = check_cache(*cache);
    if (s != CIDER_OK) return s;
    const int64_t width = static_cast<int64_t>(cache->heads) * cache->head_dim;
    if (!k || !v || !slots || !valid_dtype(dtype) || layer < 0 || layer >= cache->layers ||
        tokens < 0 || tokens > kMaxDim / cache->heads || k_stride < width || v_stride < width ||
        k_stride % 8 != 0 || v_stride % 8 != 0)
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!cache_aligned(*cache) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
      return CIDER_ERR_MISALIGNED;
    int* err = nullptr;
    s = device(&err, nullptr);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_kv_append(layer_of(*cache, layer), k, k_stride, v, v_stride,
                                               dtype == CIDER_BF16, slots, tokens, err,
                                               static_cast<cudaStream_t>(stream)));
  });
}

cider_status_t cider_kv_read(const cider_kv_cache_t* cache, int64_t layer, const int32_t* table,
                             int64_t table_width, const int32_t* starts, const int32_t* offsets,
                             int64_t requests, int64_t tokens, void* k, void* v, int dtype,
                             void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!cache) return CIDER_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || requests == 0 || cache->pages == 0 || cache->layers == 0) return CIDER_OK;
    cider_status_t s = check_cache(*cache);
    if (s != CIDER_OK) return s;
    if (!table || !starts || !offsets || !k || !v || !valid_dtype(dtype) || layer < -1 ||
        layer >= cache->layers || tokens < 0 || tokens > kMaxDim / cache->heads || requests < 0 ||
        requests > kMaxDim || table_width < 1)
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!cache_aligned(*cache) || !aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4) ||
        !aligned(starts, 4) || !aligned(offsets, 4))
      return CIDER_ERR_MISALIGNED;
    int* err = nullptr;
    int sms = 0;
    s = device(&err, &sms);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_kv_read(
        layer_of(*cache, layer < 0 ? 0 : layer), layer < 0 ? cache->layers : 1, table, table_width,
        starts, offsets, static_cast<int>(requests), tokens, k, v, dtype == CIDER_BF16, err, sms,
        static_cast<cudaStream_t>(stream)));
  });
}

cider_status_t cider_kv_compact(const cider_kv_cache_t* cache, const int32_t* table,
                                int64_t table_width, const int32_t* starts, const int32_t* path,
                                int64_t path_width, const int32_t* kept, int64_t requests,
                                void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!cache) return CIDER_ERR_INVALID_ARGUMENT;
    if (requests == 0 || cache->pages == 0 || cache->layers == 0) return CIDER_OK;
    cider_status_t s = check_cache(*cache);
    if (s != CIDER_OK) return s;
    if (!table || !starts || !path || !kept || requests < 0 || requests > kMaxDim ||
        table_width < 1 || path_width < 1 || path_width > cider::kMaxNodes)
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!cache_aligned(*cache) || !aligned(table, 4) || !aligned(starts, 4) || !aligned(path, 4) ||
        !aligned(kept, 4))
      return CIDER_ERR_MISALIGNED;
    int* err = nullptr;
    s = device(&err, nullptr);
    if (s != CIDER_OK) return s;
    return cuda_status(cider::launch_kv_compact(
        layer_of(*cache, 0), cache->layers, table, table_width, starts, path,
        static_cast<int>(path_width), kept, static_cast<int>(requests), err,
        static_cast<cudaStream_t>(stream)));
  });
}

cider_status_t cider_tree_attention(const cider_kv_cache_t* cache, int64_t layer, const void* q,
                                    int64_t q_stride, int dtype, int64_t tokens, int64_t q_heads,
                                    const int32_t* table, int64_t table_width,
                                    const int32_t* lengths, const int32_t* offsets,
                                    int64_t requests, int64_t max_nodes, const int64_t* tree,
                                    float scale, void* out, void* stream) {
  return guarded([&]() -> cider_status_t {
    if (!cache) return CIDER_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || requests == 0 || cache->pages == 0 || cache->layers == 0) return CIDER_OK;
    cider_status_t s = check_cache(*cache);
    if (s != CIDER_OK) return s;
    if (!q || !table || !lengths || !offsets || !out || !valid_dtype(dtype) || layer < 0 ||
        layer >= cache->layers || tokens < 0 || q_heads < 1 || q_heads > kMaxGrid ||
        q_heads % cache->heads != 0 || tokens > kMaxDim / q_heads || requests < 0 ||
        requests > kMaxDim || table_width < 1 || max_nodes < 1 || max_nodes > cider::kMaxNodes ||
        q_stride < q_heads * cache->head_dim || q_stride % 8 != 0 || !isfinite(scale))
      return CIDER_ERR_INVALID_ARGUMENT;
    if (!cache_aligned(*cache) || !aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) ||
        !aligned(lengths, 4) || !aligned(offsets, 4) || !aligned(tree, 8))
      return CIDER_ERR_MISALIGNED;
    cider::AttendArgs a;
    int sms = 0;
    s = device(&a.err, &sms);
    if (s != CIDER_OK) return s;
    a.cache = layer_of(*cache, layer);
    a.q = q;
    a.q_stride = q_stride;
    a.rows = tokens;
    a.q_heads = static_cast<int>(q_heads);
    a.table = table;
    a.table_width = table_width;
    a.lengths = lengths;
    a.offsets = offsets;
    a.requests = static_cast<int>(requests);
    a.max_nodes = static_cast<int>(max_nodes);
    a.tree = tree;
    a.scale = scale;
    a.out = out;
    return cuda_status(
        cider::launch_attend(a, dtype == CIDER_BF16, sms, static_cast<cudaStream_t>(stream)));
  });
}

cider_status_t cider_verify_drafts(const void* logits, int64_t logits_stride, int dtype,
                                   const int32_t* tokens, const int32_t* parents,
                                   const int32_t* offsets, int64_t requests, int64_t nodes,
                                   int64_t vocab, int64_t max_nodes, const float* uniforms,
                                   const float* noise, const float* draft,
                                   const float* temperature, int32_t* count, int32_t* path,
                                   int32_t* next, void* stream) {
  return verify(logits, logits_stride, dtype, tokens, parents, offsets, requests, nodes, vocab,
                max_nodes, uniforms, noise, draft, temperature, count, path, next, stream,
                cider::kKernelWaitTimeoutNs, -1);
}

cider_status_t cider_debug_verify_timeout(const void* logits, int64_t logits_stride, int dtype,
                                          const int32_t* tokens, const int32_t* parents,
                                          const int32_t* offsets, int64_t requests, int64_t nodes,
                                          int64_t vocab, int64_t max_nodes, const float* uniforms,
                                          const float* noise, const float* draft,
                                          const float* temperature, int32_t* count, int32_t* path,
                                          int32_t* next, int64_t wait_us, int32_t silent,
                                          void* stream) {
  if (wait_us < 1 || wait_us > 100000 || silent < -1) return CIDER_ERR_INVALID_ARGUMENT;
  return verify(logits, logits_stride, dtype, tokens, parents, offsets, requests, nodes, vocab,
                max_nodes, uniforms, noise, draft, temperature, count, path, next, stream,
                static_cast<uint64_t>(wait_us) * 1000, silent);
}

}  // extern "C"
