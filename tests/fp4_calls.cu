// The entry points of 4-bit floating point over launchers that write down what they are asked for: which
// kernels a call launches, on which memory.  Host code only; tests/test_fp4_calls.py builds and reads it.
#include "fp4_api.cu"

#include <vector>

namespace {

struct Settings {
  uint8_t* scratch = nullptr;   // where scratch memory is said to lie
  int sms = 152;
  bool fits = false;            // whether the kernel for few tokens can quantize x itself
} settings;

struct Record {
  int64_t kind;   // 0 scratch, 1 quantization, 2 product by the kernel for few tokens, 3 on pairs
  int64_t bytes;  // of scratch
  const void *wide, *codes, *scales, *row;                 // read: x in 16 bits, or quantized
  const void *y, *to_codes, *to_scales, *to_row;           // written
  int64_t stride, M, N, K, gated, dependent;
};
std::vector<Record> records;

cudaError_t record(int kind, const cider::FpProduct& p) {
  records.push_back({kind, 0, p.wide_x, p.x.codes, p.x.scales, p.x.row, p.q_codes ? nullptr : p.y, p.q_codes,
                     p.q_scales, nullptr, p.x_stride, p.M, p.N, p.K, p.is_gated, p.after_launch});
  return cudaSuccess;
}

}  // namespace

namespace cider {

cider_status_t check_device(int* dev, int* sms) {
  if (dev) *dev = 0;
  if (sms) *sms = settings.sms;
  return CIDER_OK;
}
ScratchSource::ScratchSource(ScratchSource&& o) noexcept : st_(o.st_), base_(o.base_), capacity_(o.capacity_) {}
ScratchSource::~ScratchSource() {}
cider_status_t ScratchSource::get(size_t bytes, void** out) {
  Record r{};
  r.bytes = static_cast<int64_t>(bytes);
  r.y = settings.scratch;
  records.push_back(r);
  *out = settings.scratch;
  return CIDER_OK;
}
cudaError_t launch_quantize_fp4(const void* x, int, int64_t stride, int64_t rows, int64_t K, int, uint8_t* codes,
                                uint8_t* scales, float* row, bool, int, cudaStream_t, bool) {
  records.push_back({1, 0, x, nullptr, nullptr, nullptr, nullptr, codes, scales, row, stride, rows, 0, K, 0, 0});
  return cudaSuccess;
}
cudaError_t launch_dequantize_fp4(const FpMat&, int64_t, int, void*, int, int, cudaStream_t) { return cudaSuccess; }
bool fp4_rows_quantizes_itself(const FpProduct&) { return settings.fits; }
cudaError_t launch_fp4_rows(const FpProduct& p) { return record(2, p); }
cudaError_t launch_fp4_pair(const FpProduct& p) { return record(3, p); }

}  // namespace cider

extern "C" {
void calls_begin(int64_t scratch, int sms, int fits) {
  settings = {reinterpret_cast<uint8_t*>(scratch), sms, fits != 0};
  records.clear();
}
int calls_made() { return static_cast<int>(records.size()); }
const void* calls_records() { return records.data(); }
}
