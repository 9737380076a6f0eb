// C ABI entry points of the 4-bit rows and the reader by request
// (include/dsa.h): host-side validation, then one launch.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cuda_runtime.h>

#include "../../include/dsa.h"
#include "kernels.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_status(bool launched) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && launched) return DSA_OK;
  if (std::getenv("DSA_DEBUG") != nullptr) std::fprintf(stderr, "dsa: launch failed: %s\n", cudaGetErrorString(e));
  return DSA_ERR_CUDA;
}

// n rows, `stride` elements apart, `unit` elements a vector access.
bool stride_ok(int64_t stride, int64_t n, int64_t unit) {
  return stride >= 0 && stride % unit == 0 && stride <= INT64_MAX / 4 / (n > 0 ? n : 1);
}

}  // namespace

extern "C" {

int dsa_kv_write_fp4(const void* kv_c_dev, int64_t kv_c_stride, const void* k_pe_dev, int64_t k_pe_stride,
                     int64_t n_rows, const int64_t* slots_dev, void* pool_dev, int64_t pool_rows,
                     int32_t* err_flag_dev, void* stream) {
  if (n_rows < 0 || pool_rows < 0) return DSA_ERR_SHAPE;
  if (n_rows == 0) return DSA_OK;
  if (kv_c_dev == nullptr || slots_dev == nullptr || pool_dev == nullptr) return DSA_ERR_NULL;
  if (pool_rows > INT64_MAX / 416 || n_rows > INT64_MAX / 2048) return DSA_ERR_SHAPE;
  if (!aligned(kv_c_dev, 16) || !aligned(k_pe_dev, 4) || !aligned(slots_dev, 8) || !aligned(pool_dev, 16) ||
      !aligned(err_flag_dev, 4))
    return DSA_ERR_ALIGN;
  if (!stride_ok(kv_c_stride, n_rows, 8) || (k_pe_dev != nullptr && !stride_ok(k_pe_stride, n_rows, 2))) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  const dsa::Fp4WriteArgs a{static_cast<const uint16_t*>(kv_c_dev), kv_c_stride, static_cast<const uint16_t*>(k_pe_dev),
                            k_pe_stride, n_rows, slots_dev, static_cast<uint8_t*>(pool_dev), pool_rows, err_flag_dev};
  cudaGetLastError();
  dsa::launch_kv_write_fp4(a, sms, static_cast<cudaStream_t>(stream));
  return launch_status(true);
}

int dsa_kv_read(const void* pool_dev, int64_t pool_rows, int layout, const int32_t* page_table_dev, int B,
                int max_pages, int page_size, const int32_t* cu_rows_dev, const int32_t* starts_dev,
                void* out_bf16_dev, int64_t out_rows, int64_t out_stride, int32_t* err_flag_dev, void* stream) {
  if (pool_rows < 0 || out_rows < 0 || out_rows > INT32_MAX) return DSA_ERR_SHAPE;
  if (dsa_kv_row_bytes(layout) == 0) return DSA_ERR_LAYOUT;
  if (out_rows == 0) return DSA_OK;
  if (pool_dev == nullptr || page_table_dev == nullptr || cu_rows_dev == nullptr || out_bf16_dev == nullptr)
    return DSA_ERR_NULL;
  if (B < 1 || B > DSA_MAX_REQUESTS || max_pages < 1 || page_size < 1 || (int64_t)max_pages * page_size > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (pool_rows < 1 || pool_rows > INT32_MAX) return DSA_ERR_SHAPE;
  if (out_stride < (layout == DSA_KV_ROPE656 || layout == DSA_KV_FP4_416 ? 576 : 512)) return DSA_ERR_SHAPE;
  if (!aligned(pool_dev, 16) || !aligned(out_bf16_dev, 16) || !aligned(page_table_dev, 4) || !aligned(cu_rows_dev, 4) ||
      !aligned(starts_dev, 4) || !aligned(err_flag_dev, 4) || !stride_ok(out_stride, out_rows, 8))
    return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  const dsa::KvReadArgs a{static_cast<const uint8_t*>(pool_dev), pool_rows, layout, page_table_dev, B, max_pages, page_size,
                          cu_rows_dev, starts_dev, static_cast<uint16_t*>(out_bf16_dev), out_rows, out_stride,
                          err_flag_dev};
  cudaGetLastError();
  return launch_status(dsa::launch_kv_read(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
