// C ABI entry points of the dense serving operators (include/dsa.h): page
// tables, rotary positions and the attention of new tokens.  Host-side
// validation, then one launch sequence; on a non-zero status other than
// DSA_ERR_CUDA nothing was launched.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cuda_runtime.h>

#include "../../include/dsa.h"
#include "chunk.cuh"
#include "dense.h"
#include "kernels.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <class... P>
bool any_null(const P*... p) {
  return (... || (p == nullptr));
}

int launch_status(bool launched) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && launched) return DSA_OK;
  if (std::getenv("DSA_DEBUG") != nullptr) std::fprintf(stderr, "dsa: launch failed: %s\n", cudaGetErrorString(e));
  return DSA_ERR_CUDA;
}

// Page table rows and requests within the sizes the kernels index with.
bool table_ok(int B, int max_pages, int page_size) {
  return B >= 1 && B <= DSA_MAX_REQUESTS && max_pages >= 1 && page_size >= 1 &&
         (int64_t)max_pages * page_size <= INT32_MAX;
}

// Where the parts of the attention's workspace begin (pointers from base on).
// Its size grows with T, H and B alone, not with the rows of a unit that they
// lead to, so that it serves every smaller call too.
size_t lay_out_chunk(dsa::ChunkWork& w, int T, int H, int B, int sms, char* base) {
  w.nc = dsa::chunk_columns(T, H, B);
  w.max_units = (int64_t)T * H / w.nc + B;     // full units, and the last of each request
  w.grid = sms;
  const size_t units = (size_t)((int64_t)T * H / dsa::kFewestRows + B);
  const size_t rows = (size_t)sms * 2 * dsa::chunk_columns(T, H, 1);
  size_t end = 0;
  auto take = [&](size_t bytes) {
    char* p = base + end;
    end += (bytes + 255) / 256 * 256;
    return p;
  };
  w.units = reinterpret_cast<dsa::ChunkUnit*>(take((units + 1) * sizeof(dsa::ChunkUnit)));
  w.splits = reinterpret_cast<dsa::ChunkSplit*>(take((size_t)sms * sizeof(dsa::ChunkSplit)));
  w.part_lse = reinterpret_cast<float*>(take(rows * sizeof(float)));
  w.part_o = reinterpret_cast<float*>(take(rows * 512 * sizeof(float)));
  return end;
}

// Radians as the fraction of a turn, in units of 2^-64 turn.  1 / 2 pi and the
// product are kept as two doubles each: a position is up to 2^31 such steps.
uint64_t turn_of(double radians) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;    // 1 / 2 pi
  double hi = radians * kHi;
  double lo = std::fma(radians, kHi, -hi) + radians * kLo;
  hi -= std::floor(hi);
  lo -= std::nearbyint(lo);
  const uint64_t whole = hi < 1.0 ? (uint64_t)std::ldexp(hi, 64) : 0;
  return whole + ((uint64_t)(int64_t)std::ldexp(lo, 62) << 2);
}

bool chunk_sizes_ok(int T, int H, int B) {
  return T >= 0 && H >= 1 && H <= 1024 && (int64_t)T * H <= INT32_MAX / 2 && B >= 1 && B <= DSA_MAX_REQUESTS;
}

}  // namespace

extern "C" {

int dsa_pages_extend(const int32_t* seq_lens_dev, const int32_t* new_lens_dev, int B, int32_t* page_table_dev,
                     int max_pages, int page_size, const int32_t* free_pages_dev, int free_cap,
                     const int32_t* free_count_dev, int32_t* free_count_out_dev, int T, int64_t* slots_dev,
                     int32_t* positions_dev, int32_t* token_seq_dev, int32_t* cu_q_dev, int32_t* kv_lens_dev,
                     int32_t* err_flag_dev, void* stream) {
  if (!table_ok(B, max_pages, page_size) || free_cap < 1 || T < 1 || T > INT32_MAX / 2) return DSA_ERR_SHAPE;
  if (any_null(seq_lens_dev, new_lens_dev, page_table_dev, free_pages_dev, free_count_dev, free_count_out_dev) ||
      any_null(slots_dev, positions_dev, token_seq_dev, cu_q_dev, kv_lens_dev))
    return DSA_ERR_NULL;
  for (const void* p : {(const void*)seq_lens_dev, (const void*)new_lens_dev, (const void*)page_table_dev,
                        (const void*)free_pages_dev, (const void*)free_count_dev, (const void*)free_count_out_dev,
                        (const void*)positions_dev, (const void*)token_seq_dev, (const void*)cu_q_dev,
                        (const void*)kv_lens_dev, (const void*)err_flag_dev})
    if (!aligned(p, 4)) return DSA_ERR_ALIGN;
  if (!aligned(slots_dev, 8)) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  const dsa::ExtendArgs a{seq_lens_dev,   new_lens_dev,       B, page_table_dev, max_pages,     page_size,
                          free_pages_dev, free_cap,           free_count_dev,    free_count_out_dev, T,
                          slots_dev,      positions_dev,      token_seq_dev,     cu_q_dev,      kv_lens_dev,
                          err_flag_dev};
  cudaGetLastError();
  return launch_status(dsa::launch_pages_extend(a, sms, static_cast<cudaStream_t>(stream)));
}

int dsa_pages_release(const uint8_t* finished_dev, const int32_t* seq_lens_dev, int B,
                      const int32_t* page_table_dev, int max_pages, int page_size, int32_t* free_pages_dev,
                      int free_cap, const int32_t* free_count_dev, int32_t* free_count_out_dev,
                      int32_t* seq_lens_out_dev, int32_t* err_flag_dev, void* stream) {
  if (!table_ok(B, max_pages, page_size) || free_cap < 1) return DSA_ERR_SHAPE;
  if (any_null(finished_dev) || any_null(seq_lens_dev, page_table_dev, free_pages_dev, free_count_dev,
                                         free_count_out_dev, seq_lens_out_dev))
    return DSA_ERR_NULL;
  for (const void* p : {(const void*)seq_lens_dev, (const void*)page_table_dev, (const void*)free_pages_dev,
                        (const void*)free_count_dev, (const void*)free_count_out_dev,
                        (const void*)seq_lens_out_dev, (const void*)err_flag_dev})
    if (!aligned(p, 4)) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  const dsa::ReleaseArgs a{finished_dev, seq_lens_dev,   B,
                           page_table_dev, max_pages,    page_size,
                           free_pages_dev, free_cap,     free_count_dev,
                           free_count_out_dev, seq_lens_out_dev, err_flag_dev};
  cudaGetLastError();
  return launch_status(dsa::launch_pages_release(a, sms, static_cast<cudaStream_t>(stream)));
}

int dsa_rope_qkv656(const dsa_rope* rope, const int32_t* positions_dev, int64_t pos_stride, int T, int H,
                    const void* q_nope_dev, int64_t q_nope_stride_t, int64_t q_nope_stride_h,
                    const void* q_pe_dev, int64_t q_pe_stride_t, int64_t q_pe_stride_h, void* q_out_dev,
                    const void* kv_c_dev, int64_t kv_c_stride, const void* k_pe_dev, int64_t k_pe_stride,
                    const int64_t* slots_dev, void* pool_dev, int64_t pool_rows, int32_t* err_flag_dev,
                    void* stream) {
  if (rope == nullptr) return DSA_ERR_NULL;
  if (T < 0 || H < 1 || T > INT32_MAX / 2 || pool_rows < 0) return DSA_ERR_SHAPE;
  if (rope->n_axes < 1 || rope->n_axes > 8 || (rope->interleaved != 0 && rope->interleaved != 1)) return DSA_ERR_SHAPE;
  dsa::RopeArgs a{};
  for (int i = 0; i < 32; ++i) {
    if (rope->axis[i] < 0 || rope->axis[i] >= rope->n_axes || !std::isfinite(rope->inv_freq[i])) return DSA_ERR_SHAPE;
    a.axis[i] = (uint8_t)rope->axis[i];
    a.turn[i] = turn_of(rope->inv_freq[i]);
  }
  if (T == 0) return DSA_OK;
  const bool q = q_pe_dev != nullptr, kv = kv_c_dev != nullptr;
  if (positions_dev == nullptr || (!q && !kv)) return DSA_ERR_NULL;
  if (q != (q_out_dev != nullptr) || (!q && q_nope_dev != nullptr)) return DSA_ERR_NULL;
  if (kv != (k_pe_dev != nullptr) || kv != (slots_dev != nullptr) || kv != (pool_dev != nullptr)) return DSA_ERR_NULL;
  if (pos_stride < 0 || pos_stride > INT64_MAX / 64) return DSA_ERR_SHAPE;
  if (!aligned(positions_dev, 4) || !aligned(err_flag_dev, 4)) return DSA_ERR_ALIGN;
  const int64_t most = INT64_MAX / 4 / T / H;
  auto stride_ok = [&](int64_t s, int64_t unit) { return s >= 0 && s <= most && s % unit == 0; };
  if (q) {
    if (!aligned(q_pe_dev, 4) || !aligned(q_out_dev, 16) || !aligned(q_nope_dev, 16)) return DSA_ERR_ALIGN;
    if (!stride_ok(q_pe_stride_t, 2) || !stride_ok(q_pe_stride_h, 2)) return DSA_ERR_ALIGN;
    if (q_nope_dev != nullptr && (!stride_ok(q_nope_stride_t, 8) || !stride_ok(q_nope_stride_h, 8)))
      return DSA_ERR_ALIGN;
  }
  if (kv) {
    if (pool_rows > INT64_MAX / 656) return DSA_ERR_SHAPE;
    if (!aligned(kv_c_dev, 16) || !aligned(k_pe_dev, 4) || !aligned(slots_dev, 8) || !aligned(pool_dev, 16))
      return DSA_ERR_ALIGN;
    if (!stride_ok(kv_c_stride, 8) || !stride_ok(k_pe_stride, 2)) return DSA_ERR_ALIGN;
  }
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  a.interleaved = rope->interleaved;
  a.mscale = rope->mscale;
  a.positions = positions_dev;
  a.pos_stride = pos_stride;
  a.T = T;
  a.H = H;
  a.q_nope = static_cast<const uint16_t*>(q_nope_dev);
  a.qn_t = q_nope_stride_t;
  a.qn_h = q_nope_stride_h;
  a.q_pe = static_cast<const uint16_t*>(q_pe_dev);
  a.qp_t = q_pe_stride_t;
  a.qp_h = q_pe_stride_h;
  a.q_out = static_cast<uint16_t*>(q_out_dev);
  a.kv_c = static_cast<const uint16_t*>(kv_c_dev);
  a.kv_stride = kv_c_stride;
  a.k_pe = static_cast<const uint16_t*>(k_pe_dev);
  a.kp_stride = k_pe_stride;
  a.slots = slots_dev;
  a.pool = static_cast<uint8_t*>(pool_dev);
  a.pool_rows = pool_rows;
  a.err = err_flag_dev;
  cudaGetLastError();
  dsa::launch_rope(a, sms, static_cast<cudaStream_t>(stream));
  return launch_status(true);
}

size_t dsa_chunk_attn_workspace_bytes(int T, int H, int B, int layout) {
  if (!chunk_sizes_ok(T, H, B) || dsa_kv_row_bytes(layout) == 0) return 0;
  int sms = 0;
  if (dsa::current_device_sms(&sms) != DSA_OK) sms = 152;
  dsa::ChunkWork w{};
  return lay_out_chunk(w, T, H, B, sms, nullptr);
}

int dsa_chunk_attn(const void* q_bf16_dev, int T, int H, int D, const void* pool_dev, int64_t pool_rows,
                   int layout, int kv_row_dim, const int32_t* page_table_dev, int B, int max_pages, int page_size,
                   const int32_t* cu_q_dev, const int32_t* kv_lens_dev, int causal, float sm_scale,
                   void* o_bf16_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes, int32_t* err_flag_dev,
                   void* stream) {
  if (T < 0 || pool_rows < 0) return DSA_ERR_SHAPE;
  if (dsa_kv_row_bytes(layout) == 0) return DSA_ERR_LAYOUT;
  const int width = layout == DSA_KV_ROPE656 ? 576 : 512;
  if (D != width || kv_row_dim != width) return DSA_ERR_ROW_WIDTH;
  if (H < 1 || H > 1024) return DSA_ERR_HEADS;
  if (T == 0) return DSA_OK;
  if (any_null(page_table_dev, cu_q_dev, kv_lens_dev) || q_bf16_dev == nullptr || pool_dev == nullptr ||
      o_bf16_dev == nullptr || lse_dev == nullptr)
    return DSA_ERR_NULL;
  if (!table_ok(B, max_pages, page_size) || !chunk_sizes_ok(T, H, B) || pool_rows < 1 || pool_rows > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (!aligned(q_bf16_dev, 16) || !aligned(pool_dev, 16) || !aligned(o_bf16_dev, 16) || !aligned(lse_dev, 4) ||
      !aligned(page_table_dev, 4) || !aligned(cu_q_dev, 4) || !aligned(kv_lens_dev, 4) || !aligned(err_flag_dev, 4))
    return DSA_ERR_ALIGN;
  if (workspace_dev == nullptr || ws_bytes < dsa_chunk_attn_workspace_bytes(T, H, B, layout)) return DSA_ERR_WORKSPACE;
  if (!aligned(workspace_dev, 256)) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  dsa::ChunkWork w{};
  lay_out_chunk(w, T, H, B, sms, static_cast<char*>(workspace_dev));
  w.wait_ns = dsa::wait_limit_ns();
  dsa::ChunkArgs& a = w.a;
  a.q = static_cast<const uint16_t*>(q_bf16_dev);
  a.T = T;
  a.H = H;
  a.q_row = width;
  a.pool = static_cast<const uint8_t*>(pool_dev);
  a.pool_rows = pool_rows;
  a.layout = layout;
  a.page_table = page_table_dev;
  a.B = B;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.cu_q = cu_q_dev;
  a.kv_lens = kv_lens_dev;
  a.causal = causal != 0;
  a.sm_scale = sm_scale;
  a.o = static_cast<uint16_t*>(o_bf16_dev);
  a.lse = lse_dev;
  a.err = err_flag_dev;
  cudaGetLastError();
  return launch_status(dsa::launch_chunk_attn(w, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
