// C ABI entry points of the dense serving operators (include/dsa.h): page
// tables, rotary positions and the attention of new tokens.  Host-side
// validation, then one launch sequence; on a non-zero status other than
// DSA_ERR_CUDA nothing was launched.
#include <algorithm>
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
// shared: with room for requests that share prefixes (a.G may still be 0).  flat:
// of 4-bit rows, with room for expanded ones where a call is large enough for it.
size_t lay_out_chunk(dsa::ChunkWork& w, dsa::FlatWork* flat, int T, int H, int B, int sms, bool shared, char* base) {
  w.nc = w.a.G > 0 ? 32 : dsa::chunk_columns(T, H, B);     // shared prefixes: rows of several requests together
  const int64_t all = (int64_t)T * H;
  w.max_units = (all / w.nc) * (w.a.G > 0 ? 2 : 1) + B + w.a.G;     // full units, and the last of each request and group
  w.grid = sms;
  const size_t units = (size_t)((all / dsa::kFewestRows + B) * (shared ? 2 : 1));
  w.joined0 = (int64_t)sms * 2 * (shared ? 32 : dsa::chunk_columns(T, H, 1));
  const size_t rows = (size_t)(w.joined0 + (shared ? 2 * std::min(all, (int64_t)B * dsa::kSharedRows) : 0));
  size_t end = 0;
  auto take = [&](size_t bytes) {
    char* p = base + end;
    end += (bytes + 255) / 256 * 256;
    return p;
  };
  w.units = take((units + 1) * (shared ? sizeof(dsa::SharedUnit) : sizeof(dsa::ChunkUnit)));
  w.splits = reinterpret_cast<dsa::ChunkSplit*>(take((size_t)sms * sizeof(dsa::ChunkSplit)));
  w.part_lse = reinterpret_cast<float*>(take(rows * sizeof(float)));
  w.part_o = reinterpret_cast<float*>(take(rows * 512 * sizeof(float)));
  if (shared) w.n_units = reinterpret_cast<int32_t*>(take(2 * sizeof(int32_t)));
  if (flat != nullptr && all >= dsa::kFlatCall) {
    const size_t requests = (size_t)std::min(B, dsa::kFlatRequests);
    flat->rows = reinterpret_cast<uint8_t*>(take((size_t)dsa::kFlatTiles * 128 * 656));
    flat->table = reinterpret_cast<int32_t*>(take((size_t)dsa::kFlatTable * sizeof(int32_t)));
    flat->cu8 = reinterpret_cast<int32_t*>(take((requests + 1) * sizeof(int32_t)));
    flat->kv8 = reinterpret_cast<int32_t*>(take(requests * sizeof(int32_t)));
    flat->cu4 = reinterpret_cast<int32_t*>(take((requests + 1) * sizeof(int32_t)));
    flat->kv4 = reinterpret_cast<int32_t*>(take(requests * sizeof(int32_t)));
  }
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

int release_pages(const dsa::ReleaseArgs& a, void* stream) {
  if (!table_ok(a.B, a.max_pages, a.page_size) || a.free_cap < 1) return DSA_ERR_SHAPE;
  if (any_null(a.finished) || any_null(a.seq_lens, a.page_table, a.free_count) ||
      any_null(a.free_pages, a.free_count_out, a.seq_lens_out))
    return DSA_ERR_NULL;
  for (const void* p : {(const void*)a.seq_lens, (const void*)a.page_table, (const void*)a.free_pages,
                        (const void*)a.free_count, (const void*)a.free_count_out, (const void*)a.seq_lens_out,
                        (const void*)a.err})
    if (!aligned(p, 4)) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  cudaGetLastError();
  return launch_status(dsa::launch_pages_release(a, sms, static_cast<cudaStream_t>(stream)));
}

bool chunk_sizes_ok(int T, int H, int B) {
  return T >= 0 && H >= 1 && H <= 1024 && (int64_t)T * H <= INT32_MAX / 2 && B >= 1 && B <= DSA_MAX_REQUESTS;
}

bool fp4(int layout) { return layout == DSA_KV_FP4_288 || layout == DSA_KV_FP4_416; }

size_t chunk_bytes(int T, int H, int B, int layout, bool shared) {
  if (!chunk_sizes_ok(T, H, B) || dsa_kv_row_bytes(layout) == 0) return 0;
  int sms = 0;
  if (dsa::current_device_sms(&sms) != DSA_OK) sms = 152;
  dsa::ChunkWork w{};
  dsa::FlatWork flat{};
  return lay_out_chunk(w, fp4(layout) ? &flat : nullptr, T, H, B, sms, shared, nullptr);
}

// Dense attention, checked and launched; shared: of dsa_prefix_attn.
int attend(const dsa::ChunkArgs& a, int kv_row_dim, bool shared, void* workspace, size_t ws_bytes, void* stream) {
  if (a.T < 0 || a.pool_rows < 0) return DSA_ERR_SHAPE;
  if (dsa_kv_row_bytes(a.layout) == 0) return DSA_ERR_LAYOUT;
  const int width = a.layout == DSA_KV_ROPE656 || a.layout == DSA_KV_FP4_416 ? 576 : 512;
  if (a.q_row != width || kv_row_dim != width) return DSA_ERR_ROW_WIDTH;
  if (a.H < 1 || a.H > 1024) return DSA_ERR_HEADS;
  if (a.T == 0) return DSA_OK;
  if (any_null(a.page_table, a.cu_q, a.kv_lens) || any_null(a.q, a.o) || any_null(a.pool) || any_null(a.lse)) return DSA_ERR_NULL;
  if (!table_ok(a.B, a.max_pages, a.page_size) || !chunk_sizes_ok(a.T, a.H, a.B) || a.pool_rows < 1 || a.pool_rows > INT32_MAX)
    return DSA_ERR_SHAPE;
  if (!aligned(a.q, 16) || !aligned(a.pool, 16) || !aligned(a.o, 16) || !aligned(a.lse, 4) || !aligned(a.page_table, 4) ||
      !aligned(a.cu_q, 4) || !aligned(a.kv_lens, 4) || !aligned(a.err, 4))
    return DSA_ERR_ALIGN;
  if (workspace == nullptr || ws_bytes < chunk_bytes(a.T, a.H, a.B, a.layout, shared)) return DSA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return DSA_ERR_ALIGN;
  int sms = 0;
  const int st = dsa::current_device_sms(&sms);
  if (st != DSA_OK) return st;
  dsa::ChunkWork w{};
  w.a = a;
  if (!dsa::sharing_possible(a, sms)) w.a.G = 0;
  dsa::FlatWork flat{};
  lay_out_chunk(w, fp4(a.layout) ? &flat : nullptr, a.T, a.H, a.B, sms, shared, static_cast<char*>(workspace));
  w.wait_ns = dsa::wait_limit_ns();
  cudaGetLastError();
  const int64_t tiles = ((int64_t)a.max_pages * a.page_size + 127) / 128;       // of a page-table row
  // (pages of fewer rows: every block of the expansion looks at all of them)
  if (flat.rows != nullptr && w.a.G == 0 && (int64_t)a.T * a.H >= (int64_t)a.B * dsa::kFlatRows && a.B <= dsa::kFlatRequests &&
      a.B * tiles <= dsa::kFlatTable && a.page_size >= 16) {
    flat.a = a;
    flat.tiles = dsa::kFlatTiles;
    flat.width = (int)tiles;
    dsa::ChunkWork w8 = w;
    w8.a.layout = a.layout == DSA_KV_FP4_416 ? DSA_KV_ROPE656 : DSA_KV_SCALED528;
    w8.a.pool = flat.rows;
    w8.a.pool_rows = dsa::kFlatTiles * 128;
    w8.a.page_table = flat.table;
    w8.a.max_pages = (int)tiles;
    w8.a.page_size = 128;
    w8.a.cu_q = flat.cu8;
    w8.a.kv_lens = flat.kv8;
    w.a.cu_q = flat.cu4;
    w.a.kv_lens = flat.kv4;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_status(dsa::launch_fp4_flat(flat, sms, s) && dsa::launch_chunk_attn(w8, s) && dsa::launch_chunk_attn(w, s));
  }
  const auto launch = w.a.G > 0 ? dsa::launch_prefix_attn : dsa::launch_chunk_attn;
  return launch_status(launch(w, static_cast<cudaStream_t>(stream)));
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
  return release_pages({finished_dev, nullptr, seq_lens_dev, B, page_table_dev, max_pages, page_size, free_pages_dev,
                        free_cap, free_count_dev, free_count_out_dev, seq_lens_out_dev, err_flag_dev},
                       stream);
}

int dsa_pages_release_own(const uint8_t* finished_dev, const int32_t* shared_pages_dev,
                          const int32_t* seq_lens_dev, int B, const int32_t* page_table_dev, int max_pages,
                          int page_size, int32_t* free_pages_dev, int free_cap, const int32_t* free_count_dev,
                          int32_t* free_count_out_dev, int32_t* seq_lens_out_dev, int32_t* err_flag_dev,
                          void* stream) {
  if (!table_ok(B, max_pages, page_size) || free_cap < 1) return DSA_ERR_SHAPE;
  if (shared_pages_dev == nullptr) return DSA_ERR_NULL;
  if (!aligned(shared_pages_dev, 4)) return DSA_ERR_ALIGN;
  return release_pages({finished_dev, shared_pages_dev, seq_lens_dev, B, page_table_dev, max_pages, page_size,
                        free_pages_dev, free_cap, free_count_dev, free_count_out_dev, seq_lens_out_dev, err_flag_dev},
                       stream);
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

size_t dsa_chunk_attn_workspace_bytes(int T, int H, int B, int layout) { return chunk_bytes(T, H, B, layout, false); }

size_t dsa_prefix_attn_workspace_bytes(int T, int H, int B, int layout) {
  return B > DSA_MAX_PREFIX_REQUESTS ? 0 : chunk_bytes(T, H, B, layout, true);
}

int dsa_chunk_attn(const void* q_bf16_dev, int T, int H, int D, const void* pool_dev, int64_t pool_rows,
                   int layout, int kv_row_dim, const int32_t* page_table_dev, int B, int max_pages, int page_size,
                   const int32_t* cu_q_dev, const int32_t* kv_lens_dev, int causal, float sm_scale,
                   void* o_bf16_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes, int32_t* err_flag_dev,
                   void* stream) {
  const dsa::ChunkArgs a{static_cast<const uint16_t*>(q_bf16_dev), T, H, D, static_cast<const uint8_t*>(pool_dev), pool_rows,
                         layout, page_table_dev, B, max_pages, page_size, cu_q_dev, kv_lens_dev, causal != 0, sm_scale,
                         static_cast<uint16_t*>(o_bf16_dev), lse_dev, err_flag_dev, nullptr, nullptr, 0};
  return attend(a, kv_row_dim, false, workspace_dev, ws_bytes, stream);
}

int dsa_prefix_attn(const void* q_bf16_dev, int T, int H, int D, const void* pool_dev, int64_t pool_rows,
                    int layout, int kv_row_dim, const int32_t* page_table_dev, int B, int max_pages,
                    int page_size, const int32_t* cu_q_dev, const int32_t* kv_lens_dev,
                    const int32_t* group_cu_dev, const int32_t* prefix_lens_dev, int G, int causal,
                    float sm_scale, void* o_bf16_dev, float* lse_dev, void* workspace_dev, size_t ws_bytes,
                    int32_t* err_flag_dev, void* stream) {
  if (G < 0 || G > B || B > DSA_MAX_PREFIX_REQUESTS) return DSA_ERR_SHAPE;
  if (G > 0 && T > 0 && any_null(group_cu_dev, prefix_lens_dev)) return DSA_ERR_NULL;
  if (!aligned(group_cu_dev, 4) || !aligned(prefix_lens_dev, 4)) return DSA_ERR_ALIGN;
  const dsa::ChunkArgs a{static_cast<const uint16_t*>(q_bf16_dev), T, H, D, static_cast<const uint8_t*>(pool_dev), pool_rows,
                         layout, page_table_dev, B, max_pages, page_size, cu_q_dev, kv_lens_dev, causal != 0, sm_scale,
                         static_cast<uint16_t*>(o_bf16_dev), lse_dev, err_flag_dev, group_cu_dev, prefix_lens_dev, G};
  return attend(a, kv_row_dim, true, workspace_dev, ws_bytes, stream);
}

}  // extern "C"
