// Internal launch interface of the dense serving operators: page tables and
// slot maps (pages.cu), rotary positions (rope.cu) and the attention of new
// tokens over everything in the paged pool (chunk_attn.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dsa.h"

namespace dsa {

struct ExtendArgs {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int B;
  int32_t* page_table;
  int max_pages, page_size;
  const int32_t* free_pages;
  int free_cap;
  const int32_t* free_count;
  int32_t* free_count_out;
  int T;
  int64_t* slots;
  int32_t* positions;
  int32_t* token_seq;
  int32_t* cu_q;
  int32_t* kv_lens;
  int32_t* err;
};
// false when a launch failed or was not made (of two, the first may have been).
bool launch_pages_extend(const ExtendArgs& a, int sms, cudaStream_t stream);

struct ReleaseArgs {
  const uint8_t* finished;
  const int32_t* seq_lens;
  int B;
  const int32_t* page_table;
  int max_pages, page_size;
  int32_t* free_pages;
  int free_cap;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* seq_lens_out;
  int32_t* err;
};
bool launch_pages_release(const ReleaseArgs& a, int sms, cudaStream_t stream);

struct RopeArgs {
  uint64_t turn[32];      // turns a position step, as a 64-bit fraction of one turn
  uint8_t axis[32];
  int interleaved;
  float mscale;
  const int32_t* positions;
  int64_t pos_stride;
  int T, H;
  const uint16_t* q_nope; // nullptr: q_out's first 512 dims are left alone
  int64_t qn_t, qn_h;
  const uint16_t* q_pe;   // nullptr: no queries
  int64_t qp_t, qp_h;
  uint16_t* q_out;
  const uint16_t* kv_c;   // nullptr: no rows
  int64_t kv_stride;
  const uint16_t* k_pe;
  int64_t kp_stride;
  const int64_t* slots;
  uint8_t* pool;
  int64_t pool_rows;
  int32_t* err;
};
void launch_rope(const RopeArgs& a, int sms, cudaStream_t stream);

struct ChunkArgs {
  const uint16_t* q;      // BF16 [T, H, q_row]
  int T, H, q_row;
  const uint8_t* pool;
  int64_t pool_rows;
  int layout;
  const int32_t* page_table;
  int B, max_pages, page_size;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int causal;
  float sm_scale;
  uint16_t* o;
  float* lse;
  int32_t* err;
};
// Query rows of a unit of the work list, 16 or 32.
constexpr int kFewestRows = 16;
int chunk_columns(int T, int H, int B);
struct ChunkWork;      // chunk.cuh
bool launch_chunk_attn(const ChunkWork& w, cudaStream_t stream);

// Limit of every bounded wait inside the attention kernels (dsa_set_wait_limit_ns).
uint64_t wait_limit_ns();

}  // namespace dsa
