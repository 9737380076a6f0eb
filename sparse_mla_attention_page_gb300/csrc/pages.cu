// Page tables and slot maps from request lengths, and the return of finished
// requests' pages.
//
// Both operators are a prefix sum over the requests followed by independent
// work per page and per token: at most a few megabytes, so a call is bound by
// its launch and one chain of dependent loads (lengths, scan, search, page id,
// store), not by bandwidth.  Every CTA forms the whole prefix sum for itself
// (reading B lengths again costs less than a round trip between CTAs) and takes
// a share of the pages and tokens, found by a binary search in shared memory.
//
// The lengths and the free count may be updated in place (captured steps), so
// they are written when every CTA has read them: by the one CTA of a small
// call, after a barrier; behind a larger grid by a second launch of one CTA
// (kFinish) that forms the sums again.  A decode step of 64 requests takes
// 4.2 us, 512 requests of up to 1024 pages released at once 7.9 us (70 us with
// the whole call in one cluster of 8 CTAs, the most that one launch can order).
#include "dense.h"
#include "dsa_common.cuh"
#include "scan.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 1024;
// Pages and tokens that one CTA takes on: 2400 token rows take 7.2 us in one
// CTA and 7.7 in a grid with its finishing launch, 8400 rows 12.6 and 7.8.
constexpr int kOneCta = 4 * kThreads;

enum Part { kBody = 1, kFinish = 2 };     // bits: pages and tokens; lengths, offsets and the free count

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page_size) {
  return (tokens + page_size - 1) / page_size;
}

__global__ void __launch_bounds__(kThreads, 1) pages_extend_kernel(const __grid_constant__ ExtendArgs a, int parts) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t sums[kThreads / 32];
  int32_t* tok0 = sm;              // first token of each request
  int32_t* page0 = sm + a.B;       // first of the call's pages of each request
  int32_t* seq = sm + 2 * a.B;
  if (parts == kFinish) asm volatile("griddepcontrol.wait;" ::: "memory");   // the body has read what is written here
  else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  const int64_t room = (int64_t)a.max_pages * a.page_size;
  const int32_t count = *static_cast<const volatile int32_t*>(a.free_count);   // read once: the output may alias it
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  bool bad = count < 0 || count > a.free_cap;
  int64_t tokens = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t s = a.seq_lens[b], n = a.new_lens[b];
    bad |= s < 0 || n < 0 || s + n > room;
    tokens += n;
    pages += pages_of(s + n, a.page_size) - pages_of(s, a.page_size);
  }
  int64_t all_tokens, all_pages;
  int64_t tok_at = block_scan<kThreads>(tokens, &all_tokens, sums), page_at = block_scan<kThreads>(pages, &all_pages, sums);
  bad |= all_tokens > a.T;
  const bool lengths_bad = __syncthreads_or(bad) != 0;
  const bool refused = lengths_bad || all_pages > count;
  for (int b = b0; b < b1; ++b) {
    const int64_t s = a.seq_lens[b], n = a.new_lens[b];
    tok0[b] = refused ? 0 : (int32_t)tok_at;
    page0[b] = refused ? 0 : (int32_t)page_at;
    seq[b] = (int32_t)s;
    tok_at += n;
    page_at += pages_of(s + n, a.page_size) - pages_of(s, a.page_size);
  }
  const int n_tok = refused ? 0 : (int)all_tokens;
  const int n_pages = refused ? 0 : (int)all_pages;
  __syncthreads();   // also: this CTA has read the lengths and the count

  if (parts & kBody) {
    bool bad_page = false;
    for (int t = gtid; t < a.T; t += gsize) {
      int64_t slot = -1;
      int pos = 0, b = -1;
      if (t < n_tok) {
        b = scan_owner(tok0, a.B, t);
        pos = seq[b] + (t - tok0[b]);
        const int p = pos / a.page_size;
        const int have = (int)pages_of(seq[b], a.page_size);
        // pages of this call are read from the stack: the table may not hold them yet
        const int32_t page = p < have ? a.page_table[(int64_t)b * a.max_pages + p]
                                      : __ldg(a.free_pages + (count - 1 - (page0[b] + p - have)));
        if (page >= 0) slot = (int64_t)page * a.page_size + (pos - p * a.page_size);
        else bad_page = true;
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
      a.token_seq[t] = b;
    }
    for (int k = gtid; k < n_pages; k += gsize) {
      const int b = scan_owner(page0, a.B, k);
      const int p = (int)pages_of(seq[b], a.page_size) + (k - page0[b]);
      const int32_t page = __ldg(a.free_pages + (count - 1 - k));
      bad_page |= page < 0;
      a.page_table[(int64_t)b * a.max_pages + p] = page;
    }
    if (bad_page) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
  }
  if (parts & kFinish) {
    if (refused && tid == 0) set_err(a.err, lengths_bad ? DSA_DEV_ERR_LENGTH : DSA_DEV_ERR_NO_PAGES);
    for (int b = tid; b <= a.B; b += kThreads) {
      const int begin = b < a.B ? tok0[b] : n_tok;
      a.cu_q[b] = begin;
      if (b < a.B) a.kv_lens[b] = seq[b] + (b + 1 < a.B ? tok0[b + 1] : n_tok) - begin;
    }
    if (tid == 0) *a.free_count_out = count - n_pages;
  }
}

__global__ void __launch_bounds__(kThreads, 1) pages_release_kernel(const __grid_constant__ ReleaseArgs a, int parts) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t sums[kThreads / 32];
  int32_t* page0 = sm;             // first of the call's pages of each request
  if (parts == kFinish) asm volatile("griddepcontrol.wait;" ::: "memory");
  else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  const int64_t room = (int64_t)a.max_pages * a.page_size;
  const int32_t count = *static_cast<const volatile int32_t*>(a.free_count);   // read once: the output may alias it
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  auto kept = [&](int b) { return a.shared != nullptr ? __ldg(a.shared + b) : 0; };
  auto back = [&](int b) -> int64_t {
    const int64_t s = a.seq_lens[b];
    return a.finished[b] && s > 0 ? max((int64_t)0, pages_of(s, a.page_size) - kept(b)) : 0;
  };
  bool bad = count < 0 || count > a.free_cap;
  int64_t pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t s = a.seq_lens[b];
    bad |= s < 0 || s > room || kept(b) < 0;
    pages += back(b);
  }
  int64_t all_pages;
  int64_t at = block_scan<kThreads>(pages, &all_pages, sums);
  const bool lengths_bad = __syncthreads_or(bad) != 0;
  const bool refused = lengths_bad || count + all_pages > a.free_cap;
  for (int b = b0; b < b1; ++b) {
    page0[b] = refused ? 0 : (int32_t)at;
    at += back(b);
  }
  const int n_pages = refused ? 0 : (int)all_pages;
  __syncthreads();   // also: this CTA has read the lengths and the count
  if (parts & kBody) {
    bool bad_page = false;
    for (int k = gtid; k < n_pages; k += gsize) {
      const int b = scan_owner(page0, a.B, k);
      const int32_t page = __ldg(a.page_table + (int64_t)b * a.max_pages + kept(b) + (k - page0[b]));
      bad_page |= page < 0;
      a.free_pages[count + k] = page;
    }
    if (bad_page) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
  }
  if (parts & kFinish) {
    if (refused && tid == 0) set_err(a.err, lengths_bad ? DSA_DEV_ERR_LENGTH : DSA_DEV_ERR_NO_PAGES);
    for (int b = tid; b < a.B; b += kThreads) a.seq_lens_out[b] = a.finished[b] && !refused ? 0 : a.seq_lens[b];
    if (tid == 0) *a.free_count_out = count + n_pages;
  }
}

// `items`: the pages and tokens there may be.
template <class Args>
bool launch(void (*kernel)(Args, int), const Args& a, int64_t items, size_t smem, int sms, cudaStream_t stream) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (items <= kOneCta) {
    cfg.gridDim = dim3(1);
    return cudaLaunchKernelEx(&cfg, kernel, a, (int)(kBody | kFinish)) == cudaSuccess;
  }
  const int64_t ctas = (items + kThreads - 1) / kThreads;
  cfg.gridDim = dim3((unsigned)(ctas < sms ? ctas : sms));
  if (cudaLaunchKernelEx(&cfg, kernel, a, (int)kBody) != cudaSuccess) return false;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1);
  return cudaLaunchKernelEx(&cfg, kernel, a, (int)kFinish) == cudaSuccess;
}

}  // namespace

bool launch_pages_extend(const ExtendArgs& a, int sms, cudaStream_t stream) {
  return launch(pages_extend_kernel, a, a.T, (size_t)a.B * 12, sms, stream);
}

bool launch_pages_release(const ReleaseArgs& a, int sms, cudaStream_t stream) {
  return launch(pages_release_kernel, a, (int64_t)a.B * a.max_pages, (size_t)a.B * 4, sms, stream);
}

}  // namespace dsa
