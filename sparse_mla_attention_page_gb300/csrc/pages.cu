// Page tables and slot maps from request lengths, and the return of finished
// requests' pages.
//
// Both operators are a prefix sum over the requests followed by independent
// work per page and per token.  The work is a few hundred kilobytes at most,
// so a call is bound by its launch and one chain of dependent loads (lengths,
// scan, search, page id, store), not by bandwidth: one launch of one
// thread-block cluster.  Every CTA forms the whole prefix sum for itself
// (reading B lengths again costs less than a round trip between CTAs) and
// takes a share of the pages and tokens, found by a binary search in shared
// memory.  The cluster barrier between the reads of the lengths and the first
// store is what lets the outputs alias the inputs (a captured step updates
// its lengths and its free count in place); a second launch in its place
// would cost more than the whole kernel.
#include <cooperative_groups.h>

#include "dense.h"
#include "dsa_common.cuh"
#include "scan.cuh"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = kScanThreads;

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page_size) {
  return (tokens + page_size - 1) / page_size;
}

__global__ void __launch_bounds__(kThreads, 1) pages_extend_kernel(const ExtendArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* tok0 = sm;              // first token of each request
  int32_t* page0 = sm + a.B;       // first of the call's pages of each request
  int32_t* seq = sm + 2 * a.B;
  cg::cluster_group cluster = cg::this_cluster();
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
  int64_t tok_at = block_scan(tokens, &all_tokens), page_at = block_scan(pages, &all_pages);
  bad |= all_tokens > a.T;
  const bool lengths_bad = __syncthreads_or(bad) != 0;
  const bool short_of_pages = !lengths_bad && all_pages > count;
  const bool refused = lengths_bad || short_of_pages;
  if (refused && gtid == 0)
    set_err(a.err, lengths_bad ? DSA_DEV_ERR_LENGTH : DSA_DEV_ERR_NO_PAGES);
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
  cluster.sync();   // every CTA has read the lengths and the count: the outputs may alias them

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
  for (int b = gtid; b <= a.B; b += gsize) {
    const int end = b < a.B ? tok0[b] : n_tok;
    a.cu_q[b] = end;
    if (b < a.B) a.kv_lens[b] = seq[b] + (b + 1 < a.B ? tok0[b + 1] : n_tok) - end;
  }
  if (gtid == 0) *a.free_count_out = count - n_pages;
}

__global__ void __launch_bounds__(kThreads, 1) pages_release_kernel(const ReleaseArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* page0 = sm;             // first of the call's pages of each request
  __shared__ int cluster_bad;      // CTA 0's is the cluster's
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  const int64_t room = (int64_t)a.max_pages * a.page_size;
  const int32_t count = *static_cast<const volatile int32_t*>(a.free_count);   // read once: the output may alias it
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  if (tid == 0) cluster_bad = 0;
  auto back = [&](int b) -> int64_t {
    const int64_t s = a.seq_lens[b];
    return a.finished[b] && s > 0 ? pages_of(s, a.page_size) : 0;
  };
  bool bad = count < 0 || count > a.free_cap;
  int64_t pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t s = a.seq_lens[b];
    bad |= s < 0 || s > room;
    pages += back(b);
  }
  int64_t all_pages;
  int64_t at = block_scan(pages, &all_pages);
  const bool lengths_bad = __syncthreads_or(bad) != 0;
  const bool no_room = !lengths_bad && count + all_pages > a.free_cap;
  const bool refused = lengths_bad || no_room;
  if (refused && gtid == 0) set_err(a.err, lengths_bad ? DSA_DEV_ERR_LENGTH : DSA_DEV_ERR_NO_PAGES);
  for (int b = b0; b < b1; ++b) {
    page0[b] = refused ? 0 : (int32_t)at;
    at += back(b);
  }
  const int n_pages = refused ? 0 : (int)all_pages;
  __syncthreads();
  // every page is looked at before any is pushed
  bool bad_page = false;
  for (int k = gtid; k < n_pages; k += gsize) {
    const int b = scan_owner(page0, a.B, k);
    bad_page |= __ldg(a.page_table + (int64_t)b * a.max_pages + (k - page0[b])) < 0;
  }
  // the flag is set up in every CTA before another one may reach it
  cluster.sync();
  if (bad_page) atomicOr(cluster.map_shared_rank(&cluster_bad, 0), 1);
  cluster.sync();   // also: every CTA has read the lengths and the count
  const bool dropped = refused || *cluster.map_shared_rank(&cluster_bad, 0) != 0;
  if (!refused && dropped && gtid == 0) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
  if (!dropped)
    for (int k = gtid; k < n_pages; k += gsize) {
      const int b = scan_owner(page0, a.B, k);
      a.free_pages[count + k] = __ldg(a.page_table + (int64_t)b * a.max_pages + (k - page0[b]));
    }
  for (int b = gtid; b < a.B; b += gsize) a.seq_lens_out[b] = a.finished[b] && !dropped ? 0 : a.seq_lens[b];
  if (gtid == 0) *a.free_count_out = dropped ? count : count + n_pages;
  cluster.sync();   // CTA 0's shared memory stays until every CTA has read the flag
}

// CTAs of the cluster (8 is the portable limit) for n pages and tokens: one
// for every four passes of its threads.
int cluster_size(int64_t n) {
  const int64_t c = (n + 4 * kThreads - 1) / (4 * kThreads);
  return c <= 1 ? 1 : c <= 2 ? 2 : c <= 4 ? 4 : 8;
}

template <class Args>
bool launch_cluster(void (*kernel)(Args), const Args& a, int ctas, size_t smem, cudaStream_t stream) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess;
}

}  // namespace

bool launch_pages_extend(const ExtendArgs& a, cudaStream_t stream) {
  return launch_cluster(pages_extend_kernel, a, cluster_size(a.T), (size_t)a.B * 12, stream);
}

bool launch_pages_release(const ReleaseArgs& a, cudaStream_t stream) {
  return launch_cluster(pages_release_kernel, a, cluster_size((int64_t)a.B * a.max_pages), (size_t)a.B * 4, stream);
}

}  // namespace dsa
