// Dense causal MLA attention of each request's new tokens over everything the
// request holds in the paged FP8 pool.
//
//   s_j = sm_scale <q, k_j>,  O = sum_j 2^(s_j' - m) v_j / l,  LSE = ln2 (m + log2 l)
//
// One block takes 32 query rows (token x head, tokens outermost) of a request
// and walks its keys in tiles of 32, dequantised into shared memory in FP32,
// with the running maximum and sum of the softmax in FP32.
#include <cuda_bf16.h>

#include "dense.h"
#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kQ = 32;           // query rows of a block
constexpr int kK = 32;           // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Query rows of request b within [0, T) and its length; false when it has none.
__device__ __forceinline__ bool request(const ChunkArgs& a, int b, int& t0, int& n, int& kv, int& err) {
  t0 = __ldg(a.cu_q + b);
  const int t1 = __ldg(a.cu_q + b + 1);
  kv = __ldg(a.kv_lens + b);
  const int64_t room = (int64_t)a.max_pages * a.page_size;
  err = 0;
  if (t0 < 0 || t1 < t0 || t1 > a.T) {
    err = DSA_DEV_ERR_LENGTH;
    n = 0;
    return false;
  }
  n = t1 - t0;
  if (kv < 0 || kv > room) {
    err = DSA_DEV_ERR_LENGTH;
    kv = kv < 0 ? 0 : (int)room;
  }
  return n > 0;
}

template <int kLayout>
__global__ void __launch_bounds__(kThreads) chunk_attn_simple_kernel(const ChunkArgs a) {
  constexpr int W = kLayout == DSA_KV_ROPE656 ? kD + kRopeDims : kD;
  constexpr int R = kLayout == DSA_KV_RAW512 ? kRawRow : kLayout == DSA_KV_SCALED528 ? kScaledRow : kRopeRow;
  constexpr int S = W + 1;
  extern __shared__ float smf[];
  float* qs = smf;                 // [kQ][S]
  float* ks = qs + kQ * S;         // [kK][S]
  __shared__ float ps[kQ][kK + 1], alpha[kQ], ms[kQ], ls[kQ];
  __shared__ int found[5], vis[kQ];
  __shared__ int64_t krow[kK];
  const int tid = threadIdx.x;
  if (tid == 0) {
    int64_t u = blockIdx.x;
    found[0] = -1;
    for (int b = 0; b < a.B; ++b) {
      int t0, n, kv, err;
      const bool some = request(a, b, t0, n, kv, err);
      if (err && blockIdx.x == 0) set_err(a.err, err);
      if (!some) continue;
      const int64_t units = ((int64_t)n * a.H + kQ - 1) / kQ;
      if (u < units && found[0] < 0) {
        found[0] = b;
        found[1] = t0;
        found[2] = n;
        found[3] = kv;
        found[4] = (int)u;
        if (blockIdx.x != 0) break;
      }
      u -= units;
    }
  }
  __syncthreads();
  if (found[0] < 0) return;
  const int b = found[0], t0 = found[1], n = found[2], kv = found[3];
  const int64_t r0 = (int64_t)found[4] * kQ;
  const int rows = (int)min((int64_t)kQ, (int64_t)n * a.H - r0);
  const int64_t g0 = (int64_t)t0 * a.H + r0;
  for (int i = tid; i < kQ * W; i += kThreads)
    qs[i / W * S + i % W] = i / W < rows ? bf16_bits_to_f32(a.q[(g0 + i / W) * W + i % W]) : 0.f;
  if (tid < kQ) {
    const int64_t v = a.causal ? (int64_t)kv - n + (r0 + tid) / a.H + 1 : kv;
    vis[tid] = tid < rows ? (int)max((int64_t)0, min(v, (int64_t)kv)) : 0;
    ms[tid] = -1e30f;
    ls[tid] = 0.f;
  }
  __syncthreads();
  const int last = vis[rows - 1];
  float acc[kQ][2] = {};
  for (int j0 = 0; j0 < last; j0 += kK) {
    if (tid < kK) {
      const int j = j0 + tid;
      krow[tid] = j < last ? resolve_row(j, a.page_table, a.B, a.max_pages, a.page_size, b, a.pool_rows, a.err) : -1;
    }
    __syncthreads();
    for (int i = tid; i < kK * W; i += kThreads) {
      const int k = i / W, d = i % W;
      float v = 0.f;
      if (krow[k] >= 0) {
        const uint8_t* row = a.pool + krow[k] * R;
        if (d < kD) {
          float f[4];
          e4m3x4_to_f32(row[d], f);
          v = f[0];
          if (kLayout != DSA_KV_RAW512) v *= *reinterpret_cast<const float*>(row + kD + d / kGroup * 4);
        } else {
          v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(row + kScaledRow + 2 * (d - kD)));
        }
      }
      ks[k * S + d] = v;
    }
    __syncthreads();
    {
      const int k = tid % kK, q0 = tid / kK;       // one key, query rows q0, q0 + 8, ...
      float s[4] = {};
      for (int d = 0; d < W; ++d) {
        const float kvv = ks[k * S + d];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = fmaf(qs[(q0 + 8 * i) * S + d], kvv, s[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = q0 + 8 * i;
        const bool see = j0 + k < vis[q] && krow[k] >= 0;
        const float x = see ? s[i] * a.sm_scale * kLog2e : -INFINITY;
        const float m = fmaxf(ms[q], warp_max(x));
        const float p = exp2f(x - m);
        const float l = warp_sum(p);
        ps[q][k] = p;
        __syncwarp();
        if (k == 0) {
          alpha[q] = exp2f(ms[q] - m);
          ls[q] = ls[q] * alpha[q] + l;
          ms[q] = m;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      acc[q][0] *= alpha[q];
      acc[q][1] *= alpha[q];
    }
    for (int k = 0; k < kK; ++k) {
      const float v0 = ks[k * S + tid], v1 = ks[k * S + tid + 256];
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const float p = ps[q][k];
        if (p != 0.f) {                            // a key that the query does not see adds nothing, NaN neither
          acc[q][0] = fmaf(p, v0, acc[q][0]);
          acc[q][1] = fmaf(p, v1, acc[q][1]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (q >= rows) break;
    const float l = ls[q], inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.o) + (g0 + q) * kD;
    o[tid] = __float2bfloat16_rn(acc[q][0] * inv);
    o[tid + 256] = __float2bfloat16_rn(acc[q][1] * inv);
    if (tid == 0) a.lse[g0 + q] = l == 0.f ? -INFINITY : (ms[q] + log2f(l)) * kLn2;
  }
}

template <int kLayout>
bool launch(const ChunkArgs& a, cudaStream_t stream) {
  constexpr int W = kLayout == DSA_KV_ROPE656 ? kD + kRopeDims : kD;
  const int smem = (kQ + kK) * (W + 1) * (int)sizeof(float);
  if (cudaFuncSetAttribute(chunk_attn_simple_kernel<kLayout>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return false;
  const int64_t units = ((int64_t)a.T * a.H + kQ - 1) / kQ + a.B;
  chunk_attn_simple_kernel<kLayout><<<(unsigned)units, kThreads, smem, stream>>>(a);
  return true;
}

}  // namespace

bool launch_chunk_attn(const ChunkArgs& a, cudaStream_t stream) {
  if (a.layout == DSA_KV_RAW512) return launch<DSA_KV_RAW512>(a, stream);
  if (a.layout == DSA_KV_SCALED528) return launch<DSA_KV_SCALED528>(a, stream);
  return launch<DSA_KV_ROPE656>(a, stream);
}

}  // namespace dsa
