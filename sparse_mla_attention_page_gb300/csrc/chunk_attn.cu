// Dense causal MLA attention of each request's new tokens over everything the
// request holds in the paged FP8 pool, on the 5th-generation tensor cores.
//
//   s_j = sm_scale log2(e) <q, k_j>,  p_j = 2^(s_j - m),  l = sum_j p_j
//   O = sum_j p_j v_j / l,            LSE = ln2 (m + log2 l)
//
// Orientation.  A unit (chunk.cuh) is NC query rows; its keys come in tiles of
// 128.  Scores are formed transposed, S^T = K Q^T (M = 128 keys, N = query
// columns), and so is the output, O^T += V^T P^T (M = 128 latent dims, four
// times, N = NC): the E4M3 rows land in shared memory once and are both the
// K-major A operand of the first product and the MN-major A operand of the
// second, with no conversion.  512 output dims of 64 query rows take half the
// tensor memory, the score buffers the other half, so NC = 64 is the widest
// unit; with 128 query rows along M instead, O alone would fill it.
//
// 16-bit data on 8-bit operands.  A BF16 query splits exactly into two E4M3
// terms (hi, and lo 16 times larger, both NC columns of one operand), times a
// power of two for each row; scores are then exact but for their FP32 sums.
// Softmax weights are written as two E4M3 terms that add up in the same
// accumulator (two K ranges): 8 significant bits, as BF16 weights would have.
// p is scaled so that the running maximum maps to 2^4 and may grow to 2^8
// before the maximum moves, which keeps E4M3's smallest step 2^-13 or less of
// the largest weight.
//
// Group scales (528- and 656-byte rows): one pass of the score product for
// each 128-dim group, multiplied by the row's scale as it is read out, and one
// P operand for each group, p s_g, against that group's block of values.  The
// running maximum is kept of s + log2(largest scale of the row), which bounds
// the entries of all four.  RoPE dims are one more pass, BF16.
//
// Warp roles (24 warps): 16 softmax (warp w: TMEM lane quarter w % 4 = 32 keys
// of the tile, column quarter w / 4), one issuing thread for each product, six
// producers that translate keys to rows and gather them with 16-byte cp.async
// into a ring of 16 KB blocks (128 keys x 128 bytes).  A block is released as
// soon as the product that reads it last has finished.
#include <atomic>
#include <cstddef>
#include <cuda_bf16.h>

#include "chunk.cuh"
#include "dsa_common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kTile = kChunkTile;
constexpr int kBlock = kTile * 128;          // bytes of a ring block
constexpr float kTop = 8.0f;                 // p never exceeds 2^kTop
constexpr float kBias = 4.0f;                // p of the key that set the maximum: 2^kBias
constexpr float kNoMax = -1.0e30f;           // maximum of a row that has seen no key (finite: 2^(-inf - m) = 0)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSmxWarps = 16, kSmxThreads = 512;
constexpr int kQkWarp = 16, kPvWarp = 17, kProdWarp0 = 18, kProdWarps = 6, kProdThreads = 192;
constexpr int kThreads = 768;
constexpr int kQuads = kTile / 4;            // producer work unit: 4 rows (one warp instruction per 128-byte piece)
constexpr int kQuadsPerWarp = (kQuads + kProdWarps - 1) / kProdWarps;
constexpr int kLaunchRegs = 80;              // registers a thread at launch (768 threads); the softmax warps then
constexpr int kSmxRegs = 96;                 // take 96 and the others give back to 48: 512 x 96 + 256 x 48 = 768 x 80
constexpr int kOtherRegs = 48;
static_assert(kSmxRegs * kSmxThreads + kOtherRegs * (kThreads - kSmxThreads) == kLaunchRegs * kThreads, "register split");
constexpr int kMeta = 4;                     // tiles whose rows and scales are kept
constexpr int kMaxBlocks = 12;
constexpr int kSmemLimit = 232448;

struct Misc {
  uint64_t full[kMaxBlocks], empty[kMaxBlocks];
  uint64_t meta_full[kMeta];       // rows (and scales) of a tile are in place
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], p_free[2];
  uint64_t q_full;                 // a segment's query operand is built
  uint64_t pv_done[2];             // all PV products of the even, the odd tiles
  uint64_t final[2];               // drain of the two issuers
  uint32_t tmem_base;
  int abort;
  __align__(16) int32_t rows[kMeta][kTile];   // pool row of each key, -1: masked
  __align__(16) float sig[2][64];  // per segment parity: log2-domain factor of each query column
  __align__(16) int vis[2][64];    // keys that it sees
  __align__(16) float mrun[2][64]; // its running maximum
  float red[4][4][16];             // [column quarter][lane quarter][column]
  float linv[64], lse[64];
};
constexpr int kMiscBytes = 5632;
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

template <int NC, int kLayout>
struct Cfg {
  static constexpr bool kScaled = kLayout != DSA_KV_RAW512;
  static constexpr bool kRope = kLayout == DSA_KV_ROPE656;
  static constexpr int R = kLayout == DSA_KV_RAW512 ? kRawRow : kLayout == DSA_KV_SCALED528 ? kScaledRow : kRopeRow;
  static constexpr int CPT = NC / 4;                 // query columns of a softmax thread
  static constexpr int G = kScaled ? 4 : 1;          // P operands of a tile
  static constexpr int NPASS = G + (kRope ? 1 : 0);  // score passes of a tile
  static constexpr int NB = kRope ? 5 : 4;           // ring blocks of a tile (RoPE first)
  static constexpr int NQ = 2 * NC;                  // columns of the query operand: hi, lo
  static constexpr int TERMS = 2;                    // E4M3 terms of P
  static constexpr int S_COLS = NQ;
  static constexpr int O_COL0 = 2 * S_COLS;
  static constexpr int TMEM_COLS = O_COL0 + 4 * NC;  // 128, 256 or 512
  static constexpr int Q_BYTES = NQ * 512;
  static constexpr int QR_BYTES = kRope ? NC * 128 : 0;
  static constexpr int P_TERM = NC * 128;            // bytes of one term
  static constexpr int P_BYTES = TERMS * P_TERM;
  static constexpr int SC_BYTES = kScaled ? kMeta * kTile * 16 : 0;
  static constexpr int FIXED = kMiscBytes + 1024 + Q_BYTES + QR_BYTES + SC_BYTES;
  static constexpr int NPB = 2;                      // P operands in flight
  static constexpr int NS_FIT = (kSmemLimit - FIXED - NPB * P_BYTES) / kBlock;
  static constexpr int NS = NS_FIT < kMaxBlocks ? NS_FIT : kMaxBlocks;
  static constexpr int Q_OFF = NS * kBlock;
  static constexpr int QR_OFF = Q_OFF + Q_BYTES;
  static constexpr int P_OFF = QR_OFF + QR_BYTES;
  static constexpr int SC_OFF = P_OFF + NPB * P_BYTES;
  static constexpr int MISC_OFF = SC_OFF + SC_BYTES;
  static constexpr int SMEM = MISC_OFF + kMiscBytes + 1024;
  static_assert(NS > NB, "a tile's blocks and one more");
  // a tile's rows are replaced kMeta tiles later, when its blocks are gone from the ring
  static_assert((NS - 1) / 4 + 1 < kMeta, "rows of a tile in use");
  static_assert(SMEM <= kSmemLimit && TMEM_COLS <= 512 && P_TERM % 1024 == 0 && QR_BYTES % 1024 == 0, "budgets");
};

// Byte offset of element (n, k) in a K-major operand of N rows whose K extent
// is split into 128-byte blocks, with the 128-byte swizzle.
template <int N>
__device__ __forceinline__ uint32_t kmajor_off(int n, int k) {
  return (k >> 7) * (N * 128) + (n >> 3) * 1024 + (n & 7) * 128 + ((((k >> 4) & 7) ^ (n & 7)) << 4) + (k & 15);
}

// Byte offset of P column n, key k in the MN-major PV operand without swizzle:
// core matrices of 8 keys x 16 columns.
template <int NC>
__device__ __forceinline__ uint32_t p_off(int n, int k) {
  return (n >> 4) * 128 + (k >> 3) * (NC * 8) + (k & 7) * 16 + (n & 15);
}

// Leaves in lane l the max (or sum) over the 32 lanes of v[l % N].
template <int N, bool kMax>
__device__ __forceinline__ float transpose_reduce(float (&v)[N], int lane) {
#pragma unroll
  for (int w = N / 2; w >= 1; w /= 2) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float send = upper ? v[k] : v[k + w];
      const float keep = upper ? v[k + w] : v[k];
      const float recv = __shfl_xor_sync(0xffffffffu, send, w);
      v[k] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  float r = v[0];
#pragma unroll
  for (int off = N; off < 32; off *= 2) {
    const float o = __shfl_xor_sync(0xffffffffu, r, off);
    r = kMax ? fmaxf(r, o) : r + o;
  }
  return r;
}

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// x * 2^e exactly for |e| up to 252.
__device__ __forceinline__ float scale_pow2(float x, int e) {
  const int e1 = e / 2, e2 = e - e1;
  return __fmul_rn(__fmul_rn(x, __int_as_float((127 + e1) << 23)), __int_as_float((127 + e2) << 23));
}

__device__ __forceinline__ uint64_t desc_add(uint64_t desc, uint32_t bytes) { return desc + (uint64_t)(bytes >> 4); }

// 32 lanes x N consecutive columns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    tmem_ld4(taddr, v);
  } else if constexpr (N == 8) {
    tmem_ld8(taddr, v);
  } else {
    static_assert(N == 16, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    tmem_st4(taddr, v);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8) {
      uint32_t t8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t8[k] = v[c + k];
      tmem_st8(taddr + c, t8);
    }
  }
}

// Two E4M3 terms of a pair of weights, p ~ hi + lo, from the FP16 value of p
// (the residual is exact in FP16).
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi2, uint32_t& lo2) {
  uint32_t p, t, r;
  uint16_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(v1), "f"(v0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(p));
  hi2 = h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(t) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(t));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(r));
  lo2 = h;
}

// N bytes (4, 8 or 16) held as pairs, to shared memory.
template <int N>
__device__ __forceinline__ void st_bytes(uint32_t addr, const uint32_t (&t)[N / 2]) {
  if constexpr (N == 16)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(t[0] | t[1] << 16), "r"(t[2] | t[3] << 16),
                 "r"(t[4] | t[5] << 16), "r"(t[6] | t[7] << 16)
                 : "memory");
  else if constexpr (N == 8)
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(t[0] | t[1] << 16), "r"(t[2] | t[3] << 16) : "memory");
  else
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(t[0] | t[1] << 16) : "memory");
}

// N consecutive values of a 16-byte aligned shared array (the same for the whole warp).
template <int N, class T>
__device__ __forceinline__ void ld_row(const T* p, T (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const int4 x = *reinterpret_cast<const int4*>(p + k);
    v[k] = reinterpret_cast<const T&>(x.x);
    v[k + 1] = reinterpret_cast<const T&>(x.y);
    v[k + 2] = reinterpret_cast<const T&>(x.z);
    v[k + 3] = reinterpret_cast<const T&>(x.w);
  }
}

// A CTA's walk through its tiles.  A segment is the part of a unit inside the
// CTA's range.  The next unit's entry is fetched while the current one is
// worked on.
struct Walk {
  ChunkUnit u, next;
  int unit, tile;
  __device__ __forceinline__ static ChunkUnit fetch(const ChunkWork& w, int i, int n_units) {
    union {
      ChunkUnit u;
      int4 v[3];
    } x;
    const int4* src = reinterpret_cast<const int4*>(w.units + (i < n_units ? i : n_units - 1));
#pragma unroll
    for (int k = 0; k < 3; ++k) x.v[k] = __ldcg(src + k);
    return x.u;
  }
  __device__ __forceinline__ Walk(const ChunkWork& w, int first_unit, int64_t t0, int n_units) {
    unit = first_unit;
    u = fetch(w, unit, n_units);
    next = fetch(w, unit + 1, n_units);
    tile = (int)(t0 - u.tile0);
  }
  __device__ __forceinline__ void advance(const ChunkWork& w, int n_units) {
    if (++tile == u.tiles) {
      tile = 0;
      u = next;
      next = fetch(w, ++unit + 1, n_units);
    }
  }
  __device__ __forceinline__ bool first(int it) const { return it == 0 || tile == 0; }
  __device__ __forceinline__ bool last(int it, int n_it) const { return it == n_it - 1 || tile == u.tiles - 1; }
};

struct Range {
  int64_t t0;
  int n_it, unit, n_units;
};

// ------------------------------------------------------------------- roles

template <int NC, int kLayout>
__device__ void producer_role(const ChunkWork& w, uint8_t* sm, Misc& ms, const Range& rg) {
  using C = Cfg<NC, kLayout>;
  const ChunkArgs& a = w.a;
  const int ptid = threadIdx.x - kProdWarp0 * 32, pw = ptid >> 5, lane = ptid & 31;
  const int rq = lane >> 3, ch = lane & 7;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  // thread -> key ptid of each tile: its page-table entry is fetched a tile ahead
  Walk cur(w, rg.unit, rg.t0, rg.n_units);
  int32_t entry = -1, off = 0;
  bool seen = false;
  auto look_up = [&]() {
    const int j = cur.tile * kTile + ptid;
    seen = ptid < kTile && j < chunk_visible(a, cur.u, cur.u.cols - 1);
    if (seen) {
      const int page = j / a.page_size;
      off = j - page * a.page_size;
      entry = __ldg(a.page_table + (int64_t)cur.u.b * a.max_pages + page);
    }
  };
  look_up();
  int slot = 0, phase = 0;
  bool ok = true;      // false once a wait gave up: keep going through every barrier
  for (int it = 0; it < rg.n_it; ++it) {
    const int m = it % kMeta;
    ok = ok && mbar_wait(smem_u32(&ms.empty[slot]), phase ^ 1, abort, w.wait_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (ptid < kTile) {
      int32_t row = -1;
      if (seen) {
        const int64_t r = (int64_t)entry * a.page_size + off;
        if (entry < 0 || r >= a.pool_rows) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
        else row = (int32_t)r;
      }
      ms.rows[m][ptid] = row;
      if (C::kScaled)
        cp_async_16_zfill(smem_u32(sm + C::SC_OFF + (m * kTile + ptid) * 16),
                          a.pool + (int64_t)(row >= 0 ? row : 0) * C::R + kD, row >= 0 ? 16u : 0u);
    }
    if (C::kScaled) cp_async_arrive_noinc(smem_u32(&ms.meta_full[m]));
    cur.advance(w, rg.n_units);
    if (it + 1 < rg.n_it) look_up();
    named_bar_sync(2, kProdThreads);
    if (ptid == 0) mbar_arrive(smem_u32(&ms.meta_full[m]));
    int32_t rows[kQuadsPerWarp];
#pragma unroll
    for (int i = 0; i < kQuadsPerWarp; ++i) {
      const int q = pw + i * kProdWarps;
      rows[i] = q < kQuads ? ms.rows[m][4 * q + rq] : -1;
    }
#pragma unroll 1
    for (int k = 0; k < C::NB; ++k) {
      if (k > 0) {
        ok = ok && mbar_wait(smem_u32(&ms.empty[slot]), phase ^ 1, abort, w.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (ok) {
        const uint32_t base = kv0 + slot * kBlock;
        const int col = (C::kRope ? (k == 0 ? kScaledRow : (k - 1) * 128) : k * 128) + ch * 16;
#pragma unroll
        for (int i = 0; i < kQuadsPerWarp; ++i) {
          const int q = pw + i * kProdWarps;
          if (q >= kQuads) break;
          const int r = 4 * q + rq;
          const uint8_t* src = a.pool + (int64_t)(rows[i] >= 0 ? rows[i] : 0) * C::R + col;
          cp_async_16_zfill(base + (r >> 3) * 1024 + (r & 7) * 128 + ((ch ^ (r & 7)) << 4), src, rows[i] >= 0 ? 16u : 0u);
        }
        cp_async_arrive_noinc(smem_u32(&ms.full[slot]));
      }
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  cp_async_wait_all();
}

// Waits (bounded) for every tcgen05 operation this thread issued, so that the
// tensor memory can be released.
__device__ __forceinline__ void drain_mma(uint32_t bar) {
  mma_commit(bar);
  volatile int no_abort = 0;
  mbar_wait(bar, 0, &no_abort, 2000000000ull);
}

template <int NC, int kLayout>
__device__ void qk_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout>;
  if ((threadIdx.x & 31) != 0) return;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  constexpr uint32_t kId = idesc_e4m3(C::NQ, false), kIdRope = idesc_bf16(NC);
  const uint64_t q_desc = sdesc_sw128(smem_u32(sm + C::Q_OFF), 16, 1024);
  Walk cur(w, rg.unit, rg.t0, rg.n_units);
  int slot = 0, phase = 0, seg = -1, si = 0;
  bool ok = true;
  for (int it = 0; it < rg.n_it && ok; ++it, cur.advance(w, rg.n_units)) {
    if (cur.first(it)) {
      ++seg;
      ok = mbar_wait(smem_u32(&ms.q_full), seg & 1, abort, w.wait_ns);
    }
#pragma unroll 1
    for (int k = 0; k < C::NB && ok; ++k) {
      const int sb = si & 1;
      const bool opens = C::kScaled || k == 0;     // first block of a score pass
      if (opens && si >= 2) ok = mbar_wait(smem_u32(&ms.s_free[sb]), ((si >> 1) - 1) & 1, abort, w.wait_ns);
      ok = ok && mbar_wait(smem_u32(&ms.full[slot]), phase, abort, w.wait_ns);
      if (!ok) break;
      fence_proxy_async_smem();   // rows landed through cp.async (generic proxy)
      tc_fence_after();
      const uint64_t ad = sdesc_sw128(kv0 + slot * kBlock, 16, 1024);
      const uint32_t d = tmem + sb * C::S_COLS;
      if (C::kRope && k == 0) {
        const uint64_t bd = sdesc_sw128(smem_u32(sm + C::QR_OFF), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(d, desc_add(ad, kk * 32), desc_add(bd, kk * 32), kIdRope, kk > 0 ? 1u : 0u);
        mma_commit(smem_u32(&ms.empty[slot]));
      } else {
        const int g = C::kRope ? k - 1 : k;
        const uint64_t bd = desc_add(q_desc, g * (C::NQ * 128));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_e4m3(d, desc_add(ad, kk * 32), desc_add(bd, kk * 32), kId, (!opens || kk > 0) ? 1u : 0u);
      }
      if (C::kScaled || k == C::NB - 1) {
        mma_commit(smem_u32(&ms.s_full[sb]));
        ++si;
      }
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  drain_mma(smem_u32(&ms.final[0]));
}

template <int NC, int kLayout>
__device__ void pv_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout>;
  if ((threadIdx.x & 31) != 0) return;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  constexpr uint32_t kId = idesc_e4m3(NC, true, true);
  const uint64_t p_desc = sdesc_mn_none(smem_u32(sm + C::P_OFF), NC * 8, 128);
  Walk cur(w, rg.unit, rg.t0, rg.n_units);
  int slot = 0, pi = 0;
  bool ok = true;
  auto step = [&]() { slot = slot + 1 == C::NS ? 0 : slot + 1; };
  for (int it = 0; it < rg.n_it && ok; ++it, cur.advance(w, rg.n_units)) {
    const bool first = cur.first(it);
    if (C::kRope) step();                          // the RoPE block is QK^T's alone
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      const int pb = pi % C::NPB;
      if (C::kScaled || g == 0) {
        ok = mbar_wait(smem_u32(&ms.p_full[pb]), (pi / C::NPB) & 1, abort, w.wait_ns);
        if (!ok) break;
        fence_proxy_async_smem();   // P and the rows were written through the generic proxy
        tc_fence_after();
      }
      const uint64_t ad = sdesc_sw128(kv0 + slot * kBlock, 1024, 1024);
      const uint64_t bd = desc_add(p_desc, pb * C::P_BYTES);
      const uint32_t d = tmem + C::O_COL0 + g * NC;
#pragma unroll
      for (int t = 0; t < C::TERMS; ++t)
#pragma unroll
        for (int js = 0; js < 4; ++js)
          mma_e4m3(d, desc_add(ad, js * 4096), desc_add(bd, t * C::P_TERM + js * 4 * (NC * 8)), kId,
                   (t > 0 || js > 0) ? 1u : (first ? 0u : 1u));
      mma_commit(smem_u32(&ms.empty[slot]));
      step();
      if (C::kScaled || g == 3) {
        mma_commit(smem_u32(&ms.p_free[pb]));
        ++pi;
      }
    }
    if (ok) mma_commit(smem_u32(&ms.pv_done[it & 1]));
  }
  drain_mma(smem_u32(&ms.final[1]));
}

// The query operand of one segment, and its columns' factors, visible keys and
// maxima.  512 threads: column tid / TPH, dims [DPT (tid % TPH), + DPT).
template <int NC, int kLayout>
__device__ __forceinline__ void build_query(const ChunkWork& w, uint8_t* sm, Misc& ms, const ChunkUnit& u, int par) {
  using C = Cfg<NC, kLayout>;
  constexpr int TPH = kSmxThreads / NC, DPT = kD / TPH, NV = DPT / 8;
  const ChunkArgs& a = w.a;
  const int col = threadIdx.x / TPH, part = threadIdx.x % TPH;
  const uint16_t* src = a.q + (u.row0 + col) * a.q_row;
  const bool live_col = col < u.cols;
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i] = live_col ? __ldg(reinterpret_cast<const uint4*>(src + part * DPT) + i) : make_uint4(0, 0, 0, 0);
  if constexpr (C::kRope) {
    const int rc = threadIdx.x >> 3, ch = threadIdx.x & 7;      // column, 16-byte chunk of its 64 RoPE dims
    if (rc < NC) {
      const uint4 x = rc < u.cols ? __ldg(reinterpret_cast<const uint4*>(a.q + (u.row0 + rc) * a.q_row + kD) + ch)
                                  : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(sm + C::QR_OFF + (rc >> 3) * 1024 + (rc & 7) * 128 + ((ch ^ (rc & 7)) << 4)) = x;
    }
  }
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f0 = fabsf(bf16_bits_to_f32(x[j] & 0xFFFFu)), f1 = fabsf(bf16_bits_to_f32(x[j] >> 16));
      amax = fmaxf(amax, fmaxf(f0, f1));
      nan |= !(f0 + f1 < INFINITY);
    }
  }
  if (nan) amax = INFINITY;
#pragma unroll
  for (int off = TPH / 2; off >= 1; off /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  int sh = 0;
  const float base = a.sm_scale * kLog2e;
  float sig = 0.f;
  const bool live = amax > 0.f && amax <= 1.0e38f;
  if (live) {
    int e;
    const float f = frexpf(amax, &e);                // amax = f 2^e, f in [0.5, 1)
    sh = f <= 0.875f ? 9 - e : 8 - e;                // largest sh with amax 2^sh <= 448
    sig = scale_pow2(base, -sh);
  } else if (amax > 0.f) {
    sig = __int_as_float(0x7FC00000);                // a row with a NaN or an infinity scores NaN
  }
  uint8_t* qb = sm + C::Q_OFF;
#pragma unroll
  for (int c = 0; c < NV / 2; ++c) {
    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
    if (live) {
      const uint32_t x[8] = {v[2 * c].x, v[2 * c].y, v[2 * c].z, v[2 * c].w,
                             v[2 * c + 1].x, v[2 * c + 1].y, v[2 * c + 1].z, v[2 * c + 1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4], yh[4];
        y[0] = scale_pow2(bf16_bits_to_f32(x[2 * i] & 0xFFFFu), sh);
        y[1] = scale_pow2(bf16_bits_to_f32(x[2 * i] >> 16), sh);
        y[2] = scale_pow2(bf16_bits_to_f32(x[2 * i + 1] & 0xFFFFu), sh);
        y[3] = scale_pow2(bf16_bits_to_f32(x[2 * i + 1] >> 16), sh);
        hi[i] = e4m3x4_satrne(y[0], y[1], y[2], y[3]);
        e4m3x4_to_f32(hi[i], yh);
        lo[i] = e4m3x4_satrne((y[0] - yh[0]) * 16.f, (y[1] - yh[1]) * 16.f, (y[2] - yh[2]) * 16.f, (y[3] - yh[3]) * 16.f);
      }
    }
    const int k0 = part * DPT + 16 * c;
    *reinterpret_cast<uint4*>(qb + kmajor_off<C::NQ>(col, k0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(qb + kmajor_off<C::NQ>(NC + col, k0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  if (part == 0) {
    ms.sig[par][col] = sig;
    ms.vis[par][col] = live_col ? chunk_visible(a, u, col) : 0;
    ms.mrun[par][col] = kNoMax;
  }
  fence_proxy_async_smem();
  warp_arrive(smem_u32(&ms.q_full));
}

template <int NC, int kLayout>
__device__ void softmax_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout>;
  constexpr int CPT = C::CPT;
  const ChunkArgs& a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, cq = warp >> 2;
  const int row = 32 * quarter + lane;                   // key of the tile = TMEM lane (dim of a block, for O)
  const int c0 = cq * CPT;                               // first column
  const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
  volatile int* abort = &ms.abort;
  float l_part[CPT];
  float m_lane = kNoMax;                                 // running maximum of column c0 + lane % CPT
  int seg = -1, si = 0, pi = 0, slot0 = 0;               // slot0: ring slot of the tile's first latent block
  bool ok = true;                                        // false once a wait gave up: keep going through every barrier
  if (C::kRope) slot0 = 1;
  Walk cur(w, rg.unit, rg.t0, rg.n_units);
  build_query<NC, kLayout>(w, sm, ms, cur.u, 0);
  for (int it = 0; it < rg.n_it; ++it) {
    const bool first = cur.first(it), last = cur.last(it, rg.n_it);
    const int m = it % kMeta;
    if (first) {
      ++seg;
      ok &= mbar_wait(smem_u32(&ms.q_full), seg & 1, abort, w.wait_ns);
      m_lane = kNoMax;
#pragma unroll
      for (int k = 0; k < CPT; ++k) l_part[k] = 0.f;
    }
    const int par = seg & 1;
    ok &= mbar_wait(smem_u32(&ms.meta_full[m]), (it / kMeta) & 1, abort, w.wait_ns);
    const int j = cur.tile * kTile + row;
    const bool valid = ms.rows[m][row] >= 0;
    float sc[4] = {1.f, 1.f, 1.f, 1.f}, lsc = 0.f;
    if (C::kScaled) {
      const float4 v = *reinterpret_cast<const float4*>(sm + C::SC_OFF + (m * kTile + row) * 16);
      sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
      const float big = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
      lsc = fminf(fmaxf(log2f(big), -100.f), 100.f);     // rows of no magnitude add next to nothing to any output
    }
    // scores
    float s2[CPT];
    bool poisoned = false;                               // a NaN byte in the row: every column's sum is NaN
#pragma unroll
    for (int pass = 0; pass < C::NPASS; ++pass) {
      const int sb = si & 1;
      ok &= mbar_wait(smem_u32(&ms.s_full[sb]), (si >> 1) & 1, abort, w.wait_ns);
      ++si;
      tc_fence_after();
      const uint32_t base = lane_base + sb * C::S_COLS + c0;
      if (C::kRope && pass == 0) {
        uint32_t v[CPT];
        tmem_ld<CPT>(base, v);
        tmem_wait_ld();
        const float rsig = a.sm_scale * kLog2e;
#pragma unroll
        for (int k = 0; k < CPT; ++k) s2[k] = __uint_as_float(v[k]) * rsig;
      } else {
        const int g = C::kRope ? pass - 1 : pass;
        uint32_t hi[CPT], lo[CPT];
        tmem_ld<CPT>(base, hi);
        tmem_ld<CPT>(base + NC, lo);
        tmem_wait_ld();
        float sg[CPT];
        ld_row<CPT>(&ms.sig[par][c0], sg);
        poisoned |= __uint_as_float(hi[0]) != __uint_as_float(hi[0]);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          const float v = fmaf(__uint_as_float(lo[k]), 0.0625f, __uint_as_float(hi[k])) * sg[k];
          s2[k] = !C::kScaled ? v : (pass == 0) ? v * sc[g] : fmaf(v, sc[g], s2[k]);
        }
      }
      tc_fence_before();
      warp_arrive(smem_u32(&ms.s_free[sb]));
    }
    // a row with an infinite or NaN scale holds infinities of both signs and NaN: it scores NaN
    const bool odd_scale = C::kScaled && !(fabsf(sc[0]) + fabsf(sc[1]) + fabsf(sc[2]) + fabsf(sc[3]) < INFINITY);
    if (odd_scale) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) s2[k] = __int_as_float(0x7FC00000);
    }
    // keys that a column does not see
    if (!__all_sync(0xffffffffu, valid && cur.tile * kTile + kTile <= ms.vis[par][0])) {
      int vis[CPT];
      ld_row<CPT>(&ms.vis[par][c0], vis);
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (!valid || j >= vis[k]) s2[k] = -INFINITY;
    }
    // Does a column's running maximum have to move?  One barrier ORs the
    // threads' answers; only then are the tile's maxima formed.
    float mr[CPT];
    ld_row<CPT>(&ms.mrun[par][c0], mr);
    bool grow = false;
#pragma unroll
    for (int k = 0; k < CPT; ++k) grow |= s2[k] + lsc > mr[k] + kTop;
    if (named_bar_red_or(1, kSmxThreads, grow)) {
      float tmp[CPT];
#pragma unroll
      for (int k = 0; k < CPT; ++k) tmp[k] = s2[k] + lsc;
      const float wmax = transpose_reduce<CPT, true>(tmp, lane);
      if (lane < CPT) ms.red[cq][quarter][lane] = wmax;
      named_bar_sync(1, kSmxThreads);
      const int cl = lane % CPT;
      const float tmax = fmaxf(fmaxf(ms.red[cq][0][cl], ms.red[cq][1][cl]), fmaxf(ms.red[cq][2][cl], ms.red[cq][3][cl]));
      float alpha_lane = 1.f;
      const bool need = tmax > m_lane + kTop;
      if (need) {
        const float to = tmax - kBias;
        alpha_lane = ex2_approx(m_lane - to);
        m_lane = to;
      }
      const unsigned moved = __ballot_sync(0xffffffffu, need);
      if (quarter == 0 && lane < CPT) ms.mrun[par][c0 + lane] = m_lane;
      if (moved) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) l_part[k] *= __shfl_sync(0xffffffffu, alpha_lane, k);
        if (!first) {      // O holds this segment's earlier tiles
          ok &= mbar_wait(smem_u32(&ms.pv_done[(it - 1) & 1]), ((it - 1) >> 1) & 1, abort, w.wait_ns);
          tc_fence_after();
#pragma unroll 1
          for (int db = 0; db < 4; ++db) {
            uint32_t v[CPT];
            tmem_ld<CPT>(lane_base + C::O_COL0 + db * NC + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < CPT; ++k)
              v[k] = __float_as_uint(__uint_as_float(v[k]) * __shfl_sync(0xffffffffu, alpha_lane, k));
            tmem_st<CPT>(lane_base + C::O_COL0 + db * NC + c0, v);
          }
          tmem_wait_st();
        }
      }
      named_bar_sync(1, kSmxThreads);
      ld_row<CPT>(&ms.mrun[par][c0], mr);
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      s2[k] = ex2_approx(s2[k] - mr[k]);
      l_part[k] += s2[k];
    }
    if (poisoned) {
      // The row counts as NaN for the columns that see it (p is NaN already);
      // with its bytes cleared, the others' weight 0 gives 0.  Each of the four
      // column quarters clears one 128-byte block of the row.
      int sl = slot0 + cq;
      if (sl >= C::NS) sl -= C::NS;
      uint4* p = reinterpret_cast<uint4*>(sm + sl * kBlock + (row >> 3) * 1024 + (row & 7) * 128);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = make_uint4(0, 0, 0, 0);
    }
    // every phase of pv_done is waited for, two tiles on, so that its parity tells the tiles apart
    if (it >= 2) ok &= mbar_wait(smem_u32(&ms.pv_done[it & 1]), ((it >> 1) - 1) & 1, abort, w.wait_ns);
    // P operands
#pragma unroll
    for (int g = 0; g < C::G; ++g) {
      const int pb = pi % C::NPB;
      uint32_t hi2[CPT / 2], lo2[CPT / 2];
#pragma unroll
      for (int k = 0; k < CPT; k += 2) {
        float v0 = s2[k], v1 = s2[k + 1];
        if (C::kScaled) {
          v0 *= sc[g];
          v1 *= sc[g];
          if (odd_scale) {                               // a weight of 0 times an infinite scale is 0
            if (s2[k] == 0.f) v0 = 0.f;
            if (s2[k + 1] == 0.f) v1 = 0.f;
          }
        }
        split2(v0, v1, hi2[k / 2], lo2[k / 2]);
      }
      if (pi >= C::NPB) ok &= mbar_wait(smem_u32(&ms.p_free[pb]), ((pi / C::NPB) - 1) & 1, abort, w.wait_ns);
      const uint32_t at = smem_u32(sm + C::P_OFF) + pb * C::P_BYTES + p_off<NC>(c0, row);
      st_bytes<CPT>(at, hi2);
      st_bytes<CPT>(at + C::P_TERM, lo2);
      fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive(smem_u32(&ms.p_full[pb]));
      ++pi;
    }
    slot0 += C::NB;
    if (slot0 >= C::NS) slot0 -= C::NS;
    // every score pass of this tile is done, so the query operand may be replaced
    if (last && it + 1 < rg.n_it) build_query<NC, kLayout>(w, sm, ms, cur.next, (seg + 1) & 1);

    if (last) {
      // denominators, O, LSE
      const float wsum = transpose_reduce<CPT, false>(l_part, lane);
      if (lane < CPT) ms.red[cq][quarter][lane] = wsum;
      named_bar_sync(1, kSmxThreads);
      if (quarter == 0 && lane < CPT) {
        const float l = (ms.red[cq][0][lane] + ms.red[cq][1][lane]) + (ms.red[cq][2][lane] + ms.red[cq][3][lane]);
        ms.linv[c0 + lane] = l == 0.f ? 0.f : 1.f / l;
        ms.lse[c0 + lane] = l == 0.f ? -INFINITY : (m_lane + log2f(l)) * kLn2;
      }
      named_bar_sync(1, kSmxThreads);
      ok &= mbar_wait(smem_u32(&ms.pv_done[it & 1]), (it >> 1) & 1, abort, w.wait_ns);
      tc_fence_after();
      const ChunkUnit& u = cur.u;
      const bool whole = u.tile0 >= rg.t0 && u.tile0 + u.tiles <= rg.t0 + rg.n_it;
      const int64_t part = ((int64_t)blockIdx.x * 2 + (rg.t0 >= u.tile0 ? 0 : 1)) * NC;
#pragma unroll 1
      for (int db = 0; db < 4; ++db) {
        uint32_t v[CPT];
        tmem_ld<CPT>(lane_base + C::O_COL0 + db * NC + c0, v);
        tmem_wait_ld();
        const int d = db * 128 + row;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          if (c0 + k >= u.cols) break;
          const float li = ms.linv[c0 + k];
          const float o = li == 0.f ? 0.f : __uint_as_float(v[k]) * li;
          if (whole) reinterpret_cast<__nv_bfloat16*>(a.o)[(u.row0 + c0 + k) * kD + d] = __float2bfloat16_rn(o);
          else w.part_o[(part + c0 + k) * kD + d] = o;
        }
      }
      if (quarter == 0 && lane < CPT && c0 + lane < u.cols) {
        if (whole) a.lse[u.row0 + c0 + lane] = ms.lse[c0 + lane];
        else w.part_lse[part + c0 + lane] = ms.lse[c0 + lane];
      }
    }
    cur.advance(w, rg.n_units);
  }
  (void)ok;
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int NC, int kLayout>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkWork w) {
  using C = Cfg<NC, kLayout>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc& ms = *reinterpret_cast<Misc*>(sm + C::MISC_OFF);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(smem_u32(&ms.full[s]), kProdThreads);
      mbar_init(smem_u32(&ms.empty[s]), 1);
    }
    for (int s = 0; s < kMeta; ++s) mbar_init(smem_u32(&ms.meta_full[s]), 1 + (C::kScaled ? kProdThreads : 0));
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.s_full[s]), 1);
      mbar_init(smem_u32(&ms.s_free[s]), kSmxWarps);
      mbar_init(smem_u32(&ms.p_full[s]), kSmxWarps);
      mbar_init(smem_u32(&ms.p_free[s]), 1);
      mbar_init(smem_u32(&ms.final[s]), 1);
    }
    mbar_init(smem_u32(&ms.q_full), kSmxWarps);
    mbar_init(smem_u32(&ms.pv_done[0]), 1);
    mbar_init(smem_u32(&ms.pv_done[1]), 1);
    ms.abort = 0;
    mbar_init_fence();
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(&ms.tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  // everything above overlapped the plan, whose list is visible from here on
  grid_dependency_wait();
  grid_launch_dependents();   // the merge: its blocks wait for the whole grid
  Range rg;
  const int64_t n_tiles = __ldcg(&w.hdr->n_tiles);
  rg.n_units = __ldcg(&w.hdr->n_units);
  const int grid = (int)(n_tiles < w.grid ? n_tiles : w.grid);
  rg.t0 = 0;
  rg.n_it = rg.unit = 0;
  if ((int)blockIdx.x < grid) {
    rg.t0 = chunk_tile_begin(blockIdx.x, n_tiles, grid);
    rg.n_it = (int)(chunk_tile_begin(blockIdx.x + 1, n_tiles, grid) - rg.t0);
    rg.unit = __ldcg(w.cta_unit + blockIdx.x);
  }
  if (rg.n_it > 0) {          // the same for the whole CTA
    if (warp < kSmxWarps) {
      regs_inc<kSmxRegs>();
      softmax_role<NC, kLayout>(w, sm, ms, tmem, rg);
    } else {
      regs_dec<kOtherRegs>();
      if (warp == kQkWarp) qk_role<NC, kLayout>(w, sm, ms, tmem, rg);
      else if (warp == kPvWarp) pv_role<NC, kLayout>(w, sm, ms, tmem, rg);
      else producer_role<NC, kLayout>(w, sm, ms, rg);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (tid == 0 && ms.abort) set_err(w.a.err, DSA_DEV_ERR_TIMEOUT);
}

template <int NC, int kLayout>
bool launch(const ChunkWork& w, cudaStream_t stream) {
  using C = Cfg<NC, kLayout>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<NC, kLayout>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return false;
    // the register re-split adds up only from exactly kLaunchRegs registers a thread
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, chunk_attn_kernel<NC, kLayout>) != cudaSuccess || fa.numRegs != kLaunchRegs)
      return false;
    configured.fetch_or(bit);
  }
  launch_chunk_plan(w, stream);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_attn_kernel<NC, kLayout>, w) != cudaSuccess) return false;
  return launch_chunk_merge(w, stream);
}

template <int NC>
bool launch_nc(const ChunkWork& w, cudaStream_t stream) {
  if (w.a.layout == DSA_KV_RAW512) return launch<NC, DSA_KV_RAW512>(w, stream);
  if (w.a.layout == DSA_KV_SCALED528) return launch<NC, DSA_KV_SCALED528>(w, stream);
  return launch<NC, DSA_KV_ROPE656>(w, stream);
}

}  // namespace

int chunk_columns(int T, int H, int B) {
  const int64_t rows = ((int64_t)T * H + B - 1) / B;     // of an average request
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

bool launch_chunk_attn(const ChunkWork& w, cudaStream_t stream) {
  if (w.nc == 16) return launch_nc<16>(w, stream);
  if (w.nc == 32) return launch_nc<32>(w, stream);
  return launch_nc<64>(w, stream);
}

}  // namespace dsa
