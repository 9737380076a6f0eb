// Dense causal MLA attention of each request's new tokens over everything the
// request holds in the paged FP8 pool, on the 5th-generation tensor cores.
//
//   s_j = sm_scale log2(e) <q, k_j>,  p_j = 2^(s_j - m),  l = sum_j p_j
//   O = sum_j p_j v_j / l,            LSE = ln2 (m + log2 l)
//
// Orientation.  A unit (chunk.cuh) is NC = 16 or 32 query rows; its keys come in
// tiles of 128.  Scores are formed transposed, S^T = K Q^T (M = 128 keys, N =
// query columns), and so is the output, O^T += V^T P^T (M = 128 latent dims,
// four times): the E4M3 rows land in shared memory once and are both the
// K-major A operand of the first product and the MN-major A operand of the
// second, with no conversion.  (With query rows along M the FP32 output of 128
// rows alone would fill the tensor memory.)  Units of 64 columns were built
// too: they read a tile once for twice the columns, but their operands leave
// room for little more than one tile of rows, and they ran 4 % (4096 tokens
// over 8192, 656-byte rows) to 8 % (prompts over raw rows) slower.
//
// 16-bit data on 8-bit operands.  A BF16 query times a power of two for its row
// splits into two E4M3 terms, q ~ hi + lo / 16, exactly where it is within
// 2^14 of the row's largest entry; softmax weights likewise, p ~ hi + lo / 16.
// The terms are columns of their own in both products, so a tile is read once
// for both.  A thread's hi and lo weights lie side by side, one store for both
// (1 % faster); its scores do not, as one load of both spills registers.
//
// Weights p = 2^(s - M) have 8 significant bits down to 2^-6 and lo's smallest
// step, 2^-13, below.  l sums them unrounded, so what rounding takes from them
// has to even out: a tail of keys below 2^-14 behind one that dominates (the
// first of a context often does) would, rounded to nearest, leave O altogether
// while l counts it (8192 keys 10 nats below one: 27 % of O; 93 % in the worst
// of the tests).  So lo is rounded behind a shift within half a step that
// differs from key to key (shift_of): as many weights go up as their size asks
// for.  It joins the multiplication by 16 and costs nothing.  What is left is
// noise: over the n tiles of a segment sqrt(128 n) 2^-14 at most, in the RMS, of
// a weight 1.  A move therefore puts the tile's largest p at 2^lift, lift =
// log2(n) / 2 - 2 for the n tiles to come, at least 1 (as a shift may cost a
// whole step instead of half of one): 0.6 % of the largest weight at most,
// however many keys there are.  Over scaled rows lift = log2(n) / 2, at least 1,
// as their operands hold s_g / S of a weight (below), and S follows the largest
// group of the largest row: a context behind a dominant key whose largest group
// is 8 times the others' comes out within 1 %, with 2 less within 2 to 3 %.  p
// may grow to 2^8.75 before M moves again (E4M3 ends at 448).  A move waits for
// the value products, 0.9 of a tile's time, and moves are the more frequent the
// higher lift is where rows differ in size: 4096 tokens over 8192 rows of 656
// bytes take 4215 us with lift 0, 4460 with 1, 4670 with this rule, and 5540 with
// lift = log2(n), which would keep the loss of rounding to nearest below 1 %.
//
// Group scales (528- and 656-byte rows): one pass of the score product for
// each 128-dim group, multiplied by the row's scale as it is read out, and one
// P operand for each group against that group's block of values.  With S the
// power of two above the row's largest scale, the reference M is one of s +
// log2 S, so that one exponential serves all four groups,
//   P_g = 2^(s + log2 S - M) (s_g / S) c_g,   l = sum 2^(s + log2 S - M) / S,
// and c_g, a power of two for each group, lifts groups that are smaller than
// their rows' largest throughout the segment.  (S and c_g are powers of two:
// nothing is rounded but P itself.)  RoPE dims are one more pass, BF16, with
// the row's power of two in the query.
//
// Warp roles: 16 softmax warps (warp w: TMEM lane quarter w % 4 = 32 keys of
// the tile, column quarter w / 4), one issuing thread for each product, and
// producers that translate keys to rows and bring them into a ring of 16 KB
// blocks (128 keys x 128 bytes).  A block is released as soon as the product
// that reads it last has finished.  Pages of a multiple of 32 rows come by TMA
// (one warp, boxes of 32 to 128 rows: a page never ends inside a box); other
// page sizes row by row with 16-byte cp.async (six warps).  us by TMA / row by
// row, pages of 16 (boxes of 16): 1024 tokens of 16 heads over 8192, raw 439 /
// 374, scaled 573 / 493, rope 650 / 615; 64 single tokens over up to 8192, raw
// 47.3 / 42.6; pages of 32 (prompts of up to 2047 tokens, raw): 213 / 235.
//
// What lies in shared memory for a key that nobody sees (the rest of a page, a
// box that was not loaded) has no effect: its weights are 0, and a row that
// holds a NaN byte is cleared before the second product reads it.
#include <atomic>
#include <cstddef>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <type_traits>

#include "chunk.cuh"
#include "chunk_plan.cuh"
#include "dsa_common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace dsa {
namespace {

using namespace tc;

constexpr int kTile = kChunkTile;
constexpr int kBlock = kTile * 128;          // bytes of a ring block
constexpr float kTop = 8.75f;                // p never exceeds 2^kTop (E4M3 ends at 448 = 2^8.8)
constexpr int kMaxLift = 8;                  // a whole power of two below it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSmxWarps = 16, kSmxThreads = 512;
constexpr int kQkWarp = 16, kPvWarp = 17, kProdWarp0 = 18;
constexpr int kProdWarps = 6, kProdThreads = 32 * kProdWarps;    // of the row-by-row form
constexpr int kQuads = kTile / 4;            // producer work unit: 4 rows (one warp instruction per 128-byte piece)
constexpr int kMeta = 4;                     // tiles whose rows and scales are kept
constexpr int kSegs = 6;                     // segments whose units are kept
constexpr int kMaxSBuf = 4;                  // score buffers
constexpr int kProdBar = 8;                  // named barriers: 1 + column quarter, producers
constexpr int kMaxBlocks = 12;
constexpr int kSmemLimit = 232448;

struct Misc {
  uint64_t full[kMaxBlocks], empty[kMaxBlocks];
  uint64_t rope_full, rope_empty;  // the tile's RoPE block (a buffer of its own: it is free long before the others)
  uint64_t meta_full[kMeta];       // rows (and scales) of a tile are in place
  uint64_t s_full[kMaxSBuf], s_free[kMaxSBuf];
  uint64_t p_full[2], p_free[2];   // a tile's P is written; its PV products are done
  uint64_t q_full;                 // a segment's query operand is built
  uint64_t final[2];               // drain of the two issuers
  ChunkUnit unit[kSegs];           // of each segment, published with its first tile's rows
  uint32_t tmem_base;
  int abort;
  int clean[kMeta];                // every key of the tile has a row
  __align__(16) int32_t rows[kMeta][kTile];   // pool row of each key (TMA: of each box's first), -1: masked
  __align__(16) float sig[2][32];  // per segment parity: log2-domain factor of each query column
  __align__(16) int vis[2][32];    // keys that it sees
  __align__(16) float nmax[2][32]; // minus its reference M
  __align__(16) float by[32], alpha[32];   // a move of the references, and its factor; at a segment's end 1 / l and LSE
  float red[4][4][8];             // [column quarter][lane quarter][column]
  float red_sc[4][4][4];           // [column quarter][lane quarter][group]
  ChunkRange range;                // the CTA's part of the tile list
};
constexpr int kMiscBytes = 5120;
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

template <int NC, int kLayout, bool kTma>
struct Cfg {
  static constexpr bool kScaled = kLayout != DSA_KV_RAW512;
  static constexpr bool kRope = kLayout == DSA_KV_ROPE656;
  static constexpr int R = kLayout == DSA_KV_RAW512 ? kRawRow : kLayout == DSA_KV_SCALED528 ? kScaledRow : kRopeRow;
  static constexpr int CPT = NC / 4;                 // query columns of a softmax thread
  // Registers: the launch gives every thread LAUNCH_REGS; the softmax warps
  // then take SMX_REGS and the others give back to OTHER_REGS.
  static constexpr int THREADS = kTma ? 640 : 32 * (kProdWarp0 + kProdWarps);
  static constexpr int LAUNCH_REGS = kTma ? 96 : 80;
  static constexpr int SMX_REGS = kTma ? 104 : 88;
  static constexpr int OTHER_REGS = (LAUNCH_REGS * THREADS - SMX_REGS * kSmxThreads) / (THREADS - kSmxThreads) / 8 * 8;
  static_assert(SMX_REGS * kSmxThreads + OTHER_REGS * (THREADS - kSmxThreads) <= LAUNCH_REGS * THREADS &&
                SMX_REGS % 8 == 0 && OTHER_REGS % 8 == 0, "register split");
  static constexpr int G = kScaled ? 4 : 1;          // P operands of a tile
  static constexpr int NPASS = G + (kRope ? 1 : 0);  // score passes of a tile (RoPE first)
  static constexpr int NQ = 2 * NC;                  // columns of the query and P operands: hi, lo
  // score buffers, each of the PG passes that are read out together
  static constexpr int PG = kScaled ? 2 : 1, S_COLS = PG * NQ;
  static constexpr int SBUF = 4 * NQ + 4 * S_COLS <= 512 ? 4 : 2;
  static constexpr int O_COL0 = SBUF * S_COLS;
  static constexpr int TMEM_USED = O_COL0 + 4 * NQ;
  static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
  static constexpr int Q_BYTES = 2 * NC * 512;
  static constexpr int QR_BYTES = kRope ? NC * 128 : 0;
  static constexpr int NPB = NC == 32 && kScaled ? 1 : 2;    // P operands (of all groups) in flight
  static constexpr int P_GROUP = 2 * NC * 128;
  static constexpr int P_BYTES = G * P_GROUP;
  static constexpr int SC_BYTES = kScaled ? kMeta * kTile * 16 : 0;
  static constexpr int ROPE_BYTES = kRope ? kBlock : 0;
  // The row-by-row producers: groups that take the blocks in turn, warps of a
  // group, quads of rows of a warp.  A block's barrier takes an arrival from
  // each thread of a group: three groups of two warps run raw and scaled rows
  // 8 and 6 % faster than one of six (1024 tokens of 16 heads over 8192: 374
  // against 405 us, 493 against 525); with the RoPE block they lose 8 %.
  static constexpr int GROUPS = kRope ? 1 : 3;
  static constexpr int GW = kProdWarps / GROUPS, QW = (kQuads + GW - 1) / GW;
  static_assert(kProdWarps % GROUPS == 0 && GW % 2 == 0, "rows of a thread share their place in the swizzle");
  static constexpr int FIXED = kMiscBytes + 1024 + Q_BYTES + QR_BYTES + SC_BYTES + ROPE_BYTES;
  static constexpr int NS_FIT = (kSmemLimit - FIXED - NPB * P_BYTES) / kBlock;
  static constexpr int NS = NS_FIT < kMaxBlocks ? NS_FIT : kMaxBlocks;
  static constexpr int ROPE_OFF = NS * kBlock;
  static constexpr int Q_OFF = ROPE_OFF + ROPE_BYTES;
  static constexpr int QR_OFF = Q_OFF + Q_BYTES;
  static constexpr int P_OFF = QR_OFF + QR_BYTES;
  static constexpr int SC_OFF = P_OFF + NPB * P_BYTES;
  static constexpr int MISC_OFF = SC_OFF + SC_BYTES;
  static constexpr int SMEM = MISC_OFF + kMiscBytes + 1024;
  static_assert(NS > 4, "a tile's blocks and one more");
  static_assert(NS * kBlock >= kPlanScratch, "the plan's scratch lies in the ring");
  // a tile's rows are replaced kMeta tiles later, when its blocks are gone from the ring
  static_assert((NS - 1) / 4 + 1 < kMeta, "rows of a tile in use");
  static_assert(SMEM <= kSmemLimit && TMEM_USED <= 512 && P_GROUP % 1024 == 0 && QR_BYTES % 1024 == 0, "budgets");
};

// Byte offset of element (n, k) in a K-major operand of N rows whose K extent
// is split into 128-byte blocks, with the 128-byte swizzle.
template <int N>
__device__ __forceinline__ uint32_t kmajor_off(int n, int k) {
  return (k >> 7) * (N * 128) + (n >> 3) * 1024 + (n & 7) * 128 + ((((k >> 4) & 7) ^ (n & 7)) << 4) + (k & 15);
}

// Byte offset of P column n, key k in the MN-major PV operand without swizzle:
// core matrices of 8 keys x 16 columns.
template <int NP>
__device__ __forceinline__ uint32_t p_off(int n, int k) {
  return (n >> 4) * 128 + (k >> 3) * (NP * 8) + (k & 7) * 16 + (n & 15);
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
  } else {
    static_assert(N == 8, "columns");
    tmem_ld8(taddr, v);
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    tmem_st4(taddr, v);
  } else {
    static_assert(N == 8, "columns");
    tmem_st8(taddr, v);
  }
}

// Two E4M3 terms of a pair of FP16 values, p ~ hi + lo / 16 (the residual is
// exact in FP16); shift is added to lo before it is rounded.
__device__ __forceinline__ void split2(uint32_t p, uint32_t shift, uint32_t& hi2, uint32_t& lo2) {
  uint32_t t, r;
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(p));
  hi2 = h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(t) : "h"(h));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(t));
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(r) : "r"(0x4C004C00u), "r"(shift));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(r));
  lo2 = h;
}

// The shift of the weights of one key: (k - 512) 2^-19, k = 1, 3, .., 1023, in
// both halves, within half of lo's smallest step, 2^-9.  The 128 keys of a tile
// get values 2^-16 apart, those of keys a power of two apart evenly spaced too,
// and of neighbours nearly so (79 / 128 is near the golden ratio); four tiles'
// values lie between each other's (634 is 2 modulo 8).
__device__ __forceinline__ uint32_t shift_base(int row) { return 8u * ((79u * row) & 127u) + 1u; }
__device__ __forceinline__ uint32_t shift_of(uint32_t base, int tile) {
  const uint32_t k = ((base + 634u * (uint32_t)tile) & 0x3FFu) | 0x6400u;     // 1024 + k
  uint32_t s = k | k << 16;
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(s) : "r"(0x66006600u));               // 1536
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(s) : "r"(0x00200020u));               // 2^-19
  return s;
}

// 2 N bytes (N = 4 or 8: both terms), held as pairs, to shared memory.
template <int N>
__device__ __forceinline__ void st_bytes(uint32_t addr, const uint32_t (&hi)[N / 2], const uint32_t (&lo)[N / 2]) {
  if constexpr (N == 8)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(hi[0] | hi[1] << 16), "r"(hi[2] | hi[3] << 16),
                 "r"(lo[0] | lo[1] << 16), "r"(lo[2] | lo[3] << 16) : "memory");
  else
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(hi[0] | hi[1] << 16), "r"(lo[0] | lo[1] << 16) : "memory");
}

// Two floats in one 64-bit register: half the instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// A CTA's part of the tile list.
struct Range {
  int64_t t0;
  int n_it;
};

// The producers' walk through a CTA's tiles.  A segment is the part of a unit
// inside the CTA's range.  What they need of the next unit is fetched while the
// current one is worked on: its request and lengths by every thread, one word
// of its entry by each of the first twelve (for the other roles).
struct Walk {
  int unit, tile, tiles, b, last;
  int next_tiles, next_b, next_last;
  int32_t word = 0, next_word = 0;
  static constexpr int kWords = sizeof(ChunkUnit) / 4;
  __device__ __forceinline__ void fetch_next(const ChunkWork& w, int ptid) {
    const ChunkUnit* u = w.units + unit + 1;     // (behind the last unit: read, never used)
    next_tiles = __ldcg(&u->tiles);
    next_b = __ldcg(&u->b);
    next_last = __ldcg(&u->last);
    if (ptid < kWords) next_word = __ldcg(reinterpret_cast<const int32_t*>(u) + ptid);
  }
  __device__ __forceinline__ Walk(const ChunkWork& w, const Misc& ms, int ptid) {
    const ChunkUnit& u = ms.unit[0];
    unit = ms.range.unit;
    tiles = u.tiles;
    b = u.b;
    last = u.last;
    tile = (int)(ms.range.t0 - u.tile0);
    fetch_next(w, ptid);
  }
  // true when the next tile starts a segment
  __device__ __forceinline__ bool advance(const ChunkWork& w, int ptid) {
    if (++tile < tiles) return false;
    tile = 0;
    tiles = next_tiles;
    b = next_b;
    last = next_last;
    word = next_word;
    ++unit;
    fetch_next(w, ptid);
    return true;
  }
};

// The other roles' position: tiles left in the segment, from the units that
// the producers published.
struct Segment {
  int seg = -1, left = 0;
  // at a tile's start; true when it is its segment's first
  __device__ __forceinline__ bool starts() const { return left == 0; }
  __device__ __forceinline__ int open(const Misc& ms, const int64_t t0, int it, int n_it) {
    ++seg;
    const ChunkUnit& u = ms.unit[seg % kSegs];
    const int tile = it == 0 ? (int)(t0 - u.tile0) : 0;
    left = min(u.tiles - tile, n_it - it);
    return tile;
  }
};

// The unit's query rows into L2, ahead of their use (one thread).
__device__ __forceinline__ void prefetch_queries(const ChunkArgs& a, const ChunkUnit& u) {
  const uint16_t* src = a.q + u.row0 * a.q_row;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"((uint32_t)(u.cols * a.q_row * 2)) : "memory");
}

struct ChunkMaps {
  CUtensorMap rows, scales;
};

// ------------------------------------------------------------------- roles

template <int NC, int kLayout, bool kTma>
__device__ void producer_role(const ChunkWork& w, uint8_t* sm, Misc& ms, const Range& rg) {
  using C = Cfg<NC, kLayout, kTma>;
  const ChunkArgs& a = w.a;
  const int ptid = threadIdx.x - kProdWarp0 * 32, pw = ptid >> 5, lane = ptid & 31;
  const int rq = lane >> 3, ch = lane & 7;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  // this thread's rows of a block: r0, r0 + 4 GW, ...; where its 16 bytes of the first one go
  const int group = pw / C::GW, gw = pw % C::GW, r0 = 4 * gw + rq;
  const uint32_t dst0 = (r0 >> 3) * 1024 + (r0 & 7) * 128 + ((ch ^ (r0 & 7)) << 4);
  int turn = 0;
  // thread -> key ptid of each tile: its page-table entry is fetched a tile ahead
  Walk cur(w, ms, ptid);
  int32_t entry = -1, off = 0;
  bool seen = false;
  auto look_up = [&]() {
    const int j = cur.tile * kTile + ptid;
    seen = ptid < kTile && j < cur.last;
    if (seen) {
      const int page = j / a.page_size;
      off = j - page * a.page_size;
      entry = __ldg(a.page_table + (int64_t)cur.b * a.max_pages + page);
    }
  };
  look_up();
  int slot = 0, phase = 0, seg = 0;
  bool ok = true;      // false once a wait gave up: keep going through every barrier
  bool opens = true;   // the tile starts a segment
  auto acquire = [&]() {
    ok = ok && mbar_wait(smem_u32(&ms.empty[slot]), phase ^ 1, abort, w.wait_ns);
    ok = __all_sync(0xffffffffu, ok);
  };
  for (int it = 0; it < rg.n_it; ++it) {
    const int m = it % kMeta;
    acquire();
    int32_t row_here = -1;
    if (ptid < kTile) {
      int32_t row = -1;
      if (seen) {
        const int64_t r = (int64_t)entry * a.page_size + off;
        if (entry < 0 || r >= a.pool_rows) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
        else row = (int32_t)r;
      }
      ms.rows[m][ptid] = row_here = row;
      if (C::kScaled)
        cp_async_16_zfill(smem_u32(sm + C::SC_OFF + (m * kTile + ptid) * 16),
                          a.pool + (int64_t)(row >= 0 ? row : 0) * C::R + kD, row >= 0 ? 16u : 0u);
    }
    // Once a wait has given up no unit is published: the softmax warps then run on,
    // so that a free slot no longer tells that the units before are done with.
    if (opens && seg > 0) ok = __all_sync(0xffffffffu, ok && *abort == 0);
    if (C::kScaled && ok) cp_async_arrive_noinc(smem_u32(&ms.meta_full[m]));
    if (opens) {       // (the first unit is the plan's)
      if (ok && seg > 0 && ptid < Walk::kWords) reinterpret_cast<int32_t*>(&ms.unit[seg % kSegs])[ptid] = cur.word;
      ++seg;
    }
    const bool opened = opens;
    opens = cur.advance(w, ptid);
    if (it + 1 < rg.n_it) look_up();
    const bool whole = named_bar_red_or(kProdBar, kProdThreads, ptid < kTile && row_here < 0) == 0;
    if (ptid == 0 && ok) {
      ms.clean[m] = whole;
      mbar_arrive(smem_u32(&ms.meta_full[m]));
      if (opened && seg > 1) prefetch_queries(a, ms.unit[(seg - 1) % kSegs]);
    }
    int32_t rows[C::QW];
    auto load_rows = [&]() {
#pragma unroll
      for (int i = 0; i < C::QW; ++i) rows[i] = gw + i * C::GW < kQuads ? ms.rows[m][r0 + 4 * C::GW * i] : -1;
    };
    if (C::GROUPS == 1) load_rows();
    // 128 bytes of every row, from byte `col` of it
    auto copy = [&](uint32_t base, int col, uint32_t bar) {
      if (C::GROUPS > 1) load_rows();
#pragma unroll
      for (int i = 0; i < C::QW; ++i) {
        if (gw + i * C::GW >= kQuads) break;
        const int32_t pr = rows[i];
        const uint8_t* src = a.pool + (int64_t)(pr >= 0 ? pr : 0) * C::R + ch * 16 + col;
        cp_async_16_zfill(base + dst0 + i * C::GW * 512, src, pr >= 0 ? 16u : 0u);
      }
      cp_async_arrive_noinc(bar);
    };
    if (C::kRope) {
      ok = ok && mbar_wait(smem_u32(&ms.rope_empty), (it & 1) ^ 1, abort, w.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) copy(smem_u32(sm + C::ROPE_OFF), kScaledRow, smem_u32(&ms.rope_full));
    }
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      if (turn == group) {
        if (k > 0) acquire();
        if (ok) copy(kv0 + slot * kBlock, k * 128, smem_u32(&ms.full[slot]));
      }
      turn = turn + 1 == C::GROUPS ? 0 : turn + 1;
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  cp_async_wait_all();
}

__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One box of the map at (x, y): x a multiple of 16 bytes.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// One warp; lane i < 128 / box translates and loads the tile's i-th box of every
// block.  The copies themselves set the pace (a box of 64 rows takes about 130
// cycles to issue, 64 bytes a clock), so each block is requested as soon as the
// product that read its slot last has finished.
template <int NC, int kLayout, bool kTma>
__device__ void tma_role(const ChunkWork& w, const ChunkMaps& maps, uint8_t* sm, Misc& ms, const Range& rg) {
  using C = Cfg<NC, kLayout, kTma>;
  const ChunkArgs& a = w.a;
  const int lane = threadIdx.x & 31, box = 1 << w.box_shift;
  const bool mine = lane < (kTile >> w.box_shift);
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm) + ((uint32_t)lane << (w.box_shift + 7));
  Walk cur(w, ms, lane);
  int32_t entry = -1, off = 0, want = 0;     // the next tile's: page-table entry, row in the page, keys seen of the box
  auto look_up = [&]() {
    const int j = cur.tile * kTile + (lane << w.box_shift);
    want = mine ? min(box, cur.last - j) : 0;
    if (want > 0) {
      const int page = j / a.page_size;
      off = j - page * a.page_size;
      entry = __ldg(a.page_table + (int64_t)cur.b * a.max_pages + page);
    }
  };
  look_up();
  int slot = 0, phase = 0, seg = 0, issued = 0, metas = 0, ropes = 0;   // (blocks, tiles' rows and RoPE blocks requested)
  bool ok = true, opens = true;
  for (int it = 0; it < rg.n_it && ok; ++it) {
    const int m = it % kMeta;
    int32_t row = -1;
    if (want > 0) {
      const int64_t r = (int64_t)entry * a.page_size + off;
      const bool out = entry < 0 || r >= a.pool_rows;
      if (!out) row = (int32_t)r;
      if (out || r + want > a.pool_rows) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
    }
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0)) << w.box_shift;   // rows to come
    const bool whole = __all_sync(0xffffffffu, !mine || (want == box && row >= 0 && (int64_t)row + box <= a.pool_rows));
    if (C::kRope) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ms.rope_empty), (it & 1) ^ 1, abort, w.wait_ns));
      if (!ok) break;
      if (lane == 0) mbar_arrive_tx(smem_u32(&ms.rope_full), n * 128);
      __syncwarp();
      if (row >= 0) tma_load(kv0 + C::ROPE_OFF, &maps.rows, kScaledRow, row, smem_u32(&ms.rope_full));
      ++ropes;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ms.empty[slot]), phase ^ 1, abort, w.wait_ns));
      if (!ok) break;
      if (lane == 0) mbar_arrive_tx(smem_u32(&ms.full[slot]), n * 128);
      __syncwarp();
      if (row >= 0) tma_load(kv0 + slot * kBlock, &maps.rows, k * 128, row, smem_u32(&ms.full[slot]));
      issued = min(issued + 1, C::NS);
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
      if (k == 0) {        // (the slot is free, so the tile kMeta before is out of the way)
        // no unit is published once a wait has given up (as in producer_role)
        if (opens && seg > 0) ok = __all_sync(0xffffffffu, *abort == 0);
        if (!ok) break;
        ++metas;
        if (mine) ms.rows[m][lane] = row;
        if (lane == 0) ms.clean[m] = whole;
        if (opens) {
          if (seg > 0 && lane < Walk::kWords) reinterpret_cast<int32_t*>(&ms.unit[seg % kSegs])[lane] = cur.word;
          __syncwarp();
          if (lane == 0 && seg > 0) prefetch_queries(a, ms.unit[seg % kSegs]);
          ++seg;
        }
        __syncwarp();
        if (lane == 0) {
          if (C::kScaled) mbar_arrive_tx(smem_u32(&ms.meta_full[m]), n * 16);
          else mbar_arrive(smem_u32(&ms.meta_full[m]));
        }
        if (C::kScaled) {
          __syncwarp();
          if (row >= 0)
            tma_load(smem_u32(sm + C::SC_OFF) + m * kTile * 16 + ((uint32_t)lane << (w.box_shift + 4)), &maps.scales, kD, row,
                     smem_u32(&ms.meta_full[m]));
        }
        opens = cur.advance(w, lane);
        if (it + 1 < rg.n_it) look_up();
      }
    }
  }
  // nothing is left in flight when the CTA ends, not even after a wait gave up
  volatile int no_abort = 0;
  for (int i = 0; i < issued; ++i) {
    if (slot == 0) phase ^= 1;
    slot = slot == 0 ? C::NS - 1 : slot - 1;
    mbar_wait(smem_u32(&ms.full[slot]), phase, &no_abort, 2000000000ull);
  }
  if (C::kRope && ropes > 0) mbar_wait(smem_u32(&ms.rope_full), (ropes - 1) & 1, &no_abort, 2000000000ull);
  if (C::kScaled)
    for (int i = max(0, metas - kMeta); i < metas; ++i)
      mbar_wait(smem_u32(&ms.meta_full[i % kMeta]), (i / kMeta) & 1, &no_abort, 2000000000ull);
}

// Waits (bounded) for every tcgen05 operation this thread issued, so that the
// tensor memory can be released.
__device__ __forceinline__ void drain_mma(uint32_t bar) {
  mma_commit(bar);
  volatile int no_abort = 0;
  mbar_wait(bar, 0, &no_abort, 2000000000ull);
}

template <int NC, int kLayout, bool kTma>
__device__ void qk_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout, kTma>;
  if ((threadIdx.x & 31) != 0) return;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  constexpr uint32_t kId = idesc_e4m3(C::NQ, false), kIdRope = idesc_bf16(NC);
  const uint64_t q_desc = sdesc_sw128(smem_u32(sm + C::Q_OFF), 16, 1024);
  Segment sg;
  int slot = 0, phase = 0, sb = 0, s_phase = 1;      // a fresh score buffer is free
  bool ok = true;
  for (int it = 0; it < rg.n_it && ok; ++it, --sg.left) {
    if (sg.starts()) {
      ok = mbar_wait(smem_u32(&ms.q_full), (sg.seg + 1) & 1, abort, w.wait_ns);
      if (!ok) break;
      sg.open(ms, rg.t0, it, rg.n_it);
    }
    // pass p: its score buffer, free when its first pass begins, handed over after its last
    auto score_buffer = [&](int p) { return p % C::PG != 0 || mbar_wait(smem_u32(&ms.s_free[sb]), s_phase, abort, w.wait_ns); };
    auto scored = [&](int p) {
      if (p % C::PG != C::PG - 1 && p != C::NPASS - 1) return;
      mma_commit(smem_u32(&ms.s_full[sb]));
      if (++sb == C::SBUF) {
        sb = 0;
        s_phase ^= 1;
      }
    };
    if (C::kRope) {
      ok = score_buffer(0) && mbar_wait(smem_u32(&ms.rope_full), it & 1, abort, w.wait_ns);
      if (!ok) break;
      if (!kTma) fence_proxy_async_smem();   // rows landed through cp.async (generic proxy)
      tc_fence_after();
      const uint64_t ad = sdesc_sw128(kv0 + C::ROPE_OFF, 16, 1024), bd = sdesc_sw128(smem_u32(sm + C::QR_OFF), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16(tmem + sb * C::S_COLS, desc_add(ad, kk * 32), desc_add(bd, kk * 32), kIdRope, kk > 0 ? 1u : 0u);
      mma_commit(smem_u32(&ms.rope_empty));
      scored(0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool opens = C::kScaled || k == 0;       // first block of a score pass
      const int p = C::kScaled ? k + (C::kRope ? 1 : 0) : 0;
      if (opens) ok = score_buffer(p);
      ok = ok && mbar_wait(smem_u32(&ms.full[slot]), phase, abort, w.wait_ns);
      if (!ok) break;
      if (!kTma) fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t ad = sdesc_sw128(kv0 + slot * kBlock, 16, 1024);
      const uint64_t bd = desc_add(q_desc, k * (C::NQ * 128));
      const uint32_t d = tmem + sb * C::S_COLS + p % C::PG * C::NQ;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        mma_e4m3(d, desc_add(ad, kk * 32), desc_add(bd, kk * 32), kId, (!opens || kk > 0) ? 1u : 0u);
      }
      if (C::kScaled || k == 3) scored(p);
      if (++slot == C::NS) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  drain_mma(smem_u32(&ms.final[0]));
}

template <int NC, int kLayout, bool kTma>
__device__ void pv_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout, kTma>;
  if ((threadIdx.x & 31) != 0) return;
  volatile int* abort = &ms.abort;
  const uint32_t kv0 = smem_u32(sm);
  constexpr uint32_t kId = idesc_e4m3(C::NQ, true, true);
  const uint64_t p_desc = sdesc_mn_none(smem_u32(sm + C::P_OFF), C::NQ * 8, 128);
  Segment sg;
  int slot = 0;
  bool ok = true;
  auto step = [&]() { slot = slot + 1 == C::NS ? 0 : slot + 1; };
  for (int it = 0; it < rg.n_it && ok; ++it, --sg.left) {
    const bool first = sg.starts();
    const int pb = it % C::NPB;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g == 0) {
        ok = mbar_wait(smem_u32(&ms.p_full[pb]), (it / C::NPB) & 1, abort, w.wait_ns);
        if (!ok) break;
        tc_fence_after();
        if (first) sg.open(ms, rg.t0, it, rg.n_it);
      }
      const uint64_t ad = sdesc_sw128(kv0 + slot * kBlock, 1024, 1024);
      const uint64_t bd = desc_add(p_desc, pb * C::P_BYTES + (C::kScaled ? g * C::P_GROUP : 0));
      const uint32_t d = tmem + C::O_COL0 + g * C::NQ;
#pragma unroll
      for (int js = 0; js < 4; ++js)
        mma_e4m3(d, desc_add(ad, js * 4096), desc_add(bd, js * 4 * (C::NQ * 8)), kId, js > 0 ? 1u : (first ? 0u : 1u));
      mma_commit(smem_u32(&ms.empty[slot]));
      step();
    }
    if (ok) mma_commit(smem_u32(&ms.p_free[pb]));
  }
  drain_mma(smem_u32(&ms.final[1]));
}

// The query operand of one segment, and its columns' factors, visible keys and
// references.  512 threads: column tid / TPH, dims [DPT (tid % TPH), + DPT).
// there: the unit was published (false: of a call that gave up, whose queries
// are not read).
template <int NC, int kLayout, bool kTma>
__device__ __forceinline__ void build_query(const ChunkWork& w, uint8_t* sm, Misc& ms, const ChunkUnit& u, bool there, int par) {
  using C = Cfg<NC, kLayout, kTma>;
  constexpr int TPH = kSmxThreads / NC, DPT = kD / TPH, NV = DPT / 8;
  const ChunkArgs& a = w.a;
  const int col = threadIdx.x / TPH, part = threadIdx.x % TPH;
  const uint16_t* src = a.q + (u.row0 + col) * a.q_row;
  const bool live_col = there && col < u.cols;
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i] = live_col ? __ldg(reinterpret_cast<const uint4*>(src + part * DPT) + i) : make_uint4(0, 0, 0, 0);
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f0 = fabsf(bf16_bits_to_f32(x[j] & 0xFFFFu)), f1 = fabsf(bf16_bits_to_f32(x[j] >> 16));
      amax = fmaxf(amax, fmaxf(f0, f1));
      nan |= !(f0 < INFINITY && f1 < INFINITY);      // (the largest two have an infinite sum)
    }
  }
  constexpr int RD = kRopeDims / TPH;                // RoPE dims: part p holds [64 p / TPH, + 64 / TPH)
  uint32_t pe[RD / 2];
  float pmax = 0.f;
  if constexpr (C::kRope) {
#pragma unroll
    for (int i = 0; i < RD / 2; ++i) {
      pe[i] = live_col ? __ldg(reinterpret_cast<const uint32_t*>(src + kD + part * RD) + i) : 0u;
      nan |= (pe[i] & 0x7F80u) == 0x7F80u || (pe[i] & 0x7F800000u) == 0x7F800000u;
      pmax = fmaxf(pmax, fmaxf(fabsf(bf16_bits_to_f32(pe[i] & 0xFFFFu)), fabsf(bf16_bits_to_f32(pe[i] >> 16))));
    }
  }
  if (nan) amax = INFINITY;
#pragma unroll
  for (int off = TPH / 2; off >= 1; off /= 2) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (C::kRope) pmax = fmaxf(pmax, __shfl_xor_sync(0xffffffffu, pmax, off));
  }
  int sh = 0;
  const float base = a.sm_scale * kLog2e;
  float sig = base;
  const bool live = amax > 0.f && amax < INFINITY;
  if (live) {
    int e;
    const float f = frexpf(amax, &e);                // amax = f 2^e, f in [0.5, 1)
    // largest sh with amax 2^sh <= 448, sig a normal number, and the RoPE dims
    // times 2^sh below 2^112 (times the rows' 64, in range)
    sh = min(f <= 0.875f ? 9 - e : 8 - e, 112);
    if (C::kRope && pmax > 0.f) sh = min(sh, 112 - (ilogbf(pmax) + 1));
    sig = scale_pow2(base, -sh);
  } else if (amax > 0.f) {
    sig = __int_as_float(0x7FC00000);                // a row with a NaN or an infinity scores NaN
  }
  uint8_t* qb = sm + C::Q_OFF;
  const float up = live ? __int_as_float((127 + sh) << 23) : 0.f;   // 2^sh, sh in [-120, 112]
#pragma unroll
  for (int c = 0; c < NV / 2; ++c) {
    uint32_t hi[4], lo[4];
    const uint32_t x[8] = {v[2 * c].x, v[2 * c].y, v[2 * c].z, v[2 * c].w,
                           v[2 * c + 1].x, v[2 * c + 1].y, v[2 * c + 1].z, v[2 * c + 1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h2[2], l2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {        // exact in FP16 down to steps of 2^-24
        const uint32_t q2 = live ? x[2 * i + j] : 0u;
        uint32_t y;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(bf16_bits_to_f32(q2 >> 16) * up), "f"(bf16_bits_to_f32(q2 & 0xFFFFu) * up));
        split2(y, 0u, h2[j], l2[j]);
      }
      hi[i] = h2[0] | h2[1] << 16;
      lo[i] = l2[0] | l2[1] << 16;
    }
    const int k0 = part * DPT + 16 * c;
    *reinterpret_cast<uint4*>(qb + kmajor_off<C::NQ>(col, k0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(qb + kmajor_off<C::NQ>(NC + col, k0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  if constexpr (C::kRope) {
    uint32_t x[RD / 2];
#pragma unroll
    for (int i = 0; i < RD / 2; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(scale_pow2(bf16_bits_to_f32(pe[i] & 0xFFFFu), sh),
                                                     scale_pow2(bf16_bits_to_f32(pe[i] >> 16), sh));
      x[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    const int byte = part * RD * 2;                  // of the column's 128
    uint8_t* dst = sm + C::QR_OFF + (col >> 3) * 1024 + (col & 7) * 128 + (((byte >> 4) ^ (col & 7)) << 4) + (byte & 15);
#pragma unroll
    for (int i = 0; i < RD / 2; ++i) reinterpret_cast<uint32_t*>(dst)[i] = x[i];
  }
  if (part == 0) {
    ms.sig[par][col] = sig;
    ms.vis[par][col] = live_col ? chunk_visible(a, u, col) : 0;
    ms.nmax[par][col] = 0.f;
  }
  fence_proxy_async_smem();
  warp_arrive(smem_u32(&ms.q_full));
}

template <int NC, int kLayout, bool kTma>
__device__ void softmax_role(const ChunkWork& w, uint8_t* sm, Misc& ms, uint32_t tmem, const Range& rg) {
  using C = Cfg<NC, kLayout, kTma>;
  constexpr int CPT = C::CPT, CP2 = CPT / 2;
  const ChunkArgs& a = w.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, cq = warp >> 2;
  const int row = 32 * quarter + lane;                   // key of the tile = TMEM lane (dim of a block, for O)
  const int c0 = cq * CPT;                               // first column
  const int bar = 1 + cq;                                // the four warps of a column quarter
  const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16) + c0;
  volatile int* abort = &ms.abort;
  uint64_t l_part[CP2];                                  // this row's share of the denominators
  float m_lane = 0.f;                                    // reference M of column c0 + lane % CPT (0: none yet)
  bool has = false;                                      // it is that of a key, or the column sees none at all
  bool pending = true;                                   // a column of the quarter still has none
  float cg[4] = {1.f, 1.f, 1.f, 1.f};                    // c_g
  int sb = 0, s_phase = 0;
  int slot0 = 0;                                         // ring slot of the tile's first block
  int tile = 0, last = 0;                                // tile of the unit, keys that anyone sees
  int full = 0;                                          // tiles that every column sees whole
  const uint32_t base = shift_base(row);
  // rows of the pool behind which this thread's key of a box would lie outside
  const int in_box = kTma ? row & ((1 << w.box_shift) - 1) : 0;
  const uint32_t row_limit = (uint32_t)max((int64_t)0, a.pool_rows - in_box);
  // PV of tile i; every tile's is waited for (NPB tiles on at the latest), so the parity tells them apart
  auto pv_wait = [&](int i) { mbar_wait(smem_u32(&ms.p_free[i % C::NPB]), (i / C::NPB) & 1, abort, w.wait_ns); };
  Segment sg;
  build_query<NC, kLayout, kTma>(w, sm, ms, ms.unit[0], true, 0);
  for (int it = 0; it < rg.n_it; ++it) {
    const bool first = sg.starts();
    const int m = it % kMeta;
    mbar_wait(smem_u32(&ms.meta_full[m]), (it / kMeta) & 1, abort, w.wait_ns);
    if (first) {
      mbar_wait(smem_u32(&ms.q_full), (sg.seg + 1) & 1, abort, w.wait_ns);
      tile = sg.open(ms, rg.t0, it, rg.n_it);
      last = ms.unit[sg.seg % kSegs].last;
      full = ms.vis[sg.seg & 1][0] / kTile;
      m_lane = 0.f;
      has = ms.vis[sg.seg & 1][c0 + lane % CPT] == 0;
      pending = true;
#pragma unroll
      for (int k = 0; k < CP2; ++k) l_part[k] = 0;
    }
    --sg.left;
    const int par = sg.seg & 1;
    const bool clean = ms.clean[m] != 0;
    // this key has a row and someone sees it
    auto row_valid = [&]() {
      return clean || ((uint32_t)ms.rows[m][row >> w.box_shift] < row_limit && tile * kTile + row < last);
    };
    float sc[4] = {1.f, 1.f, 1.f, 1.f};
    float lsc = 0.f, inv = 1.f;                          // log2 S and 1 / S, S = 2^(e - 126)
    bool odd_scale = false;
    if (C::kScaled) {
      const float4 v = *reinterpret_cast<const float4*>(sm + C::SC_OFF + (m * kTile + row) * 16);
      sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
      const uint32_t big = max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                               max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
      odd_scale = big >= 0x7F800000u;
      const int e = min(max((int)(big >> 23), 66), 252); // S within 2^-60 .. 2^126
      lsc = (float)(e - 126);
      inv = __int_as_float((253 - e) << 23);
    }
    // scores: the passes' sums, then times the column's factor
    uint64_t s2[CP2];
    bool poisoned = false;                               // a NaN byte in the row: every column's sum is NaN
#pragma unroll
    for (int p = 0; p < C::NPASS; ++p) {
      if (p % C::PG == 0) {
        mbar_wait(smem_u32(&ms.s_full[sb]), s_phase, abort, w.wait_ns);
        tc_fence_after();
      }
      const bool rope = C::kRope && p == 0;
      const bool two = !rope;
      const int g = C::kRope ? p - 1 : p;
      const uint32_t at = lane_base + sb * C::S_COLS + p % C::PG * C::NQ;
      const uint64_t f2 = pack2(sc[rope ? 0 : g], sc[rope ? 0 : g]);
      uint32_t v[CPT], lo[CPT];
      tmem_ld<CPT>(at, v);
      if (two) tmem_ld<CPT>(at + NC, lo);
      tmem_wait_ld();
      if (p % C::PG == C::PG - 1 || p == C::NPASS - 1) {
        tc_fence_before();
        warp_arrive(smem_u32(&ms.s_free[sb]));
      }
      if (!rope) poisoned |= __uint_as_float(v[0]) != __uint_as_float(v[0]);
#pragma unroll
      for (int k = 0; k < CPT; k += 2) {
        uint64_t t = pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        if (two) t = fma2(pack2(__uint_as_float(lo[k]), __uint_as_float(lo[k + 1])), pack2(0.0625f, 0.0625f), t);
        uint64_t& d = s2[k / 2];
        if (!C::kScaled || rope) d = t;
        else if (p == 0) d = mul2(t, f2);
        else d = fma2(t, f2, d);
      }
      if (p % C::PG == C::PG - 1 || p == C::NPASS - 1) {
        if (++sb == C::SBUF) {
          sb = 0;
          s_phase ^= 1;
        }
      }
    }
    // x = s + log2 S - M
    float x[CPT];
    {
      float sig[CPT], nm[CPT];
      ld_row<CPT>(&ms.nmax[par][c0], nm);
      ld_row<CPT>(&ms.sig[par][c0], sig);
#pragma unroll
      for (int k = 0; k < CPT; k += 2) {
        uint64_t o = pack2(nm[k], nm[k + 1]);
        if (C::kScaled) o = add2(o, pack2(lsc, lsc));
        unpack2(fma2(s2[k / 2], pack2(sig[k], sig[k + 1]), o), x[k], x[k + 1]);
      }
    }
    // a row with an infinite or NaN scale holds infinities of both signs and NaN: it scores NaN
    if (odd_scale) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) x[k] = __int_as_float(0x7FC00000);
    }
    // keys that a column does not see
    if (!clean || tile >= full) {
      const bool valid = row_valid();
      const int j = tile * kTile + row;
      int vis[CPT];
      ld_row<CPT>(&ms.vis[par][c0], vis);
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (!valid || j >= vis[k]) x[k] = -INFINITY;
    }
    // Does a column's reference have to move, or a c_g?  (A reference moves
    // for its own column only, so that a row's rounding does not hang on its
    // neighbours'.)  One barrier of
    // the column quarter's warps ORs the threads' answers; only then are the
    // tile's maxima formed.
    float top = x[0];
#pragma unroll
    for (int k = 1; k < CPT; ++k) top = fmaxf(top, x[k]);
    bool grow = pending || top > kTop;
    // P's factors s_g / S c_g, at most 1 (what lies there for a row that nobody
    // sees, or for one that scores NaN, is cut to finite values: p is 0, or NaN)
    float f[C::G];
    auto factors = [&]() {
#pragma unroll
      for (int g = 0; g < C::G; ++g) f[g] = sc[g] * inv * cg[g];
    };
    if (C::kScaled) {
      factors();
      grow |= fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1 % C::G])), fmaxf(fabsf(f[2 % C::G]), fabsf(f[3 % C::G]))) > 1.f;
    }
    if (named_bar_red_or(bar, 128, grow)) {
      float tmp[CPT];
#pragma unroll
      for (int k = 0; k < CPT; ++k) tmp[k] = x[k];
      const float wmax = transpose_reduce<CPT, true>(tmp, lane);
      if (lane < CPT) ms.red[cq][quarter][lane] = wmax;
      if (C::kScaled) {
        const bool counts = !odd_scale && row_valid();
        float t4[4];                                     // s_g / S
#pragma unroll
        for (int g = 0; g < 4; ++g) t4[g] = counts ? fabsf(sc[g]) * inv : 0.f;
        const float wsc = transpose_reduce<4, true>(t4, lane);
        if (lane < 4) ms.red_sc[cq][quarter][lane] = wsc;
      }
      named_bar_sync(bar, 128);
      const int cl = lane % CPT;
      const float tmax = fmaxf(fmaxf(ms.red[cq][0][cl], ms.red[cq][1][cl]), fmaxf(ms.red[cq][2][cl], ms.red[cq][3][cl]));
      const float lift = (float)min(max(1, (31 - __clz(sg.left + 1)) / 2 - (C::kScaled ? 0 : 2)), kMaxLift);
      const bool need = has ? tmax > kTop : tmax > -INFINITY;
      const float by = need ? tmax - lift : 0.f; // M moves by this much
      const float alpha_lane = need ? (has ? ex2_approx(-by) : 0.f) : 1.f;   // (nothing summed before the first key)
      has |= need;
      m_lane += by;
      bool moved = __any_sync(0xffffffffu, need);
      float beta[4] = {1.f, 1.f, 1.f, 1.f};
      if (C::kScaled) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float mx = fmaxf(fmaxf(ms.red_sc[cq][0][g], ms.red_sc[cq][1][g]), fmaxf(ms.red_sc[cq][2][g], ms.red_sc[cq][3][g]));
          if (pending || mx * cg[g] > 1.f) {             // c_g: the reciprocal of the power of two above mx
            const int e = max((int)((__float_as_uint(mx) + 0x7FFFFFu) >> 23), 127 - 24);
            const float c = __int_as_float((254 - e) << 23);
            beta[g] = c / cg[g];
            cg[g] = c;
            moved = true;
          }
        }
      }
      pending = __any_sync(0xffffffffu, !has);
      if (quarter == 0 && lane < CPT) {
        ms.nmax[par][c0 + lane] = -m_lane;
        ms.by[c0 + lane] = by;
        ms.alpha[c0 + lane] = alpha_lane;
      }
      named_bar_sync(bar, 128);
      if (moved) {
        if (C::kScaled) factors();
        float al[CPT];
        ld_row<CPT>(&ms.by[c0], al);
#pragma unroll
        for (int k = 0; k < CPT; ++k) x[k] -= al[k];
        ld_row<CPT>(&ms.alpha[c0], al);
#pragma unroll
        for (int k = 0; k < CP2; ++k) l_part[k] = mul2(l_part[k], pack2(al[2 * k], al[2 * k + 1]));
        if (!first) {      // O holds this segment's earlier tiles
          pv_wait(it - 1);
          tc_fence_after();
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            const float bg = g == 0 ? beta[0] : g == 1 ? beta[1] : g == 2 ? beta[2] : beta[3];
            const uint32_t at = lane_base + c0 + C::O_COL0 + g * C::NQ;
            uint32_t v[CPT], lo[CPT];                    // hi, lo
            tmem_ld<CPT>(at, v);
            tmem_ld<CPT>(at + CPT, lo);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
              v[k] = __float_as_uint(__uint_as_float(v[k]) * (al[k] * bg));
              lo[k] = __float_as_uint(__uint_as_float(lo[k]) * (al[k] * bg));
            }
            tmem_st<CPT>(at, v);
            tmem_st<CPT>(at + CPT, lo);
          }
          tmem_wait_st();
        }
      }
    }
    const uint64_t inv2 = pack2(inv, inv);
    uint32_t p2[CP2];                                    // P operands come from the FP16 values of the weights (11 significant bits)
#pragma unroll
    for (int k = 0; k < CP2; ++k) {
      const float p0 = ex2_approx(x[2 * k]), p1 = ex2_approx(x[2 * k + 1]);
      l_part[k] = C::kScaled ? fma2(pack2(p0, p1), inv2, l_part[k]) : add2(l_part[k], pack2(p0, p1));
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p2[k]) : "f"(p1), "f"(p0));
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
    const uint32_t shift = shift_of(base, tile);
    const int pb = it % C::NPB;
    const uint32_t at = smem_u32(sm + C::P_OFF) + pb * C::P_BYTES;
#pragma unroll
    for (int g = 0; g < C::G; ++g) {
      uint32_t hi2[CP2], lo2[CP2];
      uint32_t f2 = 0;
      if (C::kScaled) {
        const float fg = fminf(fmaxf(f[g], -1.f), 1.f);
        asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(f2) : "f"(fg));
      }
#pragma unroll
      for (int k = 0; k < CP2; ++k) {
        uint32_t v = p2[k];
        if (C::kScaled) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(f2));
        split2(v, shift, hi2[k], lo2[k]);
      }
      if (g == 0 && it >= C::NPB)
        pv_wait(it - C::NPB);
      st_bytes<CPT>(at + g * C::P_GROUP + p_off<C::NQ>(2 * c0, row), hi2, lo2);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    warp_arrive(smem_u32(&ms.p_full[pb]));
    slot0 += 4;
    if (slot0 >= C::NS) slot0 -= C::NS;
    ++tile;
    if (sg.left > 0) continue;
    const ChunkUnit& u = ms.unit[sg.seg % kSegs];
    // Every score pass of this tile is done, so the query operand may be replaced.
    // The next unit is there if no wait gave up so far: one that did leaves the
    // flag set (its own result says less, as a barrier further on may be a whole
    // number of phases behind).  Else the column quarter, whose threads share
    // named barriers, leaves together.  (Each wait's result kept, or the quarter
    // leaving from within the tile, take 2 to 6 % of the kernel's time.)
    bool there = true;
    if (it + 1 < rg.n_it) {
      mbar_wait(smem_u32(&ms.meta_full[(it + 1) % kMeta]), ((it + 1) / kMeta) & 1, abort, w.wait_ns);
      there = *abort == 0;
      build_query<NC, kLayout, kTma>(w, sm, ms, ms.unit[(sg.seg + 1) % kSegs], there, par ^ 1);
    }
    // the segment's end: denominators, O, LSE
    float lsum[CPT];
#pragma unroll
    for (int k = 0; k < CP2; ++k) unpack2(l_part[k], lsum[2 * k], lsum[2 * k + 1]);
    const float wsum = transpose_reduce<CPT, false>(lsum, lane);
    if (lane < CPT) ms.red[cq][quarter][lane] = wsum;
    if (named_bar_red_or(bar, 128, !there)) break;
    if (quarter == 0 && lane < CPT) {
      const float l = (ms.red[cq][0][lane] + ms.red[cq][1][lane]) + (ms.red[cq][2][lane] + ms.red[cq][3][lane]);
      ms.by[c0 + lane] = l == 0.f ? 0.f : 1.f / l;
      ms.alpha[c0 + lane] = l == 0.f ? -INFINITY : (m_lane + log2f(l)) * kLn2;
    }
    named_bar_sync(bar, 128);
    pv_wait(it);
    tc_fence_after();
    const bool whole = u.tile0 >= rg.t0 && u.tile0 + u.tiles <= rg.t0 + rg.n_it;
    const int64_t part = ((int64_t)blockIdx.x * 2 + (rg.t0 >= u.tile0 ? 0 : 1)) * NC;
    const int cols = u.cols - c0;                        // of this thread's columns
    const int64_t row0 = u.row0;
    float li[CPT];
    ld_row<CPT>(&ms.by[c0], li);
    // block db's outputs of this thread's columns, normalised
    auto read_block = [&](int db, float (&y)[CPT]) {
      uint32_t v[CPT], lo[CPT];
      tmem_ld<CPT>(lane_base + c0 + C::O_COL0 + db * C::NQ, v);
      tmem_ld<CPT>(lane_base + c0 + C::O_COL0 + db * C::NQ + CPT, lo);
      tmem_wait_ld();
      const float unlift = C::kScaled ? __int_as_float((254 << 23) - __float_as_int(cg[db])) : 1.f;   // 1 / c_g
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        y[k] = li[k] == 0.f ? 0.f : fmaf(__uint_as_float(lo[k]), 0.0625f, __uint_as_float(v[k])) * (li[k] * unlift);
    };
    if (whole) {
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.o) + (row0 + c0) * kD + row;
#pragma unroll
      for (int db = 0; db < 4; ++db) {
        float y[CPT];
        read_block(db, y);
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          if (k < cols) o[k * kD + db * 128] = __float2bfloat16_rn(y[k]);
      }
    } else {
      float* o = w.part_o + (part + c0) * kD + row;
#pragma unroll
      for (int db = 0; db < 4; ++db) {
        float y[CPT];
        read_block(db, y);
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          if (k < cols) o[k * kD + db * 128] = y[k];
      }
    }
    if (quarter == 0 && lane < CPT && lane < cols) {
      if (whole) a.lse[row0 + c0 + lane] = ms.alpha[c0 + lane];
      else w.part_lse[part + c0 + lane] = ms.alpha[c0 + lane];
    }
  }
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int NC, int kLayout, bool kTma>
__global__ void __launch_bounds__(Cfg<NC, kLayout, kTma>::THREADS, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkWork w, const __grid_constant__ ChunkMaps maps) {
  using C = Cfg<NC, kLayout, kTma>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc& ms = *reinterpret_cast<Misc*>(sm + C::MISC_OFF);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(smem_u32(&ms.full[s]), kTma ? 1 : 32 * C::GW);
      mbar_init(smem_u32(&ms.empty[s]), 1);
    }
    for (int s = 0; s < kMeta; ++s) mbar_init(smem_u32(&ms.meta_full[s]), 1 + (C::kScaled && !kTma ? kProdThreads : 0));
    for (int s = 0; s < C::SBUF; ++s) {
      mbar_init(smem_u32(&ms.s_full[s]), 1);
      mbar_init(smem_u32(&ms.s_free[s]), kSmxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.p_full[s]), kSmxWarps);
      mbar_init(smem_u32(&ms.p_free[s]), 1);
      mbar_init(smem_u32(&ms.final[s]), 1);
    }
    mbar_init(smem_u32(&ms.rope_full), kTma ? 1 : 32 * C::GW);
    mbar_init(smem_u32(&ms.rope_empty), 1);
    mbar_init(smem_u32(&ms.q_full), kSmxWarps);
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
  // everything above may overlap the kernel in front; what it wrote is visible from here on
  grid_dependency_wait();
  chunk_plan<C::THREADS>(w, sm, ms.range, ms.unit[0]);
  fence_proxy_async_smem();   // the plan's scratch becomes the ring
  __syncthreads();
  grid_launch_dependents();   // the merge: its blocks wait for the whole grid
  Range rg;
  rg.t0 = ms.range.t0;
  rg.n_it = (int)(ms.range.t1 - rg.t0);
  if (rg.n_it > 0) {          // the same for the whole CTA
    if (warp < kSmxWarps) {
      regs_inc<C::SMX_REGS>();
      softmax_role<NC, kLayout, kTma>(w, sm, ms, tmem, rg);
    } else {
      regs_dec<C::OTHER_REGS>();
      if (warp == kQkWarp) qk_role<NC, kLayout, kTma>(w, sm, ms, tmem, rg);
      else if (warp == kPvWarp) pv_role<NC, kLayout, kTma>(w, sm, ms, tmem, rg);
      else if constexpr (!kTma) producer_role<NC, kLayout, kTma>(w, sm, ms, rg);
      else if (warp == kProdWarp0) tma_role<NC, kLayout, kTma>(w, maps, sm, ms, rg);
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

template <int NC, int kLayout, bool kTma>
bool launch(const ChunkWork& w, const ChunkMaps& maps, cudaStream_t stream) {
  using C = Cfg<NC, kLayout, kTma>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<NC, kLayout, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return false;
    // the register re-split adds up only from exactly LAUNCH_REGS registers a thread
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, chunk_attn_kernel<NC, kLayout, kTma>) != cudaSuccess || fa.numRegs != C::LAUNCH_REGS)
      return false;
    configured.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_attn_kernel<NC, kLayout, kTma>, w, maps) != cudaSuccess) return false;
  // units of one tile are not spread over CTAs
  return (int64_t)w.a.max_pages * w.a.page_size <= kTile || launch_chunk_merge(w, stream);
}

// The driver's tensor map encoder (the library does not link the driver).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// The pool as a matrix of bytes: boxes of `rows` rows and `width` bytes.
bool encode_rows(CUtensorMap* map, const ChunkArgs& a, int row_bytes, int width, int rows, bool swizzle) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)a.pool_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)rows};
  const cuuint32_t steps[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.pool), dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NC, int kLayout>
bool launch_layout(const ChunkWork& w, const ChunkMaps& maps, cudaStream_t stream) {
  return w.box_shift > 0 ? launch<NC, kLayout, true>(w, maps, stream) : launch<NC, kLayout, false>(w, maps, stream);
}

template <int NC>
bool launch_nc(const ChunkWork& w, const ChunkMaps& maps, cudaStream_t stream) {
  if (w.a.layout == DSA_KV_RAW512) return launch_layout<NC, DSA_KV_RAW512>(w, maps, stream);
  if (w.a.layout == DSA_KV_SCALED528) return launch_layout<NC, DSA_KV_SCALED528>(w, maps, stream);
  return launch_layout<NC, DSA_KV_ROPE656>(w, maps, stream);
}

}  // namespace

// 16 rows where the average request has no more, else 32: half the columns
// need less of everything but the rows' bytes, two units of 16 read the rows
// twice.  us with 16 / 32, 64 requests of up to 8192 rows: 16 heads, raw 40.6 /
// 43.4, rope 52.4 / 58.8; 24 heads, raw 57.3 / 45.9, rope 81.9 / 61.1; one of
// 131072: 16 heads, raw 21.7 / 23.3; 32 heads 29.3 / 23.8.
int chunk_columns(int T, int H, int B) {
  const int64_t rows = ((int64_t)T * H + B - 1) / B;     // of an average request
  return rows <= kFewestRows ? kFewestRows : 32;
}

bool launch_chunk_attn(const ChunkWork& work, cudaStream_t stream) {
  if (work.grid > kMaxCtas) return false;      // (the merge's limit, before anything is launched)
  ChunkWork w = work;
  // the largest power of two that divides the page and the tile: a box (rows
  // one by one where that is below 32, see above)
  const int page = w.a.page_size;
  int shift = 0;
  while (shift < 7 && page % (2 << shift) == 0) ++shift;
  w.box_shift = shift >= 5 ? shift : 0;
  w.unit_cost = chunk_unit_cost(w.a.layout);
  ChunkMaps maps{};
  if (w.box_shift > 0) {
    const int row_bytes = w.a.layout == DSA_KV_RAW512 ? kRawRow : w.a.layout == DSA_KV_SCALED528 ? kScaledRow : kRopeRow;
    if (!encode_rows(&maps.rows, w.a, row_bytes, 128, 1 << w.box_shift, true)) return false;
    if (w.a.layout != DSA_KV_RAW512 && !encode_rows(&maps.scales, w.a, row_bytes, 16, 1 << w.box_shift, false)) return false;
  }
  return w.nc == 16 ? launch_nc<16>(w, maps, stream) : launch_nc<32>(w, maps, stream);
}

}  // namespace dsa
