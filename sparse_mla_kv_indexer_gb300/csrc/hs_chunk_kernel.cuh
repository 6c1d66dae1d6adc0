// Attention of a chunk of new tokens over the paged cache (prefill, the input of a later
// turn, dense decode): every query token attends to every cached row below its limit. SHARED: of
// requests that share their first positions (hs_prefix.cu), over the blocks that a kernel before has listed.
//
// "Serving GLM-5.3 with PCP, DCP and Hybrid HiSparse" (vLLM blog Part 2), footnote 1: QK
// over 576 dims (512 latent, 64 rope), PV over the 512 latent dims, every row serving all
// heads. Per token j and head h, over the positions t < limit_j of its request:
//   z_t = sm_scale * q_jh . k_t,  o = sum_t softmax(z)_t v_t,  lse = log sum_t exp z_t.
//
// Work. A (token, head) pair is a row; a block is 128 rows (128 / H tokens of one segment);
// a tile is a block against one page of 64 cached rows. The tiles of all blocks, in order,
// and a block's fixed cost (its queries, its outputs) before its first tile, are dealt in
// equal contiguous ranges to the pairs of SMs, so that one token over a long context and a
// long prompt both fill the GPU. A range cuts at most two blocks; their parts go to the
// workspace (fp32 sums, maxima) and chunk_merge_kernel joins them in a fixed order. Every
// CTA finds its range itself from the segments and limits.
//
// Split of a block over a pair. The output of 128 rows is 128 x 512 fp32, all of one SM's
// tensor memory, with no room for scores; so two CTAs form a pair (tcgen05.mma of
// cta_group::2, M = 128): each holds every other row, 256 columns of tensor memory for their
// output, and supplies half of each B operand: the keys of half the page for QK, half the
// output dims for PV. The full rate of M = 128 then needs one copy of Q (64 rows, 72 KB),
// and shared memory holds two stages of everything else.
//
// Roles (640 threads per CTA, five warpgroups):
//   warps 0-7   softmax: a thread has one row and 16 keys of the tile (in the output: one
//               128-dim group); four threads share a row
//   warps 8-15  cache rows -> fp16 operands, loaded one tile ahead into registers.
//               K: the e4m3 codes of this CTA's 32 rows as fp16 (exact), and the rope;
//               V: code x scale of all 64 rows for this CTA's two 128-dim groups
//   warp 16     tensor memory; in the pair's first CTA the tcgen05.mma issue for both
//   warp 17     the pieces (block, pages) of this pair's range and their tiles' rows, ahead of the
//               other roles
// Tile t:  QK   S_g = Q_g K_g^T for the four 128-value groups and the rope (five
//               accumulators), so that s = sum_g scale_g S_g + S_rope is exact up to fp32
//          softmax  running maximum with a lazy rescale (the reference moves when a row
//               exceeds it by more than 2^8), P = 2^(z - m + 7) in fp16, sums in fp32
//          PV   O += P V, in tensor memory for the whole piece
// QK(t+1) is issued before PV(t), so the softmax of one tile runs under the products of
// its neighbours.
//
// Numbers. K codes are exact in fp16, and rope and bf16 queries from 2^-17 to 65504 in magnitude
// (off by 2^-25 at most below: their last bits, or all, lie under fp16's smallest step); V is 4 code scale, a
// product in fp32, rounded once to fp16; P keeps 11 bits from 2^15 down to 2^-14, that is
// to 2^-21 of the row's largest (the shift by 2^7 buys seven binades under a dominant row).
// Scores, maxima, sums and the output accumulate in fp32. A row with a NaN code, or rope
// beyond fp16, scores NaN or infinity and is not seen; nor is one whose score is beyond 2^22.
//
// Measured on a GB300: 753 tokens over 74,913 rows with 64 heads 8.9 ms, 0.88 PFLOP/s, 47 % of
// the measured bf16 rate; per tile of a pair 1.52 us, against 0.73 us of its products alone
// (1,416 cycles: 36 of 25 for QK, which its shared-memory reads bound, and 8 of 64 for PV).
// What bounds it is the work around them: 6,500 warp instructions per tile and SM (0.54 a
// cycle and scheduler), half of them the conversion of K and V, and 1,490 shared-memory wavefronts
// besides the 1,246 of the products, in 2,990 cycles. With parts of it left out one at a time (8 x 129 tokens over
// 20,001 rows, 3.40 ms): V's scaling 10 %, three of four loads of scales 7 %, three quarters of V's or K's stores
// 5 and 4 %, four of five accumulator reads or the exchange of maxima nothing. More converter
// warps cost more instructions than they hide: K and V on eight warps each 7 to 11 % more time, K one tile
// ahead of V on the same warps 3 to 5 %. How the roles' instructions interleave moves every long
// case by 1 to 3 % and the ragged one by up to 12 %, in either direction, for changes that do
// nothing else (the order of two waits, a constant). One token over 131,072 rows takes 62 us (13 us
// at the copy rate): 27 tiles a pair of 1.6 us, 12 us before the first and 5 us of merge.
#pragma once

#include <cuda_fp8.h>
#include <math.h>

#include <atomic>

#include "hs_chunk.cuh"

namespace hs {

namespace {

constexpr int CK_THREADS = 640;
constexpr int CK_SM_WARPS = 8, CK_SM = CK_SM_WARPS * 32;         // softmax
constexpr int CK_CONV_WARP0 = 8, CK_CONV_WARPS = 8;               // conversion
constexpr int CK_MMA_WARP = 16, CK_PLAN_WARP = 17;
// Registers per thread: 96 at the launch (five warpgroups), then shifted between warpgroups,
// whose sum stays within the launch's.
constexpr int CK_REGS = 96, CK_SM_REGS = 96, CK_CONV_REGS = 104, CK_MISC_REGS = 80;
// The softmax keeps what it was launched with; asking for more than the others free would wait
// without end.
static_assert(CK_SM_REGS == CK_REGS && 2 * CK_SM_REGS + 2 * CK_CONV_REGS + CK_MISC_REGS <= CK_THREADS / 128 * CK_REGS,
              "register shares");
constexpr int CK_ROWS = 128;       // rows of a block
constexpr int CK_HALF = 64;        // rows of a block per CTA
constexpr int CK_BLOCK_COST = 3;   // what a block costs besides its pages, in pages
constexpr int CK_MIN_COST = CK_BLOCK_COST + 2;   // least cost of a pair's range
constexpr int CK_RING = 4;         // pieces the planning warp runs ahead
constexpr int CK_TILES = 4;        // tiles it runs ahead
constexpr int CK_SCL = 4;          // tiles of scales held
constexpr int CK_SCL_G = 68 * 4;   // bytes from one group's 64 scales to the next (other banks for the same row)
constexpr int CK_SCL_T = 4 * CK_SCL_G;
// shared memory
constexpr int CK_QATOM = CK_HALF * 128;            // 64 rows x 64 dims fp16
constexpr int CK_KATOM = 32 * 128;                 // 32 keys x 64 dims
constexpr int CK_VATOM = 64 * 128;                 // 64 keys x 64 dims
constexpr int CK_KSTAGE = 9 * CK_KATOM;            // 36,864
constexpr int CK_VSTAGE = 4 * CK_VATOM;            // 32,768
constexpr int CK_OFF_Q = 0;
constexpr int CK_OFF_K = 9 * CK_QATOM;
constexpr int CK_OFF_V = CK_OFF_K + 2 * CK_KSTAGE;
constexpr int CK_OFF_P = CK_OFF_V + 2 * CK_VSTAGE;
constexpr int CK_OFF_SCL = CK_OFF_P + CK_HALF * 128;           // float [CK_SCL][4][64 of 68]
constexpr int CK_OFF_RED = CK_OFF_SCL + CK_SCL * CK_SCL_T;   // float [2][4][64]
constexpr int CK_OFF_RING = CK_OFF_RED + 2 * 256 * 4;          // Piece [CK_RING]
constexpr int CK_PIECE_BYTES = 32;
constexpr int CK_OFF_TILES = CK_OFF_RING + CK_RING * CK_PIECE_BYTES;   // Tile [CK_TILES]
constexpr int CK_OFF_BAR = CK_OFF_TILES + CK_TILES * CK_PIECE_BYTES;
enum Bar { B_KF = 0, B_VF = 2, B_PF = 4, B_SD = 6, B_PD = 8, B_SR = 10, B_FIN = 11, B_RF = 12, B_RE = 12 + CK_RING,
           B_TF = 12 + 2 * CK_RING, B_TE = B_TF + CK_TILES, B_SC = B_TE + CK_TILES, B_SE = B_SC + CK_SCL,
           B_N = B_SE + CK_SCL };
constexpr int CK_OFF_MISC = CK_OFF_BAR + B_N * 8;   // tensor-memory slot, dead flag, plan scalars
constexpr int CK_SMEM = CK_OFF_MISC + 64 + 1024;
static_assert(CK_SMEM <= 232448, "shared memory budget");
// tensor memory: O [2][128 columns], then a ring of eight score accumulators of 32 columns, of
// which a tile takes five: the next tile's first three are written while this one's are read
constexpr uint32_t CK_TM_O = 0, CK_TM_S = 256;
// the plan's arrays, in the operand buffers before the roles start
constexpr int CK_PLAN_START = 0;                                        // int [HS_CHUNK_MAX_SEGMENTS + 1]
constexpr int CK_PLAN_BLK = CK_PLAN_START + (HS_CHUNK_MAX_SEGMENTS + 1) * 4;
constexpr int CK_MAX_BLOCKS = HS_CHUNK_MAX_SEGMENTS + HS_CHUNK_MAX_TOKENS / 2;
constexpr int CK_MAX_CHUNKS = (CK_MAX_BLOCKS + CK_THREADS - 1) / CK_THREADS;
constexpr int CK_PLAN_SUM = CK_PLAN_BLK + (HS_CHUNK_MAX_SEGMENTS + 1) * 4;   // int [CK_MAX_CHUNKS]
constexpr int CK_PLAN_WARP_TMP = CK_PLAN_SUM + CK_MAX_CHUNKS * 4;       // int [32]
static_assert(CK_PLAN_WARP_TMP + 32 * 4 <= CK_OFF_SCL, "plan arrays");

constexpr float CK_LOG2E = 1.4426950408889634f;
constexpr float CK_V_FACTOR = 4.f, CK_V_SHIFT = 2.f;   // V is held times this; its log2
constexpr float CK_MAX_SCALE = 36.5f;      // 4 x 448 x scale < 65504
constexpr float CK_RESCALE_LOG2 = 8.f;     // the reference maximum moves beyond this
constexpr float CK_P_SHIFT = 7.f;          // P = 2^(z - m + 7) <= 2^15
// Largest score in log2 units: m and 7 - m are each rounded by at most 2^-3 then, and a P of
// 2^15 times those 2^(1/4) stays below fp16's largest. Far beyond, P would overflow.
constexpr float CK_MAX_Z = 4194304.f;      // 2^22
// A row's reference may lie as far below, and further until its end: scores next to the border keep
// their weights (P at most 2^15 times 2^(1/2) there), and those below -2^23, whose reference is
// CK_LOW, have the weight 0 that they have next to any score in range. A row that ends with a
// reference below -2^22 is reported.
constexpr float CK_LOW_Z = -8388608.f;     // -2^23
constexpr float CK_LOW = -3.0e38f;
constexpr float CK_MAX_SM_SCALE = 1e20f;   // times any score of finite operands (1e12): finite

__device__ __forceinline__ bool only_low(float m) { return m > -INFINITY && m < -CK_MAX_Z; }

// A pair's partial results: for each of its two cut blocks 128 rows of unnormalised
// outputs and (reference in log2 units, sum); and the block that starts in its range and
// ends in a later pair's.
struct ChunkCut {
  int32_t tok0, n_tok, last_pair, pad;
};
struct ChunkWork {
  ChunkCut* cut;     // [pairs]
  float2* stats;     // [pairs][2][128]
  float* part;       // [pairs][2][128][512]
};
constexpr int64_t CK_SLOT_ROWS = 2 * CK_ROWS;
// Where four output dims (4 c4 .. + 3) of a row lie among its slot's, in 16 bytes: every c4's of four rows of one CTA
// next to one another. A warp of the attention, which has every other row, then stores 64 contiguous bytes for four of
// its lanes (16 bytes of 32 rows' own lines took 6 us when all SMs wrote their cut blocks at once, now 3), and the joins,
// which take four rows at a time, read 8 KB in one run.
__device__ __forceinline__ size_t part_unit(size_t row, int c4) {
  return (((row >> 3) * 2 + (row & 1)) * 128 + c4) * 4 + ((row >> 1) & 3);
}
// The j-th row of four that are next to one another.
__device__ __forceinline__ int quad_row(int four, int j) { return (four >> 1) * 8 + (four & 1) + 2 * j; }
__host__ __device__ inline int64_t work_stats_at(int pairs) { return ((int64_t)pairs * 16 + 255) / 256 * 256; }
__host__ __device__ inline int64_t work_part_at(int pairs) { return work_stats_at(pairs) + (int64_t)pairs * CK_SLOT_ROWS * 8; }
inline int64_t work_bytes_for(int pairs) { return work_part_at(pairs) + (int64_t)pairs * CK_SLOT_ROWS * 512 * 4; }
__host__ __device__ inline ChunkWork work_at(void* base, int pairs) {
  uint8_t* b = static_cast<uint8_t*>(base);
  return {reinterpret_cast<ChunkCut*>(b), reinterpret_cast<float2*>(b + work_stats_at(pairs)),
          reinterpret_cast<float*>(b + work_part_at(pairs))};
}

// hs_prefix_attention: its blocks are listed by a kernel before (prefix_plan_kernel), since a token can be
// in two of them, one of the positions its group shares and one of its own. Their sums then go to the
// workspace when the block is whole, too. Two 16-byte words of a block:
//   tok0, n_tok, req (-1: a bad request), limit (the largest of the block's tokens, within the pages)
//   first page, end page, cap (positions from here on are not of this block), cost of the blocks before
struct PlanBlock {
  int4 a, b;
};
constexpr int CK_NO_CAP = 0x7FFFFFFF;
struct PairStart {     // a pair's range: its first block (and its index), how far into its cost it starts, its units of cost
  int block, into, n, pad;
  PlanBlock first;
};
struct SharedWork {
  PairStart* start;    // [pairs]
  PlanBlock* blocks;   // [max_blocks]
  int2* of_token;      // [tokens]: what is to be joined of its blocks of shared positions, and of its own (ToJoin)
  float2* stats;       // as of ChunkWork
  float* part;
  float2* whole_stats; // [2][tokens * heads]: of shared blocks, of the others
  float* whole;        // [2][tokens * heads][512]
};
__host__ __device__ inline int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }
// Its arrays in a workspace (base null: their offsets; `end`: its bytes).
__host__ __device__ inline SharedWork shared_at(void* base, int pairs, int64_t tokens, int64_t rows, int64_t max_blocks, int64_t* end) {
  uint8_t* b = static_cast<uint8_t*>(base);
  SharedWork w;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return b + here;
  };
  w.start = reinterpret_cast<PairStart*>(take(pairs * (int64_t)sizeof(PairStart)));
  w.blocks = reinterpret_cast<PlanBlock*>(take(max_blocks * (int64_t)sizeof(PlanBlock)));
  w.of_token = reinterpret_cast<int2*>(take(tokens * 8));
  w.stats = reinterpret_cast<float2*>(take(pairs * CK_SLOT_ROWS * 8));
  w.part = reinterpret_cast<float*>(take(pairs * CK_SLOT_ROWS * 512 * 4));
  w.whole_stats = reinterpret_cast<float2*>(take(2 * rows * 8));
  w.whole = reinterpret_cast<float*>(take(2 * rows * 512 * 4));
  if (end) *end = at;
  return w;
}

struct ChunkArgs {
  int layer, n_seg, n_tok, pairs;
  int small;         // at most 32 segments and blocks: one warp plans
  const int32_t *seg_req, *seg_start, *limit;
  const void* q;
  long long q_tok, q_head;
  float scale_log2;
  void* out;
  long long o_tok, o_head;
  float* lse;
  void* work;
  // hs_prefix_attention alone
  int n_groups, max_blocks;
  const int32_t *group_start, *group_len;
};
__device__ __forceinline__ SharedWork shared_work(const ChunkArgs& A, int heads) {
  return shared_at(A.work, A.pairs, A.n_tok, (int64_t)A.n_tok * heads, A.max_blocks, nullptr);
}

// One block's pages [pg0, pg1) of one pair's range, two 16-byte words in the ring:
//   tok0, n_tok (tokens of the block; -1: no more pieces), req (-1: a bad request, nothing is
//   read), limit (the largest of the block's tokens)
//   pg0, pg1, slot (-1: the whole block, else the workspace slot 0 or 1; 2 and 3: a whole block of shared
//   positions, and of the others of a token that has both), cap (PlanBlock's)
struct Piece {
  int4 a, b;
  __device__ int tok0() const { return a.x; }
  __device__ int n_tok() const { return a.y; }
  __device__ int req() const { return a.z; }
  __device__ int pg0() const { return b.x; }
  __device__ int pg1() const { return b.y; }
  __device__ int slot() const { return b.z; }
};

// One tile in its ring, two 16-byte words: the address of its 64 rows (8 bytes), how many of
// them some token sees (-1: no more tiles), whether it begins a piece; then the piece's tok0
// and n_tok.

// Named barrier over n threads that ORs `flag` across them: a role whose threads saw a wait
// run out stops as one, and no thread is left behind at a barrier.
__device__ __forceinline__ bool bar_any(int id, int n, bool flag) {
  int out;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(out)
      : "r"(flag ? 1 : 0), "r"(id), "r"(n)
      : "memory");
  return out != 0;
}
__device__ __forceinline__ void arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive on a barrier of either CTA of the pair (cluster address). What the arrival announces to
// the issue of the products (operands, scores read) lies in the arriving CTA's own shared or
// tensor memory, behind the proxy and tcgen05 fences before it, and is read there by the tensor
// core: no data crosses the pair through this barrier, and its scope is the default one. Words
// that threads of a CTA hand to one another (pieces, tiles, scales) go through barriers of that
// CTA alone: the way round over the other CTA would not order them. A release at cluster scope
// measured 1,400 cycles per arrival (four per tile).
__device__ __forceinline__ void arrive_cluster(uint32_t cbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cbar) : "memory");
}
// Shared memory by 32-bit address: the aligned base is computed as an integer, from which the
// compiler would make generic accesses with 64-bit addresses.
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for a phase: false after `seconds` (or when another role of this CTA gave up),
// with HS_ERR_TIMEOUT recorded. Each lane has its own answer, and one may give up where the
// others still see the phase end; so that none waits for it at a warp's barrier, the softmax's
// lanes go on to a vote at their next barrier, and a converter's lane ends there and then (the
// barriers of warp, CTA and cluster wait for threads that have not ended). Inlined: a call here
// makes its callers keep their operands across it in local memory, which does not fit beside
// 228 KB of shared memory.
__device__ __forceinline__ bool ck_wait_slow(uint32_t bar, uint32_t parity, int32_t* status, uint32_t dead, int seconds) {
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (lds32(dead)) return false;
      if (globaltimer() - t0 > (uint64_t)seconds * WAIT_NS) {
        set_status(status, HS_ERR_TIMEOUT);
        sts32(dead, 1);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool ck_wait(uint32_t bar, uint32_t parity, int32_t* status, uint32_t dead, int seconds = 2) {
  if (try_wait(bar, parity)) return true;
  return ck_wait_slow(bar, parity, status, dead, seconds);
}
// The same for a whole warp, one answer for all of its lanes. (A vote at every wait of the
// softmax and the converters, or a converter that goes on, costs 1.2 to 1.6 % of a long call.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int32_t* status, uint32_t dead, int seconds = 2) {
  return __all_sync(0xffffffffu, ck_wait(bar, parity, status, dead, seconds));
}

// Registers of the calling warpgroup, down (freed at once) or up (waits for freed ones).
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// ---- tcgen05 over the pair -----------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// One lane of a converged warp, the same at every call. The issuing loop runs on the whole
// warp with warp-uniform operands and only the instruction itself is predicated: issued by
// one lane of a diverged warp, each tcgen05.mma takes 57 cycles to issue (its descriptors
// are moved to uniform registers one by one), against 25 that the smallest of them needs.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(p));
  return p != 0;
}
// The operands are the low words of their descriptors (address / 16, leading offset); the
// high word is the same for all.
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t desc_hi,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(desc_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once every MMA issued so far completes.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// The same on this CTA's barrier alone.
__device__ __forceinline__ void umma_commit_own(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Scores as the fragments of a warp-wide product: lane l gets of 32 rows l / 4 + 8 i (i = 0 .. 3) the columns 2 c, 2 c + 1
// (c = l % 4; r[8 (i / 2) + 2 (i % 2)], + 1) and 8 + 2 c, 9 + 2 c (+ 4, + 5) of 16.
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, uint32_t* r) {
#pragma unroll
  for (int b = 0; b < 2; ++b)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[8 * b]), "=r"(r[8 * b + 1]), "=r"(r[8 * b + 2]), "=r"(r[8 * b + 3]), "=r"(r[8 * b + 4]),
                   "=r"(r[8 * b + 5]), "=r"(r[8 * b + 6]), "=r"(r[8 * b + 7])
                 : "r"(taddr + ((uint32_t)(16 * b) << 16)));
}
// Four 8 x 8 matrices of 16-bit values, in such fragments, to rows of 16 bytes: lane l has the address of row l.
__device__ __forceinline__ void store_frag4(uint32_t a, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Where a key's scale lies among its group's: in order, or the four keys of a lane's fragments next to one another.
template <bool FRAGMENTS>
__device__ __forceinline__ int scale_place(int key) {
  return FRAGMENTS ? (key & ~15) + 4 * ((key >> 1) & 3) + 2 * ((key >> 3) & 1) + (key & 1) : key;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- conversions ----------------------------------------------------------------------
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 e4m3x2_to_h2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}
__device__ __forceinline__ void codes_to_f16(uint4 v, uint4& lo, uint4& hi) {
  lo = make_uint4(h2_bits(e4m3x2_to_h2(v.x & 0xFFFFu)), h2_bits(e4m3x2_to_h2(v.x >> 16)),
                  h2_bits(e4m3x2_to_h2(v.y & 0xFFFFu)), h2_bits(e4m3x2_to_h2(v.y >> 16)));
  hi = make_uint4(h2_bits(e4m3x2_to_h2(v.z & 0xFFFFu)), h2_bits(e4m3x2_to_h2(v.z >> 16)),
                  h2_bits(e4m3x2_to_h2(v.w & 0xFFFFu)), h2_bits(e4m3x2_to_h2(v.w >> 16)));
}
// 4 x code x scale in fp16: the product in fp32, rounded once (the factor keeps two more bits of
// the smallest; it leaves the output again with the sum). Products of fp16 parts of the scale are
// not exact enough: the second part of a small scale is lost under fp16's smallest step, times a
// code of up to 448. (Those products took 4 % less of a long call; with 2^-8 code and 2^10 scale, also
// fp16, nearly exact, they take 1 % more; a branch on the scales to choose between them 0 to 20 % more.)
// A NaN code becomes a finite value: its row's scores are NaN, so it is not seen, and 0 x it has to be 0.
__device__ __forceinline__ uint32_t scaled2(uint32_t two, float scale4) {
  const float2 c = __half22float2(e4m3x2_to_h2(two));
  float a, b;
  unpack(mul2(f2(__float_as_uint(c.x), __float_as_uint(c.y)), f2(scale4)), a, b);
  return h2_bits(__hmin2(__floats2half2_rn(a, b), __half2half2(__ushort_as_half(0x7BFF))));
}
__device__ __forceinline__ void codes_to_scaled_f16(uint4 v, float scale, uint4& lo, uint4& hi) {
  const float s = CK_V_FACTOR * scale;
  lo = make_uint4(scaled2(v.x & 0xFFFFu, s), scaled2(v.x >> 16, s), scaled2(v.y & 0xFFFFu, s), scaled2(v.y >> 16, s));
  hi = make_uint4(scaled2(v.z & 0xFFFFu, s), scaled2(v.z >> 16, s), scaled2(v.w & 0xFFFFu, s), scaled2(v.w >> 16, s));
}
// Eight bf16 -> fp16 (exact from 2^-17 on); *bad when one is beyond its largest.
__device__ __forceinline__ uint4 bf16x8_to_f16(uint4 v, bool* bad) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = h2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)));
    *bad |= (o[i] & 0x7C00u) == 0x7C00u || (o[i] & 0x7C000000u) == 0x7C000000u;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
template <typename T>
__device__ __forceinline__ uint4 q_to_f16(uint4 v, bool* bad) {
  if constexpr (sizeof(T) == 2 && !__is_same(T, __half)) {
    return bf16x8_to_f16(v, bad);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) *bad |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
    return v;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (__is_same(T, __half)) {
    return h2_bits(__floats2half2_rn(a, b));
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// ---- the plan -------------------------------------------------------------------------
// Inclusive scan over the CTA's threads (sum or maximum); tmp: 32 ints; returns the
// inclusive value, *total the whole.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto op = [](int a, int b) { return MAX ? max(a, b) : a + b; };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = op(v, u);
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  int w = lane < CK_THREADS / 32 ? tmp[lane] : 0;   // the warps' totals (values are >= 0)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = op(w, u);
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return warp == 0 ? v : op(before, v);
}

__device__ __forceinline__ int clamp_limit(const Dev& D, int l, bool* bad) {
  if (l < 0 || l > D.max_ctx) {
    *bad = true;
    return 0;
  }
  return l;
}

// Tokens and largest limit of block b of a segment [t0, t1).
__device__ __forceinline__ int block_limit(const Dev& D, const int32_t* limit, int t0, int t1, bool* bad) {
  int m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)   // at most 128 / 16 tokens
    if (t0 + i < t1) m = max(m, clamp_limit(D, __ldg(limit + t0 + i), bad));
  return m;
}
__device__ __forceinline__ int pages_of(int limit) { return max(1, (limit + PAGE - 1) / PAGE); }

struct Range {
  int seg, seg_t0, seg_t1;   // the segment of the first block, clamped
  int tok0;                  // the first block's first token
  int into;                  // how far into its cost the range starts
  int at;                    // the range's first unit of cost
  int n;                     // its units
  int per_pair;              // units of each pair's range
};

// This pair's range. All threads of the CTA take part; sm: the operand buffers.
__device__ Range plan_range(const Dev& D, const ChunkArgs& A, int pair, int tpb, uint8_t* sm, int32_t* found) {
  int* start = reinterpret_cast<int*>(sm + CK_PLAN_START);
  int* blk = reinterpret_cast<int*>(sm + CK_PLAN_BLK);
  int* sums = reinterpret_cast<int*>(sm + CK_PLAN_SUM);
  int* tmp = reinterpret_cast<int*>(sm + CK_PLAN_WARP_TMP);
  const int tid = threadIdx.x;
  bool bad = false;
  // segment starts, clamped to [0, n_tok] and to ascend
  const int per = (A.n_seg + CK_THREADS) / CK_THREADS;   // of the n_seg + 1 starts
  const int lo = min(tid * per, A.n_seg + 1), hi = min(lo + per, A.n_seg + 1);
  int m = 0, total;
  for (int i = lo; i < hi; ++i) {
    const int s = __ldg(A.seg_start + i), c = min(max(s, 0), A.n_tok);
    m = max(m, c);
    bad |= c != s || m != c;
    start[i] = m;
  }
  const int upto = block_scan<true>(m, tmp, &total);
  // exclusive maximum of the threads before
  int before = __shfl_up_sync(0xffffffffu, upto, 1);
  __syncthreads();
  if ((tid & 31) == 31) tmp[tid >> 5] = upto;
  __syncthreads();
  if ((tid & 31) == 0) before = tid == 0 ? 0 : tmp[(tid >> 5) - 1];
  for (int i = lo; i < hi; ++i) {
    bad |= start[i] < before;
    start[i] = max(start[i], before);
  }
  __syncthreads();
  // blocks before each segment
  int nb = 0;
  for (int i = lo; i < min(hi, A.n_seg); ++i) nb += (start[i + 1] - start[i] + tpb - 1) / tpb;
  int n_blocks;
  int at = block_scan<false>(nb, tmp, &n_blocks) - nb;
  for (int i = lo; i < min(hi, A.n_seg); ++i) {
    blk[i] = at;
    at += (start[i + 1] - start[i] + tpb - 1) / tpb;
  }
  if (tid == 0) blk[A.n_seg] = n_blocks;
  __syncthreads();
  // the cost of as many blocks at a time as the CTA has threads
  auto segment_of = [&](int b) {   // the last segment whose first block is <= b (never an empty one)
    int l = 0, h = A.n_seg;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (blk[mid] <= b) l = mid; else h = mid;
    }
    return l;
  };
  auto cost_of = [&](int b, bool* bad_id) {
    const int s = segment_of(b), t0 = start[s] + (b - blk[s]) * tpb;
    return CK_BLOCK_COST + pages_of(block_limit(D, A.limit, t0, min(t0 + tpb, start[s + 1]), bad_id));
  };
  const int chunks = (n_blocks + CK_THREADS - 1) / CK_THREADS;
  int all = 0, t = 0, end = 0;   // this thread's block of the last chunk: its cost, and that up to it
  for (int c = 0; c < chunks; ++c) {
    const int b = c * CK_THREADS + tid;
    int sum;
    t = b < n_blocks ? cost_of(b, &bad) : 0;
    end = all + block_scan<false>(t, tmp, &sum);
    if (tid == 0) sums[c] = sum;
    all += sum;
  }
  if (bad) set_status(D.status, HS_ERR_BAD_ID);
  Range r = {};
  r.per_pair = max((all + A.pairs - 1) / A.pairs, CK_MIN_COST);
  r.at = pair * r.per_pair;
  r.n = min(r.per_pair, all - r.at);
  __syncthreads();
  if (r.n <= 0) {
    r.n = 0;
    return r;
  }
  // the block that holds the range's first unit
  int c = 0, first = 0;
  while (first + sums[c] <= r.at) first += sums[c++];
  const int b = c * CK_THREADS + tid;
  if (c != chunks - 1) {
    bool ignore = false;
    t = b < n_blocks ? cost_of(b, &ignore) : 0;
    int sum;
    end = first + block_scan<false>(t, tmp, &sum);
  }
  if (t > 0 && end - t <= r.at && r.at < end) {
    const int s = segment_of(b);
    found[0] = s;
    found[1] = start[s];
    found[2] = start[s + 1];
    found[3] = start[s] + (b - blk[s]) * tpb;
    found[4] = r.at - (end - t);
  }
  __syncthreads();
  r.seg = found[0];
  r.seg_t0 = found[1];
  r.seg_t1 = found[2];
  r.tok0 = found[3];
  r.into = found[4];
  return r;
}

// The same for at most 32 segments and 32 blocks, by one warp without a barrier (3 us of a
// short call); lane b keeps block b.
struct WarpPlan {
  int tok0, tok1, req, limit;   // of this lane's block
};
__device__ Range plan_range_warp(const Dev& D, const ChunkArgs& A, int pair, int tpb, WarpPlan& mine) {
  const int lane = threadIdx.x & 31;
  auto all_max = [&](int v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    return v;
  };
  auto all_sum = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  bool bad = false;
  int s = 0, e = 0, req = -1;
  if (lane < A.n_seg) {
    const int s0 = __ldg(A.seg_start + lane), e0 = __ldg(A.seg_start + lane + 1);
    req = __ldg(A.seg_req + lane);
    s = min(max(s0, 0), A.n_tok);
    e = min(max(e0, 0), A.n_tok);
    bad = s != s0 || e != e0 || e < s;
  }
  const int start = all_max(s), end = max(start, e);
  const int before_seg = __shfl_up_sync(0xffffffffu, start, 1);
  bad |= lane > 0 && lane < A.n_seg && s < before_seg;
  const int nb = lane < A.n_seg ? (end - start + tpb - 1) / tpb : 0;
  const int upto = all_sum(nb), blk = upto - nb, n_blocks = __shfl_sync(0xffffffffu, upto, 31);
  int seg = 0;
  for (int i = 1; i < A.n_seg; ++i)
    if (__shfl_sync(0xffffffffu, blk, i) <= lane) seg = i;
  mine.tok0 = __shfl_sync(0xffffffffu, start, seg) + (lane - __shfl_sync(0xffffffffu, blk, seg)) * tpb;
  mine.tok1 = min(mine.tok0 + tpb, __shfl_sync(0xffffffffu, end, seg));
  mine.req = __shfl_sync(0xffffffffu, req, seg);
  mine.limit = lane < n_blocks ? block_limit(D, A.limit, mine.tok0, mine.tok1, &bad) : 0;
  if (bad) set_status(D.status, HS_ERR_BAD_ID);
  const int cost = lane < n_blocks ? CK_BLOCK_COST + pages_of(mine.limit) : 0;
  const int cost_end = all_sum(cost), all = __shfl_sync(0xffffffffu, cost_end, 31);
  Range r = {};
  r.per_pair = max((all + A.pairs - 1) / A.pairs, CK_MIN_COST);
  r.at = pair * r.per_pair;
  r.n = max(0, min(r.per_pair, all - r.at));
  const unsigned after = __ballot_sync(0xffffffffu, cost_end > r.at);
  r.seg = after ? __ffs(after) - 1 : 0;   // here the block
  r.into = r.at - __shfl_sync(0xffffffffu, cost_end - cost, r.seg);
  return r;
}

template <typename T, bool SHARED>
__global__ void __launch_bounds__(CK_THREADS, 1) chunk_attention_kernel(const Dev D, const ChunkArgs A) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // at the same offset in both CTAs: the dynamic shared memory of one kernel starts at one address
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t tslot = sbase + CK_OFF_MISC, dead = tslot + 4;
  int32_t* found = reinterpret_cast<int32_t*>(smem + CK_OFF_MISC) + 2;
  const uint32_t there = sbase + CK_OFF_MISC + 32;   // int [CK_SCL]: whether a tile's page exists
  auto bar = [&](int i) { return sbase + CK_OFF_BAR + 8 * i; };
  auto piece_at = [&](uint32_t slot) {
    const uint32_t at = sbase + CK_OFF_RING + slot * CK_PIECE_BYTES;
    const uint4 a = lds128(at), b = lds128(at + 16);
    return Piece{make_int4(a.x, a.y, a.z, a.w), make_int4(b.x, b.y, b.z, b.w)};
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x & 1;
  const int pair = blockIdx.x >> 1;
  const int H = D.n_heads, hs = 31 - __clz(H), tpb = CK_ROWS >> hs;   // 16, 32 or 64 heads

  if (warp == CK_MMA_WARP) tmem_alloc_pair(tslot, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_KF + i), 2 * CK_CONV_WARPS);
      mbar_init(bar(B_VF + i), 2 * CK_CONV_WARPS);
      mbar_init(bar(B_PF + i), 2 * CK_SM_WARPS);
      mbar_init(bar(B_SD + i), 1);
      mbar_init(bar(B_PD + i), 1);
    }
    for (int i = 0; i < CK_SCL; ++i) {
      mbar_init(bar(B_SC + i), 2);
      mbar_init(bar(B_SE + i), CK_SM_WARPS);
    }
    mbar_init(bar(B_SR), 2 * CK_SM_WARPS);
    mbar_init(bar(B_FIN), 1);
    for (int i = 0; i < CK_RING; ++i) {
      mbar_init(bar(B_RF + i), 1);
      mbar_init(bar(B_RE + i), CK_SM_WARPS + (rank == 0 ? 1 : 0));
    }
    for (int i = 0; i < CK_TILES; ++i) {
      mbar_init(bar(B_TF + i), 1);
      mbar_init(bar(B_TE + i), CK_CONV_WARPS);
    }
    fence_mbar_init();
    sts32(dead, 0);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = lds32(tslot);
  griddep_wait();
  griddep_launch();   // only the merge of this call depends on it, and waits for its end

  Range R = {};
  if (!SHARED && !A.small) {
    R = plan_range(D, A, pair, tpb, smem, found);
    __syncthreads();   // the plan's arrays are done with
  }

  if (warp >= CK_MMA_WARP) {
    regs_dec<CK_MISC_REGS>();
    if (warp == CK_PLAN_WARP) {
    // ------------------------------- pieces of the range -------------------------------
    const uint8_t* const kv = D.kv[A.layer];
    WarpPlan mine = {};
    SharedWork W = {};
    PlanBlock next = {};   // SHARED: the block `seg`, the workspace's list read one block ahead
    if constexpr (SHARED) {
      W = shared_work(A, H);
      const PairStart s = W.start[pair];
      R.seg = s.block, R.into = s.into, R.n = s.n;
      next = s.first;
    } else {
      if (A.small) R = plan_range_warp(D, A, pair, tpb, mine);
    }
    int seg = R.seg, t0 = R.tok0, seg_end = R.seg_t1, into = R.into, left = R.n, at = R.at;
    uint32_t k = 0, t = 0;
    int entries = -1;
    ChunkCut cut = {0, 0, 0, 0};
    bool ok = true;
    for (;; ++k) {
      int4 pa = make_int4(0, -1, -1, 0), pb = make_int4(0, 0, -1, 0);
      if constexpr (SHARED) {
        while (left > 0 && pa.y < 0) {
          const PlanBlock B = next;
          const int pages = B.b.y - B.b.x, end = min(pages > 0 ? CK_BLOCK_COST + pages : 0, into + left);
          const int p0 = max(into - CK_BLOCK_COST, 0), p1 = max(end - CK_BLOCK_COST, 0);
          if (p1 > p0) {
            const bool whole = p0 == 0 && p1 == pages;
            const int kind = B.b.z != CK_NO_CAP ? 2 : B.b.x > 0 ? 3 : -1;
            pa = B.a;
            pb = make_int4(B.b.x + p0, B.b.x + p1, whole ? kind : p0 == 0 ? 1 : 0, B.b.z);
          }
          left -= end - into;
          into = 0;
          ++seg;
          if (left > 0) next = W.blocks[seg];
        }
      }
      while (!SHARED && left > 0 && pa.y < 0) {   // the range's next pages: none of a block whose fixed cost it ends in
        int t1, r, lim;
        if (A.small) {
          t0 = __shfl_sync(0xffffffffu, mine.tok0, seg);
          t1 = __shfl_sync(0xffffffffu, mine.tok1, seg);
          r = __shfl_sync(0xffffffffu, mine.req, seg);
          lim = __shfl_sync(0xffffffffu, mine.limit, seg);
        } else {
          bool ignore = false;
          t1 = min(t0 + tpb, seg_end);
          r = __ldg(A.seg_req + seg);
          lim = block_limit(D, A.limit, t0, t1, &ignore);
        }
        const bool bad = r < 0 || r >= D.max_requests;
        const int n_pages = pages_of(lim);
        if (bad && lane == 0) set_status(D.status, HS_ERR_BAD_ID);
        const int end = min(CK_BLOCK_COST + n_pages, into + left), used = end - into;
        const int p0 = max(into - CK_BLOCK_COST, 0), p1 = max(end - CK_BLOCK_COST, 0);
        if (p1 > p0) {
          const bool whole = p0 == 0 && p1 == n_pages;
          pa = make_int4(t0, t1 - t0, bad ? -1 : r, bad ? 0 : lim);
          pb = make_int4(p0, p1, whole ? -1 : p0 == 0 ? 1 : 0, 0);
          if (p0 == 0 && !whole) cut = {t0, t1 - t0, (at - into + CK_BLOCK_COST + n_pages - 1) / R.per_pair, 0};
        }
        left -= used;
        at += used;
        into = 0;
        t0 = t1;
        if (A.small) ++seg;
        while (!A.small && left > 0 && t0 >= seg_end) {   // the next segment with tokens
          ++seg;
          t0 = seg_end;
          seg_end = max(seg_end, min(max(__ldg(A.seg_start + seg + 1), 0), A.n_tok));
        }
      }
      if (pa.y > 0 && k > 0) {   // the queries of the next pieces on their way to L2
        for (int c = lane; c < CK_HALF * 9; c += 32) {
          const int r = c / 9, gr = 2 * r + (int)rank, tk = gr >> hs;
          if (tk < pa.y)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(A.q) + (pa.x + tk) * A.q_tok +
                                                          (gr & (H - 1)) * A.q_head + (c - r * 9) * 64));
        }
      }
      const uint32_t slot = k % CK_RING;
      // a piece may be a whole context read over the host link: a long bound
      if (k >= CK_RING) ok = warp_wait(bar(B_RE + slot), (k / CK_RING - 1) & 1, D.status, dead, 30);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t dst = sbase + CK_OFF_RING + slot * CK_PIECE_BYTES;
        sts128(dst, make_uint4(pa.x, pa.y, pa.z, pa.w));
        sts128(dst + 16, make_uint4(pb.x, pb.y, pb.z, pb.w));
        arrive_local(bar(B_RF + slot));
      }
      __syncwarp();
      for (int pg = pb.x; pg < pb.y || pa.y < 0; ++pg, ++t) {
        const uint32_t ts = t % CK_TILES, dst = sbase + CK_OFF_TILES + ts * CK_PIECE_BYTES;
        if (((pg - pb.x) & 31) == 0)   // 32 block-table entries at a time, one per lane
          entries = pa.z >= 0 && pg + lane < pb.y ? __ldg(D.bt + (size_t)pa.z * D.max_pages + pg + lane) : -1;
        const int entry = __shfl_sync(0xffffffffu, entries, (pg - pb.x) & 31);
        int n_rows = pa.y < 0 ? -1 : pa.z >= 0 ? max(0, min(PAGE, pa.w - pg * PAGE)) : 0;
        const uint8_t* rows = kv;
        if (n_rows > 0) {
          if (entry >= 0 && entry < D.num_pages) {
            rows = kv + (size_t)entry * PAGE * ROW;
          } else {
            int err = HS_OK;
            rows = page_rows(D, A.layer, pa.z, pg, &err);
            if (!rows) {
              if (lane == 0) set_status(D.status, err);
              n_rows = 0;
            }
          }
        }
        if (t >= CK_TILES) ok = warp_wait(bar(B_TE + ts), (t / CK_TILES - 1) & 1, D.status, dead, 30);
        if (!ok) break;
        if (lane == 0) {
          const uint64_t at = reinterpret_cast<uint64_t>(rows);
          sts128(dst, make_uint4((uint32_t)at, (uint32_t)(at >> 32), (uint32_t)n_rows, pg == pb.x));
          sts128(dst + 16, make_uint4(pa.x, pa.y, 0, 0));
          arrive_local(bar(B_TF + ts));
        }
        __syncwarp();
        if (pa.y < 0) break;
      }
      if (!ok || pa.y < 0) break;
    }
    if (!SHARED && lane == 0 && rank == 0) work_at(A.work, A.pairs).cut[pair] = cut;
    } else if (warp == CK_MMA_WARP) {
    // ---------------------------------- MMA issue ----------------------------------
    if (rank == 0) {
      const uint32_t idesc_qk = idesc_f16(128, 64, false, false, false);
      const uint32_t idesc_pv = idesc_f16(128, 256, false, true, false);
      const uint32_t base = __shfl_sync(0xffffffffu, sbase, 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
      // low words of the descriptors of the operands' first parts; steps add address / 16
      const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 0, 1024) >> 32);
      uint32_t qd = (uint32_t)smem_desc_sw128(base + CK_OFF_Q, 16, 1024), kd = (uint32_t)smem_desc_sw128(base + CK_OFF_K, 16, 1024);
      uint32_t pd = (uint32_t)smem_desc_sw128(base + CK_OFF_P, 16, 1024), vd = (uint32_t)smem_desc_sw128(base + CK_OFF_V, CK_VATOM, 1024);
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const uint32_t slot = k % CK_RING;
        ok = warp_wait(bar(B_RF + slot), (k / CK_RING) & 1, D.status, dead, 30);
        if (!ok) break;
        const Piece p = piece_at(slot);
        const int n_tok = __shfl_sync(0xffffffffu, p.n_tok(), 0), n = __shfl_sync(0xffffffffu, p.pg1() - p.pg0(), 0);
        if (lane == 0) arrive_local(bar(B_RE + slot));
        __syncwarp();
        if (n_tok < 0) break;
        for (int i = 0; i <= n; ++i) {
          if (i < n) {
            const uint32_t t = it + i, st = t & 1;
            ok = warp_wait(bar(B_KF + st), (t >> 1) & 1, D.status, dead);
            if (!ok) break;
            tc_fence_after();
            asm volatile("" : "+r"(qd), "+r"(kd));   // the 36 descriptors are added up here, not kept in registers
            const uint32_t ks = kd + st * (CK_KSTAGE / 16);
            auto qk = [&](int g) {
#pragma unroll
              for (int kk = 0; kk < (g < 4 ? 8 : 4); ++kk) {
                const int atom = 2 * g + (kk >> 2);
                umma_f16_pair(tm + CK_TM_S + ((5 * t + g) & 7) * 32, qd + (atom * CK_QATOM + (kk & 3) * 32) / 16,
                              ks + (atom * CK_KATOM + (kk & 3) * 32) / 16, hi, idesc_qk, kk > 0);
              }
            };
            if (elect_lane()) {
              qk(0);
              qk(1);
              qk(2);
            }
            __syncwarp();
            // the other two take accumulators of the tile before, once its scores have been read
            if (t > 0) ok = warp_wait(bar(B_SR), (t - 1) & 1, D.status, dead);
            if (!ok) break;
            tc_fence_after();
            if (elect_lane()) {
              qk(3);
              qk(4);
              umma_commit_pair(bar(B_SD + st));
            }
            __syncwarp();
          }
          if (i > 0) {
            const uint32_t t = it + i - 1, st = t & 1;
            ok = warp_wait(bar(B_VF + st), (t >> 1) & 1, D.status, dead) &&
                 warp_wait(bar(B_PF + st), (t >> 1) & 1, D.status, dead);
            if (!ok) break;
            tc_fence_after();
            asm volatile("" : "+r"(pd), "+r"(vd));
            const uint32_t vs = vd + st * (CK_VSTAGE / 16);
            const uint32_t add = i > 1 ? 1u : 0u;
            if (elect_lane()) {
#pragma unroll
              for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_f16_pair(tm + CK_TM_O + g * 128, pd + kk * 2, vs + (g * 2 * CK_VATOM + kk * 2048) / 16, hi, idesc_pv,
                                kk > 0 ? 1u : add);
              umma_commit_pair(bar(B_PD + st));
            }
            __syncwarp();
          }
        }
        it += n;
      }
    }
    }
  } else if (warp >= CK_CONV_WARP0) {
    regs_inc<CK_CONV_REGS>();
    // ------------------------------ cache rows to operands ------------------------------
    const int ct = tid - CK_CONV_WARP0 * 32;
    bool bad_range = false;
    uint32_t it = 0;
    // the tile whose rows are in registers
    const uint8_t* rows = nullptr;
    int n_rows = 0, tok0 = 0, n_tok = 0;
    bool more = true, first = true;         // first: it begins a piece
    auto advance = [&](uint32_t t) {
      const uint32_t ts = t % CK_TILES, at = sbase + CK_OFF_TILES + ts * CK_PIECE_BYTES;
      more = warp_wait(bar(B_TF + ts), (t / CK_TILES) & 1, D.status, dead, 30);
      if (!more) return;
      const uint4 x = lds128(at);
      rows = reinterpret_cast<const uint8_t*>((uint64_t)x.x | (uint64_t)x.y << 32);
      n_rows = (int)x.z;
      first = x.w != 0;
      more = n_rows >= 0;
      if (first) {
        const uint4 y = lds128(at + 16);
        tok0 = (int)y.x, n_tok = (int)y.y;
      }
      __syncwarp();
      if (lane == 0) arrive_local(bar(B_TE + ts));
    };
    const float sign = A.scale_log2 < 0.f ? -1.f : 1.f;
    auto good_scale = [&](float s) {        // times the sign of sm_scale, for the scores
      if (fabsf(s) < CK_MAX_SCALE) return s * sign;
      bad_range = true;
      return 0.f;
    };
    // Q's rows, once the products of the previous piece have read theirs: copied as they are, then
    // each thread converts what it copied. Of 256 threads, a thread's next chunk is 3 rows and
    // 40 chunks on.
    int qr, qc;
    auto q_first = [&]() { qr = ct / 72, qc = ct % 72; };
    auto q_next = [&]() {
      qr += 3;
      qc += 40;
      if (qc >= 72) qc -= 72, ++qr;
    };
    auto q_at = [&]() { return sbase + CK_OFF_Q + (qc >> 3) * CK_QATOM + sw128_chunk(qr, qc & 7); };
    auto copy_q = [&]() {
      if (it > 0 && !ck_wait(bar(B_SD + ((it - 1) & 1)), ((it - 1) >> 1) & 1, D.status, dead)) return false;
      const T* q = static_cast<const T*>(A.q) + (long long)tok0 * A.q_tok;
      q_first();
#pragma unroll 1
      for (int k = 0; k < 18; ++k, q_next()) {
        const int gr = 2 * qr + (int)rank, tk = gr >> hs, h = gr & (H - 1);
        if (tk < n_tok) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(q_at()), "l"(q + tk * A.q_tok + h * A.q_head + qc * 8)
                       : "memory");
        } else {
          sts128(q_at(), make_uint4(0, 0, 0, 0));
        }
      }
      return true;
    };
    auto convert_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      bool bad = false;
      q_first();
      const int mine = (n_tok << hs) * 36;   // chunks of this CTA's rows that are a token's; the others are 0
#pragma unroll 1
      for (int k = 0; k * 256 < mine; k += 3) {
        uint32_t dst[3];
        uint4 v[3];
#pragma unroll
        for (int i = 0; i < 3; ++i, q_next()) {
          dst[i] = q_at();
          v[i] = lds128(dst[i]);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint4 f = q_to_f16<T>(v[i], &bad);
          if constexpr (!__is_same(T, __half)) sts128(dst[i], f);
        }
      }
      if (bad) {   // rare: which tokens' they are, for it is no error in one that sees nothing
        q_first();
#pragma unroll 1
        for (int k = 0; k < 18; ++k, q_next()) {
          bool here = false, ignore = false;
          q_to_f16<__half>(lds128(q_at()), &here);
          if (here) bad_range |= clamp_limit(D, __ldg(A.limit + tok0 + ((2 * qr + (int)rank) >> hs)), &ignore) > 0;
        }
      }
    };
    // K: 16-byte parts (16 codes) of this CTA's 32 rows: a warp has 16 parts of 8 rows, two rows at
    // a time, and 8 neighbouring threads 4 parts of two rows, whose chunks of fp16 (a part is two)
    // the swizzle puts on 8 different bank groups. (128 contiguous bytes per 8 threads read with a
    // third fewer L1 wavefronts, but need the chunks of half the threads exchanged: 1 % slower.)
    // V: the 16 parts of the groups 2 rank and 2 rank + 1 of all 64 rows: the warps that have
    // them for this CTA's rows take them again, the others read the other half page's.
    const uint32_t kf0 = mapa(bar(B_KF), 0), vf0 = mapa(bar(B_VF), 0);   // the first CTA's
    const int cw = ct >> 5, pv = 4 * (lane >> 3) + (lane & 3), row0 = 8 * (cw >> 1) + ((lane >> 2) & 1);   // rows row0 + 2 k
    const bool own_v = (cw & 1) == (int)rank;
    const int part = 16 * (cw & 1) + pv, base_row = (int)rank * 32, rope_row = ct >> 3;
    const int row_v = (own_v ? base_row : 32 - base_row) + row0;
    const uint32_t k_at = (part >> 2) * CK_KATOM + sw128_chunk(row0, (pv & 3) * 2),
                   rope_at = 8 * CK_KATOM + sw128_chunk(rope_row, ct & 7),
                   v_at = (pv >> 2) * CK_VATOM + sw128_chunk(row_v, (pv & 3) * 2);
    const uint32_t src = (base_row + row0) * ROW + part * 16, src_v = row_v * ROW + (16 * (int)rank + pv) * 16,
                   src_rope = (base_row + rope_row) * ROW + (33 + (ct & 7)) * 16, src_sc = (ct & 63) * ROW + LATENT;
    const uint32_t sc_v = sbase + CK_OFF_SCL + (2 * (int)rank + (pv >> 3)) * CK_SCL_G + scale_place<SHARED>(row_v) * 4;
    const uint4 z = make_uint4(0, 0, 0, 0);
    uint4 own[4], val[4], rope = z, sc = z;
    auto ld16 = [&](uint32_t at) { return __ldg(reinterpret_cast<const uint4*>(rows + at)); };
    auto load_k = [&]() {
      if (n_rows == PAGE) {
#pragma unroll
        for (int k = 0; k < 4; ++k) own[k] = ld16(src + k * 2 * ROW);
        rope = ld16(src_rope);
        if (ct < PAGE) sc = ld16(src_sc);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) own[k] = base_row + row0 + 2 * k < n_rows ? ld16(src + k * 2 * ROW) : z;
        rope = base_row + rope_row < n_rows ? ld16(src_rope) : z;
        if (ct < PAGE) sc = ct < n_rows ? ld16(src_sc) : z;
      }
    };
    auto load_v = [&]() {
      if (own_v) return;
      if (n_rows == PAGE) {
#pragma unroll
        for (int k = 0; k < 4; ++k) val[k] = ld16(src_v + k * 2 * ROW);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) val[k] = row_v + 2 * k < n_rows ? ld16(src_v + k * 2 * ROW) : z;
      }
    };
    advance(0);
    if (more) {
      load_k();
      load_v();
      copy_q();   // nothing to wait for: on its way while K is converted
    }
    while (more) {
      const uint32_t st = it & 1;
      // the softmax has read the scales of four tiles before
      if (ct < PAGE && it >= CK_SCL && !ck_wait(bar(B_SE + it % CK_SCL), (it / CK_SCL - 1) & 1, D.status, dead)) return;
      if (it >= 2 && !ck_wait(bar(B_SD + st), ((it - 2) >> 1) & 1, D.status, dead)) return;
      if (ct < PAGE) {
        const uint32_t x = sbase + CK_OFF_SCL + (it % CK_SCL) * CK_SCL_T + scale_place<SHARED>(ct) * 4;
        sts32(x, __float_as_uint(good_scale(__uint_as_float(sc.x))));
        sts32(x + CK_SCL_G, __float_as_uint(good_scale(__uint_as_float(sc.y))));
        sts32(x + 2 * CK_SCL_G, __float_as_uint(good_scale(__uint_as_float(sc.z))));
        sts32(x + 3 * CK_SCL_G, __float_as_uint(good_scale(__uint_as_float(sc.w))));
        if (ct == 0) sts32(there + (it % CK_SCL) * 4, n_rows > 0);
        __syncwarp();
        if (lane == 0) arrive_local(bar(B_SC + it % CK_SCL));
      }
      const uint32_t kt = sbase + CK_OFF_K + st * CK_KSTAGE;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 lo, hi;
        codes_to_f16(own[k], lo, hi);
        const uint32_t d = (kt + k_at + k * 256) ^ (k * 32);
        sts128(d, lo);
        sts128(d ^ 16, hi);
      }
      {
        const uint32_t w[4] = {rope.x, rope.y, rope.z, rope.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = h2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)));
        // bf16 magnitudes of 0x4780 = 65,536 and above, infinities and NaN carry into bit 15
        const uint32_t m = 0x7FFF7FFFu, c = 0x38803880u;
        bad_range |= ((((w[0] & m) + c) | ((w[1] & m) + c) | ((w[2] & m) + c) | ((w[3] & m) + c)) & 0x80008000u) != 0;
        sts128(kt + rope_at, make_uint4(o[0], o[1], o[2], o[3]));
      }
      if (first) {
        if (it > 0 && !copy_q()) return;
        convert_q();
      }
      // the stores complete behind the wait for the next tile's place, and V's behind the next loads:
      // the fences then wait 200 cycles less each (3 % of a long call)
      advance(it + 1);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(kf0 + 8 * st);
      if (own_v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) val[k] = own[k];
      }
      if (more) load_k();
      if (it >= 2 && !ck_wait(bar(B_PD + st), ((it - 2) >> 1) & 1, D.status, dead)) return;
      if (!ck_wait(bar(B_SC + it % CK_SCL), (it / CK_SCL) & 1, D.status, dead)) return;
      const uint32_t vt = sbase + CK_OFF_V + st * CK_VSTAGE + v_at, scv = sc_v + (it % CK_SCL) * CK_SCL_T;
      uint32_t sv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) sv[k] = lds32(scv + k * (SHARED ? 16 : 8));   // of rows row_v + 2 k
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 lo, hi;
        codes_to_scaled_f16(val[k], __uint_as_float(sv[k]) * sign, lo, hi);
        const uint32_t d = (vt + k * 256) ^ (k * 32);
        sts128(d, lo);
        sts128(d ^ 16, hi);
      }
      if (more) load_v();
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(vf0 + 8 * st);
      ++it;
    }
    if (bad_range) set_status(D.status, HS_ERR_RANGE);
  } else {
    // ------------------------------ softmax and output ------------------------------
    // four warps of 32 rows: `half` (tensor-memory lanes 64 half ..) and `sub` (columns). A thread has one row and the
    // warp's 16 keys. SHARED, where blocks are full: four keys of four rows, so that it needs 16 scales, not 64, and keeps
    // the reference of one of them, `mine` (lane 4 k + i of the four rows k + 8 i); in the output its row is `row`,
    // whose keeper is lane `keeper`. (8 x 129 tokens of 20,001 rows 3.40 -> 3.27 ms, and 753 of 74,913 without
    // groups 8.85 -> 8.53 ms, but 32 single tokens, whose blocks are half empty, 770 -> 829 us.)
    const int quad = warp & 3, sub = warp >> 2, half = quad >> 1, row0 = (quad & 1) * 32, row = row0 + lane;
    const int mine = SHARED ? row0 + (lane >> 2) + 8 * (lane & 3) : row, keeper = 4 * (lane & 7) + (lane >> 3), four = lane & ~3;
    const int key0 = half * 32 + sub * 16;       // the warp's 16 keys of the page
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_col = lanes + CK_TM_S + sub * 16, o_col = lanes + CK_TM_O + sub * 128;
    const uint32_t pf0 = mapa(bar(B_PF), 0), sr0 = mapa(bar(B_SR), 0);
    const uint32_t p_lo = sbase + CK_OFF_P + sw128_chunk(row, key0 >> 3),
                   p_hi = sbase + CK_OFF_P + sw128_chunk(row, (key0 >> 3) + 1);
    const int gr = 2 * row + (int)rank, tk = gr >> hs, h = gr & (H - 1), tk_mine = (2 * mine + (int)rank) >> hs;
    const uint32_t red_row = sbase + CK_OFF_RED + mine * 4, red_mine = red_row + (half * 2 + sub) * 256;
    auto red_at = [&](uint32_t at) { return __uint_as_float(lds32(at)); };
    uint32_t it = 0;
    // s is held times the sign of sm_scale (in the scales, and here for the rope), so that its
    // maximum is the maximum of z; a scale of 0 becomes one that leaves every z at 0 but that
    // of an unseen key, -inf
    const float scale = fmaxf(fabsf(A.scale_log2), 1e-37f), sign = A.scale_log2 < 0.f ? -1.f : 1.f;
    bool ok = true, dead_all = false, bad_range = false;
    for (uint32_t kp = 0;; ++kp) {
      const uint32_t slot = kp % CK_RING;
      ok &= ck_wait(bar(B_RF + slot), (kp / CK_RING) & 1, D.status, dead, 30);
      if (bar_any(2 + (quad & 1), CK_SM / 2, !ok)) break;
      const Piece P = piece_at(slot);
      __syncwarp();
      if (lane == 0) arrive_local(bar(B_RE + slot));
      if (P.n_tok() < 0) break;
      const bool live = tk < P.n_tok();
      int lim = 0;   // of row `mine`
      if ((SHARED ? tk_mine < P.n_tok() : live) && P.req() >= 0) {
        bool ignore = false;
        lim = clamp_limit(D, __ldg(A.limit + P.tok0() + (SHARED ? tk_mine : tk)), &ignore);
        if constexpr (SHARED) lim = min(lim, P.b.w);
      }
      if (SHARED && tk_mine >= P.n_tok()) lim = CK_NO_CAP;   // a row of no token, whose queries are 0, need not be masked
      if ((2 * (quad & 1) * 32 + (int)rank) >> hs >= P.n_tok()) {
        // none of these 32 rows is a token's (nor of the other three warps'): their P is 0, and
        // what the products make of it is not read
        sts128(p_lo, make_uint4(0, 0, 0, 0));
        sts128(p_hi, make_uint4(0, 0, 0, 0));
        fence_proxy_async();
        for (int pg = P.pg0(); pg < P.pg1(); ++pg, ++it) {
          const uint32_t st = it & 1;
          ok &= ck_wait(bar(B_SD + st), (it >> 1) & 1, D.status, dead);
          __syncwarp();
          if (lane == 0) {
            arrive_cluster(sr0);
            arrive_local(bar(B_SE + it % CK_SCL));
            arrive_cluster(pf0 + 8 * st);
          }
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        if (it > 0) ok &= ck_wait(bar(B_PD + ((it - 1) & 1)), ((it - 1) >> 1) & 1, D.status, dead);
        continue;
      }
      float m = -INFINITY;   // the reference of row `mine` (in its four warps alike)
      float l = 0.f;         // this thread's sum; SHARED: of its four rows
      F2 sum[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
      // of one value for each of the four rows in four lanes, what the lanes make of row `mine`
      auto join4 = [&](const float (&r)[4], auto op) {
        const bool hi = lane & 2, lo = lane & 1;
        const float a = op(hi ? r[2] : r[0], __shfl_xor_sync(0xffffffffu, hi ? r[0] : r[2], 2));
        const float b = op(hi ? r[3] : r[1], __shfl_xor_sync(0xffffffffu, hi ? r[1] : r[3], 2));
        return op(lo ? b : a, __shfl_xor_sync(0xffffffffu, lo ? a : b, 1));
      };
      for (int pg = P.pg0(); pg < P.pg1(); ++pg, ++it) {
        const uint32_t st = it & 1;
        ok &= ck_wait(bar(B_SC + it % CK_SCL), (it / CK_SCL) & 1, D.status, dead);   // over long before the products are
        uint4 x0, x1, x2, x3;
        if constexpr (SHARED) {   // this thread's scales, before the scores are waited for
          const uint32_t sc = sbase + CK_OFF_SCL + (it % CK_SCL) * CK_SCL_T + key0 * 4 + (lane & 3) * 16;
          x0 = lds128(sc), x1 = lds128(sc + CK_SCL_G), x2 = lds128(sc + 2 * CK_SCL_G), x3 = lds128(sc + 3 * CK_SCL_G);
        }
        ok &= ck_wait(bar(B_SD + st), (it >> 1) & 1, D.status, dead);
        tc_fence_after();
        F2 s2[8];   // scores, times the sign of sm_scale, in pairs of keys; SHARED: row i's of keys 2 c, 2 c + 1, then 8 + 2 c, 9 + 2 c
        float s[16];
        if constexpr (SHARED) {
          auto add_group = [&](const uint32_t* a, const uint4& x, bool set) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* v = a + 8 * (i >> 1) + 2 * (i & 1);
              const F2 p = f2(v[0], v[1]), q = f2(v[4], v[5]);
              s2[2 * i] = set ? mul2(f2(x.x, x.y), p) : fma2(f2(x.x, x.y), p, s2[2 * i]);
              s2[2 * i + 1] = set ? mul2(f2(x.z, x.w), q) : fma2(f2(x.z, x.w), q, s2[2 * i + 1]);
            }
          };
          {
            uint32_t a[48];
#pragma unroll
            for (int g = 0; g < 3; ++g) tmem_ld_frag16(s_col + ((5 * it + g) & 7) * 32, a + 16 * g);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 3; ++g) add_group(a + 16 * g, g == 0 ? x0 : g == 1 ? x1 : x2, g == 0);
          }
          {
            uint32_t a[32];
            tmem_ld_frag16(s_col + ((5 * it + 3) & 7) * 32, a);
            tmem_ld_frag16(s_col + ((5 * it + 4) & 7) * 32, a + 16);
            tmem_wait_ld();
            add_group(a, x3, false);
            const uint32_t one = __float_as_uint(sign);
            add_group(a + 16, make_uint4(one, one, one, one), false);
#pragma unroll
            for (int j = 0; j < 8; ++j) unpack(s2[j], s[2 * j], s[2 * j + 1]);
          }
        } else {
          const uint32_t sc = sbase + CK_OFF_SCL + (it % CK_SCL) * CK_SCL_T + key0 * 4;
          {
            uint32_t a[48];
#pragma unroll
            for (int g = 0; g < 3; ++g) tmem_ld16(s_col + ((5 * it + g) & 7) * 32, *reinterpret_cast<uint32_t(*)[16]>(a + 16 * g));
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 3; ++g)
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const uint4 x = lds128(sc + g * CK_SCL_G + j * 4);
                const uint32_t* v = a + 16 * g + j;
                s2[j / 2] = g == 0 ? mul2(f2(x.x, x.y), f2(v[0], v[1])) : fma2(f2(x.x, x.y), f2(v[0], v[1]), s2[j / 2]);
                s2[j / 2 + 1] = g == 0 ? mul2(f2(x.z, x.w), f2(v[2], v[3])) : fma2(f2(x.z, x.w), f2(v[2], v[3]), s2[j / 2 + 1]);
              }
          }
          {
            uint32_t a[32];
            tmem_ld16(s_col + ((5 * it + 3) & 7) * 32, *reinterpret_cast<uint32_t(*)[16]>(a));
            tmem_ld16(s_col + ((5 * it + 4) & 7) * 32, *reinterpret_cast<uint32_t(*)[16]>(a + 16));
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const uint4 x = lds128(sc + 3 * CK_SCL_G + j * 4);
              s2[j / 2] = fma2(f2(x.x, x.y), f2(a[j], a[j + 1]), s2[j / 2]);
              s2[j / 2 + 1] = fma2(f2(x.z, x.w), f2(a[j + 2], a[j + 3]), s2[j / 2 + 1]);
            }
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              s2[j / 2] = fma2(f2(a[16 + j], a[17 + j]), f2(sign), s2[j / 2]);
              unpack(s2[j / 2], s[j], s[j + 1]);
            }
          }
        }
        const int seen = lds32(there + (it % CK_SCL) * 4) ? lim - pg * PAGE - key0 : 0;   // of the warp's keys, by row `mine`
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {   // the score accumulators may be written again, and the scales
          arrive_cluster(sr0);
          arrive_local(bar(B_SE + it % CK_SCL));
        }
        float mt;
        if constexpr (SHARED) {
          if (__any_sync(0xffffffffu, seen < 16)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = __shfl_sync(0xffffffffu, seen, four + i) - 2 * (lane & 3);
#pragma unroll
              for (int j = 0; j < 4; ++j) s[4 * i + j] = (j & 1) + 8 * (j >> 1) < n ? s[4 * i + j] : -INFINITY;
            }
          }
          float r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = max_nan(max3_nan(s[4 * i], s[4 * i + 1], s[4 * i + 2]), s[4 * i + 3]);
          if (!(max_nan(max3_nan(r[0], r[1], r[2]), r[3]) * scale < CK_MAX_Z)) {   // a value that is not finite (or a query beyond fp16), or too large a score: not seen
            bad_range = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[i] = -INFINITY;
#pragma unroll
              for (int j = 4 * i; j < 4 * i + 4; ++j) {
                if (!(s[j] * scale < CK_MAX_Z)) s[j] = -INFINITY;
                r[i] = fmaxf(r[i], s[j]);
              }
            }
          }
          mt = join4(r, [](float a, float b) { return fmaxf(a, b); });
        } else {
          if (seen < 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] = j < seen ? s[j] : -INFINITY;
          }
          mt = max_nan(s[0], s[1]);
#pragma unroll
          for (int j = 2; j < 16; j += 2) mt = max3_nan(mt, s[j], s[j + 1]);
          if (!(mt * scale < CK_MAX_Z)) {   // a value that is not finite (or a query beyond fp16), or too large a score: not seen
            bad_range = true;
            mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (!(s[j] * scale < CK_MAX_Z)) s[j] = -INFINITY;
              mt = fmaxf(mt, s[j]);
            }
          }
        }
        const uint32_t buf = (it & 1) * 1024;
        sts32(red_mine + buf, __float_as_uint(mt));
        if (bar_any(2 + (quad & 1), CK_SM / 2, !ok)) {   // the four warps of these 32 rows
          dead_all = true;
          break;
        }
        mt = fmaxf(fmaxf(red_at(red_row + buf), red_at(red_row + buf + 256)), fmaxf(red_at(red_row + buf + 512), red_at(red_row + buf + 768)));
        mt *= scale;
        float f = 1.f;
        if (mt > m + CK_RESCALE_LOG2) {   // also the first finite maximum, when m is -inf
          f = ex2_approx(m - mt);
          m = mt > CK_LOW_Z ? mt : CK_LOW;
        }
        const float off = m > CK_LOW_Z ? CK_P_SHIFT - m : 0.f;   // no score beside which one counts: every weight is 0
        uint32_t ph[8];
        if constexpr (SHARED) {
          if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = mul2(sum[i], f2(__shfl_sync(0xffffffffu, f, four + i)));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 o2 = f2(__shfl_sync(0xffffffffu, off, four + i));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float p0, p1;
              unpack(fma2(f2(__float_as_uint(s[4 * i + 2 * j]), __float_as_uint(s[4 * i + 2 * j + 1])), f2(scale), o2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              sum[i] = fma2(f2(__float_as_uint(p0), __float_as_uint(p1)), f2(1.f), sum[i]);
              ph[4 * j + i] = h2_bits(__floats2half2_rn(p0, p1));   // of keys 0 .. 7, then 8 .. 15
            }
          }
        } else {
          F2 ls2 = f2(0.f);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float p0, p1;
            unpack(fma2(f2(__float_as_uint(s[j]), __float_as_uint(s[j + 1])), f2(scale), f2(off)), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            ls2 = fma2(f2(__float_as_uint(p0), __float_as_uint(p1)), f2(1.f), ls2);
            ph[j >> 1] = h2_bits(__floats2half2_rn(p0, p1));
          }
          float ls, ls_hi;
          unpack(ls2, ls, ls_hi);
          ls += ls_hi;
          l = l * f + ls;
        }
        // PV(t - 1) has read P and written O
        if (it > 0) ok = ck_wait(bar(B_PD + ((it - 1) & 1)), ((it - 1) >> 1) & 1, D.status, dead);
        tc_fence_after();
        if (pg > P.pg0() && __any_sync(0xffffffffu, f != 1.f)) {
          if constexpr (SHARED) f = __shfl_sync(0xffffffffu, f, keeper);
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_col + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(o_col + c, o);
          }
          tmem_wait_st();
        }
        if constexpr (SHARED) {
          __syncwarp();
          store_frag4(p_lo, ph);
          store_frag4(p_hi, ph + 4);
        } else {
          sts128(p_lo, make_uint4(ph[0], ph[1], ph[2], ph[3]));
          sts128(p_hi, make_uint4(ph[4], ph[5], ph[6], ph[7]));
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(pf0 + 8 * st);
      }
      // left at the barrier above, the four warps of a row alike, or at the piece's end: then one more
      if (dead_all) break;
      ok &= ck_wait(bar(B_PD + ((it - 1) & 1)), ((it - 1) >> 1) & 1, D.status, dead);
      tc_fence_after();
      const uint32_t buf = (it & 1) * 1024;
      if constexpr (SHARED) {
        float r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float hi;
          unpack(sum[i], r[i], hi);
          r[i] += hi;
        }
        l = join4(r, [](float a, float b) { return a + b; });
      }
      sts32(red_mine + buf, __float_as_uint(l));
      if (bar_any(2 + (quad & 1), CK_SM / 2, !ok)) break;
      l = (red_at(red_row + buf) + red_at(red_row + buf + 256)) + (red_at(red_row + buf + 512) + red_at(red_row + buf + 768));
      if constexpr (SHARED) {   // from row `mine` to row `row`
        l = __shfl_sync(0xffffffffu, l, keeper);
        m = __shfl_sync(0xffffffffu, m, keeper);
      }
      l *= CK_V_FACTOR;   // as O
      m -= CK_P_SHIFT + CK_V_SHIFT;
      const int dim = (2 * half + sub) * 128;      // this thread's output dims
      if (P.slot() < 0) {
        if (only_low(m)) l = 0.f, bad_range = true;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        // 16 columns at a time through this warp's quarter of its rows' P (free until the next
        // exchange of maxima), so that two lanes store 32 bytes of one row
        const uint32_t stage = sbase + CK_OFF_P + (quad & 1) * 4096 + (half * 2 + sub) * 1024;
        const uint32_t put = stage + lane * 32 + ((lane >> 2) & 1) * 16;
        T* const out0 = static_cast<T*>(A.out) + dim + (lane & 1) * 8;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          uint32_t o[16];
          tmem_ld16(o_col + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint4 v;
            v.x = pack2<T>(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv);
            v.y = pack2<T>(__uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
            v.z = pack2<T>(__uint_as_float(o[j + 4]) * inv, __uint_as_float(o[j + 5]) * inv);
            v.w = pack2<T>(__uint_as_float(o[j + 6]) * inv, __uint_as_float(o[j + 7]) * inv);
            sts128(put ^ (j * 2), v);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = (lane >> 1) + 16 * i, g = 2 * ((quad & 1) * 32 + r) + (int)rank, k = g >> hs;
            const uint4 v = lds128(stage + r * 32 + (((lane & 1) ^ ((r >> 2) & 1)) * 16));
            if (k < P.n_tok())
              *reinterpret_cast<uint4*>(out0 + (P.tok0() + (long long)k) * A.o_tok + (g & (H - 1)) * A.o_head + c) = v;
          }
          __syncwarp();
        }
        if (A.lse && live && dim == 0)
          A.lse[(size_t)(P.tok0() + tk) * H + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      } else {
        float* part;
        float2* stats;
        size_t at = ((size_t)pair * 2 + P.slot()) * CK_ROWS + gr;
        if constexpr (SHARED) {
          const SharedWork W = shared_work(A, H);
          const bool whole = P.slot() >= 2;
          part = whole ? W.whole : W.part;
          stats = whole ? W.whole_stats : W.stats;
          if (whole) at = ((size_t)(P.slot() - 2) * A.n_tok + P.tok0()) * H + gr;
        } else {
          const ChunkWork W = work_at(A.work, A.pairs);
          part = W.part;
          stats = W.stats;
        }
        uint4* const dst = reinterpret_cast<uint4*>(part) + part_unit(at, dim / 4);
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          uint32_t o[16];
          tmem_ld16(o_col + c, o);
          tmem_wait_ld();
          if (live) {
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[(c / 4 + j) * 4] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        if (live && dim == 0) stats[at] = make_float2(m, l);
      }
      tc_fence_before();   // O may be written again once the next tile's P has arrived
    }
    if (bad_range) set_status(D.status, HS_ERR_RANGE);
  }
  __syncthreads();
  if (rank == 0 && warp == CK_MMA_WARP) {   // every issued MMA has completed before TMEM is freed
    if (elect_lane()) umma_commit_own(bar(B_FIN));
    __syncwarp();
    for (int i = 0; i < 4096 && !try_wait(bar(B_FIN), 0); ++i) __nanosleep(200);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // neither CTA's memory is touched by the other any more
  tc_fence_after();
  if (warp == CK_MMA_WARP) tmem_dealloc_pair(tmem, 512);
}

constexpr int CM_SLICES = 4, CM_THREADS = 128 * CM_SLICES;   // of the kernels that join parts

template <typename T, bool SHARED>
inline hs_status launch_attention_pairs(hs_pool* p, const ChunkArgs& a, cudaStream_t st) {
  if (ensure_kernel_attrs(chunk_attention_kernel<T, SHARED>, CK_SMEM) != HS_OK) return HS_ERR_CUDA;
  // the register shares were counted against a launch of CK_REGS per thread
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, chunk_attention_kernel<T, SHARED>) != cudaSuccess) return HS_ERR_CUDA;
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < CK_REGS) return HS_ERR_CUDA;
  return launch_pdl(chunk_attention_kernel<T, SHARED>, dim3(2 * a.pairs), dim3(CK_THREADS), CK_SMEM, st, 2, p->d, a);
}

inline bool stride_ok(int64_t s, int64_t least) { return s >= least && s < (1ll << 40) && s % 8 == 0; }

// The checks that both calls share; need: bytes of workspace.
inline hs_status check_attention(hs_pool* p, int32_t layer, int32_t n_seg, const int32_t* d_seg_req, const int32_t* d_seg_start, int32_t n,
                          int32_t most_tokens, const int32_t* d_limit, int32_t dtype, const void* d_q, int64_t q_tok,
                          int64_t q_head, float sm_scale, const void* d_out, int64_t o_tok, int64_t o_head, const float* d_lse,
                          const void* d_work, int64_t work_bytes, int64_t need) {
  if (!p || layer < 0 || layer >= p->cfg.n_layers || n_seg < 0 || n_seg > HS_CHUNK_MAX_SEGMENTS || n < 0 || n > most_tokens ||
      (dtype != HS_BF16 && dtype != HS_FP16) || !on_pool_device(p))
    return HS_ERR_INVALID;
  if (n == 0 || n_seg == 0) return HS_OK;
  const auto aligned = [](const void* x) { return x && (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (!d_seg_req || !d_seg_start || !d_limit || !aligned(d_q) || !aligned(d_out) || !aligned(d_work) || !words_ok(d_seg_req) ||
      !words_ok(d_seg_start) || !words_ok(d_limit) || !words_ok(d_lse) || work_bytes < need ||
      !(fabsf(sm_scale) <= CK_MAX_SM_SCALE))
    return HS_ERR_INVALID;
  if (!stride_ok(q_tok, 0) || !stride_ok(q_head, 0) || !stride_ok(o_tok, LATENT) || !stride_ok(o_head, LATENT))
    return HS_ERR_INVALID;
  return HS_OK;
}

inline int chunk_pairs() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }

}  // namespace

}  // namespace hs
