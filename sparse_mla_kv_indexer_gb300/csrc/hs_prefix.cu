// Attention of requests that share their first positions: which blocks there are, the join of a token's two
// parts, and the call. The kernel is hs_chunk_kernel.cuh's, which reads its blocks from the list made here.
//
// With q a token and head, S the shared positions and R its own, and n, l, o of each part relative to its own
// maximum m:   out = (2^(m_S - m) o_S + 2^(m_R - m) o_R) / (2^(m_S - m) l_S + 2^(m_R - m) l_R),  m = max(m_S, m_R).
// The rows S are converted to the products' operands once for 128 / H tokens of the group, instead of once for each
// segment: of 96 single tokens with 16 heads an eighth of the tiles. With 64 heads two tokens fill a block.
//
// Measured on a GB300: 64 single tokens behind 32,768 shared rows, 64 heads, 370 us (hs_chunk_attention for the same
// tokens 676 us), of which the plan 5, the attention 355 (223 tiles a pair of 1.48 us, 11 us before the first), the
// join 10; 96 behind 131,009 rows, 16 heads, 547 us (3.93 ms). The products' floors are 154 and 229 us: what bounds
// it is the tile's work around them, as hs_chunk_kernel.cuh has it.
#include "hs_chunk_kernel.cuh"

namespace hs {

namespace {

// ---- requests that share their first positions ------------------------------------------
// The blocks of hs_prefix_attention. A group's whole shared pages are a unit of all its tokens, whatever
// segments they are of; the other pages are a unit per segment. Each unit is cut into blocks of 128 / H
// tokens.
// When it pays. Reading a group's shared pages once saves the tiles of (sum of ceil(t_i / tpb) - ceil(sum
// t_i / tpb)) blocks over them (t_i: tokens of its segments, tpb: tokens of a block). It costs each of the
// shared blocks its start and queries, PP_START pages, and every row two partial sums that are written and read again,
// PP_ROWS pages for 128 rows. A group that saves less, like long segments of 64 heads whose blocks are full anyway, is
// read by each segment alone. Measured, shared against alone, below the border and on it, where what is saved is
// what it costs: 200 groups of two single tokens, 16 heads, 5 pages 86 and 84 us, 6 pages 88 and 94; 200 of four single
// tokens, 64 heads, 13 pages 296 and 288, 14 pages 304 and 315; 100 of three times five tokens, 32 heads, 24 pages 363
// and 362, 27 pages 390 and 401.
constexpr int PP_START = 3, PP_ROWS = 11;
constexpr int PP_LIMITS = 4096;    // limits of so many tokens are kept in shared memory
// The plan's threads: 256 for so many segments, groups and blocks, else 1,024. The whole call with either: of 7 blocks at
// most 20.6 and 21.5 us, of 162 38.5 and 39.5, of 271 44.2 and 44.5, of 645 83.7 and 81.4, of 1,051 112 and 102.
constexpr int PP_FEW = 256;
// shared memory, in ints: segment starts [n_seg + 1], requests [n_seg] and shared pages [n_seg], group starts
// [n_groups + 1], lengths [n_groups] and the segment through whose request each group reads [n_groups], blocks before
// each unit [n_groups + n_seg + 1], limits
inline int plan_ints(int n_seg, int n_groups, int n_tok) {
  return 4 * n_seg + 4 * n_groups + 3 + (n_tok <= PP_LIMITS ? n_tok : 0);
}

// Clamps the values v[0 .. n) to [0, most] and to ascend. All threads; returns whether some of this thread's were not.
template <int THREADS>
__device__ __forceinline__ bool clamp_starts(int* v, int n, int most, int* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  int before = 0;
  for (int base = 0; base < n; base += THREADS) {
    const int i = base + threadIdx.x, s = i < n ? v[i] : 0;
    int m = min(max(s, 0), most);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m = max(m, u);
    }
    if (lane == 31) tmp[warp] = m;
    __syncthreads();
    int w = lane < THREADS / 32 ? tmp[lane] : 0;
    const int all = __reduce_max_sync(0xffffffffu, w);
    if (lane >= warp) w = 0;
    m = max(max(m, before), __reduce_max_sync(0xffffffffu, w));
    before = max(before, all);
    if (i < n) {
      bad |= s != m;
      v[i] = m;
    }
    __syncthreads();
  }
  return bad;
}
// Exclusive sum over the CTA's threads; *total the whole.
template <int THREADS>
__device__ __forceinline__ int plan_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  const int w = lane < THREADS / 32 ? tmp[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, w);
  const int ahead = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  __syncthreads();
  return s - v + ahead;
}

// Where the parts of one of a token's blocks lie, in one word (0: there are none, or the attention wrote the
// output itself): a whole block's in the rows of all tokens, a cut one's in the slots of n pairs from `first` on,
// at the token's place in its block.
struct ToJoin {
  int n, first, place;
  bool whole;
};
__device__ __forceinline__ int join_word(const ToJoin& j) { return j.n | j.first << 12 | j.place << 24 | (j.whole ? 1 << 30 : 0); }
__device__ __forceinline__ ToJoin join_of(int w) { return {w & 0xFFF, w >> 12 & 0xFFF, w >> 24 & 0xF, (w >> 30 & 1) != 0}; }

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) prefix_plan_kernel(const Dev D, const ChunkArgs A) {
  extern __shared__ int plan[];
  __shared__ int tmp[32];
  griddep_wait();
  griddep_launch();   // only the attention of this call depends on it, and waits for its end
  const int tid = threadIdx.x, tpb = CK_ROWS / D.n_heads, units = A.n_groups + A.n_seg;
  int* const start = plan;
  int* const req = start + A.n_seg + 1;
  int* const shared = req + A.n_seg;
  int* const group = shared + A.n_seg;
  int* const length = group + A.n_groups + 1;
  int* const reader = length + A.n_groups;
  int* const before = reader + A.n_groups;
  int* const limits = before + units + 1;
  const bool kept = A.n_tok <= PP_LIMITS;
  const SharedWork W = shared_work(A, D.n_heads);
  // everything that the plan goes by, read at once
  for (int i = tid; i <= A.n_seg; i += THREADS) {
    start[i] = __ldg(A.seg_start + i);
    if (i < A.n_seg) req[i] = __ldg(A.seg_req + i), shared[i] = 0;
  }
  if (A.n_groups > 0)
    for (int i = tid; i <= A.n_groups; i += THREADS) {
      group[i] = __ldg(A.group_start + i);
      if (i < A.n_groups) length[i] = __ldg(A.group_len + i);
    }
  if (kept)
    for (int j = tid; j < A.n_tok; j += THREADS) limits[j] = __ldg(A.limit + j);
  for (int j = tid; j < A.n_tok; j += THREADS) W.of_token[j] = make_int2(0, 0);
  __syncthreads();
  bool bad = clamp_starts<THREADS>(start, A.n_seg + 1, A.n_tok, tmp);
  if (A.n_groups > 0) bad |= clamp_starts<THREADS>(group, A.n_groups + 1, A.n_seg, tmp);
  auto blocks_of = [&](int tokens) { return (tokens + tpb - 1) / tpb; };
  // the groups that share, a warp each
  for (int g = tid >> 5; g < A.n_groups; g += THREADS / 32) {
    const int lane = tid & 31, s0 = group[g], s1 = group[g + 1], len = length[g];
    const bool fits = len >= 0 && len <= D.max_ctx;
    bad |= !fits;
    int alone = 0, first = A.n_seg;
    bool valid = true;   // a segment of a bad request sees nothing, and so shares nothing
    for (int i = s0 + lane; i < s1; i += 32) {
      const int n = blocks_of(start[i + 1] - start[i]), r = req[i];
      alone += n;
      if (n > 0) first = min(first, i), valid &= r >= 0 && r < D.max_requests;
    }
    alone = __reduce_add_sync(0xffffffffu, alone);
    first = __reduce_min_sync(0xffffffffu, first);
    valid = __all_sync(0xffffffffu, valid);
    const int tokens = start[s1] - start[s0], together = blocks_of(tokens), pages = fits && valid ? len / PAGE : 0;
    const bool pays = (long long)(alone - together) * pages >= together * PP_START + (tokens * D.n_heads * PP_ROWS + CK_ROWS - 1) / CK_ROWS;
    if (lane == 0) reader[g] = first, before[g] = pays ? together : 0;
    if (pays)
      for (int i = s0 + lane; i < s1; i += 32) shared[i] = pages;
  }
  for (int i = tid; i < A.n_seg; i += THREADS) before[A.n_groups + i] = blocks_of(start[i + 1] - start[i]);
  __syncthreads();
  int n_blocks = 0;
  for (int base = 0; base < units; base += THREADS) {
    const int u = base + tid, v = u < units ? before[u] : 0;
    int sum;
    const int at = plan_scan<THREADS>(v, tmp, &sum);
    if (u < units) before[u] = n_blocks + at;
    n_blocks += sum;
  }
  if (tid == 0) before[units] = n_blocks;
  __syncthreads();
  int cost = 0;
  PlanBlock B;
  for (int base = 0; base < n_blocks; base += THREADS) {
    const int b = base + tid;
    B = {make_int4(0, 0, -1, 0), make_int4(0, 0, CK_NO_CAP, 0)};
    if (b < n_blocks) {
      int l = 0, h = units;   // the last unit whose first block is <= b (never one without blocks)
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (before[mid] <= b) l = mid; else h = mid;
      }
      const bool of_group = l < A.n_groups;
      const int seg = of_group ? reader[l] : l - A.n_groups, end = start[of_group ? group[l + 1] : seg + 1];
      const int pages = shared[seg], r = req[seg];
      const bool bad_req = r < 0 || r >= D.max_requests;
      bad |= bad_req;
      B.a.x = start[seg] + (b - before[l]) * tpb;
      B.a.y = min(tpb, end - B.a.x);
      B.a.z = bad_req ? -1 : r;
      int lim = 0;
      if (kept) {
        for (int j = 0; j < B.a.y; ++j) lim = max(lim, clamp_limit(D, limits[B.a.x + j], &bad));
      } else {
        lim = block_limit(D, A.limit, B.a.x, B.a.x + B.a.y, &bad);
      }
      if (of_group) {
        B.b.y = min(pages, pages_of(lim));
        B.b.z = pages * PAGE;
        B.a.w = bad_req ? 0 : min(lim, pages * PAGE);
      } else {
        B.b.x = pages;
        B.b.y = pages > 0 ? max(pages, pages_of(lim)) : pages_of(lim);
        B.a.w = bad_req ? 0 : lim;
      }
    }
    const int n = B.b.y - B.b.x;
    int sum;
    B.b.w = cost + plan_scan<THREADS>(n > 0 ? CK_BLOCK_COST + n : 0, tmp, &sum);
    cost += sum;
    if (b < n_blocks) W.blocks[b] = B;
  }
  if (bad) set_status(D.status, HS_ERR_BAD_ID);
  const int per_pair = max((cost + A.pairs - 1) / A.pairs, CK_MIN_COST);
  for (int p = tid; p < A.pairs; p += THREADS)
    if (p * per_pair >= cost) W.start[p] = {0, 0, 0, 0, {make_int4(0, 0, -1, 0), make_int4(0, 0, CK_NO_CAP, 0)}};
  // the ranges that begin in each block, and what is joined of its tokens: the last blocks first, which are at hand
  for (int base = (n_blocks - 1) / THREADS * THREADS, last = base; base >= 0; base -= THREADS) {
    const int b = base + tid;
    if (b >= n_blocks) continue;
    if (base != last) B = W.blocks[b];
    const int pages = B.b.y - B.b.x;
    if (pages <= 0) continue;
    for (int p = (B.b.w + per_pair - 1) / per_pair; p * per_pair < B.b.w + CK_BLOCK_COST + pages; ++p)
      W.start[p] = {b, p * per_pair - B.b.w, min(per_pair, cost - p * per_pair), 0, B};
    const int c = B.b.w + CK_BLOCK_COST, first = c / per_pair, n = (c + pages - 1) / per_pair - first + 1;
    const bool of_group = B.b.z != CK_NO_CAP;
    if (n == 1 && !of_group && B.b.x == 0) continue;
    for (int j = 0; j < B.a.y; ++j)
      (of_group ? W.of_token[B.a.x + j].x : W.of_token[B.a.x + j].y) = join_word({n, first, j, n == 1});
  }
}

// Joins what the blocks of a token left in the workspace, in the order of its blocks and pairs: of a token
// with two blocks both, of one with a cut block its parts. A CTA has four rows of a token that lie next to one
// another; WIDE (few rows, of many parts each) a quarter of their dims, the parts dealt to four slices of 128
// threads. The CTAs go through the tasks in steps of the grid and look up 32 tokens at a time, for most may have
// nothing to join.
constexpr int PM_AHEAD = 4;   // parts whose loads are in flight (51,200 rows of two parts 71 us; six and two CTAs on an SM 84)
template <typename T, bool WIDE>
__global__ void __launch_bounds__(CM_THREADS, 3) prefix_merge_kernel(const Dev D, const ChunkArgs A) {
  __shared__ float4 acc[WIDE ? CM_SLICES : 1][128];
  __shared__ float2 ml[CM_SLICES][4];
  griddep_wait();
  const int tid = threadIdx.x, slice = WIDE ? tid >> 7 : 0, quad = tid & 3, lane = tid & 31, H = D.n_heads;
  const SharedWork W = shared_work(A, H);
  const int per_token = WIDE ? H : H / 4, tasks = A.n_tok * per_token, rows = A.n_tok * H;
  for (int base = blockIdx.x; base < tasks; base += 32 * gridDim.x) {
    const int mine = base + lane * gridDim.x;
    const int2 of = mine < tasks ? W.of_token[mine / per_token] : make_int2(0, 0);
    for (unsigned todo = __ballot_sync(0xffffffffu, (of.x | of.y) != 0); todo; todo &= todo - 1) {
      const int k = __ffs(todo) - 1, task = base + k * gridDim.x, row = quad_row(WIDE ? task >> 2 : task, quad);
      const int col = WIDE ? (task & 3) * 32 + (tid >> 2 & 31) : tid >> 2;
      const ToJoin x = join_of(__shfl_sync(0xffffffffu, of.x, k)), y = join_of(__shfl_sync(0xffffffffu, of.y, k));
      const int tok = task / per_token, h = row - tok * H, n = x.n + y.n;
      const int step = WIDE ? CM_SLICES : 1;
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = WIDE ? slice : 0; i < n; i += PM_AHEAD * step) {
        float2 s[PM_AHEAD];
        float4 v[PM_AHEAD];
#pragma unroll
        for (int u = 0; u < PM_AHEAD; ++u) {
          const int q = i + u * step;
          s[u] = make_float2(-INFINITY, 0.f);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (q >= n) continue;
          const bool shared = q < x.n, whole = shared ? x.whole : y.whole;
          const int j = shared ? q : q - x.n, first = shared ? x.first : y.first, place = shared ? x.place : y.place;
          const size_t at = whole ? (size_t)(shared ? 0 : rows) + row
                                  : ((size_t)(first + j) * 2 + (j == 0 ? 1 : 0)) * CK_ROWS + place * H + h;
          s[u] = (whole ? W.whole_stats : W.stats)[at];
          v[u] = reinterpret_cast<const float4*>(whole ? W.whole : W.part)[part_unit(at, col)];
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < PM_AHEAD; ++u) mn = fmaxf(mn, s[u].x);
        if (mn == -INFINITY) continue;
        const float f = exp2f(m - mn);
        m = mn;
        l *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int u = 0; u < PM_AHEAD; ++u) {
          const float w = exp2f(s[u].x - mn);   // 0 of a part that sees nothing, whose sums are 0
          l += w * s[u].y;
          o.x += w * v[u].x, o.y += w * v[u].y, o.z += w * v[u].z, o.w += w * v[u].w;
        }
      }
      if (WIDE) {
        acc[slice][tid & 127] = o;
        if ((tid & 127) < 4) ml[slice][quad] = make_float2(m, l);
        __syncthreads();
        if (slice == 0) {
          m = fmaxf(fmaxf(ml[0][quad].x, ml[1][quad].x), fmaxf(ml[2][quad].x, ml[3][quad].x));
          l = 0.f;
          o = make_float4(0.f, 0.f, 0.f, 0.f);
          if (m > -INFINITY) {
#pragma unroll
            for (int u = 0; u < CM_SLICES; ++u) {
              const float w = exp2f(ml[u][quad].x - m);
              const float4 v = acc[u][tid];
              l += w * ml[u][quad].y;
              o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
            }
          }
        }
      }
      if (!WIDE || slice == 0) {
        if (only_low(m)) {
          l = 0.f;
          if (col == 0) set_status(D.status, HS_ERR_RANGE);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T* op = static_cast<T*>(A.out) + tok * A.o_tok + h * A.o_head + col * 4;
        *reinterpret_cast<uint2*>(op) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
        if (A.lse && col == 0) A.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      if (WIDE) __syncthreads();   // the slices' sums are read
    }
  }
}

int prefix_blocks(int n_tok, int n_seg, int n_groups, int tpb) { return n_seg + n_groups + 2 * (n_tok / tpb) + 1; }

// Rows up to which a CTA of the join has a quarter of their dims and deals their parts to four slices. The whole call so
// and with all dims and no slices: 128 rows behind 131,072 81 and 107 us, 256 rows 116 and 129, 768 rows 283 and 285, 1,024
// rows 371 and 368; behind 8,192 (64 heads) 768 rows 42.6 and 44.0, 1,024 rows 50.2 and 47.8; behind 640 384 rows 27.7 and
// 28.3, 768 rows 30.1 and 28.3, 1,024 rows 31.6 and 27.9.
constexpr int PM_WIDE_ROWS = 768;
template <typename T>
hs_status launch_prefix(hs_pool* p, const ChunkArgs& a, cudaStream_t st) {
  const int smem = plan_ints(a.n_seg, a.n_groups, a.n_tok) * 4;
  hs_status s;
  if (a.max_blocks <= PP_FEW) {
    s = launch_pdl(prefix_plan_kernel<256>, dim3(1), dim3(256), smem, st, 0, p->d, a);
  } else {
    s = ensure_kernel_attrs(prefix_plan_kernel<1024>, smem);
    if (s == HS_OK) s = launch_pdl(prefix_plan_kernel<1024>, dim3(1), dim3(1024), smem, st, 0, p->d, a);
  }
  if (s == HS_OK) s = launch_attention_pairs<T, true>(p, a, st);
  if (s != HS_OK) return s;
  const int rows = a.n_tok * p->cfg.n_heads, most = 3 * num_sms();   // resident at once
  const auto grid = [&](int tasks) { return dim3(tasks < most ? tasks : most); };
  if (rows <= PM_WIDE_ROWS)
    return launch_pdl(prefix_merge_kernel<T, true>, grid(rows), dim3(CM_THREADS), 0, st, 0, p->d, a);
  return launch_pdl(prefix_merge_kernel<T, false>, grid(rows / 4), dim3(CM_THREADS), 0, st, 0, p->d, a);
}

}  // namespace

}  // namespace hs

using namespace hs;

namespace {
int64_t prefix_bytes(const hs_pool* p, int n_tok, int n_seg, int n_groups, int* max_blocks) {
  const int heads = p->cfg.n_heads, blocks = prefix_blocks(n_tok, n_seg, n_groups, CK_ROWS / heads);
  int64_t end = 0;
  shared_at(nullptr, chunk_pairs(), n_tok, (int64_t)n_tok * heads, blocks, &end);
  if (max_blocks) *max_blocks = blocks;
  return end;
}
bool prefix_sizes_ok(int32_t n_tok, int32_t n_seg, int32_t n_groups) {
  return n_tok >= 0 && n_tok <= HS_PREFIX_MAX_TOKENS && n_seg >= 0 && n_seg <= HS_CHUNK_MAX_SEGMENTS && n_groups >= 0 &&
         n_groups <= HS_PREFIX_MAX_GROUPS;
}
}  // namespace

extern "C" hs_status hs_prefix_workspace(const hs_pool* p, int32_t n_tok, int32_t n_seg, int32_t n_groups, int64_t* bytes) {
  if (!p || !bytes || !prefix_sizes_ok(n_tok, n_seg, n_groups) || !on_pool_device(p)) return HS_ERR_INVALID;
  *bytes = prefix_bytes(p, n_tok, n_seg, n_groups, nullptr);
  return HS_OK;
}

extern "C" hs_status hs_prefix_attention(hs_pool* p, int32_t layer, int32_t n_groups, const int32_t* d_group_start,
                                         const int32_t* d_group_len, int32_t n_seg, const int32_t* d_seg_req,
                                         const int32_t* d_seg_start, int32_t n, const int32_t* d_limit, int32_t dtype,
                                         const void* d_q, int64_t q_tok, int64_t q_head, float sm_scale, void* d_out,
                                         int64_t o_tok, int64_t o_head, float* d_lse, void* d_work, int64_t work_bytes,
                                         hs_stream_t stream) {
  CallRange nvtx_range("hs_prefix_attention");
  if (!p || !prefix_sizes_ok(n, n_seg, n_groups)) return HS_ERR_INVALID;
  int max_blocks = 0;
  const int64_t need = prefix_bytes(p, n, n_seg, n_groups, &max_blocks);
  const hs_status s = check_attention(p, layer, n_seg, d_seg_req, d_seg_start, n, HS_PREFIX_MAX_TOKENS, d_limit, dtype, d_q, q_tok,
                                      q_head, sm_scale, d_out, o_tok, o_head, d_lse, d_work, work_bytes, need);
  if (s != HS_OK) return s;
  if (n > 0 && n_seg > 0 && n_groups > 0 &&
      (!d_group_start || !d_group_len || !words_ok(d_group_start) || !words_ok(d_group_len)))
    return HS_ERR_INVALID;
  p->settled_rows = nullptr;
  if (n == 0 || n_seg == 0) return HS_OK;
  const ChunkArgs a = {layer, n_seg, n, chunk_pairs(), 0, d_seg_req, d_seg_start, d_limit, d_q, q_tok, q_head, sm_scale * CK_LOG2E,
                       d_out, o_tok, o_head, d_lse, d_work, n_groups, max_blocks, d_group_start, d_group_len};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == HS_BF16 ? launch_prefix<__nv_bfloat16>(p, a, st) : launch_prefix<__half>(p, a, st);
}
