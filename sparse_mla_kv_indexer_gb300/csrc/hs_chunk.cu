// Attention of a chunk of new tokens over the paged cache (prefill, the input of a later turn, dense
// decode): the join of cut blocks' parts and the call. The kernel is hs_chunk_kernel.cuh's.
#include "hs_chunk_kernel.cuh"

namespace hs {

namespace {

// The rows of cut blocks: out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the parts,
// in pair order, for four rows that lie next to one another at a time. WIDE (few cuts, of many parts
// each): CTA (four rows and a quarter of their dims, k) of the k-th cut, its parts dealt to four slices of
// 128 threads. Otherwise CTA (four rows, p) of the cut of pair p.
constexpr int CM_WIDE_CUTS = 32;
template <typename T, bool WIDE>
__global__ void __launch_bounds__(CM_THREADS) chunk_merge_kernel(const Dev D, const ChunkArgs A) {
  __shared__ float4 acc[CM_SLICES][128];
  __shared__ float2 ml[CM_SLICES][4];
  __shared__ int mine;
  griddep_wait();
  const ChunkWork W = work_at(A.work, A.pairs);
  const int tid = threadIdx.x, slice = WIDE ? tid >> 7 : 0, H = D.n_heads;
  const int col = WIDE ? (blockIdx.x & 3) * 32 + (tid >> 2 & 31) : tid >> 2;
  const int row = quad_row(WIDE ? blockIdx.x >> 2 : blockIdx.x, tid & 3);
  int p = blockIdx.y;
  if (WIDE) {   // the blockIdx.y-th pair that has a cut
    if (tid == 0) mine = A.pairs;
    __syncthreads();
    if (tid < 32) {
      int before = 0;
      for (int i = tid; i - tid < A.pairs; i += 32) {
        const bool has = i < A.pairs && W.cut[i].n_tok > 0;
        const unsigned b = __ballot_sync(0xffffffffu, has);
        if (has && before + __popc(b & ((1u << tid) - 1)) == (int)blockIdx.y) mine = i;
        before += __popc(b);
      }
    }
    __syncthreads();
    p = mine;
    if (p >= A.pairs) return;
  }
  const ChunkCut cut = W.cut[p];
  if (row >= cut.n_tok * H) return;   // all of the CTA's rows, or none
  auto part_at = [&](int i) { return ((size_t)i * 2 + (i == p ? 1 : 0)) * CK_ROWS + row; };
  const int step = WIDE ? CM_SLICES : 1;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = p + (WIDE ? slice : 0); i <= cut.last_pair; i += 8 * step) {
    // eight parts at a time, all of their loads in flight
    float2 s[8];
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = i + u * step <= cut.last_pair;
      s[u] = in ? W.stats[part_at(i + u * step)] : make_float2(-INFINITY, 0.f);
      v[u] = in ? reinterpret_cast<const float4*>(W.part)[part_unit(part_at(i + u * step), col)] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < 8; ++u) mn = fmaxf(mn, s[u].x);
    if (mn == -INFINITY) continue;
    const float f = exp2f(m - mn);
    m = mn;
    l *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = exp2f(s[u].x - mn);
      l += w * s[u].y;
      o.x += w * v[u].x, o.y += w * v[u].y, o.z += w * v[u].z, o.w += w * v[u].w;
    }
  }
  if (WIDE) {
    const int j = tid & 3;
    acc[slice][tid & 127] = o;
    if ((tid & 127) < 4) ml[slice][j] = make_float2(m, l);
    __syncthreads();
    if (slice > 0) return;
    m = fmaxf(fmaxf(ml[0][j].x, ml[1][j].x), fmaxf(ml[2][j].x, ml[3][j].x));
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m > -INFINITY) {
#pragma unroll
      for (int u = 0; u < CM_SLICES; ++u) {
        const float w = exp2f(ml[u][j].x - m);
        const float4 v = acc[u][tid];
        l += w * ml[u][j].y;
        o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
      }
    }
  }
  if (only_low(m)) {
    l = 0.f;
    if (col == 0) set_status(D.status, HS_ERR_RANGE);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int tok = cut.tok0 + row / H, h = row % H;
  T* op = static_cast<T*>(A.out) + tok * A.o_tok + h * A.o_head + col * 4;
  *reinterpret_cast<uint2*>(op) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
  // the outputs carry CK_V_FACTOR, and so do the sums
  if (A.lse && col == 0) A.lse[(size_t)tok * H + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T>
hs_status launch_chunk(hs_pool* p, const ChunkArgs& a, cudaStream_t st) {
  const hs_status s = launch_attention_pairs<T, false>(p, a, st);
  if (s != HS_OK) return s;
  // a pair has at most one cut, and there are no more cuts than blocks
  const int tpb = CK_ROWS / p->cfg.n_heads;
  const long long blocks = (long long)a.n_seg + a.n_tok / tpb;
  const int cuts = blocks < a.pairs ? (int)blocks : a.pairs;
  const long long rows = (long long)a.n_tok * p->cfg.n_heads;
  const int grid_rows = rows < CK_ROWS ? (int)rows : CK_ROWS;
  if (cuts <= CM_WIDE_CUTS)
    return launch_pdl(chunk_merge_kernel<T, true>, dim3(grid_rows, cuts), dim3(CM_THREADS), 0, st, 0, p->d, a);
  return launch_pdl(chunk_merge_kernel<T, false>, dim3(grid_rows / 4, a.pairs), dim3(CM_THREADS), 0, st, 0, p->d, a);
}

}  // namespace

}  // namespace hs

using namespace hs;

extern "C" hs_status hs_chunk_workspace(const hs_pool* p, int64_t* bytes) {
  if (!p || !bytes || !on_pool_device(p)) return HS_ERR_INVALID;
  *bytes = work_bytes_for(chunk_pairs());
  return HS_OK;
}

extern "C" hs_status hs_chunk_attention(hs_pool* p, int32_t layer, int32_t n_seg, const int32_t* d_seg_req,
                                        const int32_t* d_seg_start, int32_t n, const int32_t* d_limit, int32_t dtype,
                                        const void* d_q, int64_t q_tok, int64_t q_head, float sm_scale, void* d_out,
                                        int64_t o_tok, int64_t o_head, float* d_lse, void* d_work, int64_t work_bytes,
                                        hs_stream_t stream) {
  CallRange nvtx_range("hs_chunk_attention");
  const int pairs = chunk_pairs();
  const hs_status s = check_attention(p, layer, n_seg, d_seg_req, d_seg_start, n, HS_CHUNK_MAX_TOKENS, d_limit, dtype, d_q, q_tok,
                                      q_head, sm_scale, d_out, o_tok, o_head, d_lse, d_work, work_bytes, work_bytes_for(pairs));
  if (s != HS_OK) return s;
  p->settled_rows = nullptr;
  if (n == 0 || n_seg == 0) return HS_OK;
  const int small = n_seg + n / (CK_ROWS / p->cfg.n_heads) <= 32;
  const ChunkArgs a = {layer, n_seg, n, pairs, small, d_seg_req, d_seg_start, d_limit, d_q, q_tok, q_head, sm_scale * CK_LOG2E,
                       d_out, o_tok, o_head, d_lse, d_work, 0, 0, nullptr, nullptr};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == HS_BF16 ? launch_chunk<__nv_bfloat16>(p, a, st) : launch_chunk<__half>(p, a, st);
}
