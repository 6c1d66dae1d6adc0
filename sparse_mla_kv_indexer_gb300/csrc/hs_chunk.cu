// Attention of a chunk of new tokens over the paged cache (prefill, the input of a later
// turn, dense decode): every query token attends to every cached row below its limit.
//
// "Serving GLM-5.3 with PCP, DCP and Hybrid HiSparse" (vLLM blog Part 2), footnote 1: QK
// over 576 dims (512 latent, 64 rope), PV over the 512 latent dims, every row serving all
// heads. Per token j and head h, over the positions t < limit_j of its request:
//   z_t = sm_scale * q_jh . k_t,  o = sum_t softmax(z)_t v_t,  lse = log sum_t exp z_t.
//
// One warp per (token, head), one pass over the rows with the running maximum and sum of
// the softmax, in fp32 throughout.
#include <cuda_fp8.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>

#include "hs_chunk.cuh"

namespace hs {

namespace {

constexpr int CK_WARPS = 8;
constexpr float CK_LOG2E = 1.4426950408889634f;
constexpr float CK_MAX_SCALE = 146.f;   // 448 x scale < 65504

__device__ __forceinline__ void values8(uint2 w, float s, float* v) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i] & 0xFFFFu), __NV_E4M3)));
    const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i] >> 16), __NV_E4M3)));
    v[4 * i] = a.x * s, v[4 * i + 1] = a.y * s, v[4 * i + 2] = b.x * s, v[4 * i + 3] = b.y * s;
  }
}

template <typename T>
__global__ void __launch_bounds__(CK_WARPS * 32)
chunk_attention_kernel(Dev D, int layer, int n_seg, const int32_t* __restrict__ seg_req,
                       const int32_t* __restrict__ seg_start, int n_tok, const int32_t* __restrict__ limit,
                       const T* __restrict__ q, long long q_tok, long long q_head, float scale_log2,
                       T* __restrict__ out, long long o_tok, long long o_head, float* __restrict__ lse_out) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * CK_WARPS + (threadIdx.x >> 5);
  const int tok = (int)(w / D.n_heads), h = (int)(w % D.n_heads);
  if (tok >= n_tok) return;
  int s = -1, lo = 0;
  for (int i = 0; i <= n_seg; ++i) {
    const int at = seg_start[i], hi = min(max(at, lo), n_tok);
    if (at != hi && lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    if (i > 0 && tok >= lo && tok < hi) s = i - 1;
    lo = hi;
  }
  if (s < 0) return;
  const int r = seg_req[s];
  int L = limit[tok];
  if (r < 0 || r >= D.max_requests || L < 0 || L > D.max_ctx) {
    if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    L = 0;
  }
  float qv[18], acc[16], m = -INFINITY, l = 0.f;
  const T* qp = q + tok * q_tok + h * q_head;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 18; ++i) {
    const int d = i < 16 ? (i >> 3) * 256 + lane * 8 + (i & 7) : LATENT + lane * 2 + (i - 16);
    qv[i] = to_f32(qp[d]);
    bad |= !(fabsf(qv[i]) < 65504.f);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int pg = 0; pg * PAGE < L; ++pg) {
    int err = HS_OK;
    const uint8_t* rows = page_rows(D, layer, r, pg, &err);
    if (!rows) {
      if (lane == 0) set_status(D.status, err);
      continue;
    }
    const int nr = min(PAGE, L - pg * PAGE);
    for (int t = 0; t < nr; ++t) {
      const uint8_t* row = rows + (size_t)t * ROW;
      const float4 s4 = *reinterpret_cast<const float4*>(row + LATENT);
      const uint32_t rw = *reinterpret_cast<const uint32_t*>(row + LATENT + 16 + lane * 4);
      float v[18];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sj = j == 0 ? (lane < 16 ? s4.x : s4.y) : (lane < 16 ? s4.z : s4.w);
        values8(*reinterpret_cast<const uint2*>(row + j * 256 + lane * 8), sj, v + 8 * j);
        bad |= !(fabsf(sj) < CK_MAX_SCALE);
      }
      v[16] = __uint_as_float(rw << 16);
      v[17] = __uint_as_float(rw & 0xFFFF0000u);
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < 18; ++i) {
        if (!(fabsf(v[i]) < 65504.f)) bad = true, v[i] = 0.f;
        z += qv[i] * v[i];
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      z *= scale_log2;
      const float mn = fmaxf(m, z), f = exp2f(m - mn), p = exp2f(z - mn);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = acc[i] * f + p * v[i];
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* op = out + tok * o_tok + h * o_head;
#pragma unroll
  for (int i = 0; i < 16; ++i) op[(i >> 3) * 256 + lane * 8 + (i & 7)] = from_f32<T>(acc[i] * inv);
  if (lse_out && lane == 0)
    lse_out[(size_t)tok * D.n_heads + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(D.status, HS_ERR_RANGE);
}

struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
};

bool stride_ok(int64_t s, int64_t least) { return s >= least && s < (1ll << 40) && s % 8 == 0; }

int64_t workspace_bytes(const hs_pool*) { return 256; }

template <typename T>
hs_status launch_chunk(hs_pool* p, int layer, int n_seg, const int32_t* d_seg_req, const int32_t* d_seg_start, int n,
                       const int32_t* d_limit, const void* d_q, int64_t q_tok, int64_t q_head, float sm_scale,
                       void* d_out, int64_t o_tok, int64_t o_head, float* d_lse, cudaStream_t st) {
  const long long warps = (long long)n * p->cfg.n_heads;
  return launch_pdl(chunk_attention_kernel<T>, dim3((unsigned)((warps + CK_WARPS - 1) / CK_WARPS)), dim3(CK_WARPS * 32), 0,
                    st, 0, p->d, layer, n_seg, d_seg_req, d_seg_start, n, d_limit, static_cast<const T*>(d_q),
                    (long long)q_tok, (long long)q_head, sm_scale * CK_LOG2E, static_cast<T*>(d_out), (long long)o_tok,
                    (long long)o_head, d_lse);
}

}  // namespace

}  // namespace hs

using namespace hs;

extern "C" hs_status hs_chunk_workspace(const hs_pool* p, int64_t* bytes) {
  if (!p || !bytes) return HS_ERR_INVALID;
  *bytes = workspace_bytes(p);
  return HS_OK;
}

extern "C" hs_status hs_chunk_attention(hs_pool* p, int32_t layer, int32_t n_seg, const int32_t* d_seg_req,
                                        const int32_t* d_seg_start, int32_t n, const int32_t* d_limit, int32_t dtype,
                                        const void* d_q, int64_t q_tok, int64_t q_head, float sm_scale, void* d_out,
                                        int64_t o_tok, int64_t o_head, float* d_lse, void* d_work, int64_t work_bytes,
                                        hs_stream_t stream) {
  CallRange nvtx_range("hs_chunk_attention");
  if (!p || layer < 0 || layer >= p->cfg.n_layers || n_seg < 0 || n_seg > HS_CHUNK_MAX_SEGMENTS || n < 0 ||
      n > HS_CHUNK_MAX_TOKENS || (dtype != HS_BF16 && dtype != HS_FP16) || !on_pool_device(p))
    return HS_ERR_INVALID;
  if (n > 0 && n_seg > 0) {
    const auto aligned = [](const void* x) { return x && (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
    if (!d_seg_req || !d_seg_start || !d_limit || !aligned(d_q) || !aligned(d_out) || !aligned(d_work) ||
        work_bytes < workspace_bytes(p) || !(fabsf(sm_scale) <= 3.0e38f))
      return HS_ERR_INVALID;
    if (!stride_ok(q_tok, 0) || !stride_ok(q_head, 0) || !stride_ok(o_tok, LATENT) || !stride_ok(o_head, LATENT))
      return HS_ERR_INVALID;
  }
  p->settled_rows = nullptr;
  if (n == 0 || n_seg == 0) return HS_OK;
  auto f = dtype == HS_BF16 ? launch_chunk<__nv_bfloat16> : launch_chunk<__half>;
  return f(p, layer, n_seg, d_seg_req, d_seg_start, n, d_limit, d_q, q_tok, q_head, sm_scale, d_out, o_tok, o_head,
           d_lse, reinterpret_cast<cudaStream_t>(stream));
}
