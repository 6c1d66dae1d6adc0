// Quantising the cache as it is written, and reading it back.
//
// "Serving GLM-5.3 with PCP, DCP and Hybrid HiSparse" (vLLM blog Part 2), footnotes 1
// and 3: a cached KV row is 512 FP8 latent values with four fp32 scales and 64 bf16
// rope values (656 bytes); an index key is 128 FP8 values with one fp32 scale. The
// pages give the formats only; the quantisation is
//   scale = amax / 448 over the 128 values of a group (1 when they are all zero),
//   code  = x / scale rounded to the nearest e4m3 value, ties to even.
// Both divisions are the correctly rounded fp32 ones: a code can differ from the one of
// unrounded arithmetic only where x / scale lies within 2^-23 of a rounding border.
//
// One warp per token. Lane l holds latent values 256 j + 8 l .. + 7 (j = 0, 1), so that
// every load and store of a warp is one contiguous run, and the 16 lanes of a half warp
// hold exactly one 128-value group.
#include <cuda_fp8.h>
#include <math.h>
#include <nvtx3/nvToolsExt.h>

#include "hs_chunk.cuh"

namespace hs {

namespace {

constexpr int CA_WARPS = 8;          // warps per CTA
constexpr float E4M3_MAX = 448.f;
constexpr float MIN_SCALE = 1.17549435e-38f;   // the smallest normal fp32: x / scale stays finite and below 448
constexpr float BF16_MAX = 3.38953139e38f;

// N consecutive values of type T (16-byte or smaller aligned accesses) as fp32, and back.
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[N]) {
  constexpr int BYTES = N * (int)sizeof(T);
  union {
    uint4 q[BYTES >= 16 ? BYTES / 16 : 1];
    uint2 d[BYTES >= 8 ? BYTES / 8 : 1];
    uint32_t w[BYTES / 4];
    T t[N];
  } u;
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) u.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (BYTES == 8) {
    u.d[0] = *reinterpret_cast<const uint2*>(p);
  } else {
    u.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32(u.t[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[N]) {
  constexpr int BYTES = N * (int)sizeof(T);
  union U {
    uint4 q[BYTES >= 16 ? BYTES / 16 : 1];
    uint2 d[BYTES >= 8 ? BYTES / 8 : 1];
    uint32_t w[BYTES / 4];
    T t[N];
    __device__ U() {}
  } u;
#pragma unroll
  for (int i = 0; i < N; ++i) u.t[i] = from_f32<T>(v[i]);
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) reinterpret_cast<uint4*>(p)[i] = u.q[i];
  } else if constexpr (BYTES == 8) {
    *reinterpret_cast<uint2*>(p) = u.d[0];
  } else {
    *reinterpret_cast<uint32_t*>(p) = u.w[0];
  }
}

// The largest finite magnitude of v; a NaN becomes 0 and an infinity counts as no
// magnitude (it saturates later); either sets *bad.
template <int N>
__device__ __forceinline__ float finite_amax(float (&v)[N], bool* bad) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float x = fabsf(v[i]);
    const bool fin = x <= 3.402823466e38f;   // false for NaN and infinity
    *bad |= !fin;
    a = fmaxf(a, fin ? x : 0.f);
    if (x != x) v[i] = 0.f;
  }
  return a;
}
__device__ __forceinline__ float scale_of(float amax) {
  return amax > 0.f ? fmaxf(__fdiv_rn(amax, E4M3_MAX), MIN_SCALE) : 1.f;
}
// Four values over a scale as four e4m3 codes.
__device__ __forceinline__ uint32_t codes4(const float* v, float scale) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(v[0], scale), __fdiv_rn(v[1], scale)), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(__fdiv_rn(v[2], scale), __fdiv_rn(v[3], scale)), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ void values4(uint32_t w, float scale, float* v) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3)));
  v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
}

template <typename T>
__global__ void __launch_bounds__(CA_WARPS * 32)
append_quantized_kernel(Dev D, int layer, int n, const int32_t* __restrict__ req_of, const int32_t* __restrict__ pos_of,
                        const T* __restrict__ latent, long long ld_latent, const T* __restrict__ rope,
                        long long ld_rope, const T* __restrict__ keys, long long ld_keys, float key_scale) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * CA_WARPS + (threadIdx.x >> 5);
  if (t >= n) return;
  const int r = req_of[t], pos = pos_of[t];
  if (r == -1) return;   // padding
  if (r < 0 || r >= D.max_requests || pos < 0 || pos >= D.max_ctx) {
    if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    return;
  }
  // the same position again in the next token: that one is written
  if (t + 1 < n && req_of[t + 1] == r && pos_of[t + 1] == pos) return;
  const size_t at = (size_t)r * D.max_pages + (pos >> 6);
  bool bad = false;
  if (latent) {
    const int pg = D.bt[at];
    if (pg < 0 || pg >= D.num_pages) {
      if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    } else {
      uint8_t* row = D.kv[layer] + ((size_t)pg * PAGE + (pos & 63)) * ROW;
      float v[2][8], rp[2], sc[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) load_f32<T, 8>(latent + t * ld_latent + j * 256 + lane * 8, v[j]);
      load_f32<T, 2>(rope + t * ld_rope + lane * 2, rp);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a = finite_amax(v[j], &bad);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        sc[j] = scale_of(a);
        *reinterpret_cast<uint2*>(row + j * 256 + lane * 8) = make_uint2(codes4(v[j], sc[j]), codes4(v[j] + 4, sc[j]));
      }
      const float s1 = __shfl_sync(0xffffffffu, sc[0], 16), s3 = __shfl_sync(0xffffffffu, sc[1], 16);
      if (lane == 0) *reinterpret_cast<float4*>(row + LATENT) = make_float4(sc[0], s1, sc[1], s3);
      finite_amax(rp, &bad);
#pragma unroll
      for (int i = 0; i < 2; ++i) rp[i] = fminf(fmaxf(rp[i], -BF16_MAX), BF16_MAX);
      store_f32<__nv_bfloat16, 2>(reinterpret_cast<__nv_bfloat16*>(row + LATENT + 16) + lane * 2, rp);
    }
  }
  if (keys) {
    const int ip = D.idx_bt[at];
    if (ip < 0 || ip >= D.num_idx_pages) {
      if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    } else {
      uint8_t* page = reinterpret_cast<uint8_t*>(D.idx[layer / D.lpi]) + (size_t)ip * D.idx_page_bytes;
      uint32_t* code = reinterpret_cast<uint32_t*>(page + (pos & 63) * IDX_DIM) + lane;
      float v[4];
      load_f32<T, 4>(keys + t * ld_keys + lane * 4, v);
      float a = finite_amax(v, &bad);
      if (D.idx_fmt == HS_IDX_FP8) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float s = scale_of(a);
        *code = codes4(v, s);
        if (lane == 0) *reinterpret_cast<float*>(page + PAGE * IDX_DIM + (pos & 63) * 4) = s;
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float q = fminf(fmaxf(rintf(__fdiv_rn(v[i], key_scale)), -127.f), 127.f);
          w |= ((uint32_t)(int)q & 0xFFu) << (8 * i);
        }
        *code = w;
      }
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(D.status, HS_ERR_RANGE);
}

template <typename T>
__global__ void __launch_bounds__(CA_WARPS * 32)
read_rows_kernel(Dev D, int layer, int n, const int32_t* __restrict__ req_of, const int32_t* __restrict__ pos_of,
                 T* __restrict__ latent, long long ld_latent, T* __restrict__ rope, long long ld_rope,
                 T* __restrict__ keys, long long ld_keys, float key_scale) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * CA_WARPS + (threadIdx.x >> 5);
  if (t >= n) return;
  const int r = req_of[t], pos = pos_of[t];
  if (r == -1) return;   // padding
  if (r < 0 || r >= D.max_requests || pos < 0 || pos >= D.max_ctx) {
    if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    return;
  }
  if (latent || rope) {
    int err = HS_OK;
    const uint8_t* page = page_rows(D, layer, r, pos >> 6, &err);
    if (!page) {
      if (lane == 0) set_status(D.status, err);
    } else {
      const uint8_t* row = page + (size_t)(pos & 63) * ROW;
      if (latent) {
        const float4 s4 = *reinterpret_cast<const float4*>(row + LATENT);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 w = *reinterpret_cast<const uint2*>(row + j * 256 + lane * 8);
          const float s = j == 0 ? (lane < 16 ? s4.x : s4.y) : (lane < 16 ? s4.z : s4.w);
          float v[8];
          values4(w.x, s, v);
          values4(w.y, s, v + 4);
          store_f32<T, 8>(latent + t * ld_latent + j * 256 + lane * 8, v);
        }
      }
      if (rope) {
        float v[2];
        load_f32<__nv_bfloat16, 2>(reinterpret_cast<const __nv_bfloat16*>(row + LATENT + 16) + lane * 2, v);
        store_f32<T, 2>(rope + t * ld_rope + lane * 2, v);
      }
    }
  }
  if (keys) {
    const int ip = D.idx_bt[(size_t)r * D.max_pages + (pos >> 6)];
    if (ip < 0 || ip >= D.num_idx_pages) {
      if (lane == 0) set_status(D.status, HS_ERR_BAD_ID);
    } else {
      const uint8_t* page = reinterpret_cast<const uint8_t*>(D.idx[layer / D.lpi]) + (size_t)ip * D.idx_page_bytes;
      const uint32_t w = *(reinterpret_cast<const uint32_t*>(page + (pos & 63) * IDX_DIM) + lane);
      float v[4];
      if (D.idx_fmt == HS_IDX_FP8) {
        values4(w, *reinterpret_cast<const float*>(page + PAGE * IDX_DIM + (pos & 63) * 4), v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i)) * key_scale;
      }
      store_f32<T, 4>(keys + t * ld_keys + lane * 4, v);
    }
  }
}

// Rows of `width` values: 16-byte aligned, a stride of whole 16-byte units that holds a row.
bool rows_ok(const void* p, int64_t ld, int width, int size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld >= width && ld < (1ll << 40) && (ld * size) % 16 == 0;
}

struct CallArgs {
  int size = 0;
  hs_status status = HS_ERR_INVALID;   // HS_OK with size 0: nothing to do
};
// The checks both calls share.
CallArgs check_call(hs_pool* p, int32_t layer, int32_t n, const int32_t* d_req, const int32_t* d_pos, int32_t dtype,
                    const void* d_latent, int64_t ld_latent, const void* d_rope, int64_t ld_rope, const void* d_keys,
                    int64_t ld_keys, float key_scale) {
  CallArgs a;
  if (!p || layer < 0 || layer >= p->cfg.n_layers || n < 0) return a;
  const int size = dtype_size(dtype);
  if (size == 0 || !on_pool_device(p)) return a;
  if (n > 0) {
    if (!d_req || !d_pos || (!d_latent && !d_rope && !d_keys)) return a;
    if (d_latent && !rows_ok(d_latent, ld_latent, LATENT, size)) return a;
    if (d_rope && !rows_ok(d_rope, ld_rope, ROPE, size)) return a;
    if (d_keys && !rows_ok(d_keys, ld_keys, IDX_DIM, size)) return a;
    // the int8 step: a normal fp32, so that neither the quotient nor the product overflows by it alone
    if (d_keys && p->d.idx_fmt == HS_IDX_INT8 && !(key_scale >= MIN_SCALE && key_scale <= 3.0e38f)) return a;
  }
  a.status = HS_OK;
  a.size = n > 0 ? size : 0;
  return a;
}

struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
};

template <typename T>
hs_status launch_append_quantized(hs_pool* p, int layer, int n, const int32_t* d_req, const int32_t* d_pos,
                                  const void* d_latent, int64_t ld_latent, const void* d_rope, int64_t ld_rope,
                                  const void* d_keys, int64_t ld_keys, float key_scale, cudaStream_t st) {
  return launch_pdl(append_quantized_kernel<T>, dim3((n + CA_WARPS - 1) / CA_WARPS), dim3(CA_WARPS * 32), 0, st, 0,
                    p->d, layer, n, d_req, d_pos, static_cast<const T*>(d_latent), (long long)ld_latent,
                    static_cast<const T*>(d_rope), (long long)ld_rope, static_cast<const T*>(d_keys),
                    (long long)ld_keys, key_scale);
}
template <typename T>
hs_status launch_read_rows(hs_pool* p, int layer, int n, const int32_t* d_req, const int32_t* d_pos, void* d_latent,
                           int64_t ld_latent, void* d_rope, int64_t ld_rope, void* d_keys, int64_t ld_keys,
                           float key_scale, cudaStream_t st) {
  return launch_pdl(read_rows_kernel<T>, dim3((n + CA_WARPS - 1) / CA_WARPS), dim3(CA_WARPS * 32), 0, st, 0, p->d,
                    layer, n, d_req, d_pos, static_cast<T*>(d_latent), (long long)ld_latent, static_cast<T*>(d_rope),
                    (long long)ld_rope, static_cast<T*>(d_keys), (long long)ld_keys, key_scale);
}

}  // namespace

}  // namespace hs

using namespace hs;

extern "C" hs_status hs_append_quantized(hs_pool* p, int32_t layer, int32_t n, const int32_t* d_req,
                                         const int32_t* d_pos, int32_t dtype, const void* d_latent, int64_t ld_latent,
                                         const void* d_rope, int64_t ld_rope, const void* d_keys, int64_t ld_keys,
                                         float key_scale, hs_stream_t stream) {
  CallRange nvtx_range("hs_append_quantized");
  const CallArgs a = check_call(p, layer, n, d_req, d_pos, dtype, d_latent, ld_latent, d_rope, ld_rope, d_keys, ld_keys,
                                key_scale);
  if (a.status != HS_OK) return a.status;
  if (n > 0 && (d_latent == nullptr) != (d_rope == nullptr)) return HS_ERR_INVALID;   // a row is written whole
  p->settled_rows = nullptr;
  if (a.size == 0) return HS_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto f = dtype == HS_BF16   ? launch_append_quantized<__nv_bfloat16>
           : dtype == HS_FP16 ? launch_append_quantized<__half>
                              : launch_append_quantized<float>;
  return f(p, layer, n, d_req, d_pos, d_latent, ld_latent, d_rope, ld_rope, d_keys, ld_keys, key_scale, st);
}

extern "C" hs_status hs_read_rows(hs_pool* p, int32_t layer, int32_t n, const int32_t* d_req, const int32_t* d_pos,
                                  int32_t dtype, void* d_latent, int64_t ld_latent, void* d_rope, int64_t ld_rope,
                                  void* d_keys, int64_t ld_keys, float key_scale, hs_stream_t stream) {
  CallRange nvtx_range("hs_read_rows");
  const CallArgs a = check_call(p, layer, n, d_req, d_pos, dtype, d_latent, ld_latent, d_rope, ld_rope, d_keys, ld_keys,
                                key_scale);
  if (a.status != HS_OK) return a.status;
  p->settled_rows = nullptr;
  if (a.size == 0) return HS_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto f = dtype == HS_BF16   ? launch_read_rows<__nv_bfloat16>
           : dtype == HS_FP16 ? launch_read_rows<__half>
                              : launch_read_rows<float>;
  return f(p, layer, n, d_req, d_pos, d_latent, ld_latent, d_rope, ld_rope, d_keys, ld_keys, key_scale, st);
}
