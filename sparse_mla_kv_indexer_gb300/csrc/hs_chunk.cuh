// Shared by the cache operators of prefill (hs_cache.cu, hs_chunk.cu): element types, checks of
// arguments and the place of a request's page.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "hs_internal.cuh"

namespace hs {

// One NVTX range per ABI call, as for the other calls.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
};

inline int dtype_size(int32_t dtype) {
  return dtype == HS_BF16 || dtype == HS_FP16 ? 2 : dtype == HS_FP32 ? 4 : 0;
}
// The pool's metadata lives on its own device, and launches go to the current one.
inline bool on_pool_device(const hs_pool* p) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == p->device;
}

// An address that 4-byte words may be read from or written to.
inline bool words_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two fp32 values in one register pair.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(uint32_t lo, uint32_t hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ void unpack(F2 a, float& lo, float& hi) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(a.v));
  lo = __uint_as_float(x);
  hi = __uint_as_float(y);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// The largest of three, NaN when one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The larger of two, NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The 64 rows of logical page `page` (0 <= page < max_pages) of request r in `layer`: the
// pool page when it is resident, else its host copy through the mapping, else null with
// *err set.
__device__ __forceinline__ const uint8_t* page_rows(const Dev& D, int layer, int r, int page, int* err) {
  const size_t at = (size_t)r * D.max_pages + page;
  const int pg = D.bt[at];
  if (pg >= 0) {
    if (pg < D.num_pages) return D.kv[layer] + (size_t)pg * PAGE * ROW;
    *err = HS_ERR_BAD_ID;
    return nullptr;
  }
  const int64_t hp = D.host_pg[at];
  if (hp >= 0 && hp < D.host_pages) return D.host + ((size_t)hp * D.n_layers + layer) * PAGE * ROW;
  *err = hp < 0 ? HS_ERR_HOST_MISSING : HS_ERR_BAD_ID;
  return nullptr;
}

}  // namespace hs
