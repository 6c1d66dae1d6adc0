// Quantising the cache as it is written, and reading it back.
//
// "Serving GLM-5.3 with PCP, DCP and Hybrid HiSparse" (vLLM blog Part 2), footnotes 1
// and 3: a cached KV row is 512 FP8 latent values with four fp32 scales and 64 bf16
// rope values (656 bytes); an index key is 128 FP8 values with one fp32 scale. The
// pages give the formats only; the quantisation is
//   scale = amax / 448 over the 128 values of a group, 2^-126 at least (1 when they are all zero),
//   code  = x / scale rounded to the nearest e4m3 value, ties to even.
// Both divisions are the correctly rounded fp32 ones: a code can differ from the one of
// unrounded arithmetic only where x / scale lies within 2^-23 of a rounding border.
//
// A warp has a run of up to 32 tokens, whose places (request -> page -> row, a chain of three
// loads) its lanes look up side by side. Then it appends token by token, the next one's values on
// their way, or reads CA_READ tokens at a time, all of their loads in flight. The runs are dealt
// so that all warps are resident at once. Lane l holds latent values 256 j + 8 l .. + 7 (j = 0, 1), so
// that every load and store of a warp is one contiguous run, and the 16 lanes of a half warp
// hold exactly one 128-value group.
//
// Measured on a GB300 (163 MB moved for 74,160 tokens of bf16, 24.5 us at the copy rate, 25.2 us
// for a plain elementwise pass over as many bytes): append 33.9 us, read back 30.9 us (fp32 values,
// 268 MB and 40 us: 44 and 54 us), against 46 and 37 us when every token's places are looked up by the warp that takes it, one chain after
// another. The append is bound by its instructions (0.6 a cycle and scheduler), the read by the
// latency between a warp's loads; one token at a time with the next one on its way reads in 34.6
// us, three or four at a time in 43 us and more. 28, 36, 48 and 64 warps per SM append in 41 (two
// tokens more per warp), 39, 39 and 39 us (two waves).
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include "hs_chunk.cuh"

namespace hs {

namespace {

constexpr int CA_WARPS = 4;          // warps per CTA
constexpr int CA_READ = 2;           // tokens of a warp at a time when reading
constexpr int CA_SM_WARPS = 32;      // warps per SM among which the tokens are dealt, up to 32 each
constexpr float E4M3_MAX = 448.f;
constexpr float MIN_SCALE = 1.17549435e-38f;   // 2^-126, the smallest normal fp32: below it amax / 448 has too few bits, or none
constexpr float BF16_MAX = 3.38953139e38f;
constexpr float BF16_OVER = 3.39617752e38f;   // BF16_MAX and half a step: from here on bf16 rounds to infinity

// N consecutive values of type T (16-byte or smaller aligned accesses) as they are stored, as
// fp32, and back.
template <typename T, int N>
struct Raw {
  union {
    uint4 q[N * (int)sizeof(T) >= 16 ? N * (int)sizeof(T) / 16 : 1];
    uint2 d;
    uint32_t w;
    T t[N];
  };
  __device__ Raw() {}
};
template <typename T, int N>
__device__ __forceinline__ void load_raw(const T* p, Raw<T, N>& u) {
  constexpr int BYTES = N * (int)sizeof(T);
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) u.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (BYTES == 8) {
    u.d = *reinterpret_cast<const uint2*>(p);
  } else {
    u.w = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <typename T, int N>
__device__ __forceinline__ void raw_f32(const Raw<T, N>& u, float (&v)[N]) {
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

// The largest magnitude of v: NaN when one is NaN, else infinite when one is infinite.
template <int N>
__device__ __forceinline__ float amax_of(const float (&v)[N]) {
  float a = max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int i = 2; i < N; i += 2) a = max3_nan(a, fabsf(v[i]), fabsf(v[i + 1]));
  return a;
}
template <int LANES>
__device__ __forceinline__ float lanes_amax(float a) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}
// x / scale for the many x of one scale: with r the correctly rounded reciprocal,
// q + r (x - q scale) rounds to the quotient as the division does (P. Markstein, IBM J. Res.
// Dev. 34(1), 1990, theorem 2, for q within one unit of it), in three operations each. Here q
// = x r is within 1.5 units, so this was enumerated in exact arithmetic: amax / 448 for all
// 2^23 significands, and all x / scale that lie beside a border of two codes (such a scale's
// significand is a multiple of 2^18 give or take 24; 200,688 quotients). x - q scale has to
// be exact, which holds far from the smallest normal numbers: smaller amax go through the
// division itself.
__device__ __forceinline__ float over(float x, float scale, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, scale, x), r, q);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}
// The rare groups (a value that is not finite, or an amax below 2^-60), out of line: a NaN
// becomes 0, an infinity what the group's scale makes the largest code: its largest finite
// magnitude, or 448 times the least scale, or times that of zeros.
__device__ __noinline__ float rare_value(float x, float amax) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? x : x != x ? 0.f : copysignf(amax > 0.f ? fmaxf(amax, E4M3_MAX * MIN_SCALE) : E4M3_MAX, x);
}
__device__ __noinline__ float rare_quotient(float x, float scale) { return __fdiv_rn(x, scale); }
// The N values that each of LANES lanes holds of one group, as N / 4 words of e4m3 codes;
// returns the group's scale. *bad: a value was not finite.
template <int N, int LANES>
__device__ __forceinline__ float quantise(float (&v)[N], uint32_t (&code)[N / 4], bool* bad) {
  float a = lanes_amax<LANES>(amax_of(v));
  if ((a >= 8.6736174e-19f && a <= FLT_MAX) || a == 0.f) {   // 2^-60
    const float scale = a > 0.f ? over(a, E4M3_MAX, 1.f / E4M3_MAX) : 1.f;
    // minus the quotients, and the signs of the codes turned: so that -0 keeps its sign (q + r (x - q
    // scale) would add +0 to it)
    const F2 r = f2(-__frcp_rn(scale)), s = f2(scale);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const F2 x = f2(__float_as_uint(v[i + k]), __float_as_uint(v[i + k + 1])), q0 = mul2(x, r);
        unpack(fma2(fma2(q0, s, x), r, q0), q[k], q[k + 1]);
      }
      code[i / 4] = e4m3x4(q[0], q[1], q[2], q[3]) ^ 0x80808080u;
    }
    return scale;
  }
  if (!(a <= FLT_MAX)) {   // the same in all lanes of the group
    *bad = true;
    a = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (fabsf(v[i]) <= FLT_MAX) a = fmaxf(a, fabsf(v[i]));
    const unsigned group = LANES == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = rare_value(v[i], a);
  }
  const float scale = a > 0.f ? fmaxf(rare_quotient(a, E4M3_MAX), MIN_SCALE) : 1.f;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    code[i / 4] = e4m3x4(rare_quotient(v[i], scale), rare_quotient(v[i + 1], scale), rare_quotient(v[i + 2], scale),
                         rare_quotient(v[i + 3], scale));
  return scale;
}
__device__ __forceinline__ void values4(uint32_t w, float scale, float* v) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3)));
  const F2 s = f2(scale);
  unpack(mul2(f2(__float_as_uint(a.x), __float_as_uint(a.y)), s), v[0], v[1]);
  unpack(mul2(f2(__float_as_uint(b.x), __float_as_uint(b.y)), s), v[2], v[3]);
}

// Where this lane's token goes or comes from: its block-table entry's index, or -1 (none,
// padding, a bad id).
struct Place {
  int r, pos;
  long long at;
};
__device__ __forceinline__ Place place_of(const Dev& D, const int32_t* req_of, const int32_t* pos_of, int t, bool in) {
  Place p = {-1, 0, -1};
  if (!in) return p;
  p.r = req_of[t], p.pos = pos_of[t];
  if (p.r == -1) return p;
  if (p.r < 0 || p.r >= D.max_requests || p.pos < 0 || p.pos >= D.max_ctx) {
    set_status(D.status, HS_ERR_BAD_ID);
    return p;
  }
  p.at = (long long)p.r * D.max_pages + (p.pos >> 6);
  return p;
}
// Whether the next token that is not padding, of the 32 behind this lane's t = base + lane, gives
// the same position again (which then is the one to be written). All lanes take part: they hold
// the 64 tokens from base on, two each.
constexpr int CA_AGAIN = 32;
__device__ __forceinline__ bool given_again(const int32_t* req_of, const int32_t* pos_of, int base, int n) {
  const int lane = threadIdx.x & 31, t = base + lane;
  const bool in0 = t < n, in1 = n - t > CA_AGAIN;
  const int r0 = in0 ? req_of[t] : -1, r1 = in1 ? req_of[t + CA_AGAIN] : -1;
  const int p0 = in0 ? pos_of[t] : 0, p1 = in1 ? pos_of[t + CA_AGAIN] : 0;
  const uint64_t live = (uint64_t)__ballot_sync(0xffffffffu, r1 != -1) << 32 | __ballot_sync(0xffffffffu, r0 != -1);
  const int ahead = __ffs((unsigned)(live >> (lane + 1))), at = (lane + ahead) & 31;   // 0: none
  const int ra0 = __shfl_sync(0xffffffffu, r0, at), ra1 = __shfl_sync(0xffffffffu, r1, at);
  const int pa0 = __shfl_sync(0xffffffffu, p0, at), pa1 = __shfl_sync(0xffffffffu, p1, at);
  const bool first = lane + ahead < 32;
  return ahead > 0 && (first ? ra0 : ra1) == r0 && (first ? pa0 : pa1) == p0;
}
template <typename P>
__device__ __forceinline__ P* shfl_ptr(P* p, int lane) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)v, lane), hi = __shfl_sync(0xffffffffu, (uint32_t)(v >> 32), lane);
  return reinterpret_cast<P*>((uint64_t)hi << 32 | lo);
}

template <typename T>
__global__ void __launch_bounds__(CA_WARPS * 32, CA_SM_WARPS / CA_WARPS)
append_quantized_kernel(const Dev D, int layer, int group, int n, int per_warp, const int32_t* __restrict__ req_of,
                        const int32_t* __restrict__ pos_of, const T* __restrict__ latent, long long ld_latent,
                        const T* __restrict__ rope, long long ld_rope, const T* __restrict__ keys, long long ld_keys,
                        float key_scale) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int base = (blockIdx.x * CA_WARPS + (threadIdx.x >> 5)) * per_warp, count = min(per_warp, n - base);
  if (count <= 0) return;
  bool bad = false;
  // this lane's token: its row and its index-key page, or null
  uint8_t *row_mine = nullptr, *page_mine = nullptr;
  int off_mine = 0;
  {
    Place p = place_of(D, req_of, pos_of, base + lane, lane < count);
    if (given_again(req_of, pos_of, base, n)) p.at = -1;
    if (p.at >= 0) {
      off_mine = p.pos & 63;
      const int pg = latent ? D.bt[p.at] : -1, ip = keys ? D.idx_bt[p.at] : -1;
      if (pg >= 0 && pg < D.num_pages) row_mine = D.kv[layer] + ((size_t)pg * PAGE + off_mine) * ROW;
      if (ip >= 0 && ip < D.num_idx_pages) page_mine = reinterpret_cast<uint8_t*>(D.idx[group]) + (size_t)ip * D.idx_page_bytes;
      if ((latent && !row_mine) || (keys && !page_mine)) set_status(D.status, HS_ERR_BAD_ID);
    }
  }
  struct In {
    Raw<T, 8> v[2];
    Raw<T, 2> rope;
    Raw<T, 4> key;
  } in[2];
  auto fetch = [&](int k, In& x) {
    if (k >= count) return;
    const long long t = base + k;
    if (latent) {
#pragma unroll
      for (int j = 0; j < 2; ++j) load_raw<T, 8>(latent + t * ld_latent + j * 256 + lane * 8, x.v[j]);
      load_raw<T, 2>(rope + t * ld_rope + lane * 2, x.rope);
    }
    if (keys) load_raw<T, 4>(keys + t * ld_keys + lane * 4, x.key);
  };
  auto put = [&](int k, const In& x) {
    if (k >= count) return;
    uint8_t* const row = shfl_ptr(row_mine, k);
    uint8_t* const page = shfl_ptr(page_mine, k);
    const int off = __shfl_sync(0xffffffffu, off_mine, k);
    if (row) {
      float sc[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[8];
        raw_f32(x.v[j], v);
        uint32_t code[2];
        sc[j] = quantise<8, 16>(v, code, &bad);
        *reinterpret_cast<uint2*>(row + j * 256 + lane * 8) = make_uint2(code[0], code[1]);
      }
      const float s1 = __shfl_sync(0xffffffffu, sc[0], 16), s3 = __shfl_sync(0xffffffffu, sc[1], 16);
      if (lane == 0) *reinterpret_cast<float4*>(row + LATENT) = make_float4(sc[0], s1, sc[1], s3);
      float rp[2];
      raw_f32(x.rope, rp);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float r = fminf(fmaxf(rp[i], -BF16_MAX), BF16_MAX);
        bad |= !(fabsf(rp[i]) < BF16_OVER);
        rp[i] = rp[i] != rp[i] ? 0.f : r;
      }
      store_f32<__nv_bfloat16, 2>(reinterpret_cast<__nv_bfloat16*>(row + LATENT + 16) + lane * 2, rp);
    }
    if (page) {
      float kv[4];
      raw_f32(x.key, kv);
      uint32_t w[1] = {0};
      if (D.idx_fmt == HS_IDX_FP8) {
        const float scale = quantise<4, 32>(kv, w, &bad);
        if (lane == 0) *reinterpret_cast<float*>(page + PAGE * IDX_DIM + off * 4) = scale;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bad |= !(fabsf(kv[i]) <= FLT_MAX);
          const float q = kv[i] != kv[i] ? 0.f : fminf(fmaxf(rintf(__fdiv_rn(kv[i], key_scale)), -127.f), 127.f);
          w[0] |= ((uint32_t)(int)q & 0xFFu) << (8 * i);
        }
      }
      *(reinterpret_cast<uint32_t*>(page + off * IDX_DIM) + lane) = w[0];
    }
  };
  if constexpr (sizeof(T) == 2) {   // the next token's values on their way while one is quantised
    fetch(0, in[0]);
    for (int k = 0; k < count; k += 2) {
      fetch(k + 1, in[1]);
      put(k, in[0]);
      fetch(k + 2, in[0]);
      put(k + 1, in[1]);
    }
  } else {   // twice the registers: they would spill
    for (int k = 0; k < count; ++k) {
      fetch(k, in[0]);
      put(k, in[0]);
    }
  }
  if (bad) set_status(D.status, HS_ERR_RANGE);
}

template <typename T>
__global__ void __launch_bounds__(CA_WARPS * 32, CA_SM_WARPS / CA_WARPS)
read_rows_kernel(const Dev D, int layer, int group, int n, int per_warp, const int32_t* __restrict__ req_of,
                 const int32_t* __restrict__ pos_of, T* __restrict__ latent, long long ld_latent, T* __restrict__ rope,
                 long long ld_rope, T* __restrict__ keys, long long ld_keys, float key_scale) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int base = (blockIdx.x * CA_WARPS + (threadIdx.x >> 5)) * per_warp, count = min(per_warp, n - base);
  if (count <= 0) return;
  // this lane's token: its row and its index-key page, or null
  const uint8_t *row_mine = nullptr, *page_mine = nullptr;
  int off_mine = 0;
  {
    const Place p = place_of(D, req_of, pos_of, base + lane, lane < count);
    if (p.at >= 0) {
      off_mine = p.pos & 63;
      int err = HS_OK;
      if (latent || rope) {
        row_mine = page_rows(D, layer, p.r, p.pos >> 6, &err);
        if (row_mine) row_mine += (size_t)off_mine * ROW;
      }
      if (keys) {
        const int ip = D.idx_bt[p.at];
        if (ip >= 0 && ip < D.num_idx_pages)
          page_mine = reinterpret_cast<const uint8_t*>(D.idx[group]) + (size_t)ip * D.idx_page_bytes;
        else if (err == HS_OK)
          err = HS_ERR_BAD_ID;
      }
      if (err != HS_OK) {   // nothing of this token is written
        set_status(D.status, err);
        row_mine = page_mine = nullptr;
      }
    }
  }
  for (int k0 = 0; k0 < count; k0 += CA_READ) {
    const uint8_t *row[CA_READ], *page[CA_READ];
    uint2 w[CA_READ][2];
    float4 s4[CA_READ];
    float ks[CA_READ];
    uint32_t rw[CA_READ], kw[CA_READ];
#pragma unroll
    for (int u = 0; u < CA_READ; ++u) {
      const int from = (k0 + u) & 31;
      row[u] = shfl_ptr(row_mine, from);
      page[u] = shfl_ptr(page_mine, from);
      const int off = __shfl_sync(0xffffffffu, off_mine, from);
      if (k0 + u >= count) row[u] = page[u] = nullptr;
      if (row[u]) {
        if (latent) {
          s4[u] = *reinterpret_cast<const float4*>(row[u] + LATENT);
#pragma unroll
          for (int j = 0; j < 2; ++j) w[u][j] = *reinterpret_cast<const uint2*>(row[u] + j * 256 + lane * 8);
        }
        if (rope) rw[u] = *(reinterpret_cast<const uint32_t*>(row[u] + LATENT + 16) + lane);
      }
      if (page[u]) {
        kw[u] = *(reinterpret_cast<const uint32_t*>(page[u] + off * IDX_DIM) + lane);
        ks[u] = D.idx_fmt == HS_IDX_FP8 ? *reinterpret_cast<const float*>(page[u] + PAGE * IDX_DIM + off * 4) : key_scale;
      }
    }
#pragma unroll
    for (int u = 0; u < CA_READ; ++u) {
      const long long t = base + k0 + u;
      if (row[u]) {
        if (latent) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float s = j == 0 ? (lane < 16 ? s4[u].x : s4[u].y) : (lane < 16 ? s4[u].z : s4[u].w);
            float v[8];
            values4(w[u][j].x, s, v);
            values4(w[u][j].y, s, v + 4);
            store_f32<T, 8>(latent + t * ld_latent + j * 256 + lane * 8, v);
          }
        }
        if (rope) {
          const float v[2] = {__uint_as_float(rw[u] << 16), __uint_as_float(rw[u] & 0xFFFF0000u)};
          store_f32<T, 2>(rope + t * ld_rope + lane * 2, v);
        }
      }
      if (page[u]) {
        float v[4];
        if (D.idx_fmt == HS_IDX_FP8) {
          values4(kw[u], ks[u], v);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(kw[u] >> (8 * i)) * ks[u];
        }
        store_f32<T, 4>(keys + t * ld_keys + lane * 4, v);
      }
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
  if (!p || layer < 0 || layer >= p->cfg.n_layers || n < 0 || n > HS_CACHE_MAX_TOKENS) return a;
  const int size = dtype_size(dtype);
  if (size == 0 || !on_pool_device(p)) return a;
  if (n > 0) {
    if (!d_req || !d_pos || !words_ok(d_req) || !words_ok(d_pos) || (!d_latent && !d_rope && !d_keys)) return a;
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

// Tokens of a warp: as many as deal them to CA_SM_WARPS warps per SM, at least `least` at a time.
int tokens_per_warp(int n, int least) {
  const int warps = num_sms() * CA_SM_WARPS, per = (n + warps - 1) / warps;
  return per < least ? least : per > 32 ? 32 : per;
}
int cache_grid(int n, int per_warp) { return (int)(((long long)n + CA_WARPS * per_warp - 1) / (CA_WARPS * per_warp)); }

template <typename T>
hs_status launch_append_quantized(hs_pool* p, int layer, int n, const int32_t* d_req, const int32_t* d_pos,
                                  const void* d_latent, int64_t ld_latent, const void* d_rope, int64_t ld_rope,
                                  const void* d_keys, int64_t ld_keys, float key_scale, cudaStream_t st) {
  const int per = tokens_per_warp(n, 1);
  return launch_pdl(append_quantized_kernel<T>, dim3(cache_grid(n, per)), dim3(CA_WARPS * 32), 0, st, 0,
                    p->d, layer, layer / p->d.lpi, n, per, d_req, d_pos, static_cast<const T*>(d_latent), (long long)ld_latent,
                    static_cast<const T*>(d_rope), (long long)ld_rope, static_cast<const T*>(d_keys),
                    (long long)ld_keys, key_scale);
}
template <typename T>
hs_status launch_read_rows(hs_pool* p, int layer, int n, const int32_t* d_req, const int32_t* d_pos, void* d_latent,
                           int64_t ld_latent, void* d_rope, int64_t ld_rope, void* d_keys, int64_t ld_keys,
                           float key_scale, cudaStream_t st) {
  const int per = tokens_per_warp(n, CA_READ);
  return launch_pdl(read_rows_kernel<T>, dim3(cache_grid(n, per)), dim3(CA_WARPS * 32), 0, st, 0, p->d,
                    layer, layer / p->d.lpi, n, per, d_req, d_pos, static_cast<T*>(d_latent), (long long)ld_latent, static_cast<T*>(d_rope),
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
