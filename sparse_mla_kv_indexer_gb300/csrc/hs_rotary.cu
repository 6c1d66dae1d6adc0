// Rotary positions of queries and keys, before they are appended or attend.
//
// "Serving GLM-5.3 with PCP, DCP and Hybrid HiSparse" (vLLM blog Part 2), footnote 1: 64 of a cached
// row's 576 dims are rope. Of every pair (a, b) of a head's rotated dims, pair i of position p:
//   (a, b) -> magnitude (a cos w - b sin w, a sin w + b cos w),   w = p f_i.
//
// Angles. In turns, p f / 2 pi mod 1 is p times a step of 2^-64 turns mod 2^64: whole numbers,
// exact for every 32-bit position, where p f in fp32 is off by 0.08 radian at a million. The step
// is f / 2 pi rounded to the nearest, so the angle is off by 2^-34 turns at most (position 2^31). Of the phase
// the nearest quarter turn is taken off (by swapping and negating), and the rest, at most an
// eighth of a turn, is rounded to its own 24 bits before sincospif: cosines and sines are as good
// near their zeros, relative to themselves, as elsewhere, and there is no table of positions to read.
//
// Work. A CTA takes a few tokens and all of their heads (part of them when there are fewer tokens
// than SMs): its threads begin with the loads of their first values, then work out the cosines and
// sines of its tokens, once for all heads, into shared memory. A thread's unit is as many pairs as
// two 16-byte loads hold: neighbours, or eight of either half of the dims (bf16).
//
// Bytes bound the large calls: 16,411 tokens of 130 heads (546 MB) take 94 us, 5.8 TB/s, where a plain contiguous
// copy of as many bytes takes 90 us measured alike (80.6 us at the copy rate). With one, two and four units
// of a thread in flight instead of three they took 9 to 30, 16 and 11 us more. A decode's token is a launch: 3.3 us on the GPU.
#include <math.h>

#include "hs_chunk.cuh"

namespace hs {

namespace {

constexpr int RO_THREADS = 512;      // at most
constexpr int RO_SOME = 256;         // what a CTA of few rows is filled up to
constexpr int RO_RESIDENT = 2;       // CTAs of as many threads on an SM, by their registers
constexpr int RO_PARTS = HS_ROTARY_MAX_PARTS;
constexpr int RO_MAX_PAIRS = HS_ROTARY_MAX_DIMS / 2;
constexpr int RO_TABLE = 2048;       // (cos, sin) of a CTA's tokens, at most
constexpr int RO_AHEAD = 3;          // units of a thread in flight

struct RotaryPart {
  const void* in;
  void* out;
  long long in_tok, in_head, out_tok, out_head;
  int first, halves;   // the part's first row among all parts' heads; layout
};
struct RotaryArgs {
  const int32_t* pos;
  const uint64_t* steps;
  int n, pairs, n_parts, heads;      // heads: of all parts together
  int tokens, rows, splits;          // of a CTA: tokens, heads; CTAs per group of tokens
  float magnitude, sign;
  RotaryPart part[RO_PARTS];
};

// cos and sin of `phase` 2^-64 turns. All 62 bits of what lies beside the nearest quarter are converted: of its upper 30
// alone a phase of 2^-26 turns (a slow pair at an early position) keeps six bits.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const float x = (float)(int64_t)(phase - ((uint64_t)quarter << 62)) * 1.0842021724855044e-19f;   // 2^-63: in half turns
  float s, c;
  sincospif(x, &s, &c);
  const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
  return make_float2(((quarter + 1) & 2) ? -u : u, (quarter & 2) ? -v : v);
}

// V pairs of one row: V neighbouring pairs, or V values of either half, as they are stored.
template <typename T, int V>
struct Unit {
  T a[V], b[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_values(T (&to)[V], const T* from) {
  if constexpr (V * sizeof(T) == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    memcpy(to, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) to[i] = from[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_values(T* to, const T (&from)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    uint4 v;
    memcpy(&v, from, 16);
    *reinterpret_cast<uint4*>(to) = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) to[i] = from[i];
  }
}
// (a, b) -> (a c - b s, a s + b c) of V pairs, two at a time; c and s in shared memory.
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float* c, const float* s) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(c + j), s4 = *reinterpret_cast<const uint4*>(s + j);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const F2 x = f2(__float_as_uint(a[j + k]), __float_as_uint(a[j + k + 1])), y = f2(__float_as_uint(b[j + k]), __float_as_uint(b[j + k + 1]));
        const F2 cc = k ? f2(c4.z, c4.w) : f2(c4.x, c4.y), ss = k ? f2(s4.z, s4.w) : f2(s4.x, s4.y);
        const F2 minus_y = f2(__float_as_uint(-b[j + k]), __float_as_uint(-b[j + k + 1]));
        unpack(fma2(x, cc, mul2(minus_y, ss)), a[j + k], a[j + k + 1]);
        unpack(fma2(x, ss, mul2(y, cc)), b[j + k], b[j + k + 1]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * c[j] - y * s[j];
      b[j] = x * s[j] + y * c[j];
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(RO_THREADS, RO_RESIDENT) rotary_kernel(const __grid_constant__ RotaryArgs A) {
  __shared__ __align__(16) float cosines[RO_TABLE], sines[RO_TABLE];
  griddep_wait();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int group = blockIdx.x / A.splits, split = blockIdx.x - group * A.splits;
  const int tok0 = group * A.tokens, n_tok = min(A.tokens, A.n - tok0);
  const int row0 = split * A.rows, n_rows = min(A.rows, A.heads - row0), all = n_tok * n_rows;
  // a thread has the same pairs of every row that it takes
  const int per_head = A.pairs / V, step = threads / per_head, mine = tid / per_head, at = (tid - mine * per_head) * V;
  struct Place {
    T* out;
    int halves, cs;   // the row's layout; where its cosines are
  };
  auto load = [&](int row, Unit<T, V>& x) {
    Place p;
    const int tk = n_tok == 1 ? 0 : row / n_rows, h = row0 + row - tk * n_rows;
    int k = 0;
#pragma unroll
    for (int i = 1; i < RO_PARTS; ++i)
      if (i < A.n_parts && h >= A.part[i].first) k = i;
    const RotaryPart& P = A.part[k];
    const long long t = tok0 + tk, hd = h - P.first;
    const int lo = P.halves ? at : 2 * at;
    p.halves = P.halves;
    p.cs = tk * A.pairs + at;
    p.out = static_cast<T*>(P.out) + t * P.out_tok + hd * P.out_head + lo;
    const T* in = static_cast<const T*>(P.in) + t * P.in_tok + hd * P.in_head + lo;
    load_values(x.a, in);
    load_values(x.b, in + (P.halves ? A.pairs : V));
    return p;
  };
  Unit<T, V> x[RO_AHEAD];
  Place p[RO_AHEAD];
#pragma unroll
  for (int i = 0; i < RO_AHEAD; ++i)
    if (mine < step && mine + i * step < all) p[i] = load(mine + i * step, x[i]);
  for (int i = tid; i < n_tok * A.pairs; i += threads) {
    const int tk = i / A.pairs;
    const float2 cs = cos_sin((uint64_t)(int64_t)A.pos[tok0 + tk] * A.steps[i - tk * A.pairs]);
    cosines[i] = cs.x * A.magnitude;
    sines[i] = cs.y * A.magnitude * A.sign;
  }
  __syncthreads();
  for (int r0 = mine < step ? mine : all; r0 < all; r0 += RO_AHEAD * step) {
    if (r0 != mine) {
#pragma unroll
      for (int i = 0; i < RO_AHEAD; ++i)
        if (r0 + i * step < all) p[i] = load(r0 + i * step, x[i]);
    }
#pragma unroll
    for (int i = 0; i < RO_AHEAD; ++i) {
      if (r0 + i * step >= all) break;
      float a[V], b[V];
      Unit<T, V> y;
      if (p[i].halves) {
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = to_f32(x[i].a[j]), b[j] = to_f32(x[i].b[j]);
        turn(a, b, cosines + p[i].cs, sines + p[i].cs);
#pragma unroll
        for (int j = 0; j < V; ++j) y.a[j] = from_f32<T>(a[j]), y.b[j] = from_f32<T>(b[j]);
      } else {   // the 2 V values in order: pair j is values 2 j and 2 j + 1
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) (j & 1 ? b : a)[j >> 1] = to_f32(j < V ? x[i].a[j] : x[i].b[j - V]);
        turn(a, b, cosines + p[i].cs, sines + p[i].cs);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) (j < V ? y.a[j] : y.b[j - V]) = from_f32<T>((j & 1 ? b : a)[j >> 1]);
      }
      store_values(p[i].out, y.a);
      store_values(p[i].out + (p[i].halves ? A.pairs : V), y.b);
    }
  }
  // The sparse attention and the indexer read their queries before they wait for this kernel's end (after which they
  // start), and those may be any tokens of this call: the last of a prefill chunk, or of requests that decode beside
  // it. So the CTA's stores are done when it ends. (16,411 tokens of 130 heads 90.8 us without this, 93.6 so, 98.0 with
  // a fence by every thread.)
  __syncthreads();
  if (tid == 0) __threadfence();
}

// Whether 16-byte accesses reach every unit of V pairs of this part.
bool wide_part(const hs_rotary_part& p, int pairs, int size) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.d_in) | reinterpret_cast<uintptr_t>(p.d_out);
  const int64_t strides = p.in_stride_token | p.in_stride_head | p.out_stride_token | p.out_stride_head;
  return (at & 15) == 0 && (strides * size & 15) == 0 && (pairs * size & 15) == 0;
}

template <typename T>
hs_status launch_rotary(RotaryArgs& a, bool wide, cudaStream_t st) {
  const int v = wide ? 16 / (int)sizeof(T) : 1, per_head = a.pairs / v, sms = num_sms();
  // tokens of a CTA: one, or of few heads as many as keep 256 threads busy; but at least a CTA for every SM
  int tokens = RO_SOME * RO_AHEAD / (a.heads * per_head);
  const int most = RO_TABLE / a.pairs, spread = (a.n + sms - 1) / sms;
  if (tokens > most) tokens = most;
  if (tokens > spread) tokens = spread;
  a.tokens = tokens < 1 ? 1 : tokens;
  const int groups = (a.n + a.tokens - 1) / a.tokens;
  // few tokens: their heads dealt to several CTAs, a unit per thread
  int rows = a.heads;
  if (groups < sms) {
    const int least = (RO_SOME + per_head * a.tokens - 1) / (per_head * a.tokens);
    const int even = (int)(((long long)a.heads * groups + sms - 1) / sms);
    rows = even > least ? even : least;
    if (rows > a.heads) rows = a.heads;
  }
  a.rows = rows;
  a.splits = (a.heads + rows - 1) / rows;
  // threads: as many as take the rows in the fewest rounds, evenly (130 rows of four units by 288 threads in one
  // round; 256 threads would begin another one for the last two rows)
  const int all = a.tokens * rows, round = RO_THREADS / per_head * RO_AHEAD, rounds = (all + round - 1) / round;
  const int step = (all + rounds * RO_AHEAD - 1) / (rounds * RO_AHEAD), threads = (step * per_head + 31) / 32 * 32;
  const dim3 grid((unsigned)((long long)groups * a.splits));
  return wide ? launch_pdl(rotary_kernel<T, 16 / (int)sizeof(T)>, grid, dim3(threads), 0, st, 0, a)
              : launch_pdl(rotary_kernel<T, 1>, grid, dim3(threads), 0, st, 0, a);
}

bool finite_positive(double x) { return x > 0 && isfinite(x); }
// A frequency as whole 2^-64 turns per position, mod 2^64, to the nearest. 1 / (2 pi) is taken in two doubles (106 bits)
// and the product's own rounding error added back, so that nothing of 163 turns, the largest, is lost: a quotient in
// double is off by 2^-46 turns there, 2^-25 at position 2^21.
uint64_t step_of(double radians) {
  constexpr double inv = 0.15915494309189535, inv_rest = -9.839338337591243e-18;
  const double x = fabs(radians), turns = x * inv, rest = fma(x, inv_rest, fma(x, inv, -turns));
  const double scaled = ldexp(turns - floor(turns), 64), whole = floor(scaled);   // below 2^64
  const uint64_t step = (uint64_t)whole + (uint64_t)llrint(scaled - whole + ldexp(rest, 64));
  return radians < 0 ? 0 - step : step;
}

}  // namespace

}  // namespace hs

using namespace hs;

extern "C" hs_status hs_rotary_steps_of(int32_t n, const double* h_frequencies, uint64_t* h_steps) {
  CallRange nvtx_range("hs_rotary_steps_of");
  if (n < 1 || n > RO_MAX_PAIRS || !h_frequencies || !h_steps) return HS_ERR_INVALID;
  for (int i = 0; i < n; ++i)
    if (!(fabs(h_frequencies[i]) <= HS_ROTARY_MAX_FREQUENCY)) return HS_ERR_INVALID;
  for (int i = 0; i < n; ++i) h_steps[i] = step_of(h_frequencies[i]);
  return HS_OK;
}

extern "C" hs_status hs_rotary_steps(const hs_rotary_config* c, uint64_t* h_steps, float* h_magnitude) {
  CallRange nvtx_range("hs_rotary_steps");
  if (!c || !h_steps || !h_magnitude) return HS_ERR_INVALID;
  const int d = c->dims, kind = c->scaling;
  if (d < 2 || d > HS_ROTARY_MAX_DIMS || d % 2 || !finite_positive(c->theta) || kind < HS_ROTARY_NONE || kind > HS_ROTARY_RAMP)
    return HS_ERR_INVALID;
  if (kind != HS_ROTARY_NONE && !finite_positive(c->factor)) return HS_ERR_INVALID;
  if (kind == HS_ROTARY_THETA && d == 2) return HS_ERR_INVALID;
  const double theta = kind == HS_ROTARY_THETA ? c->theta * pow(c->factor, d / (d - 2.0)) : c->theta;
  double low = 0, high = 0, magnitude = 1;
  if (kind == HS_ROTARY_RAMP) {
    if (!(c->theta > 1) || !finite_positive(c->original_ctx) || !finite_positive(c->beta_fast) || !finite_positive(c->beta_slow) ||
        !isfinite(c->magnitude))
      return HS_ERR_INVALID;
    // the pair that turns beta times over the original context
    auto pair_at = [&](double beta) { return d * log(c->original_ctx / (beta * 6.283185307179586477)) / (2 * log(c->theta)); };
    low = fmax(floor(pair_at(c->beta_fast)), 0);
    high = fmin(ceil(pair_at(c->beta_slow)), d - 1);
    magnitude = 1 + c->magnitude * log(c->factor);
  }
  double f[RO_MAX_PAIRS];
  for (int i = 0; i < d / 2; ++i) {
    f[i] = pow(theta, -2.0 * i / d);
    if (kind == HS_ROTARY_LINEAR) f[i] /= c->factor;
    if (kind == HS_ROTARY_RAMP) {
      const double part = fmin(fmax((i - low) / fmax(high - low, 0.001), 0), 1);
      f[i] = f[i] * (1 - part) + f[i] / c->factor * part;
    }
    if (!(fabs(f[i]) <= HS_ROTARY_MAX_FREQUENCY)) return HS_ERR_INVALID;
  }
  if (!(fabs(magnitude) <= 3.0e38)) return HS_ERR_INVALID;
  *h_magnitude = (float)magnitude;
  return hs_rotary_steps_of(d / 2, f, h_steps);
}

extern "C" hs_status hs_rotary(hs_pool* p, int32_t n, const int32_t* d_pos, int32_t dims, const uint64_t* d_steps,
                               float magnitude, int32_t inverse, int32_t dtype, int32_t n_parts,
                               const hs_rotary_part* parts, hs_stream_t stream) {
  CallRange nvtx_range("hs_rotary");
  const int size = dtype_size(dtype);
  if (!p || n < 0 || n > HS_CACHE_MAX_TOKENS || dims < 2 || dims > HS_ROTARY_MAX_DIMS || dims % 2 || size == 0 ||
      !isfinite(magnitude) || n_parts < 1 || n_parts > RO_PARTS || !parts || !on_pool_device(p))
    return HS_ERR_INVALID;
  RotaryArgs a = {};
  a.pos = d_pos, a.steps = d_steps, a.n = n, a.pairs = dims / 2, a.n_parts = n_parts;
  a.magnitude = magnitude, a.sign = inverse ? -1.f : 1.f;
  bool wide = true;
  for (int i = 0; i < n_parts; ++i) {
    const hs_rotary_part& q = parts[i];
    if (q.heads < 1 || q.heads > HS_ROTARY_MAX_HEADS || (q.layout != HS_ROTARY_PAIRS && q.layout != HS_ROTARY_HALVES))
      return HS_ERR_INVALID;
    const auto stride = [](int64_t s, int64_t least) { return s >= least && s < (1ll << 40); };
    if (!stride(q.in_stride_token, 0) || !stride(q.in_stride_head, 0) || !stride(q.out_stride_token, n > 1 ? dims : 0) ||
        !stride(q.out_stride_head, q.heads > 1 ? dims : 0))
      return HS_ERR_INVALID;
    if (n > 0) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(q.d_in) | reinterpret_cast<uintptr_t>(q.d_out);
      if (!q.d_in || !q.d_out || at % size) return HS_ERR_INVALID;
      // in place: every unit is read by the thread that writes it
      if (q.d_in == q.d_out && ((n > 1 && q.in_stride_token != q.out_stride_token) ||
                                (q.heads > 1 && q.in_stride_head != q.out_stride_head)))
        return HS_ERR_INVALID;
    }
    a.part[i] = {q.d_in, q.d_out, q.in_stride_token, q.in_stride_head, q.out_stride_token, q.out_stride_head, a.heads,
                 q.layout == HS_ROTARY_HALVES};
    a.heads += q.heads;
    wide &= wide_part(q, a.pairs, size);
  }
  if (n > 0 && (!d_pos || !words_ok(d_pos) || !d_steps || (reinterpret_cast<uintptr_t>(d_steps) & 7))) return HS_ERR_INVALID;
  p->settled_rows = nullptr;
  if (n == 0) return HS_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == HS_BF16   ? launch_rotary<__nv_bfloat16>(a, wide, st)
         : dtype == HS_FP16 ? launch_rotary<__half>(a, wide, st)
                            : launch_rotary<float>(a, wide, st);
}
