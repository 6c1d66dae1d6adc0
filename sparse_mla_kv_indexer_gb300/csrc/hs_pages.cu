// Pages that requests share: forks of a request, copies and moves of pages, and the tables read back.
//
// "vLLM introduces Hybrid HiSparse hybrid sparse offloading for GLM 5.3" (vLLM blog Part 1), section
// "How it works": the block table holds real blocks and empty placeholders, and hot-buffer pages come
// from the same pool. So a request can begin with another one's pages by naming them, and a page can go
// anywhere in the pool as long as every table that names it follows.
//
// All of it is copying: bytes read once and written once bound the large calls, launches the small ones. 2,500
// pages of 4 layers and 2 indexers (924 MB) move in 157 us, 11 of them for the check, the copies at 6.3 TB/s
// (136 us in all at the copy rate); 48 forks of three prompts, 8 layers, take 7 us.
#include <math.h>

#include "hs_chunk.cuh"
#include "hs_pages.cuh"

namespace hs {

namespace {

constexpr int KV_CHUNKS = PAGE * ROW / 16;        // 2,624 16-byte chunks of a page of one layer

// ---- forks ----------------------------------------------------------------------------
// A fork is several CTAs: of its table entries, of its last page's rows in each layer, of its index keys
// in each indexer layer. Each finds for itself whether the fork may be made: no fork writes what decides
// that (a destination is nobody's source).
constexpr int FK_THREADS = 256;
constexpr int FK_ENTRIES = 4;                      // table entries of a thread
struct ForkArgs {
  int n, table_ctas;
  const int32_t *src, *dst, *len, *tail, *idx_tail;
};

__global__ void __launch_bounds__(FK_THREADS) fork_kernel(const Dev D, const ForkArgs A) {
  griddep_wait();
  const int i = blockIdx.y, tid = threadIdx.x;
  const int src = A.src[i], dst = A.dst[i], len = A.len[i];
  const int tail = A.tail[i], idx_tail = A.idx_tail ? A.idx_tail[i] : -1;
  const int whole = len >> 6, rows = len & 63;
  bool bad = false;
  for (int j = tid; j < A.n; j += FK_THREADS) {
    const int from = A.src[j], n = A.len[j];
    const bool other = j != i;
    bad |= from == dst || (other && A.dst[j] == dst);
    if (rows == 0 || (n & 63) == 0) continue;
    bad |= other && (A.tail[j] == tail || (A.idx_tail && A.idx_tail[j] == idx_tail));
    // a page that this call copies rows from is nobody's to write: its reader may come before or after
    if (from >= 0 && from < D.max_requests && n > 0 && n <= D.max_ctx) {
      const size_t at = (size_t)from * D.max_pages + (n >> 6);
      bad |= D.bt[at] == tail || (A.idx_tail && D.idx_bt[at] == idx_tail);
    }
  }
  if (src < 0 || src >= D.max_requests || dst < 0 || dst >= D.max_requests || len < 0 || len > D.max_ctx) bad = true;
  const uint8_t* page = nullptr;    // of the CTA's layer
  int from_idx = -1, err = HS_OK;
  const int piece = blockIdx.x - A.table_ctas;     // < 0: table entries; then layers, then indexer layers
  if (!bad && rows) {
    const size_t at = (size_t)src * D.max_pages + whole;
    page = page_rows(D, piece >= 0 && piece < D.n_layers ? piece : 0, src, whole, &err);
    bad |= tail < 0 || tail >= D.num_pages;
    if (A.idx_tail) {
      from_idx = D.idx_bt[at];
      bad |= idx_tail < 0 || idx_tail >= D.num_idx_pages || from_idx < 0 || from_idx >= D.num_idx_pages;
    }
    if (bad) err = HS_ERR_BAD_ID;
  }
  const int any = __syncthreads_or(bad);
  if (any || err != HS_OK) {
    if (blockIdx.x == 0 && tid == 0) set_status(D.status, any ? HS_ERR_BAD_ID : err);
    return;
  }
  if (piece < 0) {
    const size_t from = (size_t)src * D.max_pages, to = (size_t)dst * D.max_pages;
    const int first = blockIdx.x * FK_THREADS * FK_ENTRIES + tid;
    int32_t b[FK_ENTRIES], x[FK_ENTRIES];
    int64_t h[FK_ENTRIES];
#pragma unroll
    for (int k = 0; k < FK_ENTRIES; ++k) {
      const int e = first + k * FK_THREADS;
      if (e < whole) b[k] = D.bt[from + e], x[k] = D.idx_bt[from + e], h[k] = D.host_pg[from + e];
    }
#pragma unroll
    for (int k = 0; k < FK_ENTRIES; ++k) {
      const int e = first + k * FK_THREADS;
      if (e < whole) D.bt[to + e] = b[k], D.idx_bt[to + e] = x[k], D.host_pg[to + e] = h[k];
    }
    if (blockIdx.x == 0 && tid == 0 && rows) {
      D.bt[to + whole] = tail;
      D.host_pg[to + whole] = -1;
      if (A.idx_tail) D.idx_bt[to + whole] = idx_tail;
    }
    // a later kernel may read the tables before it waits for this one's end (which it starts after)
    __threadfence();
  } else if (rows) {
    const bool kv = piece < D.n_layers;
    const uint4* from;
    uint4* to;
    int chunks;
    if (kv) {
      from = reinterpret_cast<const uint4*>(page);
      to = reinterpret_cast<uint4*>(D.kv[piece] + (size_t)tail * PAGE * ROW);
      chunks = rows * ROW_CHUNKS;
    } else {
      if (!A.idx_tail) return;
      int8_t* keys = D.idx[piece - D.n_layers];
      from = reinterpret_cast<const uint4*>(keys + (size_t)from_idx * D.idx_page_bytes);
      to = reinterpret_cast<uint4*>(keys + (size_t)idx_tail * D.idx_page_bytes);
      chunks = rows * (IDX_DIM / 16);
      if (D.idx_fmt == HS_IDX_FP8 && tid < rows)   // the keys' scales, behind the page's keys
        reinterpret_cast<uint32_t*>(to)[PAGE * IDX_DIM / 4 + tid] =
            reinterpret_cast<const uint32_t*>(from)[PAGE * IDX_DIM / 4 + tid];
    }
    constexpr int AHEAD = 11;   // of 63 x 41 chunks, 256 threads: all in flight at once
    uint4 v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (tid + k * FK_THREADS < chunks) v[k] = from[tid + k * FK_THREADS];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (tid + k * FK_THREADS < chunks) to[tid + k * FK_THREADS] = v[k];
    static_assert(63 * ROW_CHUNKS <= AHEAD * FK_THREADS, "chunks of a last page");
  }
}

// ---- copies and moves -----------------------------------------------------------------
// Two launches: which copies are made, then the copies themselves, with the tables' entries beside them. Of few
// copies (at most CP_FEW of either kind) every CTA of the second finds that out for itself, and looks table entries up
// in a hash table of its own: a launch less. 7 pages of 4 layers moved, one call after the other, in 10.3 us instead
// of 12.5; on the GPU, caches flushed, 7 pages copied in 8.2 instead of 10.2, 64 in 10.2 to 12.3 instead of 12.3;
// moved, with the tables of 256 requests of 2^20 tokens, 7 in 22.5 either way and 64 in 24.6 to 26.6 instead of 26.6.
// So at 64 the two are about alike. Comparing each entry with all the moved pages took 43 and 197 there.
constexpr int CP_THREADS = 512, CP_WARPS = CP_THREADS / 32;
struct CopyList {
  int n, pages;               // copies; pages of this kind in the pool
  const int32_t *from, *to;
};
struct CopyArgs {
  CopyList kv, idx;
  int remap, remap_ctas, kv_ctas;   // CTAs of the second launch: tables, then KV pages, then index pages
};

// Every copy against all the others of its kind, a warp each, from shared memory: at most 4,096 x 8,192
// comparisons of whole numbers over the whole GPU are less than building a table of the pages in every CTA was
// (10 us for 2,500 pages; the search for an entry's page in it 20 us). With remap the copies that are made are
// marked in the pool's array of pages, with a number of the call's own, so that nothing has to be cleared. The number
// is taken here, by the last CTA that has read the one before: whether or not the copies are launched, no later call
// has it again, and finds marks of its own alone.
__global__ void __launch_bounds__(CP_THREADS) check_copies_kernel(const Dev D, const CopyArgs A) {
  extern __shared__ int32_t named[];
  griddep_wait();
  const bool kv = blockIdx.y == 0;
  const CopyList L = kv ? A.kv : A.idx;
  __shared__ uint32_t number;
  if (A.remap && threadIdx.x == 0) {
    uint32_t* const e = copy_epoch(D);
    const uint32_t mine = __ldcg(e) + 1;
    number = mine;
    __threadfence();
    if (atomicAdd(e + 1, 1) == gridDim.x * gridDim.y - 1) e[0] = mine, e[1] = 0;
  }
  int32_t *const from = named, *const to = named + L.n;
  #pragma unroll 8
  for (int i = threadIdx.x; i < L.n; i += CP_THREADS) from[i] = L.from[i], to[i] = L.to[i];
  __syncthreads();
  const int epoch = A.remap ? (int)number : 0;
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x * CP_WARPS + (threadIdx.x >> 5); i < L.n; i += gridDim.x * CP_WARPS) {
    const int f = from[i], d = to[i];
    int sources = 0, dests = 0, chained = 0;
#pragma unroll 4
    for (int j = lane; j < L.n; j += 32) {
      const int fj = from[j];
      sources += fj == f;
      chained |= fj == d;
      dests += to[j] == d;
    }
    sources = __reduce_add_sync(0xffffffffu, sources);
    dests = __reduce_add_sync(0xffffffffu, dests);
    chained = __reduce_or_sync(0xffffffffu, chained);
    const bool ok = f >= 0 && f < L.pages && d >= 0 && d < L.pages && dests == 1 && !chained && (!A.remap || sources == 1);
    if (lane == 0) {
      copy_made_flags(D, kv)[i] = ok;
      if (!ok) set_status(D.status, HS_ERR_BAD_ID);
      else if (A.remap) page_map(D, kv)[f] = make_int2(epoch, d);
    }
  }
}

// A warp's unit is 1/8 of a page of one layer (5,248 bytes) or 1/2 of an index page of one indexer layer,
// all of its loads in flight at once, and the next unit's pages beside them.
constexpr int CP_KV_SLICES = 8, CP_IDX_SLICES = 2, CP_AHEAD = 11;
static_assert(KV_CHUNKS / CP_KV_SLICES <= 32 * CP_AHEAD && HS_IDX_FP8_PAGE_BYTES / 16 / CP_IDX_SLICES <= 32 * CP_AHEAD, "unit");
constexpr int RM_ENTRIES = 8;      // table entries of a thread at a time

struct MarkedPages {      // where a page went: the call's marks in the pool's array
  const int2* map;
  int pages, epoch;
  __device__ int at(int page) const {
    if (page < 0 || page >= pages) return -1;
    const int2 m = map[page];
    return m.x == epoch ? m.y : -1;
  }
};
constexpr int CP_FEW = 64;
struct FewCopies {        // in shared memory; `from` is -1 of copies that are not made
  int32_t from[CP_FEW], to[CP_FEW];
};
constexpr int CP_SLOTS = 1024;
struct FewPages {         // where a page went: open addressing in shared memory, at most CP_FEW of CP_SLOTS taken
  int2* slots;
  __device__ int at(int page) const {
    if (page < 0) return -1;
    for (int h = page & (CP_SLOTS - 1);; h = (h + 1) & (CP_SLOTS - 1)) {   // ends at the first free slot
      const int2 m = slots[h];
      if (m.x == page) return m.y;
      if (m.x < 0) return -1;
    }
  }
};
// All threads: the copies that are made into an empty table.
__device__ __forceinline__ void few_slots(int2* slots, const FewCopies& c, int n) {
  __syncthreads();
  for (int i = threadIdx.x; i < CP_SLOTS; i += CP_THREADS) slots[i] = make_int2(-1, -1);
  __syncthreads();
  const int i = threadIdx.x;
  if (i < n && c.from[i] >= 0) {   // sources differ
    int h = c.from[i] & (CP_SLOTS - 1);
    while (atomicCAS(&slots[h].x, -1, c.from[i]) != -1) h = (h + 1) & (CP_SLOTS - 1);
    slots[h].y = c.to[i];
  }
  __syncthreads();
}
// All threads: the copies of a list that are made, by the rules above; whether this thread's is one that is not.
__device__ __forceinline__ bool few_made(FewCopies& c, const CopyList& L, bool remap) {
  const int i = threadIdx.x;
  const int f = i < L.n ? L.from[i] : -1, d = i < L.n ? L.to[i] : -1;
  __syncthreads();
  if (i < L.n) c.from[i] = f, c.to[i] = d;
  __syncthreads();
  int sources = 0, dests = 0, chained = 0;
  if (i < L.n)
    for (int j = 0; j < L.n; ++j) {
      const int fj = c.from[j];
      sources += fj == f;
      chained |= fj == d;
      dests += c.to[j] == d;
    }
  const bool ok = f >= 0 && f < L.pages && d >= 0 && d < L.pages && dests == 1 && !chained && (!remap || sources == 1);
  __syncthreads();
  if (i < L.n && !ok) c.from[i] = -1;
  __syncthreads();
  return i < L.n && !ok;
}
// The entries of a table that name a moved page.
template <typename Pages>
__device__ __forceinline__ void remap_table(int32_t* entries, long long n, const Pages& moved, int cta, int ctas) {
  const long long stride = (long long)ctas * CP_THREADS;
  for (long long e0 = (long long)cta * CP_THREADS + threadIdx.x; e0 < n; e0 += RM_ENTRIES * stride) {
    int32_t v[RM_ENTRIES], to[RM_ENTRIES];
#pragma unroll
    for (int k = 0; k < RM_ENTRIES; ++k) v[k] = e0 + k * stride < n ? entries[e0 + k * stride] : -1;
#pragma unroll
    for (int k = 0; k < RM_ENTRIES; ++k) to[k] = moved.at(v[k]);
#pragma unroll
    for (int k = 0; k < RM_ENTRIES; ++k)
      if (to[k] >= 0) entries[e0 + k * stride] = to[k];
  }
}

template <bool FEW>
__global__ void __launch_bounds__(CP_THREADS, 2) copy_pages_kernel(const Dev D, const CopyArgs A) {
  __shared__ FewCopies few;
  griddep_wait();
  int cta = blockIdx.x;
  if (cta < A.remap_ctas) {
    const long long n = (long long)D.max_requests * D.max_pages, hot = (long long)D.max_requests * D.n_groups * D.hot_pages_max;
    auto remap = [&](bool kv, const auto& moved) {
      remap_table(kv ? D.bt : D.idx_bt, n, moved, cta, A.remap_ctas);
      if (kv) remap_table(D.hot_pages, hot, moved, cta, A.remap_ctas);
    };
    if constexpr (FEW) {
      __shared__ int2 slots[CP_SLOTS];
      for (int kind = 0; kind < 2; ++kind) {
        const CopyList L = kind == 0 ? A.kv : A.idx;
        if (L.n == 0) continue;
        few_made(few, L, true);
        few_slots(slots, few, L.n);
        remap(kind == 0, FewPages{slots});
      }
    } else {
      const int epoch = (int)copy_epoch(D)[0];
      if (A.kv.n > 0) remap(true, MarkedPages{page_map(D, true), D.num_pages, epoch});
      if (A.idx.n > 0) remap(false, MarkedPages{page_map(D, false), D.num_idx_pages, epoch});
    }
    __threadfence();   // as the forks'
    return;
  }
  cta -= A.remap_ctas;
  const bool kv = cta < A.kv_ctas;
  const CopyList L = kv ? A.kv : A.idx;
  const uint8_t* const ok = copy_made_flags(D, kv);
  const int ctas = kv ? A.kv_ctas : gridDim.x - A.remap_ctas - A.kv_ctas;
  if (!kv) cta -= A.kv_ctas;
  if constexpr (FEW) {
    if (few_made(few, L, A.remap) && cta == 0) set_status(D.status, HS_ERR_BAD_ID);
  }
  const int lane = threadIdx.x & 31, slices = kv ? CP_KV_SLICES : CP_IDX_SLICES, per_page = (kv ? D.n_layers : D.n_groups) * slices;
  const int page_bytes = kv ? PAGE * ROW : D.idx_page_bytes, chunks = page_bytes / 16 / slices;
  const int units = L.n * per_page, step = ctas * CP_WARPS;   // at most 4,096 x 64 x 8
  int u = cta * CP_WARPS + (threadIdx.x >> 5);
  if (u >= units) return;
  int i = u / per_page, f, d;
  bool made;
  auto look_up = [&]() {
    if constexpr (FEW) {
      f = few.from[i], d = few.to[i], made = f >= 0;
    } else {
      f = L.from[i], d = L.to[i], made = ok[i];
    }
  };
  look_up();
  while (u < units) {
    const int r = u - i * per_page, layer = r / slices, slice = r - layer * slices;
    uint8_t* const pages = kv ? D.kv[layer] : reinterpret_cast<uint8_t*>(D.idx[layer]);
    const uint4* const from = reinterpret_cast<const uint4*>(pages + (size_t)(made ? f : 0) * page_bytes) + slice * chunks;
    uint4* const to = reinterpret_cast<uint4*>(pages + (size_t)(made ? d : 0) * page_bytes) + slice * chunks;
    uint4 v[CP_AHEAD];
#pragma unroll
    for (int k = 0; k < CP_AHEAD; ++k)
      if (made && lane + 32 * k < chunks) v[k] = __ldcs(from + lane + 32 * k);
    const bool now = made;
    u += step;
    if (u < units) {
      i = u / per_page;
      look_up();
    }
#pragma unroll
    for (int k = 0; k < CP_AHEAD; ++k)
      if (now && lane + 32 * k < chunks) __stcs(to + lane + 32 * k, v[k]);
  }
}

// ---- the tables -----------------------------------------------------------------------
__global__ void __launch_bounds__(256) get_pages_kernel(const Dev D, int n, const int32_t* __restrict__ req, int first, int count,
                                                        int32_t* bt, int32_t* idx, int64_t* host) {
  griddep_wait();
  const long long total = (long long)n * count, stride = (long long)gridDim.x * blockDim.x;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < total; e += stride) {
    const int i = (int)(e / count), r = req[i];
    const bool ok = r >= 0 && r < D.max_requests;
    if (!ok) set_status(D.status, HS_ERR_BAD_ID);
    const size_t at = (size_t)(ok ? r : 0) * D.max_pages + first + (e - (long long)i * count);
    if (bt) bt[e] = ok ? D.bt[at] : -1;
    if (idx) idx[e] = ok ? D.idx_bt[at] : -1;
    if (host) host[e] = ok ? D.host_pg[at] : -1;
  }
}

}  // namespace

}  // namespace hs

using namespace hs;

extern "C" hs_status hs_fork_requests(hs_pool* p, int32_t n, const int32_t* d_src, const int32_t* d_dst, const int32_t* d_len,
                                      const int32_t* d_tail, const int32_t* d_idx_tail, hs_stream_t stream) {
  CallRange nvtx_range("hs_fork_requests");
  if (!p || n < 0 || n > p->cfg.max_requests || !on_pool_device(p)) return HS_ERR_INVALID;
  if (n > 0 && (!d_src || !d_dst || !d_len || !d_tail || !words_ok(d_src) || !words_ok(d_dst) || !words_ok(d_len) ||
                !words_ok(d_tail) || !words_ok(d_idx_tail)))
    return HS_ERR_INVALID;
  p->settled_rows = nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int table_ctas = (p->d.max_pages + FK_THREADS * FK_ENTRIES - 1) / (FK_THREADS * FK_ENTRIES);
  if (n == 0) return HS_OK;
  if (n > 65535) return HS_ERR_INVALID;   // the grid's second dimension
  const ForkArgs a = {n, table_ctas, d_src, d_dst, d_len, d_tail, d_idx_tail};
  return launch_pdl(fork_kernel, dim3(table_ctas + p->d.n_layers + p->d.n_groups, n), dim3(FK_THREADS), 0, st, 0, p->d, a);
}

extern "C" hs_status hs_copy_pages(hs_pool* p, int32_t n, const int32_t* d_from, const int32_t* d_to, int32_t n_idx,
                                   const int32_t* d_idx_from, const int32_t* d_idx_to, int32_t remap, hs_stream_t stream) {
  CallRange nvtx_range("hs_copy_pages");
  if (!p || n < 0 || n > HS_COPY_MAX_PAGES || n_idx < 0 || n_idx > HS_COPY_MAX_PAGES || !on_pool_device(p)) return HS_ERR_INVALID;
  if (n > 0 && (!d_from || !d_to || !words_ok(d_from) || !words_ok(d_to))) return HS_ERR_INVALID;
  if (n_idx > 0 && (!d_idx_from || !d_idx_to || !words_ok(d_idx_from) || !words_ok(d_idx_to))) return HS_ERR_INVALID;
  p->settled_rows = nullptr;
  if (n == 0 && n_idx == 0) return HS_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CopyArgs a = {};
  a.kv = {n, p->cfg.num_pages, d_from, d_to};
  a.idx = {n_idx, p->cfg.num_idx_pages, d_idx_from, d_idx_to};
  a.remap = remap != 0;
  const int sms = num_sms(), most_listed = n > n_idx ? n : n_idx, checks = (most_listed + CP_WARPS - 1) / CP_WARPS;
  const bool few = most_listed <= CP_FEW;
  if (!few) {
    const hs_status s = launch_pdl(check_copies_kernel, dim3(checks < sms ? checks : sms, 2), dim3(CP_THREADS), most_listed * 8, st, 0, p->d, a);
    if (s != HS_OK) return s;
  }
  // CTAs for both kinds by their bytes, two on an SM
  const long long kv_units = (long long)n * p->d.n_layers * CP_KV_SLICES, idx_units = (long long)n_idx * p->d.n_groups * CP_IDX_SLICES;
  const long long kv_bytes = (long long)n * p->d.n_layers * PAGE * ROW, idx_bytes = (long long)n_idx * p->d.n_groups * p->d.idx_page_bytes;
  const auto ctas_for = [&](long long units, long long bytes) -> int {
    if (units == 0) return 0;
    const long long share = (long long)(2.0 * sms * bytes / (kv_bytes + idx_bytes)), need = (units + CP_WARPS - 1) / CP_WARPS;
    const long long c = share < 1 ? 1 : share;
    return (int)(c < need ? c : need);
  };
  a.kv_ctas = ctas_for(kv_units, kv_bytes);
  if (remap) {
    const long long entries = (long long)p->cfg.max_requests * p->d.max_pages, each = CP_THREADS * RM_ENTRIES;
    a.remap_ctas = (int)((entries + each - 1) / each < sms ? (entries + each - 1) / each : sms);
  }
  const int ctas = a.remap_ctas + a.kv_ctas + ctas_for(idx_units, idx_bytes);
  return few ? launch_pdl(copy_pages_kernel<true>, dim3(ctas), dim3(CP_THREADS), 0, st, 0, p->d, a)
             : launch_pdl(copy_pages_kernel<false>, dim3(ctas), dim3(CP_THREADS), 0, st, 0, p->d, a);
}

extern "C" hs_status hs_get_pages(hs_pool* p, int32_t n, const int32_t* d_req, int32_t first, int32_t count, int32_t* d_bt,
                                  int32_t* d_idx, int64_t* d_host, hs_stream_t stream) {
  CallRange nvtx_range("hs_get_pages");
  if (!p || n < 0 || first < 0 || count < 0 || (long long)first + count > p->d.max_pages || n > HS_CACHE_MAX_TOKENS ||
      !on_pool_device(p))
    return HS_ERR_INVALID;
  if (n > 0 && count > 0 && (!d_req || !words_ok(d_req) || !words_ok(d_bt) || !words_ok(d_idx) ||
                             (reinterpret_cast<uintptr_t>(d_host) & 7)))
    return HS_ERR_INVALID;
  p->settled_rows = nullptr;
  if (n == 0 || count == 0 || (!d_bt && !d_idx && !d_host)) return HS_OK;
  const long long need = ((long long)n * count + 255) / 256, most = (long long)num_sms() * 8;
  return launch_pdl(get_pages_kernel, dim3((unsigned)(need < most ? need : most)), dim3(256), 0,
                    reinterpret_cast<cudaStream_t>(stream), 0, p->d, n, d_req, first, count, d_bt, d_idx, d_host);
}
