// pages.cu -- the pages of the caches: reserve, fork, free, compact and copy
// (include/stv.h, stv_page_*).
//
// The books (refs, tables, counts) live on the device and one CTA changes
// them: it checks the whole call first, so that a call with anything wrong
// changes nothing.  Free pages are found without a free list: a bit per page
// (refs > 0) in shared memory with a running count per 32 pages, after which
// the r-th free or the r-th live page is a binary search, so every new page is
// the lowest free one and nothing depends on the order of atomics.  Fork,
// compact and copy leave a list of (source, destination) pages in the
// workspace, which a second launch copies in every layer.
//
// Bounds: the books are a few dependent global round trips and barriers in
// one CTA (latency); the copies are bound by HBM, two bytes moved per byte of
// page.
#include <string.h>

#include <algorithm>

#include "stv_device.cuh"

namespace stv {
namespace {

constexpr int kMaxPages = 1 << 18;
constexpr int kMaxPoolSeqs = 4096;
constexpr int kBookThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 16384;  // per work item of the copy kernel
constexpr size_t kListOffset = 16;

struct BookParams {
  stv_page_pool pool;
  const int32_t* seqs;  // reserve, free: the list; fork: the sources
  const int32_t* dst;   // fork
  int32_t* ctx;
  int n, extra;
  int32_t* n_copies;  // workspace
  int2* list;         // workspace: (source, destination)
  int32_t* map;
  int32_t* n_live;
  int32_t* status;
};

// Exclusive scan of one int per thread over the CTA; *total gets the sum.
__device__ __forceinline__ int block_scan(int x, int* total) {
  __shared__ int warp_sum[kBookThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // warp_sum may still be read from a scan before
  if (lane == 31) warp_sum[w] = incl;
  __syncthreads();
  const int ws = warp_sum[lane];
  int wincl = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, wincl, o);
    if (lane >= o) wincl += y;
  }
  *total = __shfl_sync(0xffffffffu, wincl, 31);
  return incl - x + __shfl_sync(0xffffffffu, wincl - ws, w);
}

// In-place exclusive scan of a[0 .. n), a[n] = the sum.  Ends with a barrier.
// Sums are 32-bit: see sum_fits.
__device__ __forceinline__ void scan_array(int* a, int n) {
  const int per = (n + kBookThreads - 1) / kBookThreads;
  const int i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += a[i];
  int total;
  int at = block_scan(sum, &total);
  for (int i = i0; i < i1; ++i) {
    const int x = a[i];
    a[i] = at;
    at += x;
  }
  if (threadIdx.x == 0) a[n] = total;
  __syncthreads();
}

// Whether n sequences with this many entries each can be added up, and stepped
// through, in 32 bits.  Sequences that hold each page once always can (2^18
// pages, 2^12 sequences); longer tables, with pages named again in them, may not.
__device__ __forceinline__ bool sum_fits(int entries, int n) {
  constexpr int64_t kMost = (int64_t)kMaxPages * kMaxPoolSeqs;
  static_assert(kMost + kMaxPoolSeqs + kBookThreads < 0x7fffffff, "no sum of pages passes 32 bits");
  return (int64_t)entries * n <= kMost;
}

// Last i in [0, n) with a[i] <= r, a ascending, a[0] <= r.
template <typename F>
__device__ __forceinline__ int last_at_most(F a, int n, int r) {
  int lo = 0, hi = n;  // a(lo) <= r < a(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a(mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int nth_bit(uint32_t m, int n) {  // position of the n-th set bit, n < popc(m)
  int at = 0;
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    const int c = __popc(m & ((1u << w) - 1u));
    if (n >= c) {
      n -= c;
      m >>= w;
      at += w;
    }
  }
  return at;
}

// Which pages are live: a bit each, and the live pages before each word.
struct LiveMap {
  uint32_t* bits;
  int* pre;  // [words + 1]
  int words, n_pages;

  static __host__ __device__ size_t bytes(int n_pages) {
    return (size_t)((n_pages + 31) / 32) * 8 + 4;
  }
  __device__ void build(void* smem, const int32_t* refs, int n) {
    n_pages = n;
    words = (n + 31) / 32;
    bits = static_cast<uint32_t*>(smem);
    pre = reinterpret_cast<int*>(bits + words);
    const int lane = threadIdx.x & 31;
#pragma unroll 8
    for (int w = threadIdx.x >> 5; w < words; w += kBookThreads / 32) {
      const int page = w * 32 + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, page < n && refs[page] > 0);
      if (lane == 0) {
        bits[w] = m;
        pre[w] = __popc(m);
      }
    }
    __syncthreads();
    scan_array(pre, words);
  }
  __device__ int live() const { return pre[words]; }
  __device__ int live_before(int page) const {
    const int w = page >> 5;
    return w >= words ? live() : pre[w] + __popc(bits[w] & ((1u << (page & 31)) - 1u));
  }
  __device__ bool is_live(int page) const { return (bits[page >> 5] >> (page & 31)) & 1u; }
  __device__ int live_page(int r) const {
    const int w = last_at_most([&](int i) { return pre[i]; }, words, r);
    return w * 32 + nth_bit(bits[w], r - pre[w]);
  }
  __device__ int free_page(int r) const {
    const int w = last_at_most([&](int i) { return i * 32 - pre[i]; }, words, r);
    return w * 32 + nth_bit(~bits[w], r - (w * 32 - pre[w]));
  }
};

// Marks sequence s in a bitmap; true when it was marked before.
__device__ __forceinline__ bool mark(uint32_t* bitmap, int s) {
  const uint32_t b = 1u << (s & 31);
  return (atomicOr(bitmap + (s >> 5), b) & b) != 0;
}

// Reports what any thread found wrong; true when the call must stop.
__device__ __forceinline__ bool call_fails(int found, int32_t* status) {
  __shared__ int all;
  if (threadIdx.x == 0) all = 0;
  __syncthreads();
  if (found) atomicOr(&all, found);
  __syncthreads();
  if (all && threadIdx.x == 0) report(status, all);
  return all != 0;
}

__global__ void __launch_bounds__(kBookThreads) page_reserve_kernel(const __grid_constant__ BookParams p) {
  extern __shared__ int smem[];
  __shared__ uint32_t named[kMaxPoolSeqs / 32];
  int* off = smem;  // [n + 1]: new pages of the sequences before
  if (threadIdx.x < kMaxPoolSeqs / 32) named[threadIdx.x] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const stv_page_pool& pool = p.pool;
  int bad = 0;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int s = p.seqs[i];
    off[i] = 0;
    if (s < 0 || s >= pool.max_seqs || mark(named, s)) {
      bad = STV_DEV_BAD_SEQ;
      continue;
    }
    const int have = pool.counts[s], c = p.ctx[s];
    const int64_t need = ((int64_t)c + p.extra + kPageTok - 1) / kPageTok;
    if (have < 0 || c < 0 || have > pool.table_stride || need > pool.table_stride)
      bad = STV_DEV_BAD_SEQ;
    else if (need > have)  // past n_pages, pages are short however many they are
      off[i] = (int)min(need - have, (int64_t)pool.n_pages + 1);
  }
  if (call_fails(bad, p.status)) return;
  scan_array(off, p.n);
  const int total = off[p.n];
  if (total == 0) return;
  LiveMap lm;
  lm.build(off + p.n + 1, pool.refs, pool.n_pages);
  if (call_fails(total > pool.n_pages - lm.live() ? STV_DEV_NO_PAGES : 0, p.status)) return;
  for (int r = threadIdx.x; r < total; r += kBookThreads) {
    const int page = lm.free_page(r);
    const int i = last_at_most([&](int k) { return off[k]; }, p.n, r);
    const int s = p.seqs[i];
    pool.tables[(int64_t)s * pool.table_stride + pool.counts[s] + (r - off[i])] = page;
    pool.refs[page] = 1;
  }
  __syncthreads();  // counts were read above
  for (int i = threadIdx.x; i < p.n; i += kBookThreads)
    if (off[i + 1] > off[i]) pool.counts[p.seqs[i]] += off[i + 1] - off[i];
}

__global__ void __launch_bounds__(kBookThreads) page_free_kernel(const __grid_constant__ BookParams p) {
  extern __shared__ int smem[];
  __shared__ uint32_t named[kMaxPoolSeqs / 32];
  int* off = smem;  // [n + 1]: pages of the sequences before
  if (threadIdx.x < kMaxPoolSeqs / 32) named[threadIdx.x] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const stv_page_pool& pool = p.pool;
  int bad = 0;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int s = p.seqs[i];
    off[i] = 0;
    if (s < 0 || s >= pool.max_seqs || mark(named, s)) {
      bad = STV_DEV_BAD_SEQ;
      continue;
    }
    const int have = pool.counts[s];
    if (have < 0 || have > pool.table_stride || !sum_fits(have, p.n)) bad = STV_DEV_BAD_SEQ; else off[i] = have;
  }
  if (call_fails(bad, p.status)) return;
  scan_array(off, p.n);
  const int total = off[p.n];
  auto entry = [&](int f) -> int32_t* {
    const int i = last_at_most([&](int k) { return off[k]; }, p.n, f);
    return pool.tables + (int64_t)p.seqs[i] * pool.table_stride + (f - off[i]);
  };
  for (int f = threadIdx.x; f < total; f += kBookThreads) {
    const int page = *entry(f);
    if (page < 0 || page >= pool.n_pages) bad = STV_DEV_BAD_PAGE;
  }
  if (call_fails(bad, p.status)) return;
  for (int f = threadIdx.x; f < total; f += kBookThreads)
    if (atomicSub(pool.refs + *entry(f), 1) < 1) bad = STV_DEV_BAD_PAGE;  // more holders than it has references
  if (call_fails(bad, p.status)) {
    for (int f = threadIdx.x; f < total; f += kBookThreads) atomicAdd(pool.refs + *entry(f), 1);
    return;
  }
  for (int f = threadIdx.x; f < total; f += kBookThreads) *entry(f) = -1;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) pool.counts[p.seqs[i]] = 0;
}

__global__ void __launch_bounds__(kBookThreads) page_fork_kernel(const __grid_constant__ BookParams p) {
  extern __shared__ int smem[];
  __shared__ uint32_t named[kMaxPoolSeqs / 32];
  int* full = smem;               // [n + 1]: shared pages of the forks before
  int* part = full + p.n + 1;     // [n + 1]: copied pages of the forks before
  if (threadIdx.x < kMaxPoolSeqs / 32) named[threadIdx.x] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const stv_page_pool& pool = p.pool;
  if (threadIdx.x == 0) *p.n_copies = 0;
  int bad = 0;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int a = p.seqs[i], b = p.dst[i];
    full[i] = part[i] = 0;
    if (a < 0 || a >= pool.max_seqs || b < 0 || b >= pool.max_seqs || mark(named, b)) {
      bad = STV_DEV_BAD_SEQ;
      continue;
    }
    const int c = p.ctx[a], have = pool.counts[a];
    const int pages = c / kPageTok + (c % kPageTok != 0);
    if (c < 0 || pages > have || have > pool.table_stride || !sum_fits(pages, p.n) || pool.counts[b] != 0) {
      bad = STV_DEV_BAD_SEQ;
      continue;
    }
    full[i] = c / kPageTok;
    part[i] = pages - full[i];
    const int32_t* row = pool.tables + (int64_t)a * pool.table_stride;
    if (part[i]) {
      const int page = row[full[i]];
      if (page < 0 || page >= pool.n_pages || pool.refs[page] < 1) bad = STV_DEV_BAD_PAGE;
    }
  }
  if (call_fails(bad, p.status)) return;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads)
    if ((named[p.seqs[i] >> 5] >> (p.seqs[i] & 31)) & 1u) bad = STV_DEV_BAD_SEQ;  // a source that is a destination
  scan_array(full, p.n);
  scan_array(part, p.n);
  const int n_full = full[p.n], n_part = part[p.n];
  for (int f = threadIdx.x; f < n_full; f += kBookThreads) {
    const int i = last_at_most([&](int k) { return full[k]; }, p.n, f);
    const int page = pool.tables[(int64_t)p.seqs[i] * pool.table_stride + (f - full[i])];
    if (page < 0 || page >= pool.n_pages || pool.refs[page] < 1) bad = STV_DEV_BAD_PAGE;
  }
  LiveMap lm;
  if (n_part) {
    lm.build(part + p.n + 1, pool.refs, pool.n_pages);
    if (n_part > pool.n_pages - lm.live()) bad |= STV_DEV_NO_PAGES;
  }
  if (call_fails(bad, p.status)) return;
  for (int f = threadIdx.x; f < n_full; f += kBookThreads) {
    const int i = last_at_most([&](int k) { return full[k]; }, p.n, f);
    const int e = f - full[i];
    const int page = pool.tables[(int64_t)p.seqs[i] * pool.table_stride + e];
    pool.tables[(int64_t)p.dst[i] * pool.table_stride + e] = page;
    atomicAdd(pool.refs + page, 1);
  }
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int a = p.seqs[i], b = p.dst[i], at = full[i + 1] - full[i];
    if (part[i + 1] > part[i]) {
      const int page = lm.free_page(part[i]);
      p.list[part[i]] = make_int2(pool.tables[(int64_t)a * pool.table_stride + at], page);
      pool.tables[(int64_t)b * pool.table_stride + at] = page;
      pool.refs[page] = 1;
    }
    pool.counts[b] = at + (part[i + 1] - part[i]);
    p.ctx[b] = p.ctx[a];
  }
  if (threadIdx.x == 0) *p.n_copies = n_part;
}

__global__ void __launch_bounds__(kBookThreads) page_compact_kernel(const __grid_constant__ BookParams p) {
  extern __shared__ int smem[];
  grid_dep_wait();
  grid_dep_launch();
  const stv_page_pool& pool = p.pool;
  LiveMap lm;
  lm.build(smem, pool.refs, pool.n_pages);
  const int n_live = lm.live(), stay = lm.live_before(n_live), moves = n_live - stay;
  for (int page = threadIdx.x; page < pool.n_pages; page += kBookThreads) {
    const bool live = lm.is_live(page);
    if (!live || page < n_live) p.map[page] = live ? page : -1;
  }
  for (int r = threadIdx.x; r < moves; r += kBookThreads) {
    const int a = lm.live_page(stay + r), b = lm.free_page(r);
    p.list[r] = make_int2(a, b);
    p.map[a] = b;
    pool.refs[b] = pool.refs[a];
    pool.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    *p.n_copies = moves;
    *p.n_live = n_live;
  }
}

// The list of stv_page_copy, when it may be carried out as it stands.
__global__ void __launch_bounds__(kBookThreads) page_copy_list_kernel(const __grid_constant__ BookParams p) {
  extern __shared__ uint32_t written[];  // a bit per page
  const int words = (p.pool.n_pages + 31) / 32;
  for (int w = threadIdx.x; w < words; w += kBookThreads) written[w] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x == 0) *p.n_copies = 0;
  int bad = 0;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int a = p.seqs[i], b = p.dst[i];
    if (a < 0 || a >= p.pool.n_pages || b < 0 || b >= p.pool.n_pages || mark(written, b)) bad = STV_DEV_BAD_PAGE;
  }
  if (call_fails(bad, p.status)) return;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
    const int a = p.seqs[i];
    if ((written[a >> 5] >> (a & 31)) & 1u) bad = STV_DEV_BAD_PAGE;
  }
  if (call_fails(bad, p.status)) return;
  for (int i = threadIdx.x; i < p.n; i += kBookThreads) p.list[i] = make_int2(p.seqs[i], p.dst[i]);
  if (threadIdx.x == 0) *p.n_copies = p.n;
}

struct CopyParams {
  uint8_t* pools[kMaxLayers];
  int n_layers;
  int64_t page_bytes;
  int pieces;   // work items per page of a layer
  int per_cta;  // adjacent work items of a CTA
  const int32_t* n_copies;
  const int2* list;
  // compact: tables whose entries follow the pages
  stv_page_pool pool;
  const int32_t* map;  // null: no tables to change
  int32_t* status;
};

// Copies the listed pages in every layer; a work item is 16 KB of one page, and
// the CTAs take them in order.  3,088 page copies (193 pages in 16 layers, 1.42
// GB moved) take 205 us, 6.9 TB/s, with one CTA per item: what is in flight
// lies close together in memory at any time.  A persistent grid whose CTAs
// stride over the items drifts apart and takes 228 us; bulk copies through
// shared memory, 210 us.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyParams p) {
  grid_dep_wait();
  grid_dep_launch();
  if (p.map) {
    const stv_page_pool& pool = p.pool;
    const int64_t entries = (int64_t)pool.max_seqs * pool.table_stride;
    for (int64_t f = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; f < entries;
         f += (int64_t)gridDim.x * kCopyThreads) {
      const int s = (int)(f / pool.table_stride), e = (int)(f - (int64_t)s * pool.table_stride);
      const int have = __ldg(pool.counts + s);
      if (have < 0 || have > pool.table_stride) {
        if (e == 0) report(p.status, STV_DEV_BAD_SEQ);
        continue;
      }
      if (e >= have) continue;
      const int page = pool.tables[f];
      const int to = page >= 0 && page < pool.n_pages ? __ldg(p.map + page) : -1;
      if (to < 0) report(p.status, STV_DEV_BAD_PAGE);
      else if (to != page) pool.tables[f] = to;
    }
  }
  const int64_t items = (int64_t)__ldg(p.n_copies) * p.n_layers * p.pieces;
  const int64_t w0 = (int64_t)blockIdx.x * p.per_cta, w1 = min(items, w0 + p.per_cta);
  for (int64_t w = w0; w < w1; ++w) {
    const int piece = (int)(w % p.pieces);
    const int64_t lw = w / p.pieces;
    const int layer = (int)(lw % p.n_layers);
    const int2 c = __ldg(p.list + lw / p.n_layers);
    const int64_t at = (int64_t)piece * kCopyBytes;
    const int n16 = (int)(min((int64_t)kCopyBytes, p.page_bytes - at) / 16);
    const uint4* src = reinterpret_cast<const uint4*>(p.pools[layer] + c.x * p.page_bytes + at);
    uint4* dst = reinterpret_cast<uint4*>(p.pools[layer] + c.y * p.page_bytes + at);
    constexpr int kPer = kCopyBytes / 16 / kCopyThreads;
    uint4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = k * kCopyThreads + threadIdx.x;
      if (i < n16) v[k] = src[i];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = k * kCopyThreads + threadIdx.x;
      if (i < n16) dst[i] = v[k];
    }
  }
}

int check_pool(const stv_page_pool* pool) {
  if (!pool || !pool->refs || !pool->tables || !pool->counts) return STV_ERR_INVALID_ARG;
  if (pool->n_pages < 1 || pool->max_seqs < 1 || pool->table_stride < 1) return STV_ERR_INVALID_ARG;
  if (pool->n_pages > kMaxPages || pool->max_seqs > kMaxPoolSeqs) return STV_ERR_SHAPE_UNSUPPORTED;
  return STV_OK;
}

size_t workspace_need(int n_pages) { return kListOffset + (size_t)n_pages * sizeof(int2); }

int check_workspace(void* workspace, size_t ws_bytes, int n_pages) {
  if (!workspace || (uintptr_t)workspace % 16) return STV_ERR_INVALID_ARG;
  return ws_bytes < workspace_need(n_pages) ? STV_ERR_WORKSPACE_TOO_SMALL : STV_OK;
}

void set_workspace(BookParams* b, void* workspace) {
  b->n_copies = static_cast<int32_t*>(workspace);
  b->list = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + kListOffset);
}

// The layers' pools as the copy kernel takes them; every pool holds n_pages.
int fill_copy(const stv_shape* shape, const stv_layer_cache* layers, int n_layers, int n_pages, CopyParams* c) {
  ShapeInfo sh;
  int rc = check_shape(shape, -1, &sh);
  if (rc) return rc;
  if (!layers || n_layers < 1 || n_layers > kMaxLayers) return STV_ERR_INVALID_ARG;
  memset(c, 0, sizeof(*c));
  for (int l = 0; l < n_layers; ++l) {
    if ((rc = check_layer(&layers[l], sh))) return rc;
    if (layers[l].n_pages < n_pages || (uintptr_t)layers[l].pool % 16) return STV_ERR_INVALID_ARG;
    c->pools[l] = layers[l].pool;
  }
  c->n_layers = n_layers;
  c->page_bytes = layers[0].page_bytes;
  c->pieces = (int)((c->page_bytes + kCopyBytes - 1) / kCopyBytes);
  return STV_OK;
}

// The largest books' shared memory (fork's).  Books that need the attribute ask
// for this much of it, always: it belongs to the function, so a smaller value
// would lower what a call of another thread on larger books has just set.
constexpr size_t kPlainSmem = 40 * 1024;
size_t most_smem() { return (size_t)(kMaxPoolSeqs + 1) * 8 + LiveMap::bytes(kMaxPages); }

template <typename... KArgs>
cudaError_t launch_book(void (*kernel)(KArgs...), size_t smem, const BookParams& b, cudaStream_t s) {
  if (smem > kPlainSmem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem());
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return e;
    }
  }
  return launch_pdl(kernel, 1, kBookThreads, smem, s, b);
}

// The grid for the copies of at most max_copies pages.
// per_cta: 1 where about as many will be listed; 4 where far fewer may be, so
// that CTAs without work cost little (a grid of twice the CTAs needed adds 18
// us to the 205 at one item each, 2 at four).
int plan_copies(CopyParams& c, int64_t max_copies, int per_cta, int* grid) {
  c.per_cta = per_cta;
  const int64_t items = std::max<int64_t>(1, max_copies * c.n_layers * c.pieces);
  const int64_t ctas = (items + per_cta - 1) / per_cta;
  if (ctas > 0x7fffffff) return STV_ERR_SHAPE_UNSUPPORTED;
  *grid = (int)ctas;
  return STV_OK;
}

template <typename... KArgs>
int launch_listed(void (*kernel)(KArgs...), size_t smem, const BookParams& b, CopyParams& c, int grid,
                  cudaStream_t s) {
  c.n_copies = b.n_copies;
  c.list = b.list;
  c.status = b.status;
  if (launch_book(kernel, smem, b, s) != cudaSuccess) return STV_ERR_CUDA;
  return launch_pdl(page_copy_kernel, grid, kCopyThreads, 0, s, c) == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}

}  // namespace
}  // namespace stv

using namespace stv;

extern "C" {

int stv_page_workspace_bytes(int n_pages, size_t* bytes) {
  if (!bytes || n_pages < 1) return STV_ERR_INVALID_ARG;
  if (n_pages > kMaxPages) return STV_ERR_SHAPE_UNSUPPORTED;
  *bytes = workspace_need(n_pages);
  return STV_OK;
}

int stv_page_reserve(const stv_page_pool* pool, const int32_t* seqs, int n, const int32_t* ctx, int extra,
                     int32_t* dev_status, stv_stream_t stream) {
  if (int rc = check_pool(pool)) return rc;
  if (n < 0 || n > pool->max_seqs || extra < 0 || (n > 0 && (!seqs || !ctx))) return STV_ERR_INVALID_ARG;
  if (n == 0) return STV_OK;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.pool = *pool;
  b.seqs = seqs;
  b.ctx = const_cast<int32_t*>(ctx);
  b.n = n;
  b.extra = extra;
  b.status = dev_status;
  const size_t smem = (size_t)(n + 1) * 4 + LiveMap::bytes(pool->n_pages);
  return launch_book(page_reserve_kernel, smem, b, (cudaStream_t)stream) == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}

int stv_page_free(const stv_page_pool* pool, const int32_t* seqs, int n, int32_t* dev_status, stv_stream_t stream) {
  if (int rc = check_pool(pool)) return rc;
  if (n < 0 || n > pool->max_seqs || (n > 0 && !seqs)) return STV_ERR_INVALID_ARG;
  if (n == 0) return STV_OK;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.pool = *pool;
  b.seqs = seqs;
  b.n = n;
  b.status = dev_status;
  return launch_book(page_free_kernel, (size_t)(n + 1) * 4, b, (cudaStream_t)stream) == cudaSuccess ? STV_OK
                                                                                                  : STV_ERR_CUDA;
}

int stv_page_fork(const stv_shape* shape, const stv_layer_cache* layers, int n_layers, const stv_page_pool* pool,
                  const int32_t* src, const int32_t* dst, int n, int32_t* ctx, void* workspace, size_t ws_bytes,
                  int32_t* dev_status, stv_stream_t stream) {
  int rc = check_pool(pool);
  if (rc) return rc;
  CopyParams c;
  if ((rc = fill_copy(shape, layers, n_layers, pool->n_pages, &c))) return rc;
  if (n < 0 || n > pool->max_seqs || (n > 0 && (!src || !dst || !ctx))) return STV_ERR_INVALID_ARG;
  if ((rc = check_workspace(workspace, ws_bytes, pool->n_pages))) return rc;
  if (n == 0) return STV_OK;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.pool = *pool;
  b.seqs = src;
  b.dst = dst;
  b.ctx = ctx;
  b.n = n;
  b.status = dev_status;
  set_workspace(&b, workspace);
  const size_t smem = (size_t)(n + 1) * 8 + LiveMap::bytes(pool->n_pages);
  int grid;
  if ((rc = plan_copies(c, n, 1, &grid))) return rc;
  return launch_listed(page_fork_kernel, smem, b, c, grid, (cudaStream_t)stream);
}

int stv_page_compact(const stv_shape* shape, const stv_layer_cache* layers, int n_layers, const stv_page_pool* pool,
                     int32_t* map, int32_t* n_live, void* workspace, size_t ws_bytes, int32_t* dev_status,
                     stv_stream_t stream) {
  int rc = check_pool(pool);
  if (rc) return rc;
  CopyParams c;
  if ((rc = fill_copy(shape, layers, n_layers, pool->n_pages, &c))) return rc;
  if (!map || !n_live) return STV_ERR_INVALID_ARG;
  if ((rc = check_workspace(workspace, ws_bytes, pool->n_pages))) return rc;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.pool = *pool;
  b.map = map;
  b.n_live = n_live;
  b.status = dev_status;
  set_workspace(&b, workspace);
  c.pool = *pool;
  c.map = map;
  int grid;
  if ((rc = plan_copies(c, pool->n_pages / 2, 4, &grid))) return rc;
  return launch_listed(page_compact_kernel, LiveMap::bytes(pool->n_pages), b, c, grid, (cudaStream_t)stream);
}

int stv_page_copy(const stv_shape* shape, const stv_layer_cache* layers, int n_layers, int n_pages,
                  const int32_t* src, const int32_t* dst, int n, void* workspace, size_t ws_bytes,
                  int32_t* dev_status, stv_stream_t stream) {
  if (n_pages < 1) return STV_ERR_INVALID_ARG;
  if (n_pages > kMaxPages) return STV_ERR_SHAPE_UNSUPPORTED;
  CopyParams c;
  int rc = fill_copy(shape, layers, n_layers, n_pages, &c);
  if (rc) return rc;
  if (n < 0 || n > n_pages || (n > 0 && (!src || !dst))) return STV_ERR_INVALID_ARG;
  if ((rc = check_workspace(workspace, ws_bytes, n_pages))) return rc;
  if (n == 0) return STV_OK;
  BookParams b;
  memset(&b, 0, sizeof(b));
  b.pool.n_pages = n_pages;
  b.seqs = src;
  b.dst = dst;
  b.n = n;
  b.status = dev_status;
  set_workspace(&b, workspace);
  const size_t smem = (size_t)((n_pages + 31) / 32) * 4;
  int grid;
  if ((rc = plan_copies(c, n, 1, &grid))) return rc;
  return launch_listed(page_copy_list_kernel, smem, b, c, grid, (cudaStream_t)stream);
}

}  // extern "C"
