// paged_attn.cuh -- what the two kernels of stv_paged_attn share: parameters,
// the cut of the work into equal shares, and the walk over a share.
//
// Work.  A unit is (entry, tokens_per consecutive new tokens of it, KV head): at
// most 16 or 128 (256) rows of Q that read the same keys.  Its keys come in tiles
// of 64 (single tokens) or 128: those of the first tokens (sinks) that lie before
// the window's first tile, then the window's (or all up to the last visible key).
// All tiles of all units, in the order (entry, unit, head, tile), each unit's after
// a few tiles' worth for its Q and its end, are cut into as many equal runs as there
// are CTAs.  A unit inside one CTA's run is finished there; a unit cut by the runs'
// borders leaves partials (O, and the running maximum and sum of each row), at most
// two per CTA, which the join kernel puts together in the runs' order.  So every
// CTA has the same work whatever the lengths, a single long sequence is spread over
// all SMs, and the result depends on the lengths alone.
//
// The lengths are on the device: each CTA works its own run out (a scan over the
// entries, one over the units), which costs about as much as one dependent load
// and saves a launch.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "stv_device.cuh"
#include "tc_util.cuh"

namespace stv {

constexpr int kSmallTile = 64;      // keys of a tile, single tokens
constexpr int kBigTile = 128;       // blocks and prompts
// K and V of such a tile move in pieces: a copy's waits and issue take some 330
// cycles, whatever its size, so 32 KB where a tile has as much.
__host__ __device__ constexpr int big_piece_bytes(int hd) { return hd == 64 ? 16384 : 32768; }
constexpr int kMaxEntries = 4096;
constexpr int kMaxCtx = 1 << 30;
constexpr int kSmallRows = 16;      // rows of Q per unit, single tokens

// A unit cut by the runs' borders: written by the CTA whose run it begins in.
struct JoinRecord {
  int row0, rows, h, last_cta;
};

struct AttnParams {
  // The pool as [hd / 64][rows][64 channels], in boxes of a tile of K and V
  // (single tokens: the same map), or of a piece of one; q as
  // [rows][heads][hd / 64][64], in boxes of a row tile's 64 channels.
  CUtensorMap map_k, map_v, map_q;
  const void* q;
  void* o;
  int64_t q_row, q_head, o_row, o_head;  // strides in elements
  const int32_t* tables;
  const int32_t* counts;
  int table_stride, max_seqs, n_pages;
  const int32_t* seqs;
  const int32_t* ctx;
  const int32_t* row_start;
  int n, n_rows, max_new;
  int hkv, G;
  int tokens_per;  // new tokens of a unit
  int tile_bits;   // log2 of a tile's keys
  int unit_cost;   // what a unit costs beside its tiles, in tiles
  int window, sinks, causal;
  float scale2;  // scale * log2(e)
  bool q_wide, o_wide;  // 16-byte loads of q, stores of o
  // workspace
  float* part;       // [2 * CTAs][part_rows][hd]
  float2* ml;        // [2 * CTAs][part_rows]
  JoinRecord* rec;   // [CTAs]
  int part_rows;
  // Failure-path test (stv_paged_attn_timeout_test): the producer stops before its
  // first copy, so that every wait for one runs out.
  bool withhold;
  int32_t* status;
};

namespace {

struct Entry {
  int s, ctx, L, row0;
  int keys;  // tokens of its pages
};

// Entry i, with no rows where anything about it is wrong.  (All loads first: two
// trips to memory, one without seqs.)
__device__ __forceinline__ Entry entry_of(const AttnParams& p, int i) {
  Entry e;
  e.s = p.seqs ? __ldg(p.seqs + i) : i;
  e.row0 = p.row_start ? __ldg(p.row_start + i) : i;
  const int r1 = p.row_start ? __ldg(p.row_start + i + 1) : i + 1;
  const int s = min(max(e.s, 0), p.max_seqs - 1);
  e.ctx = __ldg(p.ctx + s);
  const int have = min(__ldg(p.counts + s), p.table_stride);
  e.keys = max(0, min(have, kMaxCtx / kPageTok * 2 - 1)) * kPageTok;
  int bad = 0;
  if (e.row0 < 0 || r1 < e.row0 || r1 > p.n_rows || r1 - e.row0 > p.max_new) bad = STV_DEV_BAD_ROW;
  else if (e.s != s || e.ctx < 0 || e.ctx > kMaxCtx) bad = STV_DEV_BAD_SEQ;
  e.L = bad ? 0 : r1 - e.row0;
  if (e.L && e.ctx + e.L > e.keys) bad = STV_DEV_BAD_PAGE;
  if (bad) report(p.status, bad);
  if (!e.L) e.ctx = e.keys = 0;
  return e;
}

// Unit u of an entry.
struct AttnUnit {
  int pos0, ntok, end;  // position of its first token, tokens, keys of the sequence that have a page
  int hi, lo;           // keys some row sees: [lo, hi), and those before `sinks`
  int n_sink, wt0;      // tiles of the first tokens; first tile of the window
  int n_tiles;
};

__device__ __forceinline__ AttnUnit unit_of(const AttnParams& p, const Entry& e, int u) {
  AttnUnit x;
  x.pos0 = e.ctx + u * p.tokens_per;
  x.ntok = min(p.tokens_per, e.L - u * p.tokens_per);
  x.end = min(e.ctx + e.L, e.keys);
  x.hi = p.causal ? min(x.pos0 + x.ntok, x.end) : x.end;
  x.lo = p.window ? max(0, x.pos0 - p.window + 1) : 0;
  x.wt0 = x.lo >> p.tile_bits;
  const int up_to = (x.hi + (1 << p.tile_bits) - 1) >> p.tile_bits;
  x.n_sink = p.window && p.sinks ? min(((p.sinks - 1) >> p.tile_bits) + 1, min(x.wt0, up_to)) : 0;
  x.n_tiles = max(1, max(0, up_to - x.wt0) + x.n_sink);  // one tile at least: it writes the rows
  return x;
}
// First key of its t-th tile.
__device__ __forceinline__ int tile_key(const AttnParams& p, const AttnUnit& x, int t) {
  return (t < x.n_sink ? t : x.wt0 + t - x.n_sink) << p.tile_bits;
}
// Whether some row may not see some key of the tile.
__device__ __forceinline__ bool tile_edge(const AttnParams& p, const AttnUnit& x, int key0) {
  const int last = key0 + (1 << p.tile_bits) - 1;
  if (last >= x.end || (p.causal && last > x.pos0)) return true;
  return p.window && key0 <= x.pos0 + x.ntok - 1 - p.window && last >= p.sinks;
}
// The keys that a row (or some row of a unit) sees: [lo, hi) and, before hi, those
// below `sinks`.
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen row_sees(const AttnParams& p, const AttnUnit& x, int pos) {
  return {p.window ? max(0, pos - p.window + 1) : 0, p.causal ? min(pos + 1, x.end) : x.end};
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
// Of 32 keys from key0 on, as bits.
__device__ __forceinline__ uint32_t bits_of(const Seen& s, int sinks, int key0) {
  return low_bits(s.hi - key0) & (~low_bits(s.lo - key0) | low_bits(sinks - key0));
}

// Exclusive scan of x over the CTA's kThreads threads; *total gets the sum.
template <int kThreads>
__device__ __forceinline__ long long cta_scan(long long x, long long* total) {
  __shared__ long long warp_sum[kThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // warp_sum may still be read from a scan before
  if (lane == 31) warp_sum[w] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < w) before += warp_sum[i];
    all += warp_sum[i];
  }
  *total = all;
  return before + incl - x;
}

// Where a CTA's run begins, and its length in tiles.
struct RunStart {
  int e, u, h, off;       // entry, unit, head, and how far into that unit (its cost first, then its tiles)
  long long left, share;  // length of the run, of a full run
};

// a / b; a 64-bit division takes a third of a microsecond.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return a >> 31 == 0 && b >> 31 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Whole CTA; scratch: n + 1 ints of shared memory, free afterwards.  Ends with
// a barrier.
template <int kThreads>
__device__ __forceinline__ RunStart run_of(const AttnParams& p, int* scratch) {
  __shared__ RunStart start;
  const int tid = threadIdx.x;
  // units of the entries before
  const int per = (p.n + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, p.n), e1 = min(e0 + per, p.n);
  long long mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int nu = (entry_of(p, e).L + p.tokens_per - 1) / p.tokens_per;
    scratch[e] = nu;
    mine += nu;
  }
  long long all;
  int at = (int)cta_scan<kThreads>(mine, &all);
  // (more units than rows: entries share rows, and their sum may be anything)
  const int n_units = all > p.n_rows ? 0 : (int)all;
  if (all > p.n_rows && tid == 0) report(p.status, STV_DEV_BAD_ROW);
  for (int e = e0; e < e1; ++e) {
    const int nu = scratch[e];
    scratch[e] = at;
    at += nu;
  }
  if (tid == 0) {
    scratch[p.n] = n_units;
    start.left = 0;
    start.share = 1;
  }
  __syncthreads();
  // tiles of the units of this thread's stretch
  const int uper = (n_units + kThreads - 1) / kThreads;
  const int g0 = min(tid * uper, n_units), g1 = min(g0 + uper, n_units);
  int first = 0;  // the entry of unit g0
  {
    int lo = 0, hi = p.n;  // scratch[lo] <= g0 < scratch[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (scratch[mid] <= g0) lo = mid; else hi = mid;
    }
    first = lo;
  }
  long long tiles = 0;
  auto walk = [&](auto&& f) {
    int e = first;
    Entry en = {};
    bool have = false;
    for (int g = g0; g < g1; ++g) {
      while (scratch[e + 1] <= g) {
        ++e;
        have = false;
      }
      if (!have) {
        en = entry_of(p, e);
        have = true;
      }
      if (!f(e, g - scratch[e], unit_of(p, en, g - scratch[e]).n_tiles + p.unit_cost)) return;
    }
  };
  walk([&](int, int, int n) {
    tiles += n;
    return true;
  });
  long long total;
  const long long before = cta_scan<kThreads>(tiles, &total) * p.hkv;
  total *= p.hkv;
  const long long share = quotient(total + gridDim.x - 1, gridDim.x);
  const long long f0 = share * blockIdx.x;
  if (f0 < total && before <= f0 && f0 < before + tiles * p.hkv) {
    long long f = before;
    walk([&](int e, int u, int n) {
      if (f0 < f + (long long)n * p.hkv) {
        start.e = e;
        start.u = u;
        start.h = (int)quotient(f0 - f, n);
        start.off = (int)(f0 - f - (long long)start.h * n);
        start.left = min(share, total - f0);
        start.share = share;
        return false;
      }
      f += (long long)n * p.hkv;
      return true;
    });
  }
  __syncthreads();
  return start;
}

// Walks a run, one unit's part after the other.
struct RunWalk {
  const AttnParams& p;
  RunStart at;
  Entry en;
  AttnUnit x;
  int t0, t1;  // tiles of this part, one at least
  bool any;

  __device__ RunWalk(const AttnParams& p_, const RunStart& s) : p(p_), at(s), any(s.left > 0) {
    if (any) {
      en = entry_of(p, at.e);
      open();
      if (t0 == t1) next();
    }
  }
  __device__ void open() {
    x = unit_of(p, en, at.u);
    const int from = at.off - p.unit_cost;
    t0 = max(0, from);
    t1 = (int)max((long long)t0, min((long long)x.n_tiles, from + at.left));
  }
  // The workspace slot of this part's partials; -1: the unit is whole.
  __device__ int slot() const {
    const int b = 2 * (int)blockIdx.x;
    return t0 ? b : t1 < x.n_tiles ? b + 1 : -1;
  }
  // The last CTA that has tiles of this unit, for a unit that begins here and
  // does not end here.
  __device__ int last_cta() const {
    const int rest = x.n_tiles - t1;  // in runs after this one
    return (int)(blockIdx.x + quotient(rest + at.share - 1, at.share));
  }
  __device__ bool next() {
    do {
      at.left -= x.n_tiles + p.unit_cost - at.off;
      at.off = 0;
      if (at.left <= p.unit_cost) return any = false;  // not a tile more
      if (++at.h == p.hkv) {
        at.h = 0;
        if (++at.u * p.tokens_per >= en.L) {
          at.u = 0;
          do {
            if (++at.e >= p.n) return any = false;
            en = entry_of(p, at.e);
          } while (en.L == 0);
        }
      }
      open();
    } while (t0 == t1);
    return true;
  }
};

// Rows of the map where tiles begin (a key's row of K; V's is 256 further), or -1
// where the sequence has no page; the next page's number is on its way ahead.
struct PageWalk {
  int s = -1, lp, page, next;

  __device__ __forceinline__ int look(const AttnParams& p, const Entry& e, int at) const {
    return at * kPageTok < e.keys ? __ldg(p.tables + (int64_t)e.s * p.table_stride + at) : -1;
  }
  __device__ __forceinline__ int row(const AttnParams& p, const Entry& e, int head, int key0) {
    const int at = key0 / kPageTok;
    if (s != e.s || at != lp) {
      page = s == e.s && at == lp + 1 ? next : look(p, e, at);
      s = e.s;
      lp = at;
      next = look(p, e, at + 1);
    }
    if (page < 0 || page >= p.n_pages) {
      report(p.status, STV_DEV_BAD_PAGE);
      return -1;
    }
    return (page * p.hkv + head) * (2 * kPageTok) + key0 % kPageTok;
  }
};

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int row, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          su32(dst)),
      "l"(map), "r"(0), "r"(row), "r"(block), "r"(su32(bar))
      : "memory");
}

// P = 2^(s - m + kLift): in fp16, whose values end at 2^16 and 2^-24, it may be up
// to 2^15 (the maximum is up to 2^8 behind), so that what a long flat tail adds is
// kept down to 2^-31 of the largest; O and the sum carry the same factor.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;

template <typename T>
struct Pack;
template <>
struct Pack<__half> {
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 floats(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
};
template <>
struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 floats(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};

// n (2, 4 or 8) adjacent outputs, as wide as o allows.
template <typename T, int n>
__device__ __forceinline__ void store_out(T* dst, const float* v, bool wide) {
  uint32_t w[n / 2];
#pragma unroll
  for (int i = 0; i < n / 2; ++i) w[i] = Pack<T>::two(v[2 * i], v[2 * i + 1]);
  if (wide) {
    if constexpr (n == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (n == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

}  // namespace

// Launchers (cudaError_t of the launch); grid: CTAs, as the workspace was cut.
cudaError_t launch_attn_small(const AttnParams& p, int hd, bool bf16, int grid, cudaStream_t s);  // paged_attn.cu
// paged_attn_tc.cu; q_tiles: tiles of 128 rows per unit (1 or 2)
cudaError_t launch_attn_tiles(const AttnParams& p, int hd, bool bf16, int q_tiles, int grid, cudaStream_t s);

}  // namespace stv
