// sample.cu -- sampling from the target's logits with temperature, top-k,
// top-p and min-p from given random numbers (include/stv.h, stv_sample).
//
// Every filter and the draw itself is a cut of one order (logit descending,
// then index ascending) at a given count or a given mass, so no sort of the
// vocabulary is needed.  A cluster of CTAs shares a row, each CTA a stretch of
// it, and sweeps it up to three times (the first time from HBM, then from L2):
//   1. the maximum (a NaN shows in it);
//      then one vector in kSample, counted by quarter octaves of w, tells how
//      far down the order the cuts lie: x >= x_cut, the row's head;
//   2. the mass of all tokens (unless top-k makes it unneeded), and of the
//      head either the tokens themselves, when they are few, or their counts
//      and masses in 2,048 bins;
//   3. the tokens of the few bins that the cuts lie in.
// The first CTA sorts the gathered tokens and makes the cuts exactly.  The
// sample only chooses x_cut: when the head turns out too short, steps 2 and 3
// run once more with every token that has any mass.
//
// Masses.  w = exp((x - max) / T) as an integer of scale 2^45.  With C =
// T ln 2 / 64, k = rint(x / C) and z = x - k C (C in two floats; the first
// product's remainder is exact), w is 2^(k / 64) from a table of 64 entries
// times e^(z / T), |z / T| <= ln 2 / 128, whose cubic is rounded to 2^-29 of w.
// Integer sums do not depend on their order, so masses, bins and tokens depend
// neither on the cluster's size nor on the batch.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "stv_device.cuh"

namespace cg = cooperative_groups;

namespace stv {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kBinsPer = kBins / kThreads;
constexpr int kList = 2048;      // tokens gathered around the cuts
constexpr int kDirect = 1400;    // a head estimated at this many tokens is gathered at once
constexpr int kCoarse = 256;     // quarter octaves of the sample
constexpr int kMaxVocab = 1 << 19;
constexpr int kShift = 14;       // w < 2^45: 2^19 tokens stay below 2^64
constexpr int kMaxCluster = 8;

struct SampleParams {
  const void* x;
  int64_t row_stride;
  int n_rows, vocab, rows_per_param;
  int stretch;       // tokens per CTA of a cluster
  int sample_every;  // 1: the sample is everything
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logprob;
  int32_t* status;
  uint32_t table[64];  // 2^30 * 2^(j / 64)
};

// What the first CTA decides for its cluster.
struct Decision {
  int done;
  int kb, pb1, pb2, mb, ub1, ub2;  // bins to gather; empty ranges where a cut is not made
};

struct Smem {
  u64 tot_mass[kBins];  // first CTA: the row's bins, then of each and all before
  u64 mass[kBins];      // this CTA's bins; first CTA later: running mass over the list
  u64 list[kList];      // (~key << 32) | index
  uint32_t tot_count[kBins];
  uint32_t count[kBins];  // this CTA's bins; first CTA later: a bin's first place in the list
  uint32_t coarse[kCoarse];
  float coarse_est[kCoarse];
  uint32_t table[64];
  float table_f[64];
  u64 red[kThreads / 32];
  u64 out, part;  // part: this CTA's share of the row's mass
  float max;
  int x_index;    // greedy: the maximum's first index in this CTA's stretch
  int found[8];
  int n_list;
  Decision d;
};

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Keys ascend with the value; -0 and +0 are one value.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ u64 entry_of(float x, int i) { return ((u64)(~key_of(x)) << 32) | (uint32_t)i; }
__device__ __forceinline__ float entry_x(u64 e) { return of_key(~(uint32_t)(e >> 32)); }

// The larger one; NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A row's temperature and maximum as the weights need them.
struct Scale {
  float max;
  float floor;         // below it w = 0 (62 octaves under the maximum)
  float base;          // 0; the maximum where x / C would leave the integers of fp32: there
                       // x - max is exact for every x >= floor
  float least;         // rint(x / C) of the floor, as kMagic + k: smaller ones count as it
  float inv_c, c_hi, c_lo, inv_t;
  int top;             // octave of the maximum
  float cut;           // the head: x >= cut
  float bin_scale;     // bins of the head, from the maximum down
};

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

__device__ __forceinline__ Scale make_scale(float max, float temp) {
  Scale sc;
  const double c = (double)temp * (0.69314718055994530942 / 64.0);
  sc.max = max;
  sc.c_hi = (float)c;
  sc.c_lo = (float)(c - (double)sc.c_hi);
  sc.inv_c = (float)(1.0 / c);
  sc.inv_t = (float)(1.0 / (double)temp);
  sc.floor = __double2float_rd((double)max - 62.0 * 64.0 * c);
  sc.base = fabsf(max) * sc.inv_c < 2097152.f ? 0.f : max;
  const float t = fmaf(max - sc.base, sc.inv_c, kMagic);
  sc.top = __float_as_int(t) >> 6;
  sc.least = t - 62.f * 64.f;
  sc.cut = sc.floor;
  sc.bin_scale = 0.f;
  return sc;
}

// w of a token that is not NaN (0 for -inf and whatever lies below the floor).
__device__ __forceinline__ u64 weigh(float x, const Scale& sc, const uint32_t* table, const float* table_f) {
  const float v = x - sc.base;
  const float t = fmaxf(fmaf(v, sc.inv_c, kMagic), sc.least);  // (at 62 octaves any z gives w = 0)
  const int kb = __float_as_int(t);
  const float k = t - kMagic;
  const float z = fmaf(k, -sc.c_lo, fmaf(k, -sc.c_hi, v)) * sc.inv_t;
  const float p = fmaf(fmaf(z, 1.f / 6.f, 0.5f), z, 1.f);  // e^z - 1 = z p
  const int j = kb & 63;
  // table_f = 2^28 2^(j/64), a quarter of the integer entry: |table_f z p| < 2^22
  const float q = fmaf(table_f[j] * z, p, kMagic);
  const uint32_t m = table[j] + ((uint32_t)(__float_as_int(q) - 0x4b400000) << 2);
  const u64 w = ((u64)m << kShift) >> (sc.top - (kb >> 6));
  // cut to even, plus one where anything is left: no bias
  const uint32_t lo = (uint32_t)w;
  return (w & 0xffffffff00000000ull) | (lo | min(lo, 1u));
}

// Bin of a token of the head.
__device__ __forceinline__ int bin_of(float x, const Scale& sc) {
  return min(kBins - 1, __float2int_rd((sc.max - x) * sc.bin_scale));
}

__device__ __forceinline__ void set_cut(Scale& sc, float cut) {
  sc.cut = fminf(fmaxf(cut, sc.floor), sc.max);
  const float range = sc.max - sc.cut;
  sc.bin_scale = range > 0.f ? fminf((float)kBins / range, 3e38f) : 0.f;
}

// Calls f(x, index) for the tokens [lo, hi) of a row, a thread's own in
// ascending order; of its 16-byte vectors only groups of 32 in `every`.
template <typename T, typename F>
__device__ __forceinline__ void sweep(const T* row, int lo, int hi, F&& f, int every = 1) {
  constexpr int VE = 16 / sizeof(T);
  const T* p = row + lo;
  const int n = hi - lo;
  const int head = min(n, (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)));
  const int n_vec = (n - head) / VE;
  if ((int)threadIdx.x < head) f(to_f(p[threadIdx.x]), lo + (int)threadIdx.x);
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  auto use = [&](const uint4& q, int i) {
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int k = 0; k < VE; ++k) f(to_f(e[k]), lo + head + i * VE + k);
  };
  if (every > 1) {
    for (int g = threadIdx.x >> 5; g * every * 32 < n_vec; g += kThreads / 32) {
      const int i = g * every * 32 + (threadIdx.x & 31);
      if (i < n_vec) use(__ldg(v + i), i);
    }
    return;
  }
  constexpr int kAhead = 4;  // loads in flight per thread
  int i = threadIdx.x;
  for (; i + (kAhead - 1) * kThreads < n_vec; i += kAhead * kThreads) {
    uint4 q[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) q[a] = __ldg(v + i + a * kThreads);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) use(q[a], i + a * kThreads);
  }
  for (; i < n_vec; i += kThreads) use(__ldg(v + i), i);
  for (int j = head + n_vec * VE + threadIdx.x; j < n; j += kThreads) f(to_f(p[j]), lo + j);
}

template <typename Op>
__device__ __forceinline__ u64 block_reduce(u64 x, u64* red, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  constexpr int kWarps = kThreads / 32;  // a power of two: the lanes read them in turn
  u64 y = red[threadIdx.x & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) y = op(y, __shfl_xor_sync(0xffffffffu, y, o));
  return y;
}
__device__ __forceinline__ u64 block_max(u64 x, u64* red) {
  return block_reduce(x, red, [](u64 a, u64 b) { return a > b ? a : b; });
}
__device__ __forceinline__ u64 block_min(u64 x, u64* red) {
  return block_reduce(x, red, [](u64 a, u64 b) { return a < b ? a : b; });
}
__device__ __forceinline__ u64 block_sum(u64 x, u64* red) {
  return block_reduce(x, red, [](u64 a, u64 b) { return a + b; });
}

// Exclusive scan of one value per thread.
__device__ __forceinline__ u64 block_scan(u64 x, u64* red) {
  const int lane = threadIdx.x & 31;
  u64 incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) red[threadIdx.x >> 5] = incl;
  __syncthreads();
  const u64 ws = lane < kThreads / 32 ? red[lane] : 0;
  u64 wi = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += y;
  }
  return incl - x + __shfl_sync(0xffffffffu, wi - ws, threadIdx.x >> 5);
}

// Counts and masses of the bins become those of each bin and all before it.
__device__ __forceinline__ void accumulate_bins(uint32_t* count, u64* mass, u64* red) {
  const int b = kBinsPer * threadIdx.x;
  u64 c = 0, m = 0;
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) {
    c += count[b + i];
    m += mass[b + i];
  }
  c = block_scan(c, red);
  m = block_scan(m, red);
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) {
    c += count[b + i];
    m += mass[b + i];
    count[b + i] = (uint32_t)c;
    mass[b + i] = m;
  }
  __syncthreads();
}

// First bin for which past(bin) holds (it holds for all later ones); kBins - 1
// if none.
template <typename F>
__device__ __forceinline__ int first_bin(F&& past, int* slot) {
  if (threadIdx.x == 0) *slot = kBins - 1;
  __syncthreads();
  for (int b = kBinsPer * threadIdx.x; b < kBinsPer * (int)(threadIdx.x + 1); ++b)
    if (past(b) && (b == 0 || !past(b - 1))) *slot = b;
  __syncthreads();
  return *slot;
}

// Sorts the first n entries of list (n <= kList) ascending.
__device__ __forceinline__ void sort_list(u64* list, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) list[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int t = threadIdx.x; t < size / 2; t += kThreads) {
        const int i = 2 * t - (t & (j - 1)), l = i + j;
        const u64 a = list[i], b = list[l];
        if ((a > b) == ((i & k) == 0)) {
          list[i] = b;
          list[l] = a;
        }
      }
      __syncthreads();
    }
}

// Running masses (inclusive) over the sorted list into s.mass.
__device__ __forceinline__ void sum_list(Smem& s, int n, const Scale& sc) {
  constexpr int kPer = kList / kThreads;
  u64 w[kPer], mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x * kPer + k;
    w[k] = i < n ? weigh(entry_x(s.list[i]), sc, s.table, s.table_f) : 0;
    mine += w[k];
  }
  u64 at = block_scan(mine, s.red);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    at += w[k];
    s.mass[threadIdx.x * kPer + k] = at;
  }
  __syncthreads();
}

// Appends a token to this CTA's list; what does not fit is only counted.
__device__ __forceinline__ void append(Smem& s, float x, int i) {
  const int at = atomicAdd(&s.n_list, 1);
  if (at < kList) s.list[at] = entry_of(x, i);
}

enum { kByCount, kMassAtLeast, kMassAbove };

// The cut of the order inside bin `b` of the head (any number of tokens): the
// first token whose rank (1, 2, ...) reaches `rank`, or whose running mass
// reaches or exceeds `target`.  *mass: the running mass with it; *entry: the
// token.  One CTA does it, over the whole row, where too many tokens share the
// cuts' bins to be gathered at once: the bin's keys are cut into 2,048 ranges
// again and again until the cut's range is short, or a single value, whose
// tokens are told apart by index.
template <typename T>
__device__ __noinline__ void find_in_bin(Smem& s, const T* row, int vocab, const Scale& sc, int b, uint32_t c_before,
                                         u64 m_before, int mode, uint32_t rank, double target, u64* mass,
                                         u64* entry) {
  auto past = [&](uint32_t c, u64 m) {
    return mode == kByCount ? c >= rank : (mode == kMassAtLeast ? (double)m >= target : (double)m > target);
  };
  uint32_t lo = 0, hi = 0xffffffffu;
  for (;;) {
    uint32_t kmin = 0xffffffffu, kmax = 0, n = 0;
    sweep(row, 0, vocab, [&](float x, int) {
      const uint32_t k = key_of(x);
      if (x >= sc.cut && k >= lo && k <= hi && bin_of(x, sc) == b) {
        kmin = min(kmin, k);
        kmax = max(kmax, k);
        ++n;
      }
    });
    kmin = (uint32_t)block_min(kmin, s.red);
    kmax = (uint32_t)block_max(kmax, s.red);
    n = (uint32_t)block_sum(n, s.red);
    if (kmin == kmax) {
      const float x = of_key(kmin);
      const u64 w = weigh(x, sc, s.table, s.table_f);
      // the t-th of n equal tokens (t >= 1): estimated, then set right
      int64_t t;
      if (mode == kByCount)
        t = (int64_t)rank - c_before;
      else
        t = w ? (int64_t)((target - (double)m_before) / (double)w) : 1;
      t = max((int64_t)1, min((int64_t)n, t));
      while (t > 1 && past(c_before + (uint32_t)t - 1, m_before + (t - 1) * w)) --t;
      while (t < (int64_t)n && !past(c_before + (uint32_t)t, m_before + t * w)) ++t;
      *mass = m_before + t * w;
      // its index: each thread counts the equals of one stretch of the row
      const int per = (vocab + kThreads - 1) / kThreads;
      const int i0 = min(vocab, (int)threadIdx.x * per), i1 = min(vocab, i0 + per);
      int mine = 0;
      for (int i = i0; i < i1; ++i) mine += key_of(to_f(row[i])) == kmin;
      int64_t left = t - (int64_t)block_scan(mine, s.red);
      if (left >= 1 && left <= mine)
        for (int i = i0; i < i1; ++i)
          if (key_of(to_f(row[i])) == kmin && --left == 0) s.out = entry_of(x, i);
      __syncthreads();
      *entry = s.out;
      return;
    }
    if (n <= kList) {
      if (threadIdx.x == 0) s.n_list = 0;
      __syncthreads();
      sweep(row, 0, vocab, [&](float x, int i) {
        const uint32_t k = key_of(x);
        if (x >= sc.cut && k >= lo && k <= hi && bin_of(x, sc) == b) append(s, x, i);
      });
      __syncthreads();
      sort_list(s.list, (int)n);
      sum_list(s, (int)n, sc);
      u64 best = n - 1;
      for (uint32_t i = threadIdx.x; i < n; i += kThreads)
        if (past(c_before + i + 1, m_before + s.mass[i])) best = min(best, (u64)i);
      best = block_min(best, s.red);
      *mass = m_before + s.mass[best];
      *entry = s.list[best];
      __syncthreads();
      return;
    }
    // 2,048 ranges of the keys kmax .. kmin, descending
    const int shift = max(0, 32 - __clz(kmax - kmin) - 11);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      s.mass[i] = 0;
      s.count[i] = 0;
    }
    __syncthreads();
    sweep(row, 0, vocab, [&](float x, int) {
      const uint32_t k = key_of(x);
      if (x >= sc.cut && k >= kmin && k <= kmax && bin_of(x, sc) == b) {
        const uint32_t at = (kmax - k) >> shift;
        atomicAdd(s.count + at, 1u);
        atomicAdd(s.mass + at, weigh(x, sc, s.table, s.table_f));
      }
    });
    __syncthreads();
    accumulate_bins(s.count, s.mass, s.red);
    const int at = first_bin([&](int i) { return past(c_before + s.count[i], m_before + s.mass[i]); }, s.found);
    if (at > 0) {
      c_before += s.count[at - 1];
      m_before += s.mass[at - 1];
    }
    const uint32_t top = kmax - ((uint32_t)at << shift);
    hi = top;
    lo = (top - kmin) < (1u << shift) ? kmin : top - ((1u << shift) - 1u);
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int c_size = (int)cluster.num_blocks(), c_rank = (int)cluster.block_rank();
  const int r = blockIdx.x / c_size;
  Smem& s0 = *cluster.map_shared_rank(&s, 0);
  if (tid < 64) {
    s.table[tid] = p.table[tid];
    s.table_f[tid] = (float)p.table[tid] * 0.25f;
  }
  if (tid < kCoarse) s.coarse[tid] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const T* row = static_cast<const T*>(p.x) + (int64_t)r * p.row_stride;
  const int lo_i = min(p.vocab, c_rank * p.stretch), hi_i = min(p.vocab, lo_i + p.stretch);
  const int pi = r / p.rows_per_param;
  const float temp = p.temperature ? __ldg(p.temperature + pi) : 1.f;
  const int top_k = p.top_k ? __ldg(p.top_k + pi) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + pi) : 1.f;
  const float min_p = p.min_p ? __ldg(p.min_p + pi) : 0.f;
  const float u = __ldg(p.u + r);

  // ---- 1. the maximum, and whether anything is wrong ----
  {
    float mx = -INFINITY;
    sweep(row, lo_i, hi_i, [&](float x, int) { mx = max_nan(mx, x); });
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float* red = reinterpret_cast<float*>(s.red);
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kThreads / 32; ++w) mx = max_nan(mx, red[w]);
      s.max = mx;
    }
  }
  cluster.sync();
  float row_max = s0.max;
  for (int c = 1; c < c_size; ++c) row_max = max_nan(row_max, cluster.map_shared_rank(&s, c)->max);
  const bool bad = !(row_max > -INFINITY && row_max < INFINITY) ||
                   !(temp == 0.f || (temp >= 0x1p-100f && temp <= 0x1p60f)) || !(top_p >= 0.f) ||
                   !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
  if (bad || temp == 0.f) {
    // the maximum's first index
    if (!bad) {
      int first = p.vocab;
      sweep(row, lo_i, hi_i, [&](float x, int i) {
        if (x == row_max) first = min(first, i);
      });
      first = (int)block_min((u64)first, s.red);
      if (tid == 0) s.x_index = first;
    }
    cluster.sync();  // (also: no CTA ends while its maximum is read)
    if (c_rank == 0 && tid == 0) {
      int id = -1;
      if (!bad) {
        id = s.x_index;
        for (int c = 1; c < c_size; ++c) id = min(id, cluster.map_shared_rank(&s, c)->x_index);
      }
      p.ids[r] = id;
      if (p.logprob) p.logprob[r] = bad ? -INFINITY : 0.f;
      if (bad) report(p.status, STV_DEV_BAD_SAMPLE);
    }
    cluster.sync();
    return;
  }
  Scale sc = make_scale(row_max, temp);
  const bool want_k = top_k > 0 && top_k < p.vocab, has_p = top_p < 1.f, want_m = min_p > 0.f;
  const bool m_only = want_m && !want_k && !has_p;  // the head is what min_p keeps
  const bool need_all = !want_k && !m_only;         // the mass of every token
  const float x_min = want_m ? __double2float_ru((double)sc.max + (double)temp * log((double)min_p)) : -INFINITY;

  // ---- the sample: how far down the cuts lie, and how many tokens that is ----
  bool direct;
  {
    const float per = 4.f / 64.f * sc.inv_c;  // quarter octaves per unit of x
    sweep(
        row, lo_i, hi_i,
        [&](float x, int) {
          const float y = (sc.max - x) * per;
          if (y < (float)(kCoarse - 8)) atomicAdd(s.coarse + (int)y, 1u);
        },
        p.sample_every);
    cluster.sync();
    const float f = (float)p.sample_every;
    if (tid < kCoarse) {
      uint32_t n = 0;
      for (int c = 0; c < c_size; ++c) n += cluster.map_shared_rank(&s, c)->coarse[tid];
      s.coarse_est[tid] = (float)n;
    }
    __syncthreads();
    if (tid < 32) {  // a warp: lane l holds eight bins, from the far end for the tail's mass
      float cnt[8], wgt[8], c8 = 0.f, w8 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cnt[i] = s.coarse_est[tid * 8 + i];
        wgt[i] = f * cnt[i] * exp2f(-0.25f * (float)(tid * 8 + i));
        c8 += cnt[i];
        w8 += wgt[i];
      }
      float c_incl = c8, w_incl = w8;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, c_incl, o), b = __shfl_up_sync(0xffffffffu, w_incl, o);
        if (tid >= o) {
          c_incl += a;
          w_incl += b;
        }
      }
      const float w_all = __shfl_sync(0xffffffffu, w_incl, 31);
      // enough: top_k tokens with four deviations of the sample's count; or a
      // tail below the first bin of under 0.7 of what the cut leaves out (the
      // maximum counts as 1, so tokens the sample missed err to this side)
      const float k_need = (float)top_k / f;
      const float enough = p.sample_every > 1 ? k_need + 4.f * sqrtf(k_need) + 8.f : k_need;
      const float left = has_p ? 1.f - top_p : 1.f - u;
      const float tail = 0.7f * left * (1.f + w_all);
      int b = kCoarse;
      float n_head = 0.f, c = c_incl - c8, w = w_incl - w8;
      for (int i = 0; i < 8; ++i) {  // the bins up to this one are enough
        c += cnt[i];
        w += wgt[i];
        const int past = tid * 8 + i + 1;
        if (m_only ? (float)past > (sc.max - x_min) * per : (want_k ? c >= enough : w_all - w <= tail)) {
          b = past;
          n_head = c;
          break;
        }
      }
      const unsigned any = __ballot_sync(0xffffffffu, b < kCoarse);
      const int src = any ? __ffs(any) - 1 : 31;
      b = __shfl_sync(0xffffffffu, b, src);
      n_head = __shfl_sync(0xffffffffu, any ? n_head : c_incl, src);
      if (tid == 0) {
        s.found[0] = b;
        s.found[1] = (int)fminf(n_head * f, 1e9f);
      }
    }
    __syncthreads();
    const int b = s.found[0];
    float cut = b < kCoarse - 8 ? sc.max - (float)b / per : sc.floor;
    if (m_only) cut = x_min;
    set_cut(sc, cut);
    direct = s.found[1] <= kDirect;
  }

  u64 total = 0;  // first CTA: the row's mass, where need_all
  u64 kept = 0, token = 0;
  for (int round = 0;; ++round) {
    if (round) {  // the head was too short: every token with any mass
      set_cut(sc, sc.floor);
      direct = false;
    }
    const bool complete = sc.cut <= sc.floor;
    // ---- 2. the mass of all, the head's tokens or bins ----
    for (int i = tid; i < kBins && !direct; i += kThreads) {
      s.count[i] = 0;
      s.mass[i] = 0;
    }
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    u64 sum = 0;
    const bool all = need_all && round == 0;
    sweep(row, lo_i, hi_i, [&](float x, int i) {
      u64 w = 0;
      if (all) {
        w = weigh(x, sc, s.table, s.table_f);
        sum += w;
      }
      if (x >= sc.cut) {
        if (direct) {
          append(s, x, i);
        } else {
          if (!all) w = weigh(x, sc, s.table, s.table_f);
          const int b = bin_of(x, sc);
          atomicAdd(s.count + b, 1u);
          atomicAdd(s.mass + b, w);
        }
      }
    });
    if (all) {
      sum = block_sum(sum, s.red);
      if (tid == 0) s.part = sum;
    }
    cluster.sync();
    if (!direct) {
      // each CTA adds up a share of the bins, for the first one
      const int per = kBins / c_size;
      for (int i = c_rank * per + tid; i < (c_rank + 1) * per; i += kThreads) {
        uint32_t c = 0;
        u64 m = 0;
        for (int k = 0; k < c_size; ++k) {
          const Smem* o = cluster.map_shared_rank(&s, k);
          c += o->count[i];
          m += o->mass[i];
        }
        s0.tot_count[i] = c;
        s0.tot_mass[i] = m;
      }
      cluster.sync();
    }
    auto c_before = [&](int b) { return b ? s.tot_count[b - 1] : 0u; };
    auto m_before = [&](int b) { return b ? s.tot_mass[b - 1] : 0ull; };
    // the tokens of every CTA's list in the first one's; false if they do not fit
    auto merge_lists = [&](int* n_out) {
      int n = s.n_list;
      bool fits = n <= kList;
      for (int c = 1; c < c_size && fits; ++c) {
        const Smem* o = cluster.map_shared_rank(&s, c);
        const int m = o->n_list;
        fits = n + m <= kList;
        for (int i = tid; i < m && fits; i += kThreads) s.list[n + i] = o->list[i];
        n += m;
      }
      __syncthreads();
      *n_out = n;
      return fits;
    };
    bool has_k = want_k;
    const bool has_m = want_m && x_min >= sc.cut;
    Decision d;
    d.done = 0;
    d.kb = d.mb = -1;
    d.pb1 = d.ub1 = 0;
    d.pb2 = d.ub2 = -1;
    if (c_rank == 0) {
      if (all) {
        total = s.part;
        for (int c = 1; c < c_size; ++c) total += cluster.map_shared_rank(&s, c)->part;
      }
      if (direct) {
        int n;
        if (merge_lists(&n) && n > 0) {
          sort_list(s.list, n);
          sum_list(s, n, sc);
          const u64 head = s.mass[n - 1];
          bool ok = true;
          if (has_k && n < top_k) {
            ok = complete;
            has_k = false;
          }
          kept = has_k ? s.mass[top_k - 1] : (need_all ? total : head);
          if (has_p) {
            const double t = (double)top_p * (double)kept;
            ok = ok && (double)head >= t;
            u64 m = ~0ull;
            for (int i = tid; i < n; i += kThreads)
              if ((double)s.mass[i] >= t) m = min(m, s.mass[i]);
            kept = min(kept, block_min(m, s.red));
          }
          if (has_m) {
            u64 w = 0;
            for (int i = tid; i < n; i += kThreads)
              if (entry_x(s.list[i]) >= x_min) w = max(w, s.mass[i]);
            kept = min(kept, block_max(w, s.red));
          }
          const double t = (double)u * (double)kept;
          ok = ok && (double)head > t;
          u64 at = n - 1;
          for (int i = tid; i < n; i += kThreads)
            if ((double)s.mass[i] > t) at = min(at, (u64)i);
          at = block_min(at, s.red);
          token = s.list[at];
          d.done = ok;
        }
      } else {
        accumulate_bins(s.tot_count, s.tot_mass, s.red);
        const uint32_t n_head = s.tot_count[kBins - 1];
        const u64 head = s.tot_mass[kBins - 1];
        bool ok = true;
        if (has_k && n_head < (uint32_t)top_k) {
          ok = complete;
          has_k = false;
        }
        // a cut's mass lies between the mass before its first bin and with its last
        u64 lo = need_all ? total : head, hi = lo;
        if (has_k) {
          d.kb = first_bin([&](int b) { return s.tot_count[b] >= (uint32_t)top_k; }, s.found);
          lo = m_before(d.kb);
          hi = s.tot_mass[d.kb];
        }
        if (has_p) {
          const double t1 = (double)top_p * (double)lo, t2 = (double)top_p * (double)hi;
          ok = ok && (double)head >= t2;
          d.pb1 = first_bin([&](int b) { return (double)s.tot_mass[b] >= t1; }, s.found + 1);
          d.pb2 = first_bin([&](int b) { return (double)s.tot_mass[b] >= t2; }, s.found + 2);
          lo = min(lo, m_before(d.pb1));
          hi = min(hi, s.tot_mass[d.pb2]);
        }
        if (has_m) {
          d.mb = x_min <= sc.max ? bin_of(x_min, sc) : 0;
          lo = min(lo, m_before(d.mb));
          hi = min(hi, s.tot_mass[d.mb]);
        }
        const double u1 = (double)u * (double)lo, u2 = (double)u * (double)hi;
        ok = ok && (double)head > u2;
        d.ub1 = first_bin([&](int b) { return (double)s.tot_mass[b] > u1; }, s.found + 3);
        d.ub2 = first_bin([&](int b) { return (double)s.tot_mass[b] > u2; }, s.found + 4);
        auto wanted = [&](int b) {
          return b == d.kb || (b >= d.pb1 && b <= d.pb2) || b == d.mb || (b >= d.ub1 && b <= d.ub2);
        };
        uint32_t mine = 0;
        for (int b = kBinsPer * tid; b < kBinsPer * (tid + 1); ++b)
          if (wanted(b)) mine += s.tot_count[b] - c_before(b);
        const uint32_t n = (uint32_t)block_sum(mine, s.red);
        if ((ok || round) && n > kList) {
          // ---- one cut after the other, without the other CTAs ----
          kept = need_all ? total : head;
          if (has_k)
            find_in_bin(s, row, p.vocab, sc, d.kb, c_before(d.kb), m_before(d.kb), kByCount, (uint32_t)top_k, 0.0,
                        &kept, &token);
          if (has_p) {
            const double t = (double)top_p * (double)kept;
            const int b = first_bin([&](int i) { return (double)s.tot_mass[i] >= t; }, s.found);
            u64 m;
            find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), kMassAtLeast, 0, t, &m, &token);
            kept = min(kept, m);
          }
          if (has_m) {
            u64 w = 0;
            sweep(row, 0, p.vocab, [&](float x, int) {
              if (x >= x_min) w += weigh(x, sc, s.table, s.table_f);
            });
            kept = min(kept, block_sum(w, s.red));
          }
          const double t = (double)u * (double)kept;
          const int b = first_bin([&](int i) { return (double)s.tot_mass[i] > t; }, s.found);
          u64 m;
          find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), kMassAbove, 0, t, &m, &token);
          d.done = 1;
        } else {
          d.done = ok || round ? 2 : 0;
        }
      }
      if (tid == 0) s.d = d;
    }
    cluster.sync();
    d = s0.d;
    if (d.done == 0 && round == 0) {
      cluster.sync();  // the decision is read before it is written again
      continue;
    }
    if (d.done != 2) break;
    // ---- 3. the tokens of the cuts' bins ----
    auto wanted = [&](int b) {
      return b == d.kb || (b >= d.pb1 && b <= d.pb2) || b == d.mb || (b >= d.ub1 && b <= d.ub2);
    };
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    sweep(row, lo_i, hi_i, [&](float x, int i) {
      if (x >= sc.cut && wanted(bin_of(x, sc))) append(s, x, i);
    });
    cluster.sync();
    if (c_rank == 0) {
      int n;
      merge_lists(&n);  // counted above: they fit
      sort_list(s.list, n);
      sum_list(s, n, sc);
      for (int i = tid; i < n; i += kThreads) {
        const int b = bin_of(entry_x(s.list[i]), sc);
        if (i == 0 || bin_of(entry_x(s.list[i - 1]), sc) != b) s.count[b] = i;
      }
      __syncthreads();
      // entry i: its bin, rank and running mass in the whole order
      auto place = [&](int i, int* b, uint32_t* rank, u64* g) {
        *b = bin_of(entry_x(s.list[i]), sc);
        const int f = s.count[*b];
        *rank = c_before(*b) + (i - f) + 1;
        *g = m_before(*b) + s.mass[i] - (f ? s.mass[f - 1] : 0ull);
      };
      // the smallest running mass among the entries that `in` admits
      auto least = [&](auto&& in) {
        u64 m = ~0ull;
        for (int i = tid; i < n; i += kThreads) {
          int b;
          uint32_t rank;
          u64 g;
          place(i, &b, &rank, &g);
          if (in(b, rank, g)) m = min(m, g);
        }
        return block_min(m, s.red);
      };
      kept = need_all ? total : s.tot_mass[kBins - 1];
      if (d.kb >= 0) kept = least([&](int b, uint32_t rank, u64) { return b == d.kb && rank == (uint32_t)top_k; });
      if (has_p) {
        const double t = (double)top_p * (double)kept;
        kept = min(kept, least([&](int, uint32_t, u64 g) { return (double)g >= t; }));
      }
      if (has_m) {
        u64 w = 0;
        for (int i = tid; i < n; i += kThreads) {
          const float x = entry_x(s.list[i]);
          if (bin_of(x, sc) == d.mb && x >= x_min) w += weigh(x, sc, s.table, s.table_f);
        }
        kept = min(kept, m_before(d.mb) + block_sum(w, s.red));
      }
      const double t = (double)u * (double)kept;
      u64 at = n - 1;
      for (int i = tid; i < n; i += kThreads) {
        int b;
        uint32_t rank;
        u64 g;
        place(i, &b, &rank, &g);
        if ((double)g > t) at = min(at, (u64)i);
      }
      at = block_min(at, s.red);
      token = s.list[at];
    }
    break;
  }
  if (c_rank == 0 && tid == 0) {
    p.ids[r] = (int32_t)(uint32_t)token;
    if (p.logprob) {
      // kept in units of the largest w
      const double m = (double)kept / (double)weigh(sc.max, sc, s.table, s.table_f);
      p.logprob[r] = (float)(((double)entry_x(token) - (double)sc.max) / (double)temp - log(m));
    }
  }
  cluster.sync();  // no CTA ends while the first one reads its list
}

template <typename T>
cudaError_t launch_sample(SampleParams& p, cudaStream_t st) {
  int sm = 0;
  if (device_sm_count(&sm) != STV_OK) return cudaErrorUnknown;
  // CTAs per row: enough to give every SM two, of 2,048 tokens at least
  int c = 1;
  while (c < kMaxCluster && (int64_t)p.n_rows * c * 2 <= 2 * sm && p.vocab / (2 * c) >= 2048) c *= 2;
  constexpr int VE = 16 / sizeof(T);
  p.stretch = ((p.vocab + c - 1) / c + VE - 1) / VE * VE;
  p.sample_every = std::max(1, std::min(8, p.vocab / 16384));
  const size_t smem = sizeof(Smem);
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_rows * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
  }
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

}  // namespace
}  // namespace stv

extern "C" int stv_sample(const void* logits, int dtype, int64_t row_stride, int n_rows, int vocab,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int rows_per_param, const float* u, int32_t* ids, float* logprob, int32_t* dev_status,
                          stv_stream_t stream) {
  using namespace stv;
  if (dtype != STV_F32 && dtype != STV_F16 && dtype != STV_BF16) return STV_ERR_INVALID_ARG;
  if (n_rows < 0 || rows_per_param < 1 || vocab < 1) return STV_ERR_INVALID_ARG;
  if (vocab > kMaxVocab) return STV_ERR_SHAPE_UNSUPPORTED;
  if (n_rows == 0) return STV_OK;
  if (n_rows > 0x7fffffff / kMaxCluster) return STV_ERR_SHAPE_UNSUPPORTED;
  if (!logits || !u || !ids || (n_rows > 1 && row_stride < vocab)) return STV_ERR_INVALID_ARG;
  if ((uintptr_t)logits % (dtype == STV_F32 ? 4 : 2)) return STV_ERR_INVALID_ARG;
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.x = logits;
  p.row_stride = row_stride;
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.rows_per_param = rows_per_param;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.ids = ids;
  p.logprob = logprob;
  p.status = dev_status;
  for (int j = 0; j < 64; ++j) p.table[j] = (uint32_t)llround(ldexp(exp2(j / 64.0), 30));
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == STV_F32   ? launch_sample<float>(p, st)
                        : dtype == STV_F16 ? launch_sample<__half>(p, st)
                                           : launch_sample<__nv_bfloat16>(p, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
