// sample.cu -- sampling from the target's logits with temperature, top-k,
// top-p and min-p from given random numbers (include/stv.h, stv_sample).
//
// Every filter and the draw itself is a cut of one order (logit descending,
// then index ascending) at a given count or a given mass, so no sort of the
// vocabulary is needed.  With y = (max - x) log2(e) / T, a token's bin is
// rint(32 y): bins follow the order, and 2,048 of them, each with its count
// and its mass, say in which bin every cut lies.  The tokens of those few
// bins are gathered, sorted in shared memory, and the cuts made exactly.
//
// Masses.  w = 2^-y as an integer of scale 2^45: y in two floats, 2^-(bin/32)
// from a table of 32 entries, 2^-r for |r| <= 1/64 as a polynomial whose
// rounding error is 2^-24 of |2^-r - 1| (2^-6.5).  Integer sums do not depend
// on their order, so bins, cuts and tokens do not either.
//
// One CTA per row: a pass for the maximum, one for the bins, one to gather
// (the last two from L2).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "stv_device.cuh"

namespace stv {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kList = 2048;      // tokens gathered around the cuts
constexpr int kMaxVocab = 1 << 19;
constexpr int kScaleBits = 44;   // w of the largest logit is 2^44; sums stay below 2^63
constexpr float kFarY = 62.f;    // beyond it w = 0 (2^-62 < 2^-45)

struct SampleParams {
  const void* x;
  int64_t row_stride;
  int n_rows, vocab, rows_per_param;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logprob;
  int32_t* status;
  uint32_t table[32];  // 2^31 * 2^(-j / 32)
};

struct Smem {
  u64 mass[kBins];    // mass of the bins, then of them and all before
  u64 list[kList];    // (~key << 32) | index
  u64 sums[kList];    // running mass over the list
  uint32_t count[kBins];
  uint32_t first[kBins];   // a bin's first place in the list
  uint32_t table[32];
  u64 red[kThreads / 32];
  u64 out;
  int found[8];
  int n_list;
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

// log2(e) / T in two floats, and the row's maximum.
struct Scale {
  float max, hi, lo;
};

struct Weight {
  int bin;
  u64 w;
};

__device__ __forceinline__ int bin_of(float x, const Scale& sc) {
  const float yh = (sc.max - x) * sc.hi;
  return yh < kFarY ? __float2int_rn(yh * 32.f) : kBins - 1;
}

__device__ __forceinline__ Weight weigh(float x, const Scale& sc, const uint32_t* table) {
  const float d = sc.max - x;
  // the part of max - x that d's rounding lost
  const float t = d - sc.max;
  const float dl = (sc.max - (d - t)) - (x + t);
  const float yh = d * sc.hi;
  Weight r;
  if (!(yh < kFarY)) {
    r.bin = kBins - 1;
    r.w = 0;
    return r;
  }
  const float yl = fmaf(dl, sc.hi, fmaf(d, sc.lo, fmaf(d, sc.hi, -yh)));
  const int k = __float2int_rn(yh * 32.f);
  const float z = fmaf((float)k, -1.f / 32.f, yh) + yl;  // |z| <= 1/64 and a little
  // 2^-z - 1
  float q = fmaf(z, 0.0096181291f, -0.055504109f);
  q = fmaf(z, q, 0.24022651f);
  q = fmaf(z, q, -0.69314718f);
  q *= z;
  const uint32_t tj = table[k & 31];
  const uint32_t m = tj + (uint32_t)__float2int_rn((float)tj * q);
  const int n = k >> 5;
  r.bin = k;
  r.w = ((((u64)m << (kScaleBits + 1 - 31)) >> n) + 1) >> 1;  // rounded
  return r;
}

// Calls f(x, index) for the row's tokens, a thread's own in ascending order.
template <typename T, typename F>
__device__ __forceinline__ void sweep(const T* row, int vocab, F&& f) {
  constexpr int VE = 16 / sizeof(T);
  const int head = min(vocab, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T));
  const int n_vec = (vocab - head) / VE;
  if ((int)threadIdx.x < head) f(to_f(row[threadIdx.x]), (int)threadIdx.x);
  const uint4* v = reinterpret_cast<const uint4*>(row + head);
  for (int i = threadIdx.x; i < n_vec; i += kThreads) {
    const uint4 q = __ldg(v + i);
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int k = 0; k < VE; ++k) f(to_f(e[k]), head + i * VE + k);
  }
  for (int i = head + n_vec * VE + threadIdx.x; i < vocab; i += kThreads) f(to_f(row[i]), i);
}

template <typename Op>
__device__ __forceinline__ u64 block_reduce(u64 x, u64* red, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  u64 y = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o; o >>= 1) y = op(y, __shfl_xor_sync(0xffffffffu, y, o));
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
  const u64 ws = red[lane];
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
  const int b = 2 * threadIdx.x;
  const u64 c0 = count[b], c1 = count[b + 1], m0 = mass[b], m1 = mass[b + 1];
  const u64 c = block_scan(c0 + c1, red);
  const u64 m = block_scan(m0 + m1, red);
  count[b] = (uint32_t)(c + c0);
  count[b + 1] = (uint32_t)(c + c0 + c1);
  mass[b] = m + m0;
  mass[b + 1] = m + m0 + m1;
  __syncthreads();
}

// First bin for which past(bin) holds (it holds for all later ones); kBins - 1
// if none.
template <typename F>
__device__ __forceinline__ int first_bin(F&& past, int* slot) {
  if (threadIdx.x == 0) *slot = kBins - 1;
  __syncthreads();
  for (int b = 2 * threadIdx.x; b < 2 * (int)threadIdx.x + 2; ++b)
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

__device__ __forceinline__ u64 entry_of(float x, int i) {
  return ((u64)(~key_of(x)) << 32) | (uint32_t)i;
}
__device__ __forceinline__ float entry_x(u64 e) { return of_key(~(uint32_t)(e >> 32)); }

// Running masses (inclusive) over the sorted list into sums.
__device__ __forceinline__ void sum_list(Smem& s, int n, const Scale& sc) {
  constexpr int kPer = kList / kThreads;
  u64 w[kPer], mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x * kPer + k;
    w[k] = i < n ? weigh(entry_x(s.list[i]), sc, s.table).w : 0;
    mine += w[k];
  }
  u64 at = block_scan(mine, s.red);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    at += w[k];
    s.sums[threadIdx.x * kPer + k] = at;
  }
  __syncthreads();
}

enum { kByCount, kMassAtLeast, kMassAbove };

// The cut of the order inside bin `b` (any number of tokens): the first token
// whose rank (1, 2, ...) reaches `rank`, or whose running mass reaches or
// exceeds `target`.  *mass: the running mass with it; *entry: the token.
// Used where too many tokens share the cuts' bins to be gathered at once:
// the bin's keys are cut into 2,048 ranges again and again until the cut's
// range is short, or a single value, whose tokens are told apart by index.
template <typename T>
__device__ void find_in_bin(Smem& s, const T* row, int vocab, const Scale& sc, int b, uint32_t c_before,
                            u64 m_before, int mode, uint32_t rank, double target, u64* mass,
                            u64* entry) {
  auto past = [&](uint32_t c, u64 m) {
    return mode == kByCount ? c >= rank : (mode == kMassAtLeast ? (double)m >= target : (double)m > target);
  };
  uint32_t lo = 0, hi = 0xffffffffu;
  uint32_t* sub_count = reinterpret_cast<uint32_t*>(s.sums);  // the list's storage is free here
  for (;;) {
    uint32_t kmin = 0xffffffffu, kmax = 0, n = 0;
    sweep(row, vocab, [&](float x, int) {
      const uint32_t k = key_of(x);
      if (x > -INFINITY && k >= lo && k <= hi && bin_of(x, sc) == b) {
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
      const u64 w = weigh(x, sc, s.table).w;
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
      sweep(row, vocab, [&](float x, int i) {
        const uint32_t k = key_of(x);
        if (x > -INFINITY && k >= lo && k <= hi && bin_of(x, sc) == b) s.list[atomicAdd(&s.n_list, 1)] = entry_of(x, i);
      });
      __syncthreads();
      sort_list(s.list, (int)n);
      sum_list(s, (int)n, sc);
      u64 best = n - 1;
      for (uint32_t i = threadIdx.x; i < n; i += kThreads)
        if (past(c_before + i + 1, m_before + s.sums[i])) best = min(best, (u64)i);
      best = block_min(best, s.red);
      *mass = m_before + s.sums[best];
      *entry = s.list[best];
      __syncthreads();
      return;
    }
    // 2,048 ranges of the keys kmax .. kmin, descending
    const int shift = max(0, 32 - __clz(kmax - kmin) - 11);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      s.list[i] = 0;
      sub_count[i] = 0;
    }
    __syncthreads();
    sweep(row, vocab, [&](float x, int) {
      const uint32_t k = key_of(x);
      if (x > -INFINITY && k >= kmin && k <= kmax && bin_of(x, sc) == b) {
        const uint32_t at = (kmax - k) >> shift;
        atomicAdd(sub_count + at, 1u);
        atomicAdd(s.list + at, weigh(x, sc, s.table).w);
      }
    });
    __syncthreads();
    accumulate_bins(sub_count, s.list, s.red);
    const int at = first_bin([&](int i) { return past(c_before + sub_count[i], m_before + s.list[i]); }, s.found);
    if (at > 0) {
      c_before += sub_count[at - 1];
      m_before += s.list[at - 1];
    }
    const uint32_t top = kmax - ((uint32_t)at << shift);
    hi = top;
    lo = max(kmin, top - ((1u << shift) - 1u));
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, r = blockIdx.x;
  if (tid < 32) s.table[tid] = p.table[tid];
  for (int i = tid; i < kBins; i += kThreads) {
    s.count[i] = 0;
    s.mass[i] = 0;
  }
  grid_dep_wait();
  grid_dep_launch();
  const T* row = static_cast<const T*>(p.x) + (int64_t)r * p.row_stride;
  const int pi = r / p.rows_per_param;
  const float temp = p.temperature ? __ldg(p.temperature + pi) : 1.f;
  const int top_k = p.top_k ? __ldg(p.top_k + pi) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + pi) : 1.f;
  const float min_p = p.min_p ? __ldg(p.min_p + pi) : 0.f;
  const float u = __ldg(p.u + r);

  // ---- the maximum, its first index, and whether anything is wrong ----
  float best = -INFINITY;
  int best_i = 0;
  bool bad = false;
  sweep(row, p.vocab, [&](float x, int i) {
    bad = bad || !(x < INFINITY);
    if (x > best) {
      best = x;
      best_i = i;
    }
  });
  const u64 top = block_min(entry_of(best, best_i), s.red);
  bad = __syncthreads_or(bad);
  Scale sc;
  sc.max = entry_x(top);
  bad = bad || !(sc.max > -INFINITY) || !(temp == 0.f || (temp >= 0x1p-100f && temp <= 0x1p60f)) || !(top_p >= 0.f) ||
        !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
  if (bad || temp == 0.f) {
    if (tid == 0) {
      p.ids[r] = bad ? -1 : (int32_t)(uint32_t)top;
      if (p.logprob) p.logprob[r] = bad ? -INFINITY : 0.f;
      if (bad) report(p.status, STV_DEV_BAD_SAMPLE);
    }
    return;
  }
  {
    const double c = 1.4426950408889634074 / (double)temp;  // 2^-60 .. 2^101: two normal floats
    sc.hi = (float)c;
    sc.lo = (float)(c - (double)sc.hi);
  }

  // ---- the bins ----
  sweep(row, p.vocab, [&](float x, int) {
    if (x > -INFINITY) {
      const Weight w = weigh(x, sc, s.table);
      atomicAdd(s.count + w.bin, 1u);
      atomicAdd(s.mass + w.bin, w.w);
    }
  });
  __syncthreads();
  accumulate_bins(s.count, s.mass, s.red);

  // ---- the bins that the cuts lie in; a cut's mass is known to lie between
  // the mass before its first and with its last ----
  auto c_before = [&](int b) { return b ? s.count[b - 1] : 0u; };
  auto m_before = [&](int b) { return b ? s.mass[b - 1] : 0ull; };
  const bool has_k = top_k > 0 && (uint32_t)top_k < s.count[kBins - 1];
  const bool has_p = top_p < 1.f, has_m = min_p > 0.f;
  int kb = 0, pb1 = 0, pb2 = 0, mb = 0;
  u64 lo = s.mass[kBins - 1], hi = lo;
  if (has_k) {
    kb = first_bin([&](int b) { return s.count[b] >= (uint32_t)top_k; }, s.found);
    lo = m_before(kb);
    hi = s.mass[kb];
  }
  if (has_p) {
    const double t1 = (double)top_p * (double)lo, t2 = (double)top_p * (double)hi;
    pb1 = first_bin([&](int b) { return (double)s.mass[b] >= t1; }, s.found + 1);
    pb2 = first_bin([&](int b) { return (double)s.mass[b] >= t2; }, s.found + 2);
    lo = min(lo, m_before(pb1));
    hi = min(hi, s.mass[pb2]);
  }
  float x_min = -INFINITY;
  if (has_m) {
    const double t = (double)sc.max + (double)temp * log((double)min_p);
    x_min = __double2float_ru(t);
    mb = x_min > -INFINITY ? bin_of(x_min, sc) : kBins - 1;
    lo = min(lo, m_before(mb));
    hi = min(hi, s.mass[mb]);
  }
  const double u1 = (double)u * (double)lo, u2 = (double)u * (double)hi;
  const int ub1 = first_bin([&](int b) { return (double)s.mass[b] > u1; }, s.found + 3);
  const int ub2 = first_bin([&](int b) { return (double)s.mass[b] > u2; }, s.found + 4);
  auto wanted = [&](int b) {
    return (has_k && b == kb) || (has_p && b >= pb1 && b <= pb2) || (has_m && b == mb) || (b >= ub1 && b <= ub2);
  };
  uint32_t mine = 0;
  for (int b = 2 * tid; b < 2 * tid + 2; ++b)
    if (wanted(b)) mine += s.count[b] - c_before(b);
  const uint32_t n = (uint32_t)block_sum(mine, s.red);

  u64 kept = s.mass[kBins - 1], token;
  if (n <= kList) {
    // ---- gather them, sort, and cut ----
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    sweep(row, p.vocab, [&](float x, int i) {
      if (x > -INFINITY && wanted(bin_of(x, sc))) s.list[atomicAdd(&s.n_list, 1)] = entry_of(x, i);
    });
    __syncthreads();
    sort_list(s.list, (int)n);
    sum_list(s, (int)n, sc);
    for (int i = tid; i < (int)n; i += kThreads) {
      const int b = bin_of(entry_x(s.list[i]), sc);
      if (i == 0 || bin_of(entry_x(s.list[i - 1]), sc) != b) s.first[b] = i;
    }
    __syncthreads();
    // entry i: its bin, rank and running mass in the whole order
    auto place = [&](int i, int* b, uint32_t* rank, u64* g) {
      *b = bin_of(entry_x(s.list[i]), sc);
      const int f = s.first[*b];
      *rank = c_before(*b) + (i - f) + 1;
      *g = m_before(*b) + s.sums[i] - (f ? s.sums[f - 1] : 0ull);
    };
    // the smallest running mass among the entries that `in` admits
    auto least = [&](auto&& in) {
      u64 m = ~0ull;
      for (int i = tid; i < (int)n; i += kThreads) {
        int b;
        uint32_t rank;
        u64 g;
        place(i, &b, &rank, &g);
        if (in(b, rank, g, i)) m = min(m, g);
      }
      return block_min(m, s.red);
    };
    if (has_k) kept = least([&](int b, uint32_t rank, u64, int) { return b == kb && rank == (uint32_t)top_k; });
    if (has_p) {
      const double t = (double)top_p * (double)kept;
      kept = min(kept, least([&](int, uint32_t, u64 g, int) { return (double)g >= t; }));
    }
    if (has_m) {
      u64 w = 0;
      for (int i = tid; i < (int)n; i += kThreads) {
        const float x = entry_x(s.list[i]);
        if (bin_of(x, sc) == mb && x >= x_min) w += weigh(x, sc, s.table).w;
      }
      kept = min(kept, m_before(mb) + block_sum(w, s.red));
    }
    const double t = (double)u * (double)kept;
    u64 at = n - 1;
    for (int i = tid; i < (int)n; i += kThreads) {
      int b;
      uint32_t rank;
      u64 g;
      place(i, &b, &rank, &g);
      if ((double)g > t) at = min(at, (u64)i);
    }
    at = block_min(at, s.red);
    token = s.list[at];
  } else {
    // ---- one cut after the other ----
    if (has_k)
      find_in_bin(s, row, p.vocab, sc, kb, c_before(kb), m_before(kb), kByCount, (uint32_t)top_k, 0.0, &kept, &token);
    if (has_p) {
      const double t = (double)top_p * (double)kept;
      const int b = first_bin([&](int i) { return (double)s.mass[i] >= t; }, s.found);
      u64 m;
      find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), kMassAtLeast, 0, t, &m, &token);
      kept = min(kept, m);
    }
    if (has_m) {
      u64 w = 0;
      sweep(row, p.vocab, [&](float x, int) {
        if (x >= x_min && x > -INFINITY) w += weigh(x, sc, s.table).w;
      });
      kept = min(kept, block_sum(w, s.red));
    }
    const double t = (double)u * (double)kept;
    const int b = first_bin([&](int i) { return (double)s.mass[i] > t; }, s.found);
    u64 m;
    find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), kMassAbove, 0, t, &m, &token);
  }
  if (tid == 0) {
    p.ids[r] = (int32_t)(uint32_t)token;
    if (p.logprob)
      p.logprob[r] = (float)(((double)entry_x(token) - (double)sc.max) / (double)temp -
                             log((double)kept * 0x1p-44));
  }
}

template <typename T>
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Smem));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  return launch_pdl(sample_kernel<T>, p.n_rows, kThreads, sizeof(Smem), st, p);
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
  for (int j = 0; j < 32; ++j) p.table[j] = (uint32_t)llround(ldexp(exp2(-j / 32.0), 31));
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == STV_F32   ? launch_sample<float>(p, st)
                        : dtype == STV_F16 ? launch_sample<__half>(p, st)
                                           : launch_sample<__nv_bfloat16>(p, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
