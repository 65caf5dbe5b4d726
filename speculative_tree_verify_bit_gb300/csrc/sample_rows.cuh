// sample_rows.cuh -- the kernel of stv_sample (see sample.cu), compiled by
// sample.cu once for each size of CTA: it is included inside a namespace that
// defines
//   kThreads, kCtasPerSm   the CTA's threads, and how many an SM holds
//   kBins, kBinBits        bins of the head, a power of two, and its logarithm
//   kList                  tokens gathered around the cuts
//   kDirect                more tokens than this are not gathered at once
//   kLeastHead             tokens, so that the sample knows what lies beneath

constexpr int kBinsPer = kBins / kThreads;
constexpr int kMost = kBins > kList ? kBins : kList;
static_assert(kBins % kThreads == 0 && kList % kThreads == 0 && kBins == 1 << kBinBits, "whole shares");

// What the first CTA decides for its cluster: the token is drawn; gather the
// bins; a cut lies past the head.
enum { kDone, kGather, kTooShort };
struct Decision {
  int done;
  int kb, pb1, pb2, mb, ub1, ub2;  // bins to gather; empty ranges where a cut is not made
  float lo[2], hi[2];              // two ranges of x that hold them (the draw's; all others)

  __device__ bool wanted(int b) const {
    return b == kb || (b >= pb1 && b <= pb2) || b == mb || (b >= ub1 && b <= ub2);
  }
};

// A row's temperature and maximum as the weights need them.
struct Scale {
  float max;
  float floor;  // 62 octaves under the maximum
  float zero;   // below it w = 0 (w of 2^-45 of the largest's octave is 0 already)
  float base;   // 0; the maximum where x / C would leave the integers of fp32: there
                // x - max is exact for every x >= floor
  float inv_c, c_hi, c_lo, inv_t;
  int top;          // octave of the maximum, plus 32 - kShift
  float cut;        // the head: x >= cut
  float bin_scale;  // bins of the head, from the maximum down
  float x_min;      // the least x that min_p keeps
};

struct alignas(16) Smem {
  u64 mass[kMost];      // this CTA's bins (low and high words apart); first CTA later:
                        // running mass over the list
  u64 list[kList];      // (~key << 32) | index
  uint32_t count[kBins];  // this CTA's bins; first CTA later: a bin's first place in the list
  uint4 ring[kBinnedStages][kThreads];  // vectors on their way in, a thread's own slots
  union {
    uint4 more[kStages - kBinnedStages][kThreads];  // the ring goes on here, or
    struct {  // first CTA: the merged lists; the row's bins, then of each and all before
      u64 tot_mass[kMost];
      uint32_t tot_count[kBins];
    };
  };
  u64 queue[kThreads / 32][64];   // a warp's tokens of the head, taken 32 at a time
  alignas(16) uint32_t coarse[kCoarse];
  uint32_t coarse_all[kCoarse];
  uint32_t table[64];  // 2^30 2^(j / 64), less four times the bits of kMagic
  float table_f[64];   // 2^28 2^(j / 64)
  u64 red[kThreads / 32];
  uint32_t red_c[kThreads / 32];
  u64 out;
  u64 slot[5];  // first CTA: the cuts' masses, the token, the tokens' mass
  double inv_t;
  float c_hi, c_lo, inv_c, m_hi, m_lo;  // see Scale; T ln min_p in two floats
  // first CTA: what the CTAs of the cluster hand it
  u64 part[kMaxCluster];      // their share of the row's mass
  int n_lists[kMaxCluster];   // tokens that they gathered
  int x_index[kMaxCluster];   // the maximum's first index in their stretch
  float cut[kMaxCluster];     // the value above which they gathered
  float max[kMaxCluster];     // (every CTA's) the maxima of the stretches
  Scale sc;       // of this CTA: its cut, until the bins have one
  int found[2];
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

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

// What does not depend on the maximum (one thread per CTA: fp64 runs at a 64th
// of the fp32 rate).
__device__ __forceinline__ void prepare_scale(Smem& s, float temp, float min_p) {
  const double c = (double)temp * (0.69314718055994530942 / 64.0), inv = 1.0 / (double)temp;
  const double m = min_p > 0.f ? (double)temp * log((double)min_p) : 0.0;
  s.inv_t = inv;
  s.c_hi = (float)c;
  s.c_lo = (float)(c - (double)s.c_hi);
  s.inv_c = (float)(inv * (64.0 / 0.69314718055994530942));
  s.m_hi = (float)m;
  s.m_lo = (float)(m - (double)s.m_hi);
}
__device__ __forceinline__ Scale make_scale(const Smem& s, float max, float min_p) {
  Scale sc;
  sc.max = max;
  sc.c_hi = s.c_hi;
  sc.c_lo = s.c_lo;
  sc.inv_c = s.inv_c;
  sc.inv_t = (float)s.inv_t;
  sc.floor = __fsub_rd(max, __fmul_ru(62.f * 64.f, s.c_hi));
  sc.zero = __fsub_rd(max, __fmul_ru(48.f * 64.f, s.c_hi));
  sc.base = fabsf(max) * sc.inv_c < 2097152.f ? 0.f : max;
  sc.top = (__float_as_int(fmaf(max - sc.base, sc.inv_c, kMagic)) >> 6) + 32 - kShift;
  sc.cut = sc.floor;
  sc.bin_scale = 0.f;
  sc.x_min = -INFINITY;
  if (min_p > 0.f) {  // the least float that is not below max + T ln min_p
    const float a = max + s.m_hi, b = a - max;
    sc.x_min = __fadd_ru(a, ((max - (a - b)) + (s.m_hi - b)) + s.m_lo);
  }
  return sc;
}

// w from rint(x / C) (the bits of kMagic + k) and the correction of 2^(k/64),
// in quarters (kMagic + q).
__device__ __forceinline__ u64 weight_of(int kb, float q, const Scale& sc, const uint32_t* table) {
  const uint32_t m = table[kb & 63] + ((uint32_t)__float_as_int(q) << 2);
  u64 w;  // m 2^14 2^-octaves; a shift by 64 or more leaves 0
  asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"((u64)m << 32), "r"(sc.top - (kb >> 6)));
  // the last bit set where anything is left: off by up to one either way, which
  // evens out over tokens that differ (equal ones are all off by the same)
  const uint32_t lo = (uint32_t)w;
  return (w & 0xffffffff00000000ull) | (lo | min(lo, 1u));
}

// w of a token that is not NaN (0 for -inf and whatever lies below the floor).
__device__ __forceinline__ u64 weigh(float x, const Scale& sc, const uint32_t* table, const float* table_f) {
  const float v = x - sc.base;
  // (far down, t is no longer kMagic + an integer; its bits are yet smaller, and w is 0 whatever z)
  const float t = fmaf(v, sc.inv_c, kMagic);
  const int kb = __float_as_int(t);
  const float k = t - kMagic;
  const float z = fmaf(k, -sc.c_lo, fmaf(k, -sc.c_hi, v)) * sc.inv_t;
  const float p = fmaf(fmaf(z, 1.f / 6.f, 0.5f), z, 1.f);  // e^z - 1 = z p
  // table_f = 2^28 2^(j/64), a quarter of the integer entry: |table_f z p| < 2^22
  const float q = fmaf(table_f[kb & 63] * z, p, kMagic);
  return weight_of(kb, q, sc, table);
}

// Two tokens at once, in paired fp32 instructions: the same operations, and so
// the same w.
__device__ __forceinline__ u64 pack2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(u64 r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 weigh_two(float xa, float xb, const Scale& sc, const uint32_t* table,
                                         const float* table_f) {
  const u64 v = add2(pack2(xa, xb), pack2(-sc.base, -sc.base));
  float ta, tb;
  unpack2(fma2(v, pack2(sc.inv_c, sc.inv_c), pack2(kMagic, kMagic)), ta, tb);
  const int ka = __float_as_int(ta), kb = __float_as_int(tb);
  const u64 k = add2(pack2(ta, tb), pack2(-kMagic, -kMagic));
  const u64 z = mul2(fma2(k, pack2(-sc.c_lo, -sc.c_lo), fma2(k, pack2(-sc.c_hi, -sc.c_hi), v)),
                     pack2(sc.inv_t, sc.inv_t));
  const u64 p = fma2(fma2(z, pack2(1.f / 6.f, 1.f / 6.f), pack2(0.5f, 0.5f)), z, pack2(1.f, 1.f));
  float qa, qb;
  unpack2(fma2(mul2(pack2(table_f[ka & 63], table_f[kb & 63]), z), p, pack2(kMagic, kMagic)), qa, qb);
  return weight_of(ka, qa, sc, table) + weight_of(kb, qb, sc, table);
}

// Bin of a token of the head.
__device__ __forceinline__ int bin_of(float x, const Scale& sc) {
  return min(kBins - 1, __float2int_rd((sc.max - x) * sc.bin_scale));
}

// floor(f * m) for f in [0, 1); *exact tells whether nothing was cut off.
__device__ __forceinline__ u64 share(float f, u64 m, bool* exact) {
  const uint32_t b = __float_as_uint(f) & 0x7fffffffu;  // -0 is 0
  const int e = (int)(b >> 23);
  const u64 frac = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = 150 - max(e, 1);  // f = frac * 2^-sh, sh in [24, 149]
  const u64 lo = frac * m, hi = __umul64hi(frac, m);
  if (sh >= 128) {
    *exact = (lo | hi) == 0;
    return 0;
  }
  if (sh >= 64) {
    *exact = lo == 0 && (sh == 64 || (hi << (128 - sh)) == 0);
    return sh == 64 ? hi : hi >> (sh - 64);
  }
  *exact = (lo << (64 - sh)) == 0;
  return (lo >> sh) | (hi << (64 - sh));
}
// The least mass that is at least f * m (f below 1), and that exceeds it.
__device__ __forceinline__ u64 at_least(float f, u64 m) {
  bool exact;
  const u64 t = share(f, m, &exact);
  return exact ? t : t + 1;
}
__device__ __forceinline__ u64 above(float f, u64 m) {
  bool exact;
  return share(f, m, &exact) + 1;
}

__device__ __forceinline__ void set_cut(Scale& sc, float cut) {
  sc.cut = fminf(fmaxf(cut, sc.floor), sc.max);
  const float range = sc.max - sc.cut;
  sc.bin_scale = range > 0.f ? fminf((float)kBins / range, 3e38f) : 0.f;
}

__device__ __forceinline__ void copy_async(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// Sweeps the tokens [lo, hi) of a row by whole warps: many(vector, its first
// index, whether this lane has one, where it lies in shared memory) for the
// 16-byte vectors, one(value, index, whether) for the ends that do not fill a
// vector (at most VE - 1 each, by the first warp).  Vectors come in through the
// thread's own slots of the ring, kAhead - 1 ahead, without taking registers
// or barriers.
template <int kAhead, typename T, typename Many, typename One>
__device__ __forceinline__ void sweep_vectors(Smem& s, const T* row, int lo, int hi, Many&& many, One&& one) {
  constexpr int VE = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const T* p = row + lo;
  const int n = hi - lo;
  const int head = min(n, (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)));
  const int n_vec = (n - head) / VE;
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  uint4* ring = &s.ring[0][threadIdx.x];
  int i = threadIdx.x;
#pragma unroll
  for (int a = 0; a < kAhead - 1; ++a) {
    if (i + a * kThreads < n_vec) copy_async(ring + a * kThreads, v + i + a * kThreads);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int at = 0, put = (kAhead - 1) * kThreads;
#pragma unroll 1
  for (; i - lane < n_vec; i += kThreads) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
    // into the slot of the vector before, which has been used
    const int next = i + (kAhead - 1) * kThreads;
    if (next < n_vec) copy_async(ring + put, v + next);
    asm volatile("cp.async.commit_group;" ::: "memory");
    many(ring[at], lo + head + i * VE, i < n_vec, ring + at);
    put = at;
    at = at == (kAhead - 1) * kThreads ? 0 : at + kThreads;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  const int rest = n - head - n_vec * VE;
  if ((int)threadIdx.x < 32) {
    const bool in = lane < head + rest;
    const int j = lane < head ? lane : lane + n_vec * VE;
    one(in ? to_f(p[j]) : -INFINITY, lo + j, in);
  }
}

// Calls f(x, index) for the tokens [lo, hi) of a row.
template <typename T, typename F>
__device__ __forceinline__ void sweep(Smem& s, const T* row, int lo, int hi, F&& f) {
  sweep_vectors<kBinnedStages>(
      s, row, lo, hi,
      [&](const uint4& q, int i, bool in, const uint4*) {
        const T* e = reinterpret_cast<const T*>(&q);
        if (in) {
#pragma unroll
          for (int k = 0; k < (int)(16 / sizeof(T)); ++k) f(to_f(e[k]), i + k);
        }
      },
      [&](float x, int i, bool in) {
        if (in) f(x, i);
      });
}

// Calls f(x) for one group of 32 vectors in `every` (and for no tokens outside
// the vectors).
template <typename T, typename F>
__device__ __forceinline__ void sweep_sample(const T* row, int lo, int hi, int every, F&& f) {
  constexpr int VE = 16 / sizeof(T);
  const T* p = row + lo;
  const int n = hi - lo;
  const int head = min(n, (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T)));
  const int n_vec = (n - head) / VE;
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 1
  for (int g = threadIdx.x >> 5; g * every * 32 < n_vec; g += kThreads / 32) {
    const int i = g * every * 32 + (threadIdx.x & 31);
    if (i < n_vec) {
      const uint4 q = __ldg(v + i);
      const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int k = 0; k < VE; ++k) f(to_f(e[k]));
    }
  }
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
__device__ __forceinline__ void accumulate_bins(uint32_t* count, u64* mass, u64* red, uint32_t* red_c) {
  const int b = kBinsPer * threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t c[kBinsPer], c_all = 0;
  u64 m[kBinsPer], m_all = 0;
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) {
    c[i] = c_all += count[b + i];
    m[i] = m_all += mass[b + i];
  }
  uint32_t ci = c_all;
  u64 mi = m_all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ci, o);
    const u64 y = __shfl_up_sync(0xffffffffu, mi, o);
    if (lane >= o) {
      ci += x;
      mi += y;
    }
  }
  if (lane == 31) {
    red_c[warp] = ci;
    red[warp] = mi;
  }
  __syncthreads();
  uint32_t c0 = ci - c_all;
  u64 m0 = mi - m_all;
  for (int w = 0; w < warp; ++w) {
    c0 += red_c[w];
    m0 += red[w];
  }
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) {
    count[b + i] = c0 + c[i];
    mass[b + i] = m0 + m[i];
  }
  __syncthreads();
}

// First bin whose running count or mass reaches t; kBins - 1 if none.  (Every
// thread searches for itself: a dozen broadcast reads, no barrier.)
template <typename V>
__device__ __forceinline__ int first_bin(const V* running, V t) {
  int lo = -1, hi = kBins - 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (running[mid] >= t) hi = mid; else lo = mid;
  }
  return hi;
}

// Sorts n entries (n <= kList) of `src` ascending into s.list, by way of
// s.mass; src may be s.list.
//
// Up to kThreads / 2: two threads count the entries that precede one.  More: an
// entry's place is the number of entries in the bins before its own (from `top`
// down, `scale` to a unit of x) and of smaller ones in it; few share a
// bin, unless they are equal.
__device__ __noinline__ void sort_list(Smem& s, const u64* src, int n, float top, float scale) {
  constexpr int kPer = kList / kThreads;
  if (n <= kThreads / 2) {
    const int i = (int)threadIdx.x >> 1;
    const u64 e = i < n ? src[i] : 0;
    int before = 0;
    if (i < n)
      for (int j = threadIdx.x & 1; j < n; j += 2) before += src[j] < e;
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    __syncthreads();
    if (i < n && !(threadIdx.x & 1)) s.list[before] = e;
    __syncthreads();
    return;
  }
#pragma unroll
  for (int k = 0; k < kBinsPer; ++k) s.count[threadIdx.x + k * kThreads] = 0;
  __syncthreads();
  u64 e[kPer];
  int bin[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < n) {
      e[k] = src[i];
      bin[k] = min(kBins - 1, __float2int_rd((top - entry_x(e[k])) * scale));
      atomicAdd(s.count + bin[k], 1u);
    }
  }
  __syncthreads();
  // counts -> first places
  uint32_t c[kBinsPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kBinsPer; ++k) {
    c[k] = s.count[kBinsPer * threadIdx.x + k];
    sum += c[k];
  }
  uint32_t at = (uint32_t)block_scan(sum, s.red);
#pragma unroll
  for (int k = 0; k < kBinsPer; ++k) {
    s.count[kBinsPer * threadIdx.x + k] = at;
    at += c[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if ((int)threadIdx.x + k * kThreads < n) s.mass[atomicAdd(s.count + bin[k], 1u)] = e[k];
  __syncthreads();
  // s.count[b] is now the end of bin b
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if ((int)threadIdx.x + k * kThreads < n) {
      const int b0 = bin[k] ? (int)s.count[bin[k] - 1] : 0, b1 = (int)s.count[bin[k]];
      int place = b0;
      for (int j = b0; j < b1; ++j) place += s.mass[j] < e[k];
      s.list[place] = e[k];
    }
  }
  __syncthreads();
}

// s.list in place, with the bins laid between its largest and smallest value.
__device__ __forceinline__ void sort_list(Smem& s, int n) {
  float top = 0.f, scale = 0.f;
  if (n > kThreads / 2) {
    u64 lo = ~0ull, hi = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      lo = min(lo, s.list[i]);
      hi = max(hi, s.list[i]);
    }
    top = entry_x(block_min(lo, s.red));
    const float low = entry_x(block_max(hi, s.red));
    scale = top > low ? fminf((float)kBins / (top - low), 3e38f) : 0.f;
  }
  sort_list(s, s.list, n, top, scale);
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

constexpr u64 kAll = ~0ull;

// The cuts and the draw among the n gathered tokens, sorted in s.list (n >= 1):
// the whole head, or (binned) the tokens of the bins that the cuts lie in.
// top_k 0, top_p 1 and has_m false: no such cut.  kept: the mass where nothing
// is cut (kAll: that of the tokens); on return the kept mass, and the token.
// False when a cut lies past the tokens.
template <int kPer, bool binned>
__device__ __noinline__ bool finish_by(Smem& s, int n, int mb, uint32_t top_k, float top_p, bool has_m, float u,
                                       u64* kept, u64* token) {
  const Scale sc = s.sc;
  constexpr u64 kNone = ~0ull;
  // a thread's tokens: adjacent ones
  const int i0 = threadIdx.x * kPer;
  float x[kPer], x_next = -INFINITY;
  u64 w[kPer], g[kPer], mine = 0;
  uint32_t rank[kPer];
  int bin[kPer], bin_prev = -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const bool in = i0 + k < n;
    x[k] = in ? entry_x(s.list[i0 + k]) : -INFINITY;
    w[k] = in ? weigh(x[k], sc, s.table, s.table_f) : 0;
    mine += w[k];
    g[k] = mine;
    rank[k] = i0 + k + 1;
    bin[k] = in && binned ? bin_of(x[k], sc) : -1;
  }
  if (i0 + kPer < n) x_next = entry_x(s.list[i0 + kPer]);
  if (binned && i0 > 0 && i0 < n) bin_prev = bin_of(entry_x(s.list[i0 - 1]), sc);
  if (threadIdx.x < 5) {
    u64 v = kNone;
    if (threadIdx.x == 2) v = binned && has_m ? (mb ? s.tot_mass[mb - 1] : 0ull) : kNone;
    s.slot[threadIdx.x] = v;
  }
  const u64 before = block_scan(mine, s.red);
#pragma unroll
  for (int k = 0; k < kPer; ++k) g[k] += before;
  if (*kept == kAll) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (i0 + k == n - 1) s.slot[4] = g[k];
    __syncthreads();
    *kept = s.slot[4];
  }
  if (binned) {
    // places and masses in the whole order: by each bin's first token
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (bin[k] >= 0 && bin[k] != (k ? bin[k - 1] : bin_prev)) {
        s.count[bin[k]] = i0 + k;
        s.mass[bin[k]] = g[k] - w[k];
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (bin[k] >= 0) {
        const int b = bin[k];
        rank[k] = (b ? s.tot_count[b - 1] : 0u) + (i0 + k - s.count[b]) + 1;
        g[k] = (b ? s.tot_mass[b - 1] : 0ull) + g[k] - s.mass[b];
      }
  }
  bool ok = true;
  if (top_k) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (i0 + k < n && rank[k] == top_k) s.slot[0] = g[k];
    __syncthreads();
    ok = s.slot[0] != kNone;
    if (ok) *kept = s.slot[0];
  }
  if (top_p < 1.f || has_m) {
    const u64 t = at_least(top_p < 1.f ? top_p : 0.f, *kept);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (i0 + k < n) {
        if (top_p < 1.f && g[k] >= t && (g[k] - w[k] < t || rank[k] == 1)) s.slot[1] = g[k];
        const float xn = k + 1 < kPer ? x[k + 1 < kPer ? k + 1 : k] : x_next;
        if (has_m && (!binned || bin[k] == mb) && x[k] >= sc.x_min && !(xn >= sc.x_min)) s.slot[2] = g[k];
      }
    __syncthreads();
    if (top_p < 1.f) ok = ok && s.slot[1] != kNone;
    *kept = min(*kept, min(s.slot[1], s.slot[2]));
  }
  const u64 t = above(u, *kept);
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (i0 + k < n && g[k] >= t && g[k] - w[k] < t) s.slot[3] = s.list[i0 + k];
  __syncthreads();
  ok = ok && s.slot[3] != kNone;
  *token = s.slot[3];
  return ok;
}

template <bool binned>
__device__ __forceinline__ bool finish(Smem& s, int n, int mb, uint32_t top_k, float top_p, bool has_m, float u,
                                       u64* kept, u64* token) {
  return n <= kThreads ? finish_by<1, binned>(s, n, mb, top_k, top_p, has_m, u, kept, token)
                       : finish_by<kList / kThreads, binned>(s, n, mb, top_k, top_p, has_m, u, kept, token);
}

// Appends tokens to this CTA's list; what does not fit is only counted.
__device__ __forceinline__ void append(Smem& s, float x, int i) {
  const int at = atomicAdd(&s.n_list, 1);
  if (at < kList) s.list[at] = entry_of(x, i);
}
__device__ __forceinline__ void append_warp(Smem& s, u64 entry, bool have) {
  const unsigned m = __ballot_sync(0xffffffffu, have);
  const int lane = threadIdx.x & 31;
  int at = 0;
  if (lane == 0 && m) at = atomicAdd(&s.n_list, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
  if (have && at < kList) s.list[at] = entry;
}

// Sums and products in two floats (48 bits).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add_pair(Pair a, Pair b) {
  const float h = a.hi + b.hi, t = h - a.hi;
  const float e = (a.hi - (h - t)) + (b.hi - t) + (a.lo + b.lo);
  const float r = h + e;
  return {r, e - (r - h)};
}
__device__ __forceinline__ Pair mul_pair(Pair a, Pair b) {
  const float h = a.hi * b.hi;
  return {h, fmaf(a.hi, b.hi, -h) + (a.hi * b.lo + a.lo * b.hi)};
}

// ln m, m >= 1, to 4e-9: m = 2^e f with f in [0.7, 1.42), and ln f =
// 2 atanh(t), t = (f - 1) / (f + 1), by its series (|t| <= 0.18; past t only
// 2^-8 of the sum is left, for which fp32 is enough).
__device__ __forceinline__ Pair ln_of(u64 m) {
  int e = 63 - __clzll((long long)m);
  const u64 top = m << (63 - e);  // f in [1, 2) as top * 2^-63
  Pair f = {(float)(uint32_t)(top >> 40) * 0x1p-23f, (float)(uint32_t)((top >> 8) & 0xffffffffu) * 0x1p-55f};
  if (f.hi > 1.4142135f) {
    f.hi *= 0.5f;
    f.lo *= 0.5f;
    ++e;
  }
  const float n = f.hi - 1.f;  // exact
  const float d = f.hi + 1.f, d1 = d - f.hi, d_lost = (f.hi - (d - d1)) + (1.f - d1);
  Pair t;
  t.hi = n / d;
  t.lo = (fmaf(-t.hi, d, n) + f.lo - t.hi * (f.lo + d_lost)) / d;
  const float t2 = t.hi * t.hi;
  float p = fmaf(t2, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(t2, p, 1.f / 9.f);
  p = fmaf(t2, p, 1.f / 7.f);
  p = fmaf(t2, p, 1.f / 5.f);
  p = fmaf(t2, p, 1.f / 3.f);
  const Pair ln_f = {2.f * t.hi, 2.f * t.lo + 2.f * t.hi * t2 * p};
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr Pair ln2 = {(float)kLn2, (float)(kLn2 - (double)(float)kLn2)};
  return add_pair(mul_pair({(float)e, 0.f}, ln2), ln_f);
}

// ln of a token's share of the kept mass: (x - max) / T - ln(kept / w of max).
__device__ __forceinline__ float log_share(float x, u64 kept, const Scale& sc, const Smem& s) {
  const float d = x - sc.max, t = d - x;
  const Pair diff = {d, (x - (d - t)) + (-sc.max - t)};
  const Pair inv = {(float)s.inv_t, (float)(s.inv_t - (double)(float)s.inv_t)};
  const Pair a = ln_of(kept), b = ln_of(weigh(sc.max, sc, s.table, s.table_f));
  Pair r = add_pair(mul_pair(diff, inv), {-a.hi, -a.lo});
  r = add_pair(r, b);
  return r.hi + r.lo;
}

// Adds one token of mass w to a bin.  The mass is kept as two words in
// separate arrays (shared memory adds 32 bits at a time); join_bins makes it
// one.
__device__ __forceinline__ void add_to_bin(Smem& s, int b, u64 w) {
  uint32_t* lo = reinterpret_cast<uint32_t*>(s.mass);
  uint32_t* hi = lo + kBins;
  atomicAdd(s.count + b, 1u);
  const uint32_t wl = (uint32_t)w, old = atomicAdd(lo + b, wl);
  const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
  if (wh) atomicAdd(hi + b, wh);
}
__device__ __forceinline__ u64 bin_mass(const Smem& s, int b) {
  const uint32_t* lo = reinterpret_cast<const uint32_t*>(s.mass);
  return ((u64)lo[kBins + b] << 32) | lo[b];
}
__device__ __forceinline__ void join_bins(Smem& s) {
  u64 m[kBinsPer];
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) m[i] = bin_mass(s, threadIdx.x + i * kThreads);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) s.mass[threadIdx.x + i * kThreads] = m[i];
  __syncthreads();
}
__device__ __forceinline__ void clear_bins(Smem& s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.count[i] = 0;
    s.mass[i] = 0;
  }
}

// What sweep_row does with the tokens x >= cut.
enum Take { kAppend, kToBins, kAppendWanted, kFirstIndex };

// Sweeps the tokens [lo, hi) of a row: the mass of all of them, where asked
// for, and the tokens x >= cut to this CTA's list (all, or those of the bins
// of s.d), to its bins, or only their least index.  Returns the thread's share
// of the mass, or its least index.
//
// A warp collects the tokens x >= cut in its queue and handles them 32 at a
// time, one per lane, so that atomics and dependent arithmetic are waited for
// once for 32 of them.
template <int kAhead, Take take, bool all, typename T>
__device__ __noinline__ u64 sweep_row(Smem& s, const T* row, int lo, int hi, float cut) {
  const Scale sc = s.sc;
  const int lane = threadIdx.x & 31;
  u64* queue = s.queue[threadIdx.x >> 5];
  constexpr bool in_ranges = take == kAppendWanted;
  const Decision& d = s.d;
  float lo0 = 0.f, hi0 = 0.f, lo1 = 0.f, hi1 = 0.f;
  if (in_ranges) {
    lo0 = d.lo[0];
    hi0 = d.hi[0];
    lo1 = d.lo[1];
    hi1 = d.hi[1];
  }
  auto near = [&](float x) { return (x >= lo0 && x <= hi0) || (x >= lo1 && x <= hi1); };
  u64 sum = take == kFirstIndex ? ~0ull : 0ull;
  int waiting = 0;  // the same in every lane
  auto handle = [&](u64 e, bool have) {
    if (take == kAppend || take == kAppendWanted) {
      if (take == kAppendWanted) have = have && d.wanted(bin_of(entry_x(e), sc));
      append_warp(s, e, have);
    } else if (have) {
      if (take == kToBins) {
        const float x = entry_x(e);
        add_to_bin(s, bin_of(x, sc), weigh(x, sc, s.table, s.table_f));
      } else {
        sum = min(sum, (u64)(uint32_t)e);
      }
    }
  };
  // (once more, after the last token, for those that still wait)
  auto put = [&](float x, int i, bool in, bool last) {
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (m || last) {
      if (in) queue[waiting + __popc(m & ((1u << lane) - 1u))] = entry_of(x, i);
      waiting += __popc(m);
      if (waiting >= 32 || last) {
        __syncwarp();
        handle(queue[lane], lane < waiting);
        const u64 e = queue[32 + lane];
        __syncwarp();
        queue[lane] = e;
        waiting -= 32;
        __syncwarp();
      }
    }
  };
  constexpr int VE = 16 / sizeof(T);
  float end_x = -INFINITY;
  int end_i = 0;
  sweep_vectors<kAhead>(
      s, row, lo, hi,
      [&](const uint4& q, int i, bool in, const uint4* slot) {
        const T* e = reinterpret_cast<const T*>(&q);
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < VE; ++k) m = fmaxf(m, to_f(e[k]));
        if (all && in && m >= sc.zero) {
#pragma unroll
          for (int k = 0; k < VE; k += 2)
            sum += weigh_two(to_f(e[k]), to_f(e[k + 1]), sc, s.table, s.table_f);
        }
        bool some = in && m >= cut;
        if (in_ranges && some) {
          some = false;
#pragma unroll
          for (int k = 0; k < VE; ++k) some = some || near(to_f(e[k]));
        }
        if (__any_sync(0xffffffffu, some)) {
#pragma unroll 1
          for (int k = 0; k < VE; ++k) {
            const float x = to_f(reinterpret_cast<const T*>(slot)[k]);
            put(x, i + k, in && x >= cut && (!in_ranges || near(x)), false);
          }
        }
      },
      [&](float x, int i, bool in) {
        if (all && in) sum += weigh(x, sc, s.table, s.table_f);
        end_x = x;
        end_i = i;
      });
  // the ends (the first warp's), and what waits: at most 31 and 32
#pragma unroll 1
  for (int k = 0; k < 2; ++k) put(end_x, end_i, k == 0 && end_x >= cut && end_x > -INFINITY, k == 1);
  return sum;
}

// The cut of the order inside bin `b` of the head (any number of tokens): the
// first token whose rank (1, 2, ...) reaches `rank`, or, where rank is 0, whose
// running mass reaches `target`.  *mass: the running mass with it; *entry: the
// token.  One CTA does it, over the whole row, where too many tokens share the
// cuts' bins to be gathered at once: the bin's keys are cut into kBins ranges
// again and again until the cut's range is short, or a single value, whose
// tokens are told apart by index.
template <typename T>
__device__ __noinline__ void find_in_bin(Smem& s, const T* row, int vocab, const Scale& sc, int b, uint32_t c_before,
                                         u64 m_before, uint32_t rank, u64 target, u64* mass, u64* entry) {
  auto past = [&](uint32_t c, u64 m) { return rank ? c >= rank : m >= target; };
  uint32_t lo = 0, hi = 0xffffffffu;
  for (;;) {
    uint32_t kmin = 0xffffffffu, kmax = 0, n = 0;
    sweep(s, row, 0, vocab, [&](float x, int) {
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
      // the t-th of n equal tokens, 1 <= t <= n
      const float x = of_key(kmin);
      const u64 w = weigh(x, sc, s.table, s.table_f);
      u64 t = 1;
      if (rank)
        t = rank - c_before;
      else if (w && target > m_before)
        t = (target - m_before + w - 1) / w;
      t = max(1ull, min((u64)n, t));
      *mass = m_before + t * w;
      // its index: each thread counts the equals of one stretch of the row
      const int per = (vocab + kThreads - 1) / kThreads;
      const int i0 = min(vocab, (int)threadIdx.x * per), i1 = min(vocab, i0 + per);
      int mine = 0;
      for (int i = i0; i < i1; ++i) mine += key_of(to_f(row[i])) == kmin;
      int64_t left = (int64_t)t - (int64_t)block_scan(mine, s.red);
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
      sweep(s, row, 0, vocab, [&](float x, int i) {
        const uint32_t k = key_of(x);
        if (x >= sc.cut && k >= lo && k <= hi && bin_of(x, sc) == b) append(s, x, i);
      });
      __syncthreads();
      sort_list(s, (int)n);
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
    // kBins ranges of the keys kmax .. kmin, descending
    const int shift = max(0, 32 - __clz(kmax - kmin) - kBinBits);
    clear_bins(s);
    __syncthreads();
    sweep(s, row, 0, vocab, [&](float x, int) {
      const uint32_t k = key_of(x);
      if (x >= sc.cut && k >= kmin && k <= kmax && bin_of(x, sc) == b)
        add_to_bin(s, (int)((kmax - k) >> shift), weigh(x, sc, s.table, s.table_f));
    });
    __syncthreads();
    join_bins(s);
    accumulate_bins(s.count, s.mass, s.red, s.red_c);
    const int at = rank ? first_bin(s.count, rank - c_before)
                        : first_bin(s.mass, target > m_before ? target - m_before : 0ull);
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int c_size = (int)cluster.num_blocks(), c_rank = (int)cluster.block_rank();
  const int r = blockIdx.x / c_size;
  Smem& s0 = *cluster.map_shared_rank(&s, 0);
  if (tid < 64) {
    s.table[tid] = p.table[tid] - ((uint32_t)__float_as_int(kMagic) << 2);
    s.table_f[tid] = (float)p.table[tid] * 0.25f;
  }
  for (int i = tid; i < kCoarse; i += kThreads) s.coarse[i] = 0;
  // shared memory of a CTA may be written by another once all have started
  cg::cluster_group::arrival_token started = cluster.barrier_arrive();
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

  const bool want_k = top_k > 0 && top_k < p.vocab, has_p = top_p < 1.f, want_m = min_p > 0.f;
  const bool m_only = want_m && !want_k && !has_p;  // the head is what min_p keeps
  const bool need_all = !want_k && !m_only;         // the mass of every token
  // top-k: the tokens that this CTA should gather, with the others four
  // deviations more than top_k; unless they are too many, or too many for
  // groups' maxima to tell (share * (1 + 0.7 share / kGroups) tokens lie above
  // the maximum that `share` groups reach)
  constexpr int VE = 16 / sizeof(T);
  constexpr float kGroups = kThreads * VE;
  float share = (float)top_k / (float)c_size;
  if (c_size > 1) share = fminf((float)top_k, share + 4.f * sqrtf(share) + 8.f);
  const bool by_groups = want_k && share * (float)c_size * (1.f + 0.7f * share / kGroups) <= (float)kDirect &&
                         share < 0.6f * kGroups;
  const bool by_sample = !by_groups && !m_only;

  // ---- 1. the groups' maxima, and whether anything is wrong ----
  if (tid == kThreads - 1) prepare_scale(s, temp, min_p);
  float top[VE];  // of this thread's tokens, by their place in a vector
#pragma unroll
  for (int k = 0; k < VE; ++k) top[k] = -INFINITY;
  float cta_max;
  {
    float ends = -INFINITY;
    sweep_vectors<kStages>(
        s, row, lo_i, hi_i,
        [&](const uint4& q, int, bool in, const uint4*) {
          const T* e = reinterpret_cast<const T*>(&q);
          if (in) {
#pragma unroll
            for (int k = 0; k < VE; ++k) top[k] = max_nan(top[k], to_f(e[k]));
          }
        },
        [&](float x, int, bool in) {
          if (in) ends = x;
        });
    float mx = ends;
#pragma unroll
    for (int k = 0; k < VE; ++k) mx = max_nan(mx, top[k]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float* red = reinterpret_cast<float*>(s.red);
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    cta_max = red[tid & (kThreads / 32 - 1)];
#pragma unroll
    for (int o = kThreads / 64; o; o >>= 1) cta_max = max_nan(cta_max, __shfl_xor_sync(0xffffffffu, cta_max, o));
    cluster.barrier_wait(std::move(started));
    if (tid < c_size) cluster.map_shared_rank(&s, tid)->max[c_rank] = cta_max;  // to every CTA
  }
  const float per = 4.f / 64.f * s.inv_c;  // quarter octaves of w to a unit of x
  if (by_sample) {
    sweep_sample(row, lo_i, hi_i, p.sample_every, [&](float x) {
      const float y = (cta_max - x) * per;
      if (y >= 0.f && y < (float)kCoarse) atomicAdd(s.coarse + (int)y, 1u);
    });
    for (int i = tid; i < kCoarse; i += kThreads) s.coarse_all[i] = 0;
  }
  cg::cluster_group::arrival_token arrived = cluster.barrier_arrive();
  // the value that about `share` of this CTA's tokens exceed: the groups'
  // maxima counted by eighths of an octave
  if (by_groups) {
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      const float y = (cta_max - top[k]) * (2.f * per);
      if (y >= 0.f && y < (float)kCoarse) atomicAdd(s.coarse + (int)y, 1u);
    }
    __syncthreads();
    if (tid < 32) {
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += n[i] = s.coarse[tid * 8 + i];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += a;
      }
      uint32_t c = incl - sum;
      int b = kCoarse;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c += n[i];
        if (b == kCoarse && (float)c >= share) b = tid * 8 + i + 1;
      }
      b = __reduce_min_sync(0xffffffffu, b);
      if (tid == 0) s.found[0] = b;
    }
  }
  cluster.barrier_wait(std::move(arrived));
  __syncthreads();
  float row_max = s.max[0];
  for (int c = 1; c < c_size; ++c) row_max = max_nan(row_max, s.max[c]);
  const bool bad = !(row_max > -INFINITY && row_max < INFINITY) ||
                   !(temp == 0.f || (temp >= 0x1p-100f && temp <= 0x1p60f)) || !(top_p >= 0.f) ||
                   !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
  if (bad || temp == 0.f) {
    // the maximum's first index
    if (!bad) {
      int first = (int)min((u64)p.vocab, sweep_row<kStages, kFirstIndex, false>(s, row, lo_i, hi_i, row_max));
      first = (int)block_min((u64)first, s.red);
      if (tid == 0) s0.x_index[c_rank] = first;
    }
    cluster.sync();
    if (c_rank == 0 && tid == 0) {
      int id = -1;
      if (!bad) {
        id = s.x_index[0];
        for (int c = 1; c < c_size; ++c) id = min(id, s.x_index[c]);
      }
      p.ids[r] = id;
      if (p.logprob) p.logprob[r] = bad ? -INFINITY : 0.f;
      if (bad) report(p.status, STV_DEV_BAD_SAMPLE);
    }
    return;
  }
  Scale sc = make_scale(s, row_max, min_p);
  const float x_min = sc.x_min;
  // ---- how far down the cuts lie ----
  bool direct = true;
  if (by_groups) {
    const int b = s.found[0];
    set_cut(sc, b < kCoarse ? cta_max - (float)b / (2.f * per) : sc.floor);
  } else if (m_only) {
    set_cut(sc, x_min);
  } else {
    // the CTAs' samples, counted from their own maxima, as the row's
    for (int i = tid; i < c_size * kCoarse; i += kThreads) {
      const int c = i / kCoarse, k = i % kCoarse;
      const uint32_t n = cluster.map_shared_rank(&s, c)->coarse[k];
      const float g = (float)k + (sc.max - s.max[c]) * per;
      if (n && g < (float)(kCoarse - 8)) atomicAdd(s.coarse_all + (int)g, n);
    }
    __syncthreads();
    const float f = (float)p.sample_every;
    if (tid < 32) {  // a warp: lane l holds eight bins
      float cnt[8], wgt[8], c8 = 0.f, w8 = 0.f, sure = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cnt[i] = (float)s.coarse_all[tid * 8 + i];
        const float w = exp2f(-0.25f * (float)(tid * 8 + i));
        wgt[i] = f * cnt[i] * w;
        c8 += cnt[i];
        w8 += wgt[i];
        // surely there: two deviations under the sample's count
        sure += fmaxf(cnt[i], f * (cnt[i] - 2.f * sqrtf(cnt[i]))) * w;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sure += __shfl_xor_sync(0xffffffffu, sure, o);
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
      // tail of under 0.7 of what the cut leaves out of the mass that is surely
      // there, the maximum's 1 with it, below a head of so many tokens that the
      // sample knows what lies beneath
      const float k_need = (float)top_k / f;
      const float enough = p.sample_every > 1 ? k_need + 4.f * sqrtf(k_need) + 8.f : k_need;
      const float left = has_p ? 1.f - top_p : 1.f - u;
      const float tail = 0.7f * left * (1.f + sure);
      int b = kCoarse;
      float c = c_incl - c8, w = w_incl - w8, n_head = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // the bins up to this one are enough
        c += cnt[i];
        w += wgt[i];
        const int past = tid * 8 + i + 1;
        if (b == kCoarse && (want_k ? c >= enough : w_all - w <= tail && c * f >= kLeastHead)) {
          b = past;
          n_head = c * f;
        }
      }
      const unsigned any = __ballot_sync(0xffffffffu, b < kCoarse);
      const int src = any ? __ffs(any) - 1 : 31;
      b = __shfl_sync(0xffffffffu, b, src);
      n_head = __shfl_sync(0xffffffffu, any ? n_head : c_incl * f, src);
      if (tid == 0) {
        s.found[0] = b;
        s.found[1] = n_head <= (float)kDirect;
      }
    }
    __syncthreads();
    const int b = s.found[0];
    direct = s.found[1];
    set_cut(sc, b < kCoarse - 8 ? sc.max - (float)b / per : sc.floor);
  }

  u64 total = 0;  // first CTA: the row's mass, where need_all
  u64 kept = 0, token = 0;
  for (int round = 0;; ++round) {
    if (round) {  // a cut lies further down: every token that has any mass
      set_cut(sc, sc.floor);
      direct = false;
    }
    bool complete = sc.cut <= sc.floor;  // the head is every token with any mass
    // ---- 2. the mass of all, the head's tokens or bins ----
    const bool binned = !direct;
    if (binned) clear_bins(s);
    if (tid == 0) {
      s.n_list = 0;
      s.sc = sc;
    }
    __syncthreads();
    {
      const bool all = need_all && round == 0;
      u64 sum = all ? (binned ? sweep_row<kStages, kToBins, true>(s, row, lo_i, hi_i, sc.cut)
                              : sweep_row<kStages, kAppend, true>(s, row, lo_i, hi_i, sc.cut))
                    : (binned ? sweep_row<kStages, kToBins, false>(s, row, lo_i, hi_i, sc.cut)
                              : sweep_row<kStages, kAppend, false>(s, row, lo_i, hi_i, sc.cut));
      if (all) {
        sum = block_sum(sum, s.red);
        if (tid == 0) s0.part[c_rank] = sum;
      } else {
        __syncthreads();
      }
    }
    if (tid == 0) {
      s0.n_lists[c_rank] = s.n_list;
      s0.cut[c_rank] = sc.cut;
    }
    cluster.sync();
    if (binned) {
      // each CTA adds up a share of the bins, for the first one
      const int per = kBins / c_size;
      for (int i = c_rank * per + tid; i < (c_rank + 1) * per; i += kThreads) {
        uint32_t c = 0;
        u64 m = 0;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < c_size) {
            const Smem* o = cluster.map_shared_rank(&s, k);
            c += o->count[i];
            m += bin_mass(*o, i);
          }
        s0.tot_count[i] = c;
        s0.tot_mass[i] = m;
      }
      cluster.sync();
    }
    auto c_before = [&](int b) { return b ? s.tot_count[b - 1] : 0u; };
    auto m_before = [&](int b) { return b ? s.tot_mass[b - 1] : 0ull; };
    // entry i of the CTAs' lists, one after the other
    auto entry = [&](int i) {
      int c = 0;
      while (i >= s.n_lists[c]) i -= s.n_lists[c++];
      return cluster.map_shared_rank(&s, c)->list[i];
    };
    Decision d;
    d.done = kTooShort;
    d.kb = d.mb = -1;
    d.pb1 = d.ub1 = 0;
    d.pb2 = d.ub2 = -1;
    bool has_m = want_m && x_min >= sc.cut;
    if (c_rank == 0) {
      if (need_all && round == 0)
        for (int c = 0; c < c_size; ++c) total += s.part[c];
      if (!binned) {
        int m = 0;
        float least = sc.cut;
        bool fits = true;
        for (int c = 0; c < c_size; ++c) {
          m += s.n_lists[c];
          fits = fits && s.n_lists[c] <= kList;
          least = fmaxf(least, s.cut[c]);  // above the largest cut every CTA has all its tokens
        }
        if (fits) {
          if (tid == 0) s.n_list = 0;
          __syncthreads();
          for (int i = tid; i - (tid & 31) < m; i += kThreads) {
            const u64 e = i < m ? entry(i) : 0ull;
            const bool in = i < m && entry_x(e) >= least;
            const unsigned mask = __ballot_sync(0xffffffffu, in);
            int at = 0;
            if ((tid & 31) == 0 && mask) at = atomicAdd(&s.n_list, __popc(mask));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << (tid & 31)) - 1u));
            if (in && at < kList) s.tot_mass[at] = e;
          }
          __syncthreads();
          const int n = s.n_list;
          if (n >= 1 && n <= kList) {
            set_cut(sc, least);
            if (tid == 0) s.sc = sc;
            complete = sc.cut <= sc.floor;
            has_m = want_m && x_min >= sc.cut;
            sort_list(s, s.tot_mass, n, sc.max, sc.bin_scale);
            // all of a complete head may be fewer than top_k
            const uint32_t k = want_k && !(complete && n < top_k) ? (uint32_t)top_k : 0u;
            kept = need_all ? total : kAll;
            if (finish<false>(s, n, 0, k, top_p, has_m, u, &kept, &token)) d.done = kDone;
          }
        }
      } else {
        accumulate_bins(s.tot_count, s.tot_mass, s.red, s.red_c);
        const uint32_t n_head = s.tot_count[kBins - 1];
        const u64 head = s.tot_mass[kBins - 1];
        const bool has_k = want_k && !(complete && n_head < (uint32_t)top_k);
        bool ok = !has_k || n_head >= (uint32_t)top_k;
        // a cut's mass lies between the mass before its first bin and with its last
        u64 lo = need_all ? total : head, hi = lo;
        if (has_k) {
          d.kb = first_bin(s.tot_count, (uint32_t)top_k);
          lo = m_before(d.kb);
          hi = s.tot_mass[d.kb];
        }
        if (has_p) {
          const u64 t = at_least(top_p, hi);
          ok = ok && head >= t;
          d.pb1 = first_bin(s.tot_mass, at_least(top_p, lo));
          d.pb2 = has_k ? first_bin(s.tot_mass, t) : d.pb1;
          lo = min(lo, m_before(d.pb1));
          hi = min(hi, s.tot_mass[d.pb2]);
        }
        if (has_m) {
          d.mb = x_min <= sc.max ? bin_of(x_min, sc) : 0;
          lo = min(lo, m_before(d.mb));
          hi = min(hi, s.tot_mass[d.mb]);
        }
        const u64 t = above(u, hi);
        ok = ok && head >= t;
        d.ub1 = first_bin(s.tot_mass, above(u, lo));
        d.ub2 = lo < hi ? first_bin(s.tot_mass, t) : d.ub1;
        // the tokens of those bins, counted once
        uint32_t n = 0;
        {
          int a[4] = {d.kb, has_p ? d.pb1 : -1, d.mb, d.ub1}, b[4] = {d.kb, d.pb2, d.mb, d.ub2};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int from = a[i], to = b[i];
#pragma unroll
            for (int j = 0; j < i; ++j) {  // less the bins of the ranges before
              if (a[j] < 0 || a[j] > to || b[j] < from) continue;
              if (a[j] <= from) from = b[j] + 1; else if (b[j] >= to) to = a[j] - 1;
            }
            if (from >= 0 && from <= to) n += s.tot_count[to] - c_before(from);
          }
        }
        if (ok || complete) d.done = kGather;
        {
          // x of a bin lies within its bounds widened by the rounding of (max - x) bin_scale
          auto high = [&](int b) { return b > 0 ? sc.max - (float)b / sc.bin_scale * 0.99999f : sc.max; };
          auto low = [&](int b) { return fmaxf(sc.cut, sc.max - (float)(b + 1) / sc.bin_scale * 1.00001f); };
          int b1 = kBins, b2 = -1;
          if (d.kb >= 0) b1 = min(b1, d.kb), b2 = max(b2, d.kb);
          if (has_p) b1 = min(b1, d.pb1), b2 = max(b2, d.pb2);
          if (d.mb >= 0) b1 = min(b1, d.mb), b2 = max(b2, d.mb);
          d.lo[0] = b2 >= 0 ? low(b2) : INFINITY;
          d.hi[0] = b2 >= 0 ? high(b1) : -INFINITY;
          d.lo[1] = low(d.ub2);
          d.hi[1] = high(d.ub1);
        }
        if (d.done == kGather && n > kList) {
          // ---- one cut after the other, without the other CTAs ----
          kept = need_all ? total : head;
          if (has_k)
            find_in_bin(s, row, p.vocab, sc, d.kb, c_before(d.kb), m_before(d.kb), (uint32_t)top_k, 0, &kept,
                        &token);
          if (has_p) {
            const u64 tp = at_least(top_p, kept);
            const int b = first_bin(s.tot_mass, tp);
            u64 m;
            find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), 0, tp, &m, &token);
            kept = min(kept, m);
          }
          if (has_m) {
            u64 w = 0;
            sweep(s, row, 0, p.vocab, [&](float x, int) {
              if (x >= x_min) w += weigh(x, sc, s.table, s.table_f);
            });
            kept = min(kept, block_sum(w, s.red));
          }
          const u64 tu = above(u, kept);
          const int b = first_bin(s.tot_mass, tu);
          u64 m;
          find_in_bin(s, row, p.vocab, sc, b, c_before(b), m_before(b), 0, tu, &m, &token);
          d.done = kDone;
        }
      }
      if (tid < c_size) cluster.map_shared_rank(&s, tid)->d = d;
    }
    cluster.sync();
    d = s.d;
    if (d.done == kTooShort) continue;
    if (d.done == kDone) break;
    // ---- 3. the tokens of the cuts' bins ----
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    sweep_row<kBinnedStages, kAppendWanted, false>(s, row, lo_i, hi_i, sc.cut);
    __syncthreads();
    if (tid == 0) s0.n_lists[c_rank] = s.n_list;
    cluster.sync();
    if (c_rank == 0) {
      int n = 0;  // at most kList, as counted above
      for (int c = 0; c < c_size; ++c) n += s.n_lists[c];
      for (int i = s.n_lists[0] + tid; i < n; i += kThreads) s.list[i] = entry(i);
      __syncthreads();
      sort_list(s, n);
      kept = need_all ? total : s.tot_mass[kBins - 1];
      if (n > 0) finish<true>(s, n, d.mb, d.kb >= 0 ? (uint32_t)top_k : 0u, top_p, has_m, u, &kept, &token);
    }
    cluster.sync();  // no CTA ends while the first one reads its list
    break;
  }
  if (c_rank == 0 && tid == 0) {
    p.ids[r] = (int32_t)(uint32_t)token;
    if (p.logprob) p.logprob[r] = log_share(entry_x(token), kept, sc, s);
  }
}
