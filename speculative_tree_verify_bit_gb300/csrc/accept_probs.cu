// accept_probs.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers, on a token tree (include/stv.h,
// stv_tree_accept_probs).
//
// A cluster of CTAs takes one sequence.  Each CTA gathers, for every node i at
// once, the target's and the draft's probability of i's token at i's parent:
// the walk down the tree then needs no memory as long as drafts are accepted.
// A rejection changes the node's whole row, R <- max(R - Z S, 0), and needs Z =
// sum R: one pass over the vocabulary, split over the cluster's warps.  Since
// max(max(p - a, 0) - b, 0) = max(p - a - b, 0), the row after any number of
// rejections is max(p - F q, 0) with one factor F, the sum of Z / sum S over
// them: R is not stored, and a pass costs the same however many there were.
// Tokens taken out of S (distinct) or of R (certain) are few and are put right
// apart; without draft rows one pass per node gives every Z.  The last token
// comes from the same sums, kept per warp: the CTA whose range holds it reads one
// warp's share again with all its threads.
//
// R, Z and the running sums are integers in units of 2^-60, so nothing depends on
// the order of threads.  A number becomes one in three steps of fp32 additions
// (x + 2 leaves the first 22 bits in the sum's last places, and so on), whose bits
// are added up in 32-bit registers: conversions to 64-bit integers run at the rate
// of the fp64 units, 2 a clock and SM.  F q is a product of fp32 pairs, off by less than
// 2^-46 of itself.  The sums saturate at 4 instead of wrapping: rows of more mass
// than that are refused.  Every CTA takes every decision from the same numbers.
//
// Bounds: the launch, two dependent loads, a pass, two cluster barriers and the
// second reading, one after the other, for few sequences (one chain over 248,320
// fp32 tokens 7.1 us; 8 trees of 16 nodes in bf16 37 us, at most six rejections at a
// node, 12,000 cycles each: the pass 6,000, barriers 2,000, the walk's own steps
// 3,500).  For many, that chain and the bytes one after the other, since all clusters
// run in step (64 chains without draft rows 17.6 us; their 64 MB take 9.4 at the copy
// bandwidth, and DRAM is busy 36 % of the time).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>
#include <utility>

#include "stv_device.cuh"

namespace stv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 524288;
constexpr uint64_t kFull = 1ull << 62;  // 4 in units of 2^-60
enum Drafts { kReplaced = 0, kDistinct = 1, kCertain = 2 };

struct AcceptParams {
  const int32_t* parent;
  const int32_t* ids;
  const void* p;
  const void* q;
  int64_t p_stride, q_stride;
  const float* u;
  int vocab, T;
  int32_t* n_commit;
  int32_t* path;
  int32_t* out_ids;
  int32_t* status;
};

// What a node's rejected children did to its row: max(p - F q, 0), F = f.x + f.y,
// but for the tokens taken out, whose R is kept here.
struct Rest {
  float2 f;
  int n_gone;
  int gone[kMaxT];
  float gone_p[kMaxT], gone_q[kMaxT];
  uint64_t gone_r[kMaxT];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ bool is_prob(float x) { return x >= 0.f && x <= 1.f; }
__device__ __forceinline__ uint64_t sat_add(uint64_t a, uint64_t b) { return min(a + b, kFull); }

// A number in [0, 2) as h 2^-22 + l 2^-44 + s 2^-60, rounded to 2^-60; sums and
// differences of a few of them stay in 32 bits.
struct Parts {
  int h, l, s;
};
__device__ __forceinline__ Parts parts_of(float x) {
  const float t = __fadd_rn(x, 2.f), r = __fsub_rn(x, __fsub_rn(t, 2.f));          // r exact, at most 2^-23
  const float t2 = __fmaf_rn(r, 4194304.f, 3.f);                                   // 2^22 r
  const float r2 = __fmaf_rn(__fsub_rn(t2, 3.f), -2.384185791015625e-7f, r);       // exact, at most 2^-45
  const float t3 = __fmaf_rn(r2, 274877906944.f, 3.f);                             // 2^38 r2
  return {__float_as_int(t) - 0x40000000, __float_as_int(t2) - 0x40400000, __float_as_int(t3) - 0x40400000};
}
__device__ __forceinline__ uint64_t whole(const Parts& x) {
  return (uint64_t)(((long long)x.h << 38) + ((long long)x.l << 16) + x.s);
}
__device__ __forceinline__ uint64_t fixed(float x) { return whole(parts_of(x)); }
// The same of a number of at most 2^-22, without h.
__device__ __forceinline__ Parts small_parts_of(float x) {
  const float t2 = __fmaf_rn(x, 4194304.f, 3.f);
  const float r2 = __fmaf_rn(__fsub_rn(t2, 3.f), -2.384185791015625e-7f, x);
  const float t3 = __fmaf_rn(r2, 274877906944.f, 3.f);
  return {0, __float_as_int(t2) - 0x40400000, __float_as_int(t3) - 0x40400000};
}

// a += max(p - F q, 0).  F q = x + w with w at most 2^-23 x; where p >= x, p - x = d + e
// exactly; d + e - w has the sign of (p - x) - w, since d is exact where w matters.
// (Each operation here is rounded by itself, and as add_above2 rounds it: the last
// token is looked for among the same numbers as a pass has added up, so the running
// sums end where the mass does.)
template <bool kOneF>
__device__ __forceinline__ void add_above(Parts& a, float p, float q, float2 f) {
  const float x = kOneF ? q : __fmul_rn(q, f.x);
  const float d = __fsub_rn(p, x);
  float e = __fsub_rn(__fsub_rn(p, d), x), w = 0.f;
  if constexpr (!kOneF) {
    w = __fmaf_rn(q, f.y, __fmaf_rn(q, f.x, -x));
    e = __fsub_rn(e, w);
  }
  const Parts y = parts_of(d), z = small_parts_of(e);
  if (d > w) {
    a.h += y.h;
    a.l += y.l + z.l;
    a.s += y.s + z.s;
  }
}
__device__ __forceinline__ uint64_t rest_of(float p, float q, float2 f) {
  if (f.x == 0.f) return fixed(p);
  Parts a = {0, 0, 0};
  if (f.x == 1.f && f.y == 0.f) add_above<true>(a, p, q, f);
  else add_above<false>(a, p, q, f);
  return whole(a);
}
// The walk's own arithmetic, one thread's, in pairs of floats (x + y, y at most
// half a place of x): about 2^-46, at a few cycles an operation where an fp64 one
// takes a hundred.  A product that goes on into a sum has to be rounded first, which
// the compiler is free not to do with * and +.
__device__ __forceinline__ float2 pair_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return make_float2(s, __fsub_rn(b, __fsub_rn(s, a)));
}
__device__ __forceinline__ float2 pair_of(uint64_t x) {  // of x units
  if (x == 0) return make_float2(0.f, 0.f);
  const int s = __clzll((long long)x);
  x <<= s;
  const uint32_t top = (uint32_t)(x >> 40), rest = (uint32_t)(x >> 8);  // 24 bits, the next 32
  const float unit = __int_as_float((127 - 36 + 16 - s) << 23);       // 2^(64 - 24 - 60 - s)
  return pair_sum(__fmul_rn((float)top, unit), __fmul_rn(__fmul_rn((float)rest, 2.3283064365386963e-10f), unit));
}
__device__ __forceinline__ float2 operator*(float2 a, float2 b) {
  const float x = __fmul_rn(a.x, b.x);
  return pair_sum(x, __fadd_rn(__fmaf_rn(a.x, b.x, -x), __fmaf_rn(a.x, b.y, __fmul_rn(a.y, b.x))));
}
__device__ __forceinline__ float2 operator/(float2 a, float2 b) {  // b > 0
  const float r = 1.f / b.x, q = __fmul_rn(a.x, r);
  const float2 back = b * make_float2(q, 0.f);
  return pair_sum(q, __fmul_rn(__fadd_rn(__fsub_rn(a.x, back.x), __fsub_rn(a.y, back.y)), r));
}
__device__ __forceinline__ float2 operator+(float2 a, float2 b) {  // both at least 0
  const bool swap = b.x > a.x;
  const float2 s = pair_sum(swap ? b.x : a.x, swap ? a.x : b.x);
  return pair_sum(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}
__device__ __forceinline__ bool operator<(float2 a, float2 b) { return a.x < b.x || (a.x == b.x && a.y < b.y); }

// VE entries of a row from entry e on, as they lie; zeros outside [0, vocab).
template <typename T>
__device__ __forceinline__ uint4 load_entries(const T* row, int e, int vocab, bool wide) {
  constexpr int VE = 16 / (int)sizeof(T);
  if (wide && e >= 0 && e + VE <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + e));
  uint4 v = make_uint4(0, 0, 0, 0);
  T* t = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < VE; ++i)
    if (e + i >= 0 && e + i < vocab) t[i] = row[e + i];
  return v;
}
template <typename T>
__device__ __forceinline__ float entry(const uint4& v, int i) {
  return to_f(reinterpret_cast<const T*>(&v)[i]);
}
// Entries i and i + 1, i even.
template <typename T>
__device__ __forceinline__ float2 entries(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
  else if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
  else return make_float2(__uint_as_float(w[i / 2] << 16), __uint_as_float(w[i / 2] & 0xffff0000u));
}
// The largest of the bit patterns so far; whether one is above 1's (or negative).
template <typename T>
__device__ __forceinline__ uint32_t most_of(uint32_t most, const uint4& v) {
  if constexpr (sizeof(T) == 4) return max(max(most, max(v.x, v.y)), max(v.z, v.w));
  else return __vmaxu2(__vmaxu2(most, __vmaxu2(v.x, v.y)), __vmaxu2(v.z, v.w));
}
template <typename T>
__device__ __forceinline__ bool above_one(uint32_t most) {
  if constexpr (sizeof(T) == 4) return most > 0x3f800000u;
  constexpr uint32_t one = std::is_same<T, __half>::value ? 0x3c00u : 0x3f80u;
  return (most & 0xffffu) > one || (most >> 16) > one;
}

// Sums of parts, two numbers an instruction (paired fp32): the bits of the sums as
// they are, their constants taken off at the end.  The steps are parts_of's and
// add_above's, so that each number counts as it does there.
struct Sums {
  uint32_t h = 0, l = 0, s = 0;
  __device__ __forceinline__ void low(float2 r) {
    const float2 three = make_float2(3.f, 3.f);
    const float2 t2 = __ffma2_rn(r, make_float2(4194304.f, 4194304.f), three);
    const float2 r2 = __ffma2_rn(__fadd2_rn(t2, make_float2(-3.f, -3.f)),
                                 make_float2(-2.384185791015625e-7f, -2.384185791015625e-7f), r);
    const float2 t3 = __ffma2_rn(r2, make_float2(274877906944.f, 274877906944.f), three);
    l += __float_as_uint(t2.x) + __float_as_uint(t2.y);
    s += __float_as_uint(t3.x) + __float_as_uint(t3.y);
  }
  __device__ __forceinline__ void add(float2 x) {
    const float2 t = __fadd2_rn(x, make_float2(2.f, 2.f)), u = __fadd2_rn(t, make_float2(-2.f, -2.f));
    h += __float_as_uint(t.x) + __float_as_uint(t.y);
    low(__ffma2_rn(u, make_float2(-1.f, -1.f), x));
  }
  // of n numbers, m of them (n, or with their errors 2 n) with low parts
  __device__ __forceinline__ uint64_t whole_of(int n, int m) const {
    return whole(Parts{(int)(h - (uint32_t)n * 0x40000000u), (int)(l - (uint32_t)m * 0x40400000u),
                       (int)(s - (uint32_t)m * 0x40400000u)});
  }
};
template <bool kOneF>
__device__ __forceinline__ void add_above2(Sums& a, float2 p, float2 q, float2 f) {
  const float2 neg = make_float2(-1.f, -1.f);
  const float2 x = kOneF ? q : __fmul2_rn(q, make_float2(f.x, f.x));
  float2 d = __ffma2_rn(x, neg, p), e = __ffma2_rn(x, neg, __ffma2_rn(d, neg, p)), w = make_float2(0.f, 0.f);
  if constexpr (!kOneF) {
    w = __ffma2_rn(q, make_float2(f.y, f.y), __ffma2_rn(q, make_float2(f.x, f.x), __fmul2_rn(x, neg)));
    e = __ffma2_rn(w, neg, e);
  }
  const bool kx = d.x > w.x, ky = d.y > w.y;
  a.add(make_float2(kx ? d.x : 0.f, ky ? d.y : 0.f));
  a.low(make_float2(kx ? e.x : 0.f, ky ? e.y : 0.f));
}

struct Share {
  uint64_t sum, draft;  // of R, of q
  int bad;
};

template <typename T, int kDrafts>
__global__ void __launch_bounds__(kThreads, kDrafts == kCertain ? 2 : 1) accept_probs_kernel(const __grid_constant__ AcceptParams p) {
  constexpr int VE = 16 / (int)sizeof(T);
  __shared__ int id[kMaxT], way[kMaxT];
  // nodes' children; nodes with good numbers; taken, if nothing was rejected before
  __shared__ uint32_t kids[kMaxT], fine, taken;
  __shared__ float uu[kMaxT], pp[kMaxT], qq[kMaxT];
  __shared__ Rest st;
  __shared__ uint64_t warp_sum[kWarps], warp_draft[kWarps];
  __shared__ int warp_bad[kWarps];
  __shared__ Share share[2][kMaxCluster];
  __shared__ int cmd, node, bad_bits;
  __shared__ uint64_t scan_sum[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  auto started = cluster.barrier_arrive();  // waited for before the first store to another CTA
  const int s = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int V = p.vocab, T_ = p.T;
  grid_dep_wait();
  grid_dep_launch();
  const T* p_rows = static_cast<const T*>(p.p) + (int64_t)s * T_ * p.p_stride;
  const T* q_rows = kDrafts == kCertain ? nullptr : static_cast<const T*>(p.q) + (int64_t)s * T_ * p.q_stride;

  if (tid < 32) {
    const bool act = tid < T_;
    const int64_t at = (int64_t)s * T_ + tid;
    const int pa = act ? __ldg(p.parent + at) : -1, x = act ? __ldg(p.ids + at) : -1;
    const float u = act ? __ldg(p.u + at) : 0.f;
    const bool bad = act && (tid == 0 ? pa != -1 : (pa < 0 || pa >= tid));
    const int any = __any_sync(0xffffffffu, bad);
    const bool there = act && tid > 0 && !any && x >= 0 && x < V;
    const float px = there ? to_f(p_rows[pa * p.p_stride + x]) : 0.f;
    float qx = 1.f;
    if constexpr (kDrafts != kCertain) qx = there ? to_f(q_rows[pa * p.q_stride + x]) : 0.f;
    id[tid] = x;
    uu[tid] = u;
    pp[tid] = px;
    qq[tid] = qx;
    kids[tid] = 0;
    __syncwarp();
    const uint32_t with = __match_any_sync(0xffffffffu, there ? pa : -1);
    if (there && lane == __ffs(with) - 1) kids[pa] = with;
    const uint32_t good = __ballot_sync(0xffffffffu, is_prob(px) && is_prob(qx) && u >= 0.f && u < 1.f);
    // u q < p, exactly, however small: two 24-bit numbers make one of 48
    const uint32_t take = __ballot_sync(0xffffffffu, (double)u * (double)qx < (double)px);
    if (tid == 0) {
      bad_bits = any ? STV_DEV_BAD_TREE : 0;
      st.f = make_float2(0.f, 0.f);
      st.n_gone = 0;
      node = 0;
      fine = good;
      taken = take;
    }
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));

  // Thread 0's place in the walk.  todo: the node's children not tried yet; z: Z (1
  // until a rejection counts); known: the warps' sums are those of the row as it is
  // now, but for the tokens taken out (certain: of p); left: R's sum, with them.
  int c = 0, depth = 0, pass = 0;
  uint32_t todo = kids[0];
  const float2 one = make_float2(1.f, 0.f), zero = make_float2(0.f, 0.f);
  float2 z = one, before_f = zero, draft_mass = one;
  uint64_t draft_all = 0, draft_sum = 0;  // what is left of the draft's mass; the last pass's sum
  bool pending = false, known = false, fresh = true;  // fresh: nothing was rejected at this node
  uint64_t left = 0;
  int v_per = 0;
  const T* prow = p_rows;
  const T* qrow = q_rows;
  int pre = 0;
  bool p_wide = false, q_wide = false;
  // What a token taken out adds to the sums (modulo 2^64).
  auto gone_adds = [&](int i) { return st.gone_r[i] - rest_of(st.gone_p[i], st.gone_q[i], st.f); };
  auto place_of = [&](int x) {
    for (int i = 0; i < st.n_gone; ++i)
      if (st.gone[i] == x) return i;
    return -1;
  };

  for (;;) {
    if (tid == 0) {
      way[0] = 0;
      cmd = 0;
      while (!cmd && !bad_bits) {
        if (pending) {  // a rejected child, and the sum after it (certain: of p)
          const int x = id[c], at = place_of(x);
          if constexpr (kDrafts == kCertain) {
            const uint64_t px = fixed(pp[c]);
            if (at < 0 && left > px) {  // else nothing would be left
              st.gone[st.n_gone] = x;
              st.gone_p[st.n_gone] = pp[c];
              st.gone_r[st.n_gone++] = 0;
              left -= px;
            }
            if (st.n_gone) z = pair_of(left);
          } else {
            if (left == 0) {  // R and Z stay
              st.f = before_f;
              known = false;
            } else {
              z = pair_of(left);
              known = true;
            }
            if constexpr (kDrafts == kDistinct) {
              if (st.n_gone == 0) draft_all = draft_sum;
              if (at < 0) {
                const uint64_t qx = fixed(qq[c]);
                draft_all = draft_all > qx ? draft_all - qx : 0;
                st.gone[st.n_gone] = x;
                st.gone_p[st.n_gone] = pp[c];
                st.gone_q[st.n_gone] = qq[c];
                st.gone_r[st.n_gone++] = rest_of(pp[c], qq[c], st.f);
              }
              draft_mass = pair_of(draft_all);
            }
          }
          pending = false;
        }
        if (!todo) {  // the last token: from the sums that there are, or a pass first
          cmd = known ? 2 : 1;
          known = true;
          break;
        }
        c = __ffs(todo) - 1;
        todo &= todo - 1;
        if (!((fine >> c) & 1u)) {
          bad_bits = STV_DEV_BAD_SAMPLE;
          break;
        }
        bool take = (taken >> c) & 1u;
        if (!fresh) {
          const int at = place_of(id[c]);
          float2 s_x = make_float2(qq[c], 0.f), r_x = make_float2(pp[c], 0.f);  // S(x), R(x), times the sum of S
          if (at >= 0) r_x = pair_of(st.gone_r[at]);
          else if (kDrafts != kCertain && st.f.x > 0.f) r_x = pair_of(rest_of(pp[c], qq[c], st.f));
          if constexpr (kDrafts == kDistinct) {
            if (st.n_gone) {
              if (at >= 0 || draft_mass.x == 0.f) s_x = zero;
              else r_x = r_x * draft_mass;
            }
          }
          take = make_float2(uu[c], 0.f) * s_x * z < r_x;
        }
        if (take) {
          node = c;
          todo = kids[c];
          way[++depth] = c;
          if (!fresh) {
            st.n_gone = 0;
            z = draft_mass = one;
            st.f = zero;
          }
          fresh = true;
          known = false;
          continue;
        }
        fresh = false;
        pending = true;
        if constexpr (kDrafts == kCertain) {
          cmd = known ? 0 : 1;
          known = true;
        } else {
          before_f = st.f;
          float2 f = z;
          if constexpr (kDrafts == kDistinct)
            if (st.n_gone) f = draft_mass.x > 0.f ? z / draft_mass : zero;
          st.f = st.f + f;
          cmd = 1;
        }
      }
    }
    __syncthreads();
    if (bad_bits || cmd == 2) break;

    // ---- a pass: sum R (and q) over the vocabulary ----
    prow = p_rows + (int64_t)node * p.p_stride;
    if constexpr (kDrafts != kCertain) qrow = q_rows + (int64_t)node * p.q_stride;
    const int mis = (int)((uintptr_t)prow % 16);
    p_wide = mis % sizeof(T) == 0;
    pre = p_wide ? mis / (int)sizeof(T) : 0;
    q_wide = kDrafts != kCertain && (int)((uintptr_t)qrow % 16) == mis && p_wide;
    const int n_vec = (V + pre + VE - 1) / VE;
    v_per = (n_vec + C * kWarps - 1) / (C * kWarps);
    const int v0 = (rank * kWarps + w) * v_per, v1 = min(n_vec, v0 + v_per);
    const float2 f = st.f;
    const bool none = f.x == 0.f, plain = f.x == 1.f && f.y == 0.f;
    uint64_t sum = 0, draft = 0;
    bool bad = false;
    constexpr int U = 4;  // vectors in flight
    for (int v = v0 + lane; v < v1; v += 32 * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const bool in = v + 32 * j < v1;
        const int e = in ? (v + 32 * j) * VE - pre : V;  // V: zeros
        a[j] = load_entries(prow, e, V, p_wide);
        if constexpr (kDrafts != kCertain)
          if (!none) b[j] = load_entries(qrow, e, V, q_wide);
      }
      uint32_t most = 0;  // of the entries' bits: above 1's, they are looked at again
      Sums part, part_q;
      const bool one_sum = kDrafts == kCertain || none;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        most = most_of<T>(most, a[j]);
        if (one_sum) {
#pragma unroll
          for (int i = 0; i < VE; i += 2) part.add(entries<T>(a[j], i));
        } else {
          most = most_of<T>(most, b[j]);
          if (plain) {
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
              const float2 y = entries<T>(b[j], i);
              add_above2<true>(part, entries<T>(a[j], i), y, f);
              if constexpr (kDrafts == kDistinct) part_q.add(y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < VE; i += 2) add_above2<false>(part, entries<T>(a[j], i), entries<T>(b[j], i), f);
          }
        }
      }
      sum = sat_add(sum, part.whole_of(U * VE, one_sum ? U * VE : 2 * U * VE));
      if constexpr (kDrafts == kDistinct)
        if (plain) draft = sat_add(draft, part_q.whole_of(U * VE, U * VE));
      if (above_one<T>(most)) {  // -0 is a probability
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            bad |= !is_prob(entry<T>(a[j], i));
            if constexpr (kDrafts != kCertain)
              if (!none) bad |= !is_prob(entry<T>(b[j], i));
          }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sum = sat_add(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      if constexpr (kDrafts == kDistinct) draft = sat_add(draft, __shfl_xor_sync(0xffffffffu, draft, o));
    }
    const int any_bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      warp_sum[w] = sum;
      warp_draft[w] = draft;
      warp_bad[w] = any_bad;
    }
    __syncthreads();
    ++pass;
    if (w == 0) {
      Share mine = {lane < kWarps ? warp_sum[lane] : 0, lane < kWarps ? warp_draft[lane] : 0,
                    lane < kWarps ? warp_bad[lane] : 0};
#pragma unroll
      for (int o = kWarps / 2; o; o >>= 1) {
        mine.sum = sat_add(mine.sum, __shfl_xor_sync(0xffffffffu, mine.sum, o));
        mine.draft = sat_add(mine.draft, __shfl_xor_sync(0xffffffffu, mine.draft, o));
        mine.bad |= __shfl_xor_sync(0xffffffffu, mine.bad, o);
      }
      if (lane < C) *cluster.map_shared_rank(&share[pass & 1][rank], lane) = mine;
    }
    cluster.sync();
    if (w == 0) {
      Share x = lane < C ? share[pass & 1][lane] : Share{0, 0, 0};
#pragma unroll
      for (int o = kMaxCluster / 2; o; o >>= 1) {
        x.sum = sat_add(x.sum, __shfl_xor_sync(0xffffffffu, x.sum, o));
        x.draft = sat_add(x.draft, __shfl_xor_sync(0xffffffffu, x.draft, o));
        x.bad |= __shfl_xor_sync(0xffffffffu, x.bad, o);
      }
      uint64_t more = 0;
      const int n_gone = kDrafts == kDistinct ? st.n_gone : 0;
      if (n_gone) {
        if (lane < n_gone) more = gone_adds(lane);
#pragma unroll
        for (int o = 16; o; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
      }
      if (lane == 0) {
        left = x.sum + more;
        draft_sum = x.draft;
        if (x.bad || x.sum >= kFull || draft_sum >= kFull || !(fine & 1u) ||
            ((kDrafts == kCertain || !pending) && left == 0))
          bad_bits = STV_DEV_BAD_SAMPLE;
      }
      __syncwarp();  // lane 0 goes on to the walk, which changes what the others have just read of st
    }
    // (thread 0's next decisions are behind this loop's first barrier; it alone reads what it wrote)
  }

  const int64_t out = (int64_t)s * T_;
  if (bad_bits) {
    if (rank == 0) {
      if (tid < T_) {
        p.path[out + tid] = -1;
        p.out_ids[out + tid] = -1;
      }
      if (tid == 0) {
        p.n_commit[s] = 0;
        report(p.status, bad_bits);
      }
    }
    return;
  }
  // ---- the last token ----
  __shared__ int depth_s;
  __shared__ uint64_t left_s;
  if (tid == 0) {
    depth_s = depth;
    left_s = left;  // the row's whole mass
  }
  if (tid < st.n_gone) {  // what the tokens taken out add to their ranges
    const int at = (st.gone[tid] + pre) / VE / v_per;
    const unsigned long long x = gone_adds(tid);
    atomicAdd(reinterpret_cast<unsigned long long*>(&share[pass & 1][at / kWarps].sum), x);
    if (at / kWarps == rank) atomicAdd(reinterpret_cast<unsigned long long*>(&warp_sum[at % kWarps]), x);
  }
  __syncthreads();
  if (rank == 0 && tid < T_) {
    p.path[out + tid] = tid <= depth_s ? way[tid] : -1;
    if (tid != depth_s) p.out_ids[out + tid] = tid < depth_s ? id[way[tid + 1]] : -1;
    if (tid == 0) p.n_commit[s] = depth_s + 1;
  }
  // u times the mass, rounded down: a whole running sum exceeds one iff it exceeds the other.
  const uint64_t target = __umul64hi(__float2ull_rz(uu[0] * 18446744073709551616.f), left_s);
  uint64_t before = 0;
  for (int i = 0; i < rank; ++i) before += share[pass & 1][i].sum;
  if (target < before || target >= before + share[pass & 1][rank].sum) return;
  int from = 0;
  for (; from < kWarps - 1; ++from) {
    if (target < before + warp_sum[from]) break;
    before += warp_sum[from];
  }
  const int n_vec = (V + pre + VE - 1) / VE;
  const int w0 = (rank * kWarps + from) * v_per, w1 = min(n_vec, w0 + v_per);
  const int m = (v_per + kThreads - 1) / kThreads;
  const int v0 = min(w1, w0 + tid * m), v1 = min(w1, v0 + m);
  const float2 f = st.f;
  const int n_gone = st.n_gone;
  // R of the entries of vector v.
  auto rest_at = [&](int v, uint64_t (&r)[VE]) {
    const int e = v * VE - pre;
    const uint4 a = load_entries(prow, e, V, p_wide);
    uint4 b = make_uint4(0, 0, 0, 0);
    if constexpr (kDrafts != kCertain)
      if (f.x != 0.f) b = load_entries(qrow, e, V, q_wide);
#pragma unroll
    for (int i = 0; i < VE; ++i) r[i] = rest_of(entry<T>(a, i), entry<T>(b, i), f);
    for (int g = 0; g < n_gone; ++g) {
      const int i = st.gone[g] - e;
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (k == i) r[k] = st.gone_r[g];
    }
  };
  uint64_t sum = 0, r[VE];
  for (int v = v0; v < v1; ++v) {
    rest_at(v, r);
#pragma unroll
    for (int i = 0; i < VE; ++i) sum += r[i];
  }
  uint64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan_sum[w] = incl;
  __syncthreads();
  for (int i = 0; i < w; ++i) before += scan_sum[i];
  before += incl - sum;
  if (target < before || target >= before + sum) return;
  for (int v = v0; v < v1; ++v) {
    if (v1 - v0 > 1) rest_at(v, r);  // else r still holds it
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (target >= before && target < before + r[i]) p.out_ids[out + depth_s] = v * VE - pre + i;
      before += r[i];
    }
  }
}

template <typename T, int kDrafts>
cudaError_t launch(const AcceptParams& p, int n_seqs, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_seqs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaSuccess;
  if (cluster > 8)
    e = cudaFuncSetAttribute(accept_probs_kernel<T, kDrafts>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, accept_probs_kernel<T, kDrafts>, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

template <typename T>
cudaError_t launch_for(const AcceptParams& p, int drafts, int n_seqs, int cluster, cudaStream_t s) {
  if (!p.q) return launch<T, kCertain>(p, n_seqs, cluster, s);
  return drafts == STV_DRAFTS_DISTINCT ? launch<T, kDistinct>(p, n_seqs, cluster, s)
                                       : launch<T, kReplaced>(p, n_seqs, cluster, s);
}

}  // namespace
}  // namespace stv

extern "C" int stv_tree_accept_probs(const int32_t* parent, const int32_t* draft_ids, const void* p, int64_t p_stride,
                                     const void* q, int64_t q_stride, int dtype, int vocab, int drafts,
                                     const float* u, int t_nodes, int n_seqs, int32_t* n_commit, int32_t* path,
                                     int32_t* out_ids, int32_t* dev_status, stv_stream_t stream) {
  using namespace stv;
  if (dtype != STV_F32 && dtype != STV_F16 && dtype != STV_BF16) return STV_ERR_INVALID_ARG;
  if (drafts != STV_DRAFTS_REPLACED && drafts != STV_DRAFTS_DISTINCT) return STV_ERR_INVALID_ARG;
  if (n_seqs < 0) return STV_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > kMaxVocab || t_nodes < 1 || t_nodes > kMaxT || n_seqs > 1 << 20)
    return STV_ERR_SHAPE_UNSUPPORTED;
  if (n_seqs == 0) return STV_OK;
  const int64_t es = dtype == STV_F32 ? 4 : 2, most = ((int64_t)1 << 48) / ((int64_t)n_seqs * t_nodes);
  if (!parent || !draft_ids || !p || !u || !n_commit || !path || !out_ids) return STV_ERR_INVALID_ARG;
  if (p_stride < vocab || p_stride > most || (uintptr_t)p % es) return STV_ERR_INVALID_ARG;
  if (q && (q_stride < vocab || q_stride > most || (uintptr_t)q % es)) return STV_ERR_INVALID_ARG;
  AcceptParams a;
  memset(&a, 0, sizeof(a));
  a.parent = parent;
  a.ids = draft_ids;
  a.p = p;
  a.q = q;
  a.p_stride = p_stride;
  a.q_stride = q_stride;
  a.u = u;
  a.vocab = vocab;
  a.T = t_nodes;
  a.n_commit = n_commit;
  a.path = path;
  a.out_ids = out_ids;
  a.status = dev_status;
  // As many CTAs for a sequence as have 4,096 entries each, while the grid stays
  // within one wave (two CTAs on an SM without draft rows, by registers; 16 in a
  // cluster find room only where there are few).
  int sm = 0;
  if (int rc = device_sm_count(&sm)) return rc;
  int cluster = kMaxCluster;
  auto fits = [&](int c) { return (int64_t)n_seqs * c <= (c > 8 || q ? sm : 2 * sm) && vocab >= 4096 * c; };
  while (cluster > 1 && !fits(cluster)) cluster /= 2;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == STV_F32   ? launch_for<float>(a, drafts, n_seqs, cluster, st)
                        : dtype == STV_F16 ? launch_for<__half>(a, drafts, n_seqs, cluster, st)
                                           : launch_for<__nv_bfloat16>(a, drafts, n_seqs, cluster, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
