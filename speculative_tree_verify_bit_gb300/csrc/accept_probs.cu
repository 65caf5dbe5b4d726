// accept_probs.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers, on a token tree (include/stv.h,
// stv_tree_accept_probs).
//
// A cluster of CTAs takes one sequence.  Each CTA gathers, for every node i at
// once, the target's and the draft's probability of i's token at i's parent:
// the walk down the tree then needs no memory as long as drafts are accepted.
// A rejection changes the node's whole row, R <- max(R - Z S, 0), and needs Z =
// sum R: one pass over the vocabulary, split over the cluster's warps.  R is
// not stored: after k rejections at a node it is computed again from p, q and
// the k factors.  The last token comes from the same sums, kept per warp: the
// CTA whose range holds it reads one warp's share again with all its threads.
//
// R, Z and the running sums are integers in units of 2^-56 (an entry of at
// least 2^-32 in fp32 is exact), so nothing depends on the order of threads.
// The sums saturate at 64 instead of wrapping: rows of more mass than that are
// refused.  Every CTA takes every decision from the same numbers.
//
// Bounds: the launch, two dependent loads, a pass, two cluster barriers and the
// second reading, one after the other, for few sequences; HBM for many.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <utility>

#include "stv_device.cuh"

namespace stv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 524288;
constexpr uint64_t kFull = 1ull << 62;  // 64 in units of 2^-56
constexpr float kUnit = 72057594037927936.f;  // 2^56
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

// What a node's rejected children do to its row.
struct Steps {
  int k;             // rejections that count
  int n_gone;        // tokens taken out of S (distinct) or R (certain)
  uint64_t mul[kMaxT];  // Z over the sum of S (set_factor)
  int shift[kMaxT];
  int gone_before[kMaxT];
  int gone[kMaxT];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ uint64_t fixed(float x) { return __float2ull_rn(x * kUnit); }
__device__ __forceinline__ bool is_prob(float x) { return x >= 0.f && x <= 1.f; }
__device__ __forceinline__ uint64_t sat_add(uint64_t a, uint64_t b) { return min(a + b, kFull); }

// f > 0 as mul / 2^64 * 2^e with mul's top bit set: s f = (s 2^6 mul / 2^64) / 2^(6 - e).
__device__ __forceinline__ void set_factor(Steps& st, int j, double f) {
  if (!(f > 0)) {
    st.mul[j] = 0;
    st.shift[j] = 6;
    return;
  }
  int e;
  const double fr = frexp(f, &e);
  st.mul[j] = (uint64_t)(fr * 9007199254740992.0) << 11;  // 2^53, then 2^64
  st.shift[j] = 6 - e;
}
__device__ __forceinline__ uint64_t times(uint64_t s, uint64_t mul, int shift) {
  const uint64_t x = __umul64hi(s << 6, mul);
  return shift >= 0 ? (shift < 64 ? x >> shift : 0) : x << min(-shift, 63);
}

// R of token y after the node's steps.
template <int kDrafts>
__device__ __forceinline__ uint64_t rest_of(float p, float q, int y, const Steps& st, int k) {
  uint64_t r = fixed(p);
  if constexpr (kDrafts == kCertain) {
    for (int j = 0; j < k; ++j)
      if (st.gone[st.gone_before[j]] == y) r = 0;
  } else {
    const uint64_t s0 = fixed(q);
    for (int j = 0; j < k; ++j) {
      uint64_t s = s0;
      if constexpr (kDrafts == kDistinct)
        for (int i = 0; i < st.gone_before[j]; ++i)
          if (st.gone[i] == y) s = 0;
      const uint64_t x = times(s, st.mul[j], st.shift[j]);
      r = r > x ? r - x : 0;
    }
  }
  return r;
}

// VE entries of a row from entry e on; zeros outside [0, vocab).
template <typename T, int VE>
__device__ __forceinline__ void load_entries(const T* row, int e, int vocab, bool wide, float (&x)[VE]) {
  if (wide && e >= 0 && e + VE <= vocab) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e));
    const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = to_f(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = e + i >= 0 && e + i < vocab ? to_f(row[e + i]) : 0.f;
  }
}

struct Share {
  uint64_t sum, draft;  // of R, of q
  int bad;
};

template <typename T, int kDrafts>
__global__ void __launch_bounds__(kThreads) accept_probs_kernel(const __grid_constant__ AcceptParams p) {
  constexpr int VE = 16 / (int)sizeof(T);
  __shared__ int par[kMaxT], id[kMaxT], way[kMaxT];
  __shared__ float uu[kMaxT], pp[kMaxT], qq[kMaxT];
  __shared__ Steps st;
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
    par[tid] = there ? pa : -1;
    id[tid] = x;
    uu[tid] = u;
    pp[tid] = there ? to_f(p_rows[pa * p.p_stride + x]) : 0.f;
    if constexpr (kDrafts != kCertain) qq[tid] = there ? to_f(q_rows[pa * p.q_stride + x]) : 0.f;
    else qq[tid] = 1.f;
    if (tid == 0) {
      bad_bits = any ? STV_DEV_BAD_TREE : 0;
      st.k = st.n_gone = 0;
      node = 0;
    }
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));

  // Thread 0's place in the walk.  z: Z (1 until a rejection counts); known:
  // the warps' sums are those of R as it is now.
  int c = 1, depth = 0, pass = 0;
  double z = 1.0, draft_mass = 1.0;
  uint64_t draft_all = 0;
  bool pending = false, known = false;
  uint64_t total = 0;
  int v_per = 0;
  const T* prow = p_rows;
  const T* qrow = q_rows;
  int pre = 0;
  bool p_wide = false, q_wide = false;

  for (;;) {
    if (tid == 0) {
      way[0] = 0;
      if (pending) {  // the sum after a rejection
        const int j = st.k - 1;
        if (total == 0) {
          --st.k;  // nothing left: R and Z stay
          known = false;
        } else {
          z = (double)total * (1.0 / 72057594037927936.0);
          known = true;
        }
        if constexpr (kDrafts != kReplaced) {
          const int x = id[c];
          bool seen = false;
          for (int i = 0; i < st.n_gone; ++i) seen |= st.gone[i] == x;
          if constexpr (kDrafts == kDistinct) {
            if (j == 0 && st.n_gone == 0) draft_all = share[pass & 1][0].draft;
            if (!seen) {
              const uint64_t out = fixed(qq[c]);
              draft_all = draft_all > out ? draft_all - out : 0;
            }
            draft_mass = (double)draft_all * (1.0 / 72057594037927936.0);
            if (!seen) st.gone[st.n_gone++] = x;
          } else {
            st.n_gone = st.k;  // the token of each rejection that counts, in turn
          }
        }
        pending = false;
        ++c;
      }
      cmd = 0;
      while (!cmd && !bad_bits) {
        while (c < T_ && par[c] != node) ++c;
        if (c >= T_) {
          cmd = known ? 2 : 1;  // the last token: from the sums that there are, or a pass first
          known = true;
          break;
        }
        const int x = id[c];
        if (!is_prob(pp[c]) || !is_prob(qq[c]) || !(uu[c] >= 0.f && uu[c] < 1.f)) {
          bad_bits = STV_DEV_BAD_SAMPLE;
          break;
        }
        double share_d = qq[c];  // S(x)
        if constexpr (kDrafts == kDistinct) {
          for (int i = 0; i < st.n_gone; ++i)
            if (st.gone[i] == x) share_d = 0;
          if (st.n_gone) share_d = draft_mass > 0 ? share_d / draft_mass : 0;
        }
        const double r = st.k ? (double)rest_of<kDrafts>(pp[c], qq[c], x, st, st.k) * (1.0 / 72057594037927936.0)
                              : (double)pp[c];
        if ((double)uu[c] * share_d * z < r) {  // accepted
          node = c;
          way[++depth] = c;
          st.k = st.n_gone = 0;
          z = draft_mass = 1.0;
          known = false;
          ++c;
          continue;
        }
        const int j = st.k++;
        if constexpr (kDrafts == kCertain) {
          st.gone[j] = x;
          st.gone_before[j] = j;
        } else {
          st.gone_before[j] = st.n_gone;
          double f = z;
          if constexpr (kDrafts == kDistinct)
            if (st.n_gone) f = draft_mass > 0 ? z / draft_mass : 0;
          set_factor(st, j, f);
        }
        pending = true;
        known = false;
        cmd = 1;
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
    const int k = st.k;
    const bool plain = kDrafts != kCertain && k == 1 && st.mul[0] == 1ull << 63 && st.shift[0] == 5;
    uint64_t sum = 0, draft = 0;
    bool bad = false;
#pragma unroll 4
    for (int v = v0 + lane; v < v1; v += 32) {
      float a[VE], b[VE];
      const int e = v * VE - pre;
      load_entries<T, VE>(prow, e, V, p_wide, a);
      if constexpr (kDrafts != kCertain) {
        if (k || kDrafts == kDistinct) load_entries<T, VE>(qrow, e, V, q_wide, b);
      }
      uint64_t part = 0, part_q = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        bad |= !is_prob(a[i]);
        if constexpr (kDrafts != kCertain) {
          if (k || kDrafts == kDistinct) bad |= !is_prob(b[i]);
        }
      }
      if (!bad) {
        if (k == 0) {
#pragma unroll
          for (int i = 0; i < VE; ++i) part += fixed(a[i]);
        } else if (plain) {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const uint64_t x = fixed(a[i]), y = fixed(b[i]);
            part += x > y ? x - y : 0;
            if constexpr (kDrafts == kDistinct) part_q += y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i) part += rest_of<kDrafts>(a[i], kDrafts == kCertain ? 0.f : b[i], e + i, st, k);
        }
      }
      sum = sat_add(sum, part);
      if constexpr (kDrafts == kDistinct) draft = sat_add(draft, part_q);
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
      for (int o = 8; o; o >>= 1) {
        mine.sum = sat_add(mine.sum, __shfl_xor_sync(0xffffffffu, mine.sum, o));
        mine.draft = sat_add(mine.draft, __shfl_xor_sync(0xffffffffu, mine.draft, o));
        mine.bad |= __shfl_xor_sync(0xffffffffu, mine.bad, o);
      }
      if (lane < C) *cluster.map_shared_rank(&share[pass & 1][rank], lane) = mine;
    }
    cluster.sync();
    if (tid == 0) {
      total = 0;
      uint64_t all = 0;
      int found = 0;
      for (int i = 0; i < C; ++i) {
        const Share x = share[pass & 1][i];
        total = sat_add(total, x.sum);
        all = sat_add(all, x.draft);
        found |= x.bad;
      }
      share[pass & 1][0].draft = all;
      if (found || total >= kFull || all >= kFull || (!pending && total == 0) || !(uu[0] >= 0.f && uu[0] < 1.f))
        bad_bits = STV_DEV_BAD_SAMPLE;
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
  // Thread 0's depth and total for all.
  __shared__ int depth_s;
  __shared__ uint64_t total_s;
  if (tid == 0) {
    depth_s = depth;
    total_s = total;
  }
  __syncthreads();
  if (rank == 0 && tid < T_) {
    p.path[out + tid] = tid <= depth_s ? way[tid] : -1;
    if (tid != depth_s) p.out_ids[out + tid] = tid < depth_s ? id[way[tid + 1]] : -1;
    if (tid == 0) p.n_commit[s] = depth_s + 1;
  }
  // u total, rounded down: a whole running sum exceeds one iff it exceeds the other.
  const uint64_t target = __umul64hi(__float2ull_rz(uu[0] * 18446744073709551616.f), total_s);
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
  const int k = st.k;
  uint64_t sum = 0;
  for (int v = v0; v < v1; ++v) {
    float a[VE], b[VE] = {};
    load_entries<T, VE>(prow, v * VE - pre, V, p_wide, a);
    if constexpr (kDrafts != kCertain)
      if (k) load_entries<T, VE>(qrow, v * VE - pre, V, q_wide, b);
#pragma unroll
    for (int i = 0; i < VE; ++i) sum += rest_of<kDrafts>(a[i], b[i], v * VE - pre + i, st, k);
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
    float a[VE], b[VE] = {};
    load_entries<T, VE>(prow, v * VE - pre, V, p_wide, a);
    if constexpr (kDrafts != kCertain)
      if (k) load_entries<T, VE>(qrow, v * VE - pre, V, q_wide, b);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const uint64_t r = rest_of<kDrafts>(a[i], b[i], v * VE - pre + i, st, k);
      if (target >= before && target < before + r) p.out_ids[out + depth_s] = v * VE - pre + i;
      before += r;
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, accept_probs_kernel<T, kDrafts>, p);
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
  // As many CTAs for a sequence as have 4,096 entries each, while the grid stays within one wave.
  int sm = 0;
  if (int rc = device_sm_count(&sm)) return rc;
  int cluster = kMaxCluster;
  while (cluster > 1 && ((int64_t)n_seqs * cluster > 2 * sm || vocab < 4096 * cluster)) cluster /= 2;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == STV_F32   ? launch_for<float>(a, drafts, n_seqs, cluster, st)
                        : dtype == STV_F16 ? launch_for<__half>(a, drafts, n_seqs, cluster, st)
                                           : launch_for<__nv_bfloat16>(a, drafts, n_seqs, cluster, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}
