// paged_attn.cu -- attention over the drafter's 16-bit paged cache
// (include/stv.h, stv_paged_attn): the kernel for single tokens, the join, and
// the entry point.
//
// Single tokens (at most 16 rows of Q per KV head).  One warp keeps a ring of
// tiles (64 keys: K and V, one TMA box each, 128-byte swizzle) full; four warps
// take 16 keys of every tile each, on their own: S = Q K^T by mma.sync (Q's
// fragments stay in registers), a running maximum that moves only when it grows
// by more than 2^8, P in the accumulator's layout as the next product's operand,
// O += P V over all channels.  Nothing is exchanged until the unit's end, where
// the four warps' O, maxima and sums are put together through shared memory.  16
// rows are what a tile's bytes need of the tensor cores to keep up with HBM many
// times over, so the split over keys, not over channels, is the one without
// barriers.  Bound by HBM; the ring holds what the SM needs in flight: 262,100 keys
// of 4 heads of 256 channels take 159 us (6,760 GB/s, the measured copy
// bandwidth), 64 ragged sequences of 173,000 keys of 128 channels in all 63 us, of
// 315,000 keys 104: 10 us more than their bytes, as a short call takes.  That is a
// chain: 1,000 keys take 9.7 us, of which the lengths and the run 2.3, the page and
// the tile 1.0, the products 1.3, the four warps' parts 1.3, the join 2.
#include <string.h>

#include <algorithm>

#include "paged_attn.cuh"

namespace stv {
namespace {

constexpr int kWorkers = 4;  // warps, 16 keys of a tile each
constexpr int kThreads = 32 * (kWorkers + 1);

template <int HD>
struct Small {
  static constexpr int kTileBytes = kSmallTile * HD * 2;  // of K, and of V
  static constexpr int kStages = HD == 256 ? 3 : 4;
  static constexpr int kCtasPerSm = HD == 256 ? 1 : HD == 128 ? 1 : 2;
  static constexpr int kQBytes = kSmallRows * HD * 2;
  static constexpr int kChunk = HD / 4;  // channels put together at a time
  static constexpr int kExchangeBytes = kWorkers * kSmallRows * kChunk * 4;
  static constexpr int kSmem = 1024 + kStages * 2 * kTileBytes + 2 * kQBytes + kExchangeBytes;
};

enum TileFlags { kFirst = 1, kLast = 2, kEdge = 4, kAbsent = 8, kStop = 16 };

// A tile as the producer hands it to the workers.
struct TileInfo {
  int flags, key0;
  int row0, rows, h, slot;  // the unit's first row of q, its rows of Q, KV head, workspace slot or -1
  AttnUnit x;
};

template <int kStages>
struct SmallShared {
  uint64_t full[kStages], empty[kStages], q_full[2], q_empty[2], met;
  TileInfo info[kStages];
  float2 ml[kWorkers][kSmallRows];
  int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, Small<HD>::kCtasPerSm)
    attn_small_kernel(const __grid_constant__ AttnParams p) {
  using K = Small<HD>;
  constexpr int kStages = K::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ SmallShared<kStages> sh;
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  uint8_t* const ring = smem;
  uint8_t* const qbuf = ring + kStages * 2 * K::kTileBytes;
  float* const exchange = reinterpret_cast<float*>(qbuf + 2 * K::kQBytes);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWorkers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 32);
      mbar_init(&sh.q_empty[i], kWorkers);
    }
    mbar_init(&sh.met, kWorkers);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  grid_dep_wait();
  grid_dep_launch();
  const RunStart start = run_of<kThreads>(p, reinterpret_cast<int*>(ring));
  fence_async_smem();  // the scratch's last reads come before the ring's copies
  __syncthreads();

  if (warp == kWorkers) {
    // =================== producer (whole warp; lane 0 issues) ===================
    RunWalk run(p, start);
    JoinRecord rec = {0, 0, 0, 0};
    PageWalk pages;
    int g = 0, n_units = 0, issued = 0;
    bool ok = true;
    for (; ok && run.any; run.next(), ++n_units) {
      const int rows = run.x.ntok * p.G, row0 = run.en.row0 + run.at.u * p.tokens_per;
      const int slot = run.slot();
      if (slot == 2 * (int)blockIdx.x + 1) rec = {row0, rows, run.at.h, run.last_cta()};
      for (int t = run.t0; ok && t < run.t1; ++t, ++g) {
        const int st = g % kStages;
        if (!(ok = !p.withhold && waitw<false>(&sh.empty[st], ((g / kStages) & 1) ^ 1, abort_flag))) break;
        const int key0 = tile_key(p, run.x, t);
        const int row = pages.row(p, run.en, run.at.h, key0);
        if (lane == 0) {
          TileInfo& i = sh.info[st];
          i.flags = (t == run.t0 ? kFirst : 0) | (t + 1 == run.t1 ? kLast : 0) | (row < 0 ? kAbsent : 0) |
                    (tile_edge(p, run.x, key0) ? kEdge : 0);
          i.key0 = key0;
          i.row0 = row0;
          i.rows = rows;
          i.h = run.at.h;
          i.slot = slot;
          i.x = run.x;
          if (row < 0) {
            mbar_arrive(&sh.full[st]);
          } else {
            mbar_expect_tx(&sh.full[st], 2 * K::kTileBytes);
            uint8_t* dst = ring + st * 2 * K::kTileBytes;
            tma_box(dst, &p.map_k, row, 0, &sh.full[st]);
            tma_box(dst + K::kTileBytes, &p.map_k, row + kPageTok, 0, &sh.full[st]);
          }
        }
        issued = g + 1;
        __syncwarp();
        if (t == run.t0) {
          // The unit's Q: 16 rows, row r of token r / G, 16-byte pieces swizzled
          // within the row; zeros past the unit's rows.
          const int b = n_units & 1;
          if (!(ok = waitw<false>(&sh.q_empty[b], ((n_units >> 1) & 1) ^ 1, abort_flag))) break;
          const uint32_t base = su32(qbuf + b * K::kQBytes);
#pragma unroll
          for (int i = 0; i < kSmallRows * HD / 8 / 32; ++i) {
            const int e = i * 32 + lane, r = e / (HD / 8), c = e % (HD / 8);
            const T* src = static_cast<const T*>(p.q) + (int64_t)(row0 + r / p.G) * p.q_row +
                           (int64_t)(run.at.h * p.G + r % p.G) * p.q_head + c * 8;
            const uint32_t dst = base + r * (HD * 2) + ((c ^ (r & 7)) << 4);
            if (r >= rows) {
              st_shared_v4(dst, 0u, 0u, 0u, 0u);
            } else if (p.q_wide) {
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
            } else {
              const uint16_t* s16 = reinterpret_cast<const uint16_t*>(src);
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = __ldg(s16 + 2 * k) | (uint32_t)__ldg(s16 + 2 * k + 1) << 16;
              st_shared_v4(dst, w[0], w[1], w[2], w[3]);
            }
          }
          // one more arrival, and that one when this lane's copies have landed; then the lane's own
          asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(su32(&sh.q_full[b])) : "memory");
          mbar_arrive(&sh.q_full[b]);
        }
      }
    }
    int oldest = max(0, issued - kStages);
    if (ok) {
      const int st = g % kStages;
      if (waitw<false>(&sh.empty[st], ((g / kStages) & 1) ^ 1, abort_flag)) {
        if (lane == 0) {
          sh.info[st].flags = kStop;
          mbar_arrive(&sh.full[st]);
        }
        oldest = max(0, issued - kStages + 1);  // the stage was free: its copy has landed
      }
    }
    if (lane == 0) {
      p.rec[blockIdx.x] = rec;
      // No copy may still be landing when the CTA exits.
      volatile int never = 0;
      for (int j = oldest; j < issued; ++j) wait1<false>(&sh.full[j % kStages], (j / kStages) & 1, &never);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // =================== workers ===================
    const int r0 = lane >> 2, kq = 2 * (lane & 3);
    const int l8 = lane & 7, lm = lane >> 3;
    uint32_t qf[HD / 16][4];
    float o[HD / 8][4];
    float m[2], l[2];
    int met = 0, n_units = 0;
    // All four warps have come here.
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.met);
      // (a poll: the others are about to come, and a suspended warp wakes up late)
      bool ok = false;
      for (uint32_t it = 0; it < kSpinLimit && !ok; ++it) ok = probe(&sh.met, met & 1);
      if (!ok) ok = wait_suspend(&sh.met, met & 1, abort_flag);
      ++met;
      return __all_sync(0xffffffffu, ok);
    };
    for (int g = 0;; ++g) {
      const int st = g % kStages;
      if (!waitw<false>(&sh.full[st], (g / kStages) & 1, abort_flag)) break;
      const TileInfo& info = sh.info[st];
      const int flags = info.flags;
      if (flags & kStop) break;
      if (flags & kFirst) {
        const int b = n_units & 1;
        if (!waitw<false>(&sh.q_full[b], (n_units >> 1) & 1, abort_flag)) break;
        const int r = (lm & 1) * 8 + l8;
        const uint32_t base = su32(qbuf + b * K::kQBytes) + r * (HD * 2);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) ldsm4(base + (((2 * ks + (lm >> 1)) ^ (r & 7)) << 4), qf[ks]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_empty[b]);
        ++n_units;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }
      if (!(flags & kAbsent)) {
        const uint32_t kbase = su32(ring + st * 2 * K::kTileBytes), vbase = kbase + K::kTileBytes;
        // S: 16 rows x 16 keys; the even and the odd 16 channels apart, so that
        // four chains of products run side by side.
        float s[2][2][4] = {};
        {
          const int key = warp * 16 + (lm >> 1) * 8 + l8;
          const uint32_t krow = kbase + key * 128;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const int c = 2 * ks + (lm & 1);
            uint32_t b[4];
            ldsm4(krow + (c >> 3) * 8192 + (((c & 7) ^ (key & 7)) << 4), b);
            mma16816<T>(s[ks & 1][0], qf[ks], b[0], b[1]);
            mma16816<T>(s[ks & 1][1], qf[ks], b[2], b[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[0][j][i] = (s[0][j][i] + s[1][j][i]) * p.scale2;
        uint32_t live = 0xfu;  // of this thread's keys of V: kq, kq + 1, kq + 8, kq + 9
        if (flags & kEdge) {
          const int k0 = info.key0 + 32 * (warp >> 1), at = 16 * (warp & 1) + kq;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sees =
                bits_of(row_sees(p, info.x, info.x.pos0 + (r0 + 8 * half) / p.G), p.sinks, k0) >> at;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (!((sees >> (8 * j + i)) & 1)) s[0][j][2 * half + i] = -INFINITY;
          }
          const uint32_t some = bits_of({info.x.lo, info.x.hi}, p.sinks, k0) >> at;
          live = (some & 3) | ((some >> 8) & 3) << 2;
        }
        uint32_t pf[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = 2 * half;
          float mx = fmaxf(fmaxf(s[0][0][i], s[0][0][i + 1]), fmaxf(s[0][1][i], s[0][1][i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const bool grows = mx > m[half] + 8.f;
          if (__any_sync(0xffffffffu, grows)) {
            float corr = 1.f;
            if (grows) {
              corr = ex2(m[half] - mx);  // 0 for the first keys
              m[half] = mx;
            }
            l[half] *= corr;
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
              o[n][i] *= corr;
              o[n][i + 1] *= corr;
            }
          }
          const float ref = (m[half] == -INFINITY ? 0.f : m[half]) - kLift<T>;
          // The sum takes P as the product takes it, rounded to the cache's type.
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = Pack<T>::two(ex2(s[0][j][i] - ref), ex2(s[0][j][i + 1] - ref));
            const float2 f = Pack<T>::floats(w);
            l[half] += f.x + f.y;
            pf[2 * j + half] = w;
          }
        }
        const uint32_t mask0 = (live & 1 ? 0xffffu : 0u) | (live & 2 ? 0xffff0000u : 0u);
        const uint32_t mask1 = (live & 4 ? 0xffffu : 0u) | (live & 8 ? 0xffff0000u : 0u);
        {
          const int key = warp * 16 + (lm & 1) * 8 + l8;
          const uint32_t vrow = vbase + key * 128;
#pragma unroll
          for (int n = 0; n < HD / 16; ++n) {
            const int c = 2 * n + (lm >> 1);
            uint32_t b[4];
            ldsm4t(vrow + (c >> 3) * 8192 + (((c & 7) ^ (key & 7)) << 4), b);
            // a key that no row sees may hold anything
            mma16816<T>(o[2 * n], pf, b[0] & mask0, b[1] & mask1);
            mma16816<T>(o[2 * n + 1], pf, b[2] & mask0, b[3] & mask1);
          }
        }
      }
      const int row0 = info.row0, rows = info.rows, h = info.h, slot = info.slot;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (!(flags & kLast)) continue;

      // ---- the unit's end: the four warps' parts ----
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
        if ((lane & 3) == 0) sh.ml[warp][r0 + 8 * half] = make_float2(m[half], l[half]);
      }
      if (!meet()) break;
      float mm[2], ll[2], fac[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float2 x[kWorkers];
        mm[half] = -INFINITY;
        ll[half] = 0.f;
#pragma unroll
        for (int i = 0; i < kWorkers; ++i) {
          x[i] = sh.ml[i][r0 + 8 * half];
          mm[half] = fmaxf(mm[half], x[i].x);
        }
        const float ref = mm[half] == -INFINITY ? 0.f : mm[half];
#pragma unroll
        for (int i = 0; i < kWorkers; ++i) ll[half] += ex2(x[i].x - ref) * x[i].y;
        fac[half] = ex2(m[half] - ref);
        if (slot < 0) fac[half] = ll[half] > 0.f ? fac[half] / ll[half] : 0.f;
      }
      if (slot >= 0 && warp == 0 && (lane & 3) == 0) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
          if (r0 + 8 * half < rows)
            p.ml[(int64_t)slot * p.part_rows + r0 + 8 * half] = make_float2(mm[half], ll[half]);
      }
      bool ok = true;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float* mine = exchange + warp * (kSmallRows * K::kChunk);
#pragma unroll
        for (int n = 0; n < K::kChunk / 8; ++n) {
          const int i = c * (K::kChunk / 8) + n;
#pragma unroll
          for (int half = 0; half < 2; ++half)
            *reinterpret_cast<float2*>(mine + (r0 + 8 * half) * K::kChunk + n * 8 + kq) =
                make_float2(o[i][2 * half] * fac[half], o[i][2 * half + 1] * fac[half]);
        }
        if (!(ok = meet())) break;
        constexpr int kEach = K::kChunk / 8;  // channels of a thread
        const int r = tid >> 3, ch = (tid & 7) * kEach;
        float v[kEach] = {};
#pragma unroll
        for (int i = 0; i < kWorkers; ++i)
#pragma unroll
          for (int k = 0; k < kEach; ++k) v[k] += exchange[i * (kSmallRows * K::kChunk) + r * K::kChunk + ch + k];
        if (r < rows) {
          const int col = c * K::kChunk + ch;
          if (slot < 0) {
            T* dst = static_cast<T*>(p.o) + (int64_t)(row0 + r / p.G) * p.o_row + (int64_t)(h * p.G + r % p.G) * p.o_head;
            store_out<T, kEach>(dst + col, v, p.o_wide);
          } else {
            float* dst = p.part + ((int64_t)slot * p.part_rows + r) * HD + col;
#pragma unroll
            for (int k = 0; k < kEach; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(v[k], v[k + 1]);
          }
        }
        if (c < 3 && !(ok = meet())) break;
      }
      if (!ok) break;
    }
  }
  __syncthreads();
  if (tid == 0 && sh.abort) report(p.status, STV_DEV_TIMEOUT);
}

// Units cut by the runs' borders: M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l
// over their parts, in the runs' order.  Block (b, j) takes rows of the unit that
// begins in CTA b's run and goes on after it; HD / 4 threads take a part of a row, so
// there are kSlots at a time: of one row (kParts: single tokens, whose parts may be
// as many as CTAs), put together through shared memory, or of as many rows.  A
// thread asks for the next kBatch parts at once.
constexpr int kJoinThreads = 256;
template <typename T, int HD, bool kParts>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kPer = 4, kTeam = HD / kPer, kSlots = kJoinThreads / kTeam, kBatch = 8;
  grid_dep_wait();
  grid_dep_launch();
  const JoinRecord rec = p.rec[blockIdx.x];
  const int slot = threadIdx.x / kTeam, ch = threadIdx.x % kTeam * kPer;
  const int r = kParts ? blockIdx.y : blockIdx.y * kSlots + slot;
  if ((kParts ? (int)blockIdx.y : (int)blockIdx.y * kSlots) >= rec.rows) return;
  const int first = blockIdx.x, n = r < rec.rows ? rec.last_cta - first + 1 : 0, step = kParts ? kSlots : 1;
  float M = -INFINITY, L = 0.f, v[kPer] = {};
  for (int i0 = kParts ? slot : 0; i0 < n; i0 += step * kBatch) {
    float2 x[kBatch];
    float4 a[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int c = first + i0 + k * step;
      x[k] = make_float2(-INFINITY, 0.f);
      if (i0 + k * step < n) {
        const int64_t at = (int64_t)(2 * c + (c == first)) * p.part_rows + r;
        x[k] = __ldg(p.ml + at);
        a[k] = __ldg(reinterpret_cast<const float4*>(p.part + at * HD + ch));
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) m = fmaxf(m, x[k].x);
    const float ref = m == -INFINITY ? 0.f : m, f0 = ex2(M - ref);
    M = m;
    L *= f0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (x[k].x == -INFINITY && x[k].y == 0.f) continue;  // not there, or without keys (NaN scores count)
      const float f = ex2(x[k].x - ref);
      L += f * x[k].y;
      v[0] += f * a[k].x;
      v[1] += f * a[k].y;
      v[2] += f * a[k].z;
      v[3] += f * a[k].w;
    }
  }
  if constexpr (kParts) {
    __shared__ float2 ml[kSlots];
    __shared__ float4 part[kSlots][kTeam];
    if (threadIdx.x % kTeam == 0) ml[slot] = make_float2(M, L);
    part[slot][threadIdx.x % kTeam] = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
    if (slot > 0) return;
    M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) M = fmaxf(M, ml[k].x);
    const float ref = M == -INFINITY ? 0.f : M;
    L = v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const float f = ex2(ml[k].x - ref);
      const float4 a = part[k][threadIdx.x];
      L += f * ml[k].y;
      v[0] += f * a.x;
      v[1] += f * a.y;
      v[2] += f * a.z;
      v[3] += f * a.w;
    }
  }
  if (r >= rec.rows) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int k = 0; k < kPer; ++k) v[k] *= inv;
  T* dst = static_cast<T*>(p.o) + (int64_t)(rec.row0 + r / p.G) * p.o_row + (int64_t)(rec.h * p.G + r % p.G) * p.o_head;
  store_out<T, kPer>(dst + ch, v, p.o_wide);
}

template <typename T, int HD>
cudaError_t launch_small(const AttnParams& p, int grid, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_small_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Small<HD>::kSmem);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  return launch_pdl(attn_small_kernel<T, HD>, grid, kThreads, Small<HD>::kSmem, s, p);
}

template <typename T, int HD>
cudaError_t launch_join(const AttnParams& p, bool small, int grid, cudaStream_t s) {
  const int rows = (int)std::min<int64_t>(p.part_rows, (int64_t)p.max_new * p.G);  // of a unit, at most
  const int slots = kJoinThreads / (HD / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)(small ? rows : (rows + slots - 1) / slots));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = small ? cudaLaunchKernelEx(&cfg, attn_join_kernel<T, HD, true>, p)
                        : cudaLaunchKernelEx(&cfg, attn_join_kernel<T, HD, false>, p);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// f<T, HD>(...) for the cache's type and head size.
#define STV_BY_TYPE(f, ...)                                                                            \
  (bf16 ? (hd == 256 ? f<__nv_bfloat16, 256>(__VA_ARGS__) : hd == 128 ? f<__nv_bfloat16, 128>(__VA_ARGS__) \
                                                                     : f<__nv_bfloat16, 64>(__VA_ARGS__)) \
        : (hd == 256 ? f<__half, 256>(__VA_ARGS__) : hd == 128 ? f<__half, 128>(__VA_ARGS__)             \
                                                              : f<__half, 64>(__VA_ARGS__)))

cudaError_t launch_attn_join(const AttnParams& p, int hd, bool bf16, bool small, int grid, cudaStream_t s) {
  return STV_BY_TYPE(launch_join, p, small, grid, s);
}

// How a call is cut: which kernel, its CTAs, and the workspace.
struct AttnPlan {
  bool small;
  int q_tiles, grid, tokens_per, part_rows;
  size_t ml_at, part_at, bytes;
};

int plan_attn(const RowShape& sh, int max_new, AttnPlan* a) {
  int sm = 0;
  if (int rc = device_sm_count(&sm)) return rc;
  a->small = (int64_t)max_new * sh.G <= kSmallRows;
  if (a->small) {
    a->grid = sm * (sh.hd == 256 ? Small<256>::kCtasPerSm : sh.hd == 128 ? Small<128>::kCtasPerSm : Small<64>::kCtasPerSm);
    a->tokens_per = kSmallRows / sh.G;
    a->part_rows = kSmallRows;
  } else {
    // Two tiles of 128 rows share each tile of keys where O of both fits
    // tensor memory and some sequence has rows for a second one.
    const int one = kMaxRows / sh.G;
    a->q_tiles = sh.hd < 256 && max_new > one ? 2 : 1;
    a->grid = sm;
    a->tokens_per = a->q_tiles * one;
    a->part_rows = a->q_tiles * kMaxRows;
  }
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  a->ml_at = up((size_t)a->grid * sizeof(JoinRecord));
  a->part_at = a->ml_at + up((size_t)2 * a->grid * a->part_rows * sizeof(float2));
  a->bytes = a->part_at + (size_t)2 * a->grid * a->part_rows * sh.hd * sizeof(float);
  return STV_OK;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

int encode(CUtensorMap* map, bool bf16, int rank, void* base, const cuuint64_t* dims, const cuuint64_t* strides,
           const cuuint32_t* box) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return STV_ERR_CUDA;
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, base, dims,
                        strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? STV_OK : STV_ERR_CUDA;
}

// The pool as [hd / 64][rows][64 channels], boxes of `keys` rows of `blocks` times 64 channels.
int make_pool_map(const stv_layer_cache* layer, const RowShape& sh, int keys, int blocks, CUtensorMap* map) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)layer->n_pages * sh.hkv * 2 * kPageTok, (cuuint64_t)sh.hd / 64};
  const cuuint64_t strides[2] = {(cuuint64_t)sh.hd * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)keys, (cuuint32_t)blocks};
  return encode(map, sh.bf16, 3, layer->pool, dims, strides, box);
}

// q as [rows][heads][hd / 64][64 channels], boxes of 64 channels of `tokens` tokens' G heads.
int make_q_map(const stv_rows* q, const RowShape& sh, int n_rows, int tokens, CUtensorMap* map) {
  const cuuint64_t dims[4] = {64, (cuuint64_t)sh.hd / 64, (cuuint64_t)sh.hq, (cuuint64_t)n_rows};
  // a stride that no step is taken along is the view's to choose: any that the map accepts
  const cuuint64_t strides[3] = {128, sh.hq > 1 ? (cuuint64_t)q->head_stride * 2 : (cuuint64_t)sh.hd * 2,
                                 n_rows > 1 ? (cuuint64_t)q->row_stride * 2 : (cuuint64_t)sh.hd * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)sh.G, (cuuint32_t)tokens};
  return encode(map, sh.bf16, 4, q->data, dims, strides, box);
}

}  // namespace

cudaError_t launch_attn_small(const AttnParams& p, int hd, bool bf16, int grid, cudaStream_t s) {
  return STV_BY_TYPE(launch_small, p, grid, s);
}

}  // namespace stv

using namespace stv;

extern "C" int stv_paged_attn_workspace_bytes(const stv_shape* shape, int max_new, size_t* bytes) {
  RowShape sh;
  if (int rc = check_row_shape(shape, &sh)) return rc;
  if (!bytes || max_new < 1) return STV_ERR_INVALID_ARG;
  AttnPlan a;
  if (int rc = plan_attn(sh, max_new, &a)) return rc;
  *bytes = a.bytes;
  return STV_OK;
}

static int paged_attn(const stv_shape* shape, const stv_attn_spec* spec, const stv_layer_cache* layer,
                      const stv_page_pool* pool, const int32_t* seqs, int n, const int32_t* ctx,
                      const int32_t* row_start, int max_new, const stv_rows* q, const stv_rows* o, int n_rows,
                      void* workspace, size_t ws_bytes, int32_t* dev_status, stv_stream_t stream, bool withhold) {
  RowShape sh;
  int rc = check_row_shape(shape, &sh);
  if (rc || (rc = check_row_layer(layer, sh))) return rc;
  if (!spec || !pool || !pool->tables || !pool->counts || !q || !o) return STV_ERR_INVALID_ARG;
  if (spec->window < 0 || spec->sinks < 0 || (spec->causal != 0 && spec->causal != 1)) return STV_ERR_INVALID_ARG;
  const float scale = spec->scale == 0.f ? 1.f / sqrtf((float)sh.hd) : spec->scale;
  const float scale2 = scale * 1.4426950408889634f;  // infinite times a score of 0 would be NaN
  if (!(scale > 0.f) || isinf(scale2)) return STV_ERR_INVALID_ARG;
  if (pool->max_seqs < 1 || pool->table_stride < 1 || n < 0 || n_rows < 0 || max_new < 1) return STV_ERR_INVALID_ARG;
  if (n > kMaxEntries || n_rows > 1 << 29) return STV_ERR_SHAPE_UNSUPPORTED;
  if (!row_start && n_rows < n) return STV_ERR_INVALID_ARG;
  if (n == 0 || n_rows == 0) return STV_OK;
  if (!ctx || !workspace || (uintptr_t)workspace % 16) return STV_ERR_INVALID_ARG;
  for (const stv_rows* v : {q, o})
    if (!rows_view_ok(v, sh.hd, n_rows) || v->heads != sh.hq || (uintptr_t)v->data % 2) return STV_ERR_INVALID_ARG;
  // o's columns may lie beside q's in the same rows, or in the same heads
  if (views_may_meet(q, o, sh.hd, n_rows, 2)) return STV_ERR_INVALID_ARG;
  if (rows_meet_pool(o, sh.hd, n_rows, layer)) return STV_ERR_INVALID_ARG;
  AttnPlan a;
  if ((rc = plan_attn(sh, max_new, &a))) return rc;
  if (ws_bytes < a.bytes) return STV_ERR_WORKSPACE_TOO_SMALL;

  AttnParams p;
  memset(&p, 0, sizeof(p));
  auto wide = [&](const stv_rows* v) {
    return (uintptr_t)v->data % 16 == 0 && (v->heads == 1 || v->head_stride % 8 == 0) &&
           (n_rows == 1 || v->row_stride % 8 == 0);
  };
  p.q = q->data;
  p.o = o->data;
  p.q_row = q->row_stride;
  p.q_head = q->head_stride;
  p.o_row = o->row_stride;
  p.o_head = o->head_stride;
  p.q_wide = wide(q);
  p.o_wide = wide(o);
  if (a.small) {
    if ((rc = make_pool_map(layer, sh, kSmallTile, sh.hd / 64, &p.map_k))) return rc;
  } else {
    if ((rc = make_pool_map(layer, sh, kBigTile, big_piece_bytes(sh.hd) / 16384, &p.map_k))) return rc;
    if ((rc = make_pool_map(layer, sh, big_piece_bytes(sh.hd) / (2 * sh.hd), sh.hd / 64, &p.map_v))) return rc;
    // (strides that a tensor map does not take: plain loads)
    if (p.q_wide && make_q_map(q, sh, n_rows, kMaxRows / sh.G, &p.map_q)) p.q_wide = false;
  }
  p.tile_bits = a.small ? 6 : 7;
  // Measured: 64 ragged single tokens of 128 channels take 86, 75, 72 and 74 us at 0, 2,
  // 4 and 8; of 256 channels 92, 86, 83 and 83 at 0, 1, 2 and 4; of 64 (8 KV heads) 93, 74,
  // 76 and 81 at 0, 4, 8 and 16.  A windowed prompt of 256 channels takes 4 % and 18 % more
  // at 2 and 1 than at 3, as much at 5; 8,192 tokens of 64 channels 374, 371, 370 and 378 us
  // at 1, 2, 3 and 5.
  p.unit_cost = a.small ? 512 / sh.hd : 3;
  p.tables = pool->tables;
  p.counts = pool->counts;
  p.table_stride = pool->table_stride;
  p.max_seqs = pool->max_seqs;
  p.n_pages = layer->n_pages;
  p.seqs = seqs;
  p.ctx = ctx;
  p.row_start = row_start;
  p.n = n;
  p.n_rows = n_rows;
  p.max_new = max_new;
  p.hkv = sh.hkv;
  p.G = sh.G;
  p.tokens_per = a.tokens_per;
  p.window = spec->window;
  p.sinks = spec->window ? spec->sinks : 0;
  p.causal = spec->causal;
  p.scale2 = scale2;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.rec = reinterpret_cast<JoinRecord*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + a.ml_at);
  p.part = reinterpret_cast<float*>(ws + a.part_at);
  p.part_rows = a.part_rows;
  p.withhold = withhold;
  p.status = dev_status;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = a.small ? launch_attn_small(p, sh.hd, sh.bf16, a.grid, st)
                          : launch_attn_tiles(p, sh.hd, sh.bf16, a.q_tiles, a.grid, st);
  if (e == cudaSuccess) e = launch_attn_join(p, sh.hd, sh.bf16, a.small, a.grid, st);
  return e == cudaSuccess ? STV_OK : STV_ERR_CUDA;
}

extern "C" int stv_paged_attn(const stv_shape* shape, const stv_attn_spec* spec, const stv_layer_cache* layer,
                              const stv_page_pool* pool, const int32_t* seqs, int n, const int32_t* ctx,
                              const int32_t* row_start, int max_new, const stv_rows* q, const stv_rows* o, int n_rows,
                              void* workspace, size_t ws_bytes, int32_t* dev_status, stv_stream_t stream) {
  return paged_attn(shape, spec, layer, pool, seqs, n, ctx, row_start, max_new, q, o, n_rows, workspace, ws_bytes,
                    dev_status, stream, false);
}

extern "C" int stv_paged_attn_timeout_test(const stv_shape* shape, const stv_attn_spec* spec,
                                           const stv_layer_cache* layer, const stv_page_pool* pool,
                                           const int32_t* seqs, int n, const int32_t* ctx, const int32_t* row_start,
                                           int max_new, const stv_rows* q, const stv_rows* o, int n_rows,
                                           void* workspace, size_t ws_bytes, int32_t* dev_status,
                                           stv_stream_t stream) {
  return paged_attn(shape, spec, layer, pool, seqs, n, ctx, row_start, max_new, q, o, n_rows, workspace, ws_bytes,
                    dev_status, stream, true);
}
