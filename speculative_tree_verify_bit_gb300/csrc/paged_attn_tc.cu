// paged_attn_tc.cu -- attention over the drafter's 16-bit paged cache
// (include/stv.h, stv_paged_attn): blocks and prompts, on the 5th-generation
// tensor cores.
//
// A unit's rows (tokens x the G heads of its KV head) fill one tile of 128 rows,
// or two that share every tile of keys (head_dim 64 and 128: O of both fits
// tensor memory, and K and V cross shared memory once for twice the products).
// Per CTA: warp 0 produces (TMA, one box per K and V tile of 64 keys, 128-byte
// swizzle, rings of their own); warp 1 issues the MMAs; four warps per row tile
// do the softmax, thread = row = TMEM lane.  S = Q K^T with Q and S in tensor
// memory; P takes S's place in 16 bits and O += P V reads V as it lies in the
// cache (keys x channels: the MN-major operand).  A step is (tile of keys, row
// tile); S has two buffers, so the tensor pipe has the next step's S to form while
// the softmax of this one runs: with two row tiles they take turns, with one the
// tiles of keys do.
//
// The pipeline runs on across units.  At a unit's end the softmax warps put the
// next unit's Q into tensor memory, then write O / l, or the partials of a unit
// that the runs' borders cut.  Keys that no row sees are cleared in V, since 0
// times what a reused page holds there could be NaN.
// Every wait is bounded; a timeout sets a CTA abort flag, every role stops,
// copies and MMAs in flight are waited for and tensor memory is freed.
#include "paged_attn.cuh"

namespace stv {
namespace {

constexpr float kRescaleThreshold = 8.f;  // log2 units
constexpr int kInfos = 8;

template <int HD, int NQ>
struct Tiles {
  static constexpr int kTileBytes = kAttnTile * HD * 2;
  static constexpr int kKStages = HD == 256 ? 3 : HD == 128 ? 5 : 6;
  static constexpr int kVStages = HD == 256 ? 4 : HD == 128 ? 5 : 6;
  static_assert(kVStages + 2 <= kInfos, "tile infos in flight");
  static constexpr int kSmem = 1024 + (kKStages + kVStages) * kTileBytes;
  static constexpr int kThreads = 64 + 128 * NQ;
  // tensor memory: Q of each row tile, two S, O of each row tile
  static constexpr uint32_t kColQ = 0, kColS = NQ * HD / 2, kColO = kColS + 128;
  static constexpr uint32_t kCols = kColO + NQ * HD <= 256 ? 256 : 512;
  static_assert(kColO + NQ * HD <= 512, "tensor memory");
};

template <int HD, int NQ>
struct TilesShared {
  uint64_t k_full[Tiles<HD, NQ>::kKStages], k_empty[Tiles<HD, NQ>::kKStages];
  uint64_t v_full[Tiles<HD, NQ>::kVStages], v_empty[Tiles<HD, NQ>::kVStages];
  uint64_t info_full[kInfos];
  uint64_t s_full[2], p_full[2], pv_done[NQ], q_ready[NQ], o_ready[NQ], o_free[NQ], mma_done;
  TileInfo info[kInfos];
  uint32_t tmem_base;
  int abort;
};

// kind::f16: f32 D, A K-major; bf16 or f16; B K-major, or MN-major (the keys x
// channels of V).
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int n, bool mn_major) {
  return idesc_f16_f32(128, n) | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) |
         (mn_major ? 1u << 16 : 0u);
}
// MN-major, 128-byte swizzle: 64 channels by 8 keys make an atom of 1,024 bytes;
// atoms of further keys 1,024 bytes apart, of further channels a 64-key block.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kAttnTile * 128 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <typename T, int HD, int NQ>
__global__ void __launch_bounds__(Tiles<HD, NQ>::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ AttnParams p) {
  using C = Tiles<HD, NQ>;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TilesShared<HD, NQ> sh;
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  uint8_t* const kring = smem;
  uint8_t* const vring = smem + KS * C::kTileBytes;
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < kInfos; ++i) mbar_init(&sh.info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.q_ready[i], 4);
      mbar_init(&sh.o_ready[i], 1);
      mbar_init(&sh.o_free[i], 4);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sh.tmem_base)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dep_wait();
  grid_dep_launch();
  const RunStart start = run_of<C::kThreads>(p, reinterpret_cast<int*>(kring));
  fence_async_smem();  // the scratch's last reads come before the ring's copies
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 0) {
    // =================== producer ===================
    if (lane == 0) {
      RunWalk run(p, start);
      JoinRecord rec = {0, 0, 0, 0};
      int g = 0, k_issued = 0, v_issued = 0;
      bool ok = true;
      for (; ok && run.any; run.next()) {
        TileInfo in;
        in.row0 = run.en.row0 + run.at.u * p.tokens_per;
        in.rows = run.x.ntok * p.G;
        in.h = run.at.h;
        in.slot = run.slot();
        in.x = run.x;
        if (in.slot == 2 * (int)blockIdx.x + 1) rec = {in.row0, in.rows, in.h, run.last_cta()};
        for (int t = run.t0; t < run.t1; ++t, ++g) {
          in.key0 = tile_key(run.x, t);
          const int row = tile_row(p, run.en.s, in.h, in.key0);
          in.flags = (t == run.t0 ? kFirst : 0) | (t + 1 == run.t1 ? kLast : 0) | (row < 0 ? kAbsent : 0) |
                     (row < 0 || tile_edge(p, run.x, in.key0) ? kEdge : 0);
          const int ks = g % KS, vs = g % VS;
          if (!(ok = wait1<false>(&sh.k_empty[ks], ((g / KS) & 1) ^ 1, abort_flag))) break;
          sh.info[g % kInfos] = in;
          mbar_arrive(&sh.info_full[g % kInfos]);
          if (row < 0) {
            mbar_arrive(&sh.k_full[ks]);
          } else {
            mbar_expect_tx(&sh.k_full[ks], C::kTileBytes);
            tma_tile(kring + ks * C::kTileBytes, &p.map, row, &sh.k_full[ks]);
          }
          ++k_issued;
          if (!(ok = wait1<false>(&sh.v_empty[vs], ((g / VS) & 1) ^ 1, abort_flag))) break;
          if (row < 0) {
            mbar_arrive(&sh.v_full[vs]);
          } else {
            mbar_expect_tx(&sh.v_full[vs], C::kTileBytes);
            tma_tile(vring + vs * C::kTileBytes, &p.map, row + kPageTok, &sh.v_full[vs]);
          }
          ++v_issued;
        }
      }
      if (ok) {
        // Tile g - VS has been done with (its infos' place is free) once its V stage is.
        if (wait1<false>(&sh.v_empty[g % VS], ((g / VS) & 1) ^ 1, abort_flag)) {
          sh.info[g % kInfos].flags = kStop;
          mbar_arrive(&sh.info_full[g % kInfos]);
        }
      }
      p.rec[blockIdx.x] = rec;
      // No copy may still be landing when the CTA exits.
      volatile int never = 0;
      for (int j = max(0, k_issued - KS); j < k_issued; ++j) wait1<false>(&sh.k_full[j % KS], (j / KS) & 1, &never);
      for (int j = max(0, v_issued - VS); j < v_issued; ++j) wait1<false>(&sh.v_full[j % VS], (j / VS) & 1, &never);
    }
  } else if (warp == 1) {
    // =================== MMA issuer (whole warp, one elected lane issues) ===================
    // Per unit: S of steps 0 and 1, then P V of step j and S of step j + 2.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t kdesc0 = desc_sw128(su32(kring)), vdesc0 = desc_mn_sw128(su32(vring));
    constexpr uint32_t kIdescQK = idesc<T>(kAttnTile, false), kIdescPV = idesc<T>(HD, true);
    int g0 = 0, n_units = 0;  // tiles of earlier units
    auto flags_of = [&](int g, int* flags) -> bool {
      if (!waitw<false>(&sh.info_full[g % kInfos], (g / kInfos) & 1, abort_flag)) return false;
      *flags = sh.info[g % kInfos].flags;
      return true;
    };
    // S of step n (tile g, row tile qt).
    auto issue_qk = [&](int g, int qt) -> bool {
      const int n = g * NQ + qt, b = n & 1, ks = g % KS;
      if (qt == 0 && !waitw<false>(&sh.k_full[ks], (g / KS) & 1, abort_flag)) return false;
      tc_after();
      const uint64_t kd = kdesc0 + (uint64_t)(ks * (C::kTileBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        mma_tmemA(tm + C::kColS + 64 * b, tm + C::kColQ + qt * (HD / 2) + 8 * kk,
                  kd + (uint64_t)((kk >> 2) * (kAttnTile * 128 >> 4) + (kk & 3) * 2), kIdescQK, kk > 0);
      if (qt == NQ - 1) tc_commit(&sh.k_empty[ks]);
      tc_commit(&sh.s_full[b]);
      return true;
    };
    bool ok = true;
    for (;;) {
      int flags;
      if (!(ok = flags_of(g0, &flags)) || (flags & kStop)) break;
      for (int qt = 0; qt < NQ && ok; ++qt) ok = waitw<false>(&sh.q_ready[qt], n_units & 1, abort_flag);
      if (!ok) break;
      tc_after();
      // the unit's last tile, as far as the infos have been read
      int known = g0, last = flags & kLast ? g0 : -1;
      auto exists = [&](int g) -> bool {  // tile g belongs to the unit
        while (last < 0 && known < g) {
          int f;
          if (!flags_of(++known, &f)) return ok = false;
          if (f & kLast) last = known;
        }
        return last < 0 || g <= last;
      };
      auto qk_step = [&](int n) {  // n: step of the unit
        const int g = g0 + n / NQ;
        if (ok && exists(g) && ok) ok = issue_qk(g, n % NQ);
      };
      qk_step(0);
      qk_step(1);
      for (int n = 0; ok; ++n) {
        const int g = g0 + n / NQ, qt = n % NQ;
        if (last >= 0 && g > last) break;
        const int step = g * NQ + qt, b = step & 1, vs = g % VS;
        if (!(ok = waitw<false>(&sh.p_full[b], (step >> 1) & 1, abort_flag))) break;
        if (qt == 0 && !(ok = waitw<false>(&sh.v_full[vs], (g / VS) & 1, abort_flag))) break;
        // the unit's first P V restarts O: the previous unit's O has been read
        if (g == g0 && n_units > 0 && !(ok = waitw<false>(&sh.o_free[qt], (n_units - 1) & 1, abort_flag))) break;
        tc_after();
        const uint64_t vd = vdesc0 + (uint64_t)(vs * (C::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kAttnTile / 16; ++kk)
          mma_tmemA(tm + C::kColO + qt * HD, tm + C::kColS + 64 * b + 8 * kk, vd + (uint64_t)(kk * (2048 >> 4)), kIdescPV,
                    (g > g0 || kk > 0));
        if (qt == NQ - 1) tc_commit(&sh.v_empty[vs]);
        tc_commit(&sh.pv_done[qt]);
        if (last >= 0 && g == last) tc_commit(&sh.o_ready[qt]);
        qk_step(n + 2);
      }
      if (!ok) break;
      g0 = last + 1;
      ++n_units;
    }
    // Every MMA issued here has finished before TMEM is freed.
    tc_commit(&sh.mma_done);
    volatile int never = 0;
    waitw<false>(&sh.mma_done, 0, &never);
  } else {
    // =================== softmax (thread = row = TMEM lane) ===================
    const int qt = (warp - 2) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const int tile_rows = p.tokens_per / NQ * p.G;  // rows of a row tile
    const int ru = qt * tile_rows + r;              // row of the unit
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_q = C::kColQ + qt * (HD / 2), col_o = C::kColO + qt * HD;
    const float c = p.scale2;
    auto load_q = [&](const TileInfo& in) {
      const bool live = r < tile_rows && ru < in.rows;
      const T* src = static_cast<const T*>(p.q) + (int64_t)(in.row0 + ru / p.G) * p.q_row +
                     (int64_t)(in.h * p.G + ru % p.G) * p.q_head;
#pragma unroll
      for (int chunk = 0; chunk < HD / 64; ++chunk) {
        uint32_t v[32];
        if (!live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        } else if (p.q_wide) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + chunk * 64) + e);
            v[4 * e] = x.x;
            v[4 * e + 1] = x.y;
            v[4 * e + 2] = x.z;
            v[4 * e + 3] = x.w;
          }
        } else {
          const uint16_t* s16 = reinterpret_cast<const uint16_t*>(src) + chunk * 64;
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __ldg(s16 + 2 * e) | (uint32_t)__ldg(s16 + 2 * e + 1) << 16;
        }
        tmem_st32(lane_addr + col_q + 32 * chunk, v);
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_ready[qt]);
    };
    auto info_of = [&](int g, TileInfo* in) -> bool {
      if (!waitw<false>(&sh.info_full[g % kInfos], (g / kInfos) & 1, abort_flag)) return false;
      *in = sh.info[g % kInfos];
      return true;
    };
    TileInfo in;
    bool ok = info_of(0, &in);
    if (ok && !(in.flags & kStop)) load_q(in);
    float m_ref = -INFINITY, l = 0.f;
    int n_units = 0;
    for (int g = 0; ok && !(in.flags & kStop); ++g) {
      const int step = g * NQ + qt, b = step & 1;
      if (!(ok = waitw<false>(&sh.s_full[b], (step >> 1) & 1, abort_flag))) break;
      tc_after();
      uint32_t sa[32], sb[32];
      tmem_ld32(lane_addr + C::kColS + 64 * b, sa);
      tmem_ld32(lane_addr + C::kColS + 64 * b + 32, sb);
      tmem_wait_ld(sa);
      tmem_wait_ld(sb);
      if (in.flags & kEdge) {
        const bool absent = in.flags & kAbsent;
        const uint64_t vis = absent ? 0ull : row_sees(p, in.x.pos0 + ru / p.G, in.x.end, in.key0);
        const uint32_t va = (uint32_t)vis, vb = (uint32_t)(vis >> 32);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          sa[e] = ((va >> e) & 1u) ? sa[e] : 0xff800000u;
          sb[e] = ((vb >> e) & 1u) ? sb[e] : 0xff800000u;
        }
        // Keys that no row sees: zeros in V, by the first row tile's warps.
        const uint64_t some = absent ? 0ull : unit_sees(p, in.x, in.key0);
        if (qt == 0 && some != ~0ull) {
          const int vs = g % VS;
          if (!(ok = waitw<false>(&sh.v_full[vs], (g / VS) & 1, abort_flag))) break;
          const uint32_t base = su32(vring + vs * C::kTileBytes);
          for (int i = r; i < kAttnTile * (HD / 8); i += 128) {
            const int key = (i >> 3) % kAttnTile;
            if (!((some >> key) & 1)) st_shared_v4(base + i * 16, 0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
      }
      // Row maximum: 3-input max, 8 independent chains.
      float mx8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(__uint_as_float(sa[e]), __uint_as_float(sb[e]));
#pragma unroll
      for (int e = 8; e < 32; e += 2) {
        mx8[(e >> 1) & 7] = max3(mx8[(e >> 1) & 7], __uint_as_float(sa[e]), __uint_as_float(sa[e + 1]));
        mx8[((e >> 1) + 4) & 7] = max3(mx8[((e >> 1) + 4) & 7], __uint_as_float(sb[e]), __uint_as_float(sb[e + 1]));
      }
      const float mx = fmaxf(max3(mx8[0], mx8[1], mx8[2]), max3(max3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
      const float m_tile = mx * c;
      float corr = 1.f;
      if (m_tile > m_ref + kRescaleThreshold) {
        if (m_ref != -INFINITY) corr = ex2(m_ref - m_tile);
        m_ref = m_tile;
        l *= corr;
      }
      // P = 2^(S c - m_ref), rounded to the cache's type, packed in key pairs into
      // S's columns; the row's sum takes it before the rounding.
      const float mref = m_ref == -INFINITY ? 0.f : m_ref;
      const float2 c2 = make_float2(c, c), nm2 = make_float2(-mref, -mref);
      float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pk[32];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 xa = __ffma2_rn(make_float2(__uint_as_float(sa[2 * e]), __uint_as_float(sa[2 * e + 1])), c2, nm2);
        const float2 xb = __ffma2_rn(make_float2(__uint_as_float(sb[2 * e]), __uint_as_float(sb[2 * e + 1])), c2, nm2);
        const float2 pa = make_float2(ex2(xa.x), ex2(xa.y)), pb = make_float2(ex2(xb.x), ex2(xb.y));
        sum4[e & 3] = __fadd2_rn(sum4[e & 3], __fadd2_rn(pa, pb));
        pk[e] = Pack<T>::two(pa.x, pa.y);
        pk[16 + e] = Pack<T>::two(pb.x, pb.y);
      }
      const float2 sum2 = __fadd2_rn(__fadd2_rn(sum4[0], sum4[1]), __fadd2_rn(sum4[2], sum4[3]));
      l += sum2.x + sum2.y;
      tmem_st32(lane_addr + C::kColS + 64 * b, pk);
      // O may be rescaled only once the row tile's previous P V has finished: the
      // one before that has (this S followed it), and the next waits for this warp,
      // so the phase is that one's or the one before.  At a unit's first tile O
      // holds nothing to rescale.
      if (!(in.flags & kFirst) && __any_sync(0xffffffffu, corr != 1.f)) {
        if (!(ok = waitw<false>(&sh.pv_done[qt], (g - 1) & 1, abort_flag))) break;
        tc_after();
        const float2 corr2 = make_float2(corr, corr);
#pragma unroll 1
        for (int chunk = 0; chunk < HD / 32; ++chunk) {
          uint32_t o[32];
          tmem_ld32(lane_addr + col_o + 32 * chunk, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), corr2);
            o[2 * e] = __float_as_uint(x.x);
            o[2 * e + 1] = __float_as_uint(x.y);
          }
          tmem_st32(lane_addr + col_o + 32 * chunk, o);
        }
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[b]);

      TileInfo next;
      if (!(ok = info_of(g + 1, &next))) break;
      if (in.flags & kLast) {
        // The next unit's Q: every S of this unit's row tile has been formed.
        if (!(next.flags & kStop)) load_q(next);
        if (!(ok = waitw<false>(&sh.o_ready[qt], n_units & 1, abort_flag))) break;
        tc_after();
        const bool live = r < tile_rows && ru < in.rows;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        float* part = nullptr;
        T* dst = nullptr;
        if (in.slot >= 0) {
          part = p.part + ((int64_t)in.slot * p.part_rows + ru) * HD;
          if (live) p.ml[(int64_t)in.slot * p.part_rows + ru] = make_float2(m_ref, l);
        } else {
          dst = static_cast<T*>(p.o) + (int64_t)(in.row0 + ru / p.G) * p.o_row +
                (int64_t)(in.h * p.G + ru % p.G) * p.o_head;
        }
#pragma unroll 1
        for (int chunk = 0; chunk < HD / 32; ++chunk) {
          uint32_t o[32];
          tmem_ld32(lane_addr + col_o + 32 * chunk, o);
          tmem_wait_ld(o);
          if (!live) continue;
          if (part) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<float4*>(part + 32 * chunk)[e] =
                  make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                              __uint_as_float(o[4 * e + 3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(o[8 * e + k]) * inv;
              store_out<T, 8>(dst + 32 * chunk + 8 * e, v, p.o_wide);
            }
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free[qt]);
        m_ref = -INFINITY;
        l = 0.f;
        ++n_units;
      }
      in = next;
    }
  }

  // ---- teardown ----
  tc_before();
  __syncthreads();
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
  if (tid == 0 && sh.abort) report(p.status, STV_DEV_TIMEOUT);
}

template <typename T, int HD, int NQ>
cudaError_t launch_one(const AttnParams& p, int grid, cudaStream_t s) {
  using C = Tiles<HD, NQ>;
  cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<T, HD, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  return launch_pdl(attn_tiles_kernel<T, HD, NQ>, grid, C::kThreads, C::kSmem, s, p);
}

template <typename T>
cudaError_t launch_for(const AttnParams& p, int hd, int q_tiles, int grid, cudaStream_t s) {
  if (hd == 256) return launch_one<T, 256, 1>(p, grid, s);
  if (hd == 128) return q_tiles == 2 ? launch_one<T, 128, 2>(p, grid, s) : launch_one<T, 128, 1>(p, grid, s);
  return q_tiles == 2 ? launch_one<T, 64, 2>(p, grid, s) : launch_one<T, 64, 1>(p, grid, s);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnParams& p, int hd, bool bf16, int q_tiles, int grid, cudaStream_t s) {
  return bf16 ? launch_for<__nv_bfloat16>(p, hd, q_tiles, grid, s) : launch_for<__half>(p, hd, q_tiles, grid, s);
}

}  // namespace stv
