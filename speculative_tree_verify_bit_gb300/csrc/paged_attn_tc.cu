// paged_attn_tc.cu -- attention over the drafter's 16-bit paged cache
// (include/stv.h, stv_paged_attn): blocks and prompts, on the 5th-generation
// tensor cores.
//
// A unit's rows (tokens x the G heads of its KV head) fill one tile of 128 rows,
// or two that share every tile of keys (head_dim 64 and 128: O of both fits
// tensor memory).  Per CTA: warp 0 produces K and V, warp 1 issues the MMAs,
// warp 2 brings Q, and from warp 4 on four warps per row tile do the softmax,
// thread = row = TMEM lane.  A tile of 128 keys makes S = Q K^T of N = 128 (an MMA
// of N = 64 takes 47 cycles, one of N = 128 74); P takes S's place in 16 bits and
// O += P V reads V as it lies in the cache (keys x channels: the MN-major
// operand).  Q is in shared memory: tensor memory holds two S and O, 512 columns.
//
// K and V pass through one ring of pieces (K: 128 keys of 64 or 128 channels, V:
// 64 or 128 keys of all channels) in the order in which the MMAs take them.  A
// step is (tile of keys, row tile); S of step n + 2 is formed after P V of step n,
// so the tensor pipe works while a softmax runs: with two row tiles they take
// turns, with one the tiles of keys do.  The order runs on across units.
//
// Keys that no row sees are cleared in V, since 0 times what a reused page holds
// there could be NaN.  Every wait is bounded; a timeout sets a CTA abort flag,
// every role stops, copies and MMAs in flight are waited for and tensor memory is
// freed.
//
// Measured (2,070 MHz maximum): an 8,192-token prompt of 24 / 4 heads of 128 takes
// 342 us, 1,206 TFLOP/s (0.63 of the measured bf16 peak); 32,768 tokens of heads of
// 256 through a window of 2,048, 1,330 us, 1,210 TFLOP/s (0.63), and 1,430 to 1,475 in a
// long row of calls, where the power limit takes the clock to 1,850 to 1,950 MHz; 2,048
// tokens over 100,000 cached ones 1,750 us with heads of 128 (0.75), 4,090 of 256 (0.64),
// 1,897 of 64 (0.46).  The tensor pipe is busy 55 % of the time.  Heads of 256: a step takes 2,500 cycles where its MMAs
// take 2,304 (K and V cross shared memory once per 128 rows, 57 bytes a cycle and
// SM), and a unit's end 8,000 more: two or three masked tiles and O on its way out.
// Heads of 128: a row tile's turn is its softmax (1,700 cycles, two row tiles' on
// the same schedulers), 250 to hand P over and 1,300 of its own MMAs; the other row
// tile's MMAs fill 1,300 of that.
#include "paged_attn.cuh"

namespace stv {
namespace {

constexpr float kRescaleThreshold = 8.f;  // log2 units
constexpr int kUnits = 16;  // units that the producer may be ahead; a unit has a tile at least

template <int HD, int NQ>
struct Tiles {
  static constexpr int kQTile = kMaxRows * HD * 2;
  static constexpr int kPiece = big_piece_bytes(HD);
  static constexpr int kPieces = kBigTile * HD * 2 / kPiece;  // of K's tile, and of V's
  static constexpr int kKBlocks = kPiece / 16384;             // blocks of 64 channels in a piece of K
  static constexpr int kVKeys = kPiece / (2 * HD);            // keys of a piece of V
  static constexpr int kAhead = 2 / NQ;      // tiles of keys that S runs ahead
  static constexpr int kStage = NQ * 16384;  // 32 rows x 128 bytes for each softmax warp: O on its way out
  // Two tiles of K and V, or one where they are large: every place in the ring is
  // known when the loop over two tiles is compiled.
  static constexpr int kDeep = HD == 256 ? 1 : 2;
  static constexpr int kRing = 2 * kPieces * kDeep;
  static_assert(kRing / kPieces / 2 + kAhead + 2 < kUnits, "units in flight");
  static constexpr int kSmem = 1024 + NQ * kQTile + kStage + kRing * kPiece;
  static constexpr int kThreads = 128 + 128 * NQ;
  // Registers: with two row tiles the block starts with 168 a thread; the first
  // four warps give up 80 of theirs, 40 more for each softmax thread, which holds a
  // row of S (128 columns) at once.
  static constexpr int kLaunchRegs = 168, kFewRegs = 88, kSoftmaxRegs = 208;
  static_assert(kFewRegs + 2 * kSoftmaxRegs == 3 * kLaunchRegs, "registers of the block");
  // tensor memory: two S (P in their first halves), O of each row tile
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr uint32_t kCols = 512;
  static_assert(NQ * HD <= 256, "tensor memory");
};

struct UnitInfo {
  int row0, rows, h, slot;  // first row of q, rows of Q, KV head, workspace slot or -1
  int t0, t1;               // tiles of this part; t1 = t0: the run has ended
  AttnUnit x;
};

template <int HD, int NQ>
struct TilesShared {
  uint64_t full[Tiles<HD, NQ>::kRing], empty[Tiles<HD, NQ>::kRing];
  uint64_t unit_full[kUnits];
  uint64_t s_full[2], p_full[2], pv_done, q_full, q_empty, o_ready[NQ], o_free[NQ], mma_done;
  UnitInfo unit[kUnits];
  uint8_t absent[32];  // of tile g % 32: no page there
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
// atoms of further keys 1,024 bytes apart, of further channels `block` bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t block) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D (TMEM) = A x B (shared-memory descriptors) (+ D when acc != 0).
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.u32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_q(void* dst, const CUtensorMap* map, int block, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          su32(dst)),
      "l"(map), "r"(0), "r"(block), "r"(head), "r"(row), "r"(su32(bar))
      : "memory");
}

template <typename T, int HD, int NQ>
__global__ void __launch_bounds__(Tiles<HD, NQ>::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ AttnParams p) {
  using C = Tiles<HD, NQ>;
  constexpr int R = C::kRing, NP = C::kPieces, kPiece = C::kPiece;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TilesShared<HD, NQ> sh;
  uint8_t* smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  uint8_t* const qbuf = smem;
  uint8_t* const ring = smem + NQ * C::kQTile;
  uint8_t* const stage = ring + R * kPiece;
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kUnits; ++i) mbar_init(&sh.unit_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&sh.o_ready[i], 1);
      mbar_init(&sh.o_free[i], 4);
    }
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.q_full, 32);
    mbar_init(&sh.q_empty, 1);
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
  const RunStart start = run_of<C::kThreads>(p, reinterpret_cast<int*>(ring));
  fence_async_smem();  // the scratch's last reads come before the ring's copies
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem_base;

  // The unit of the n-th entry, once it is known.
  auto unit_at = [&](int n, UnitInfo* u) -> bool {
    if (!waitw<false>(&sh.unit_full[n % kUnits], (n / kUnits) & 1, abort_flag)) return false;
    *u = sh.unit[n % kUnits];
    return true;
  };

  if (warp < 4) {
  if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFewRegs));
  if (warp == 0) {
    // =================== producer of K and V ===================
    if (lane == 0) {
      RunWalk run(p, start);
      JoinRecord rec = {0, 0, 0, 0};
      PageWalk pages;
      int g = 0, n_units = 0, st = 0, n_issued = 0;
      uint32_t ph = 1;
      int v_rows[C::kAhead + 1];  // of tiles whose K is on its way
      bool ok = true;
      auto issue = [&](int row, bool v) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (!ok || !(ok = !p.withhold && wait1<false>(&sh.empty[st], ph, abort_flag))) return;
          uint8_t* dst = ring + st * kPiece;
          if (row < 0) {
            mbar_arrive(&sh.full[st]);
          } else {
            mbar_expect_tx(&sh.full[st], kPiece);
            if (v) tma_box(dst, &p.map_v, row + kPageTok + i * C::kVKeys, 0, &sh.full[st]);
            else tma_box(dst, &p.map_k, row, i * C::kKBlocks, &sh.full[st]);
          }
          ++n_issued;
          if (++st == R) {
            st = 0;
            ph ^= 1u;
          }
        }
      };
      for (; ok && run.any; run.next(), ++n_units) {
        UnitInfo& u = sh.unit[n_units % kUnits];
        u.row0 = run.en.row0 + run.at.u * p.tokens_per;
        u.rows = run.x.ntok * p.G;
        u.h = run.at.h;
        u.slot = run.slot();
        u.t0 = run.t0;
        u.t1 = run.t1;
        u.x = run.x;
        if (u.slot == 2 * (int)blockIdx.x + 1) rec = {u.row0, u.rows, u.h, run.last_cta()};
        mbar_arrive(&sh.unit_full[n_units % kUnits]);
        for (int t = run.t0; ok && t < run.t1; ++t, ++g) {
          const int row = pages.row(p, run.en, run.at.h, tile_key(p, run.x, t));
          sh.absent[g % 32] = row < 0;
          issue(row, false);
#pragma unroll
          for (int i = C::kAhead; i > 0; --i) v_rows[i] = v_rows[i - 1];
          v_rows[0] = row;
          if (g + 1 >= C::kAhead && ok) issue(v_rows[C::kAhead - 1], true);
        }
      }
      if (C::kAhead == 2 && g > 0 && ok) {  // V of tile g is the (2 g + kAhead)-th, the last one too
        issue(-1, false);
        if (ok) issue(v_rows[0], true);
      }
      if (ok) {
        // (the place of a unit kUnits ago, which is done with)
        sh.unit[n_units % kUnits].t0 = sh.unit[n_units % kUnits].t1 = 0;
        mbar_arrive(&sh.unit_full[n_units % kUnits]);
      }
      p.rec[blockIdx.x] = rec;
      // No copy may still be landing when the CTA exits.
      volatile int never = 0;
      for (int j = max(0, n_issued - R); j < n_issued; ++j) wait1<false>(&sh.full[j % R], (j / R) & 1, &never);
    }
  } else if (warp == 1) {
    // =================== MMA issuer (whole warp, one elected lane issues) ===================
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t kIdescQK = idesc<T>(kBigTile, false), kIdescPV = idesc<T>(HD, true);
    const uint64_t qdesc = desc_sw128(su32(qbuf)), kdesc = desc_sw128(su32(ring));
    const uint64_t vdesc = desc_mn_sw128(su32(ring), C::kVKeys * 128);
    // Whatever the loop's course hangs on is read from lane 0, so that the compiler
    // knows the warp to stay together: descriptors are then kept once for the warp
    // (an MMA takes 140 cycles to issue otherwise).  What a step waits for is probed
    // at once, ahead of the issue.
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    int qk_unit = 0, qk_left = 0;    // units whose S has begun; tiles of the last one still to come
    int pv_unit = 0, pv_left = 0;    // the same for P V
    bool pv_first = false, ok = true;
    // K or V of a tile lies in pieces st, st + 1, ...; ph: their phase.
    auto landed = [&](int st, uint32_t ph) -> uint32_t {
      uint32_t y = 1;
#pragma unroll
      for (int i = 0; i < NP; ++i) y &= probe(&sh.full[st + i], ph);
      return y;
    };
    auto wait_landed = [&](int st, uint32_t ph) -> bool {
      bool y = true;
#pragma unroll 1
      for (int i = 0; i < NP && y; ++i) y = waitw<false>(&sh.full[st + i], ph, abort_flag);
      return y;
    };
    // Whether the run has another tile for S; at a unit's first, its Q is waited for.
    auto more_qk = [&]() -> bool {
      if (qk_left > 0) return true;
      UnitInfo u;
      if (!(ok = unit_at(qk_unit, &u))) return false;
      qk_left = same(u.t1 - u.t0);
      if (qk_left == 0) return false;  // the run has ended
      return ok = waitw<false>(&sh.q_full, qk_unit++ & 1, abort_flag);
    };
    // S of a step (K of its tile is at st and has landed).
    auto issue_qk = [&](int qt, int b, int st) {
      if (qt == 0) --qk_left;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t kd = kdesc + (uint64_t)((st + i) * (kPiece >> 4));
        const uint64_t qd = qdesc + (uint64_t)(qt * (C::kQTile >> 4) + i * (kPiece >> 4));
#pragma unroll
        for (int kk = 0; kk < 4 * C::kKBlocks; ++kk) {
          const int at = (kk >> 2) * (16384 >> 4) + (kk & 3) * 2;
          mma_smem(tm + C::kColS + 128 * b, qd + at, kd + at, kIdescQK, i > 0 || kk > 0);
        }
        if (qt == NQ - 1) tc_commit(&sh.empty[st + i]);
      }
      tc_commit(&sh.s_full[b]);
      if (qt == NQ - 1 && qk_left == 0) tc_commit(&sh.q_empty);
    };
    // In the ring: K of the first tiles, then V of tile g (the (2 g + A)-th) and K of
    // tile g + A; A = kAhead.
    constexpr int A = C::kAhead, D = C::kDeep;
    bool more = true;
    int tiles_left = 0;  // of those whose S has been issued
#pragma unroll
    for (int i = 0; i < A; ++i) {
      if (!more || !(more = more_qk()) || !(more = ok = wait_landed(i * NP, 0))) continue;
      tc_after();
#pragma unroll
      for (int qt = 0; qt < NQ; ++qt) issue_qk(qt, (i * NQ + qt) & 1, i * NP);
      ++tiles_left;
    }
    for (int g0 = 0; ok && tiles_left > 0; g0 += 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!ok || tiles_left == 0) break;
        const int g = g0 + j;
        const int v_st = (2 * j + A) % (2 * D) * NP, k_st = (2 * j + A + 1) % (2 * D) * NP;
        const uint32_t v_ph = ((2 * g + A) / (2 * D)) & 1, k_ph = ((2 * g + A + 1) / (2 * D)) & 1;
        if ((pv_first = pv_left == 0)) {
          UnitInfo u;
          if (!(ok = unit_at(pv_unit, &u))) break;
          pv_left = same(u.t1 - u.t0);
          ++pv_unit;
        }
        --pv_left;
        --tiles_left;
#pragma unroll
        for (int qt = 0; qt < NQ; ++qt) {
          const int b = NQ == 2 ? qt : j;
          const uint32_t ph = (NQ == 2 ? g : g >> 1) & 1;
          // all that the step waits for, looked at once
          const uint32_t seen_p = probe(&sh.p_full[b], ph);
          const uint32_t seen_v = qt == 0 ? landed(v_st, v_ph) : 1u, seen_k = qt == 0 ? landed(k_st, k_ph) : 1u;
          if (!__all_sync(0xffffffffu, seen_p & seen_v)) {
            if (qt == 0 && !(ok = wait_landed(v_st, v_ph))) break;
            if (!(ok = waitw<false>(&sh.p_full[b], ph, abort_flag))) break;
          }
          // the unit's first P V restarts O: the previous unit's O has been read
          if (pv_first && pv_unit > 1 && !(ok = waitw<false>(&sh.o_free[qt], (pv_unit - 2) & 1, abort_flag))) break;
          tc_after();
#pragma unroll
          for (int kk = 0; kk < kBigTile / 16; ++kk) {  // 16 keys
            const int st = v_st + kk * 16 / C::kVKeys, in = kk * 16 % C::kVKeys;
            mma_tmemA(tm + C::kColO + qt * HD, tm + C::kColS + 128 * b + 8 * kk,
                      vdesc + (uint64_t)(st * (kPiece >> 4) + in * (128 >> 4)), kIdescPV, !pv_first || kk > 0);
            if (in + 16 == C::kVKeys && qt == NQ - 1) tc_commit(&sh.empty[st]);
          }
          if (NQ == 1) tc_commit(&sh.pv_done);
          if (pv_left == 0) tc_commit(&sh.o_ready[qt]);
          if (qt == 0 && more) {
            more = more_qk();
            if (!ok) break;
            if (more) {
              ++tiles_left;
              if (!__all_sync(0xffffffffu, seen_k) && !(ok = wait_landed(k_st, k_ph))) break;
            }
          }
          if (more) issue_qk(qt, b, k_st);
        }
      }
    }
    // Every MMA issued here has finished before TMEM is freed.
    tc_commit(&sh.mma_done);
    volatile int never = 0;
    waitw<false>(&sh.mma_done, 0, &never);
  } else if (warp == 2) {
    // =================== Q ===================
    // K-major tiles [hd / 64][128 rows][128 bytes], row r of token r / G.  Rows
    // past a row tile's keep what they held: a row's sums are its own.
    const int tile_tokens = p.tokens_per / NQ, tile_rows = tile_tokens * p.G;
    int asked = 0;  // units whose Q has been asked for
    for (int n = 0;; ++n) {
      UnitInfo u;
      if (!unit_at(n, &u) || u.t1 == u.t0) break;
      if (n > 0 && !waitw<false>(&sh.q_empty, (n - 1) & 1, abort_flag)) break;
      if (p.q_wide) {
        if (lane == 0) {
          mbar_expect_tx(&sh.q_full, NQ * (HD / 64) * tile_rows * 128);
          for (int qt = 0; qt < NQ; ++qt)
            for (int i = 0; i < HD / 64; ++i)
              tma_q(qbuf + qt * C::kQTile + i * 16384, &p.map_q, i, u.h * p.G, u.row0 + qt * tile_tokens, &sh.q_full);
        } else {
          mbar_arrive(&sh.q_full);
        }
      } else {
        for (int e = lane; e < u.rows * (HD / 8); e += 32) {
          const int ru = e / (HD / 8), c = e % (HD / 8), qt = ru / tile_rows, r = ru % tile_rows;
          const uint16_t* src = static_cast<const uint16_t*>(p.q) + (int64_t)(u.row0 + ru / p.G) * p.q_row +
                                (int64_t)(u.h * p.G + ru % p.G) * p.q_head + c * 8;
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = __ldg(src + 2 * k) | (uint32_t)__ldg(src + 2 * k + 1) << 16;
          st_shared_v4(su32(qbuf) + qt * C::kQTile + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[0], w[1],
                       w[2], w[3]);
        }
        fence_async_smem();
        mbar_arrive(&sh.q_full);
      }
      asked = n + 1;
    }
    // (the MMA warp has seen it land, unless the CTA aborted)
    volatile int never = 0;
    if (asked) wait1<false>(&sh.q_full, (asked - 1) & 1, &never);
  }
  } else {
    if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // =================== softmax (thread = row = TMEM lane) ===================
    const int qt = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const int tile_rows = p.tokens_per / NQ * p.G;  // rows of a row tile
    const int ru = qt * tile_rows + r;              // row of the unit
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_o = C::kColO + qt * HD;
    const float c = p.scale2;
    // A unit's end: its O is ready, or about to be.
    struct Ended {
      bool any = false, cut;
      float l;
      int64_t at;  // where this thread's row goes, in elements; -1: nowhere
    } ended;
    int n_ended = 0;
    // Writes O of the unit that has ended.  It is taken out of tensor memory at once,
    // so that the next unit's P V may start, and leaves through shared memory, 128
    // bytes of each of the warp's rows at a time (64 columns of o, 32 of the
    // partials; 16-byte pieces swizzled), so that whole lines of four rows go out
    // together.
    auto write_out = [&]() -> bool {
      if (!waitw<false>(&sh.o_ready[qt], n_ended & 1, abort_flag)) return false;
      ++n_ended;
      tc_after();
      const uint32_t mine = su32(stage) + (warp - 4) * 4096;
      const int piece = lane & 7;
      int64_t to[8];  // of the rows that this thread stores a piece of
#pragma unroll
      for (int i = 0; i < 8; ++i) to[i] = __shfl_sync(0xffffffffu, ended.at, 4 * i + (lane >> 3));
      // 128 bytes of the warp's rows: w, a thread's row's.  put(i, x): 16 bytes of row to[i].
      auto through = [&](const uint32_t* w, auto&& put) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          st_shared_v4(mine + lane * 128 + ((e ^ (lane & 7)) << 4), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        __syncwarp();
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                       : "r"(mine + row * 128 + ((piece ^ (row & 7)) << 4)) : "memory");
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (to[i] >= 0) put(i, x[i]);
        __syncwarp();
      };
      auto free_o = [&]() {
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free[qt]);
      };
      if (ended.cut) {
#pragma unroll 1
        for (int col = 0; col < HD; col += 32) {
          uint32_t o[32];
          tmem_ld32(lane_addr + col_o + col, o);
          tmem_wait_ld(o);
          if (col + 32 == HD) free_o();
          float* dst = p.part + col + 4 * piece;
          through(o, [&](int i, const uint4& x) { *reinterpret_cast<uint4*>(dst + to[i]) = x; });
        }
        return true;
      }
      const float inv = ended.l > 0.f ? 1.f / ended.l : 0.f;
      // (of 256 channels the registers hold a quarter at a time)
      constexpr int kHold = HD == 256 ? 128 : HD;
#pragma unroll 1
      for (int col = 0; col < HD; col += kHold) {
        uint32_t out[kHold / 2];
#pragma unroll
        for (int i = 0; i < kHold / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(lane_addr + col_o + col + 32 * i, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            out[16 * i + e] = Pack<T>::two(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        }
        if (col + kHold == HD) free_o();
#pragma unroll
        for (int i = 0; i < kHold / 64; ++i) {
          uint16_t* dst = static_cast<uint16_t*>(p.o) + col + 64 * i + 8 * piece;
          if (p.o_wide) {
            through(out + 32 * i, [&](int j, const uint4& x) { *reinterpret_cast<uint4*>(dst + to[j]) = x; });
          } else {
            through(out + 32 * i, [&](int j, const uint4& x) {
              uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                dst[to[j] + k] = (uint16_t)y[0];
                y[0] = __funnelshift_r(y[0], y[1], 16);
                y[1] = __funnelshift_r(y[1], y[2], 16);
                y[2] = __funnelshift_r(y[2], y[3], 16);
                y[3] >>= 16;
              }
            });
          }
        }
      }
      return true;
    };

    int g = 0;
    bool ok = true;
    for (int n_units = 0; ok; ++n_units) {
      if (!(ok = waitw<false>(&sh.unit_full[n_units % kUnits], (n_units / kUnits) & 1, abort_flag))) break;
      const UnitInfo& u = sh.unit[n_units % kUnits];  // stays as it is until the unit's end
      const int t0 = u.t0, t1 = u.t1;
      if (t1 == t0) break;
      const bool live = r < tile_rows && ru < u.rows;
      const Seen sees = row_sees(p, u.x, u.x.pos0 + ru / p.G), some = {u.x.lo, u.x.hi};
      // Some row may not see some key of a tile that goes on to `full_to` or further,
      // or begins at `full_from` or before (and is not all among the first tokens).
      const int full_to = p.causal ? min(u.x.pos0 + 1, u.x.end) : u.x.end;
      const int full_from = p.window ? u.x.pos0 + u.x.ntok - 1 - p.window : -1;
      const int n_sink = u.x.n_sink, skip = u.x.wt0 - n_sink;
      float m_ref = -INFINITY, l = 0.f;
      for (int t = t0; t < t1; ++t, ++g) {
        const int n = g * NQ + qt, b = n & 1;
        const int key0 = (t < n_sink ? t : t + skip) * kBigTile;
        if (!(ok = waitw<false>(&sh.s_full[b], (n >> 1) & 1, abort_flag))) break;
        tc_after();
        const uint32_t col_s = lane_addr + C::kColS + 128 * b;
        const bool absent = sh.absent[g % 32];
        bool all_seen = true;  // by some row each
        if (absent || key0 + kBigTile > full_to || (key0 <= full_from && key0 + kBigTile > p.sinks)) {
          // Columns that the row does not see go back as -inf, 32 at a time (a loop:
          // this path is cold, and a long one waits for its instructions).
          uint32_t all = ~0u;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint32_t vis = absent ? 0u : bits_of(sees, p.sinks, key0 + 32 * i);
            all &= absent ? 0u : bits_of(some, p.sinks, key0 + 32 * i);
            if (__all_sync(0xffffffffu, vis == ~0u)) continue;
            uint32_t x[32];
            tmem_ld32(col_s + 32 * i, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = ((vis >> e) & 1u) ? x[e] : 0xff800000u;
            tmem_st32(col_s + 32 * i, x);
          }
          tmem_wait_st();
          all_seen = all == ~0u;
        }
        uint32_t s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(col_s + 32 * i, s + 32 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_wait_ld(s + 32 * i);
        // The row's maximum: 3-input max, 8 independent chains.
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[8 + e]));
#pragma unroll
        for (int e = 16; e < 128; e += 2)
          mx8[(e >> 1) & 7] = max3(mx8[(e >> 1) & 7], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float mx = fmaxf(max3(mx8[0], mx8[1], mx8[2]), max3(max3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float m_tile = mx * c;
        const bool grows = m_tile > m_ref + kRescaleThreshold;
        if (__any_sync(0xffffffffu, grows)) {
          float corr = 1.f;
          if (grows) {
            if (m_ref != -INFINITY) corr = ex2(m_ref - m_tile);
            m_ref = m_tile;
            l *= corr;
          }
          // O may be rescaled only once the row tile's previous P V has finished.  With
          // two row tiles this S followed it; with one, this S followed the P V before
          // that, and the next waits for this warp, so the phase is that one's or the
          // one before.  At a unit's first tile O holds nothing to rescale.
          if (t > t0) {
            if (NQ == 1) {
              if (!(ok = waitw<false>(&sh.pv_done, (g - 1) & 1, abort_flag))) break;
              tc_after();
            }
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
        }
        // P = 2^(S c - m_ref + kLift), rounded to the cache's type, packed in key pairs into
        // S's columns.  The row's sum takes it before the rounding: as rounded, where a
        // large key's own rounding cancels, an 8,192-token prompt of 128 channels takes 381
        // us for 342 and one of 256 through a window 388 for 329.
        const float mref = (m_ref == -INFINITY ? 0.f : m_ref) - kLift<T>;
        const float2 c2 = make_float2(c, c), nm2 = make_float2(-mref, -mref);
        float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(s[64 * half + 2 * e]), __uint_as_float(s[64 * half + 2 * e + 1])), c2, nm2);
            const float2 v = make_float2(ex2(x.x), ex2(x.y));
            sum4[e & 3] = __fadd2_rn(sum4[e & 3], v);
            pk[e] = Pack<T>::two(v.x, v.y);
          }
          tmem_st32(col_s + 32 * half, pk);
        }
        // Keys that no row sees: zeros in V, by the first row tile's warps.  (V comes
        // late, so this is the last thing before P is handed over.)
        if (qt == 0 && !all_seen) {
          const int p0 = (2 * g + C::kAhead) * NP;
#pragma unroll 1
          for (int i = 0; i < NP && ok; ++i) ok = waitw<false>(&sh.full[(p0 + i) % R], ((p0 + i) / R) & 1, abort_flag);
          if (!ok) break;
          // thread: 16 bytes of keys r / 8 + 16 m in every block of 64 channels
          constexpr int kPer = C::kVKeys / 16;  // of those keys in a piece
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const uint32_t at = su32(ring) + (p0 + i) % R * kPiece + r * 16;
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
              const int k = key0 + (r >> 3) + 16 * (i * kPer + m);
              if (!absent && k < some.hi && (k >= some.lo || k < p.sinks)) continue;
#pragma unroll
              for (int cb = 0; cb < HD / 64; ++cb) st_shared_v4(at + m * 2048 + cb * (C::kVKeys * 128), 0u, 0u, 0u, 0u);
            }
          }
          fence_async_smem();
        }
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[b]);
        const float2 sum2 = __fadd2_rn(__fadd2_rn(sum4[0], sum4[1]), __fadd2_rn(sum4[2], sum4[3]));
        l += sum2.x + sum2.y;
        // With two row tiles the unit before is written once this one's first P is on
        // its way (an 8,192-token prompt takes 4 % less); with one, whose MMAs have a step
        // more at hand, at once (2 % less).
        if (ended.any) {
          if (!(ok = write_out())) break;
          ended.any = false;
        }
      }
      if (!ok) break;
      ended.any = true;
      ended.cut = u.slot >= 0;
      ended.l = l;
      ended.at = -1;
      if (live) {
        if (ended.cut) p.ml[(int64_t)u.slot * p.part_rows + ru] = make_float2(m_ref, l);
        ended.at = ended.cut ? ((int64_t)u.slot * p.part_rows + ru) * HD
                             : (int64_t)(u.row0 + ru / p.G) * p.o_row + (int64_t)(u.h * p.G + ru % p.G) * p.o_head;
      }
      if (NQ == 1) {
        if (!(ok = write_out())) break;
        ended.any = false;
      }
    }
    if (ok && ended.any) write_out();
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
  static_assert(C::kSmem + sizeof(TilesShared<HD, NQ>) + 512 <= 232448, "shared memory per CTA");
  cudaError_t e = cudaFuncSetAttribute(attn_tiles_kernel<T, HD, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  if (NQ == 2) {
    // The softmax warps wait for the registers that the others give up: the block
    // must have been compiled to start with as many as the split adds up to.
    static const int regs = [] {
      cudaFuncAttributes a;
      if (cudaFuncGetAttributes(&a, attn_tiles_kernel<T, HD, NQ>) == cudaSuccess) return a.numRegs;
      (void)cudaGetLastError();
      return 0;
    }();
    if (regs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
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
