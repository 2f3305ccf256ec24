// The ring forward with capped scores or a bias by distance.  Each ra_scored_fwd_*.cu makes it for one
// kind of change, so that they compile side by side.
//
// The plain forward (ra_fwd.cuh: its tiles, its loads and its order of products) with twice the softmax threads.
// A cap makes a score cost 8 instructions where a plain one costs 5, and the two softmax warps that a scheduler had
// then kept the tensor cores waiting: they issue one instruction in 2.6 cycles between them, because each
// instruction waits for the one before and their long straight code for its fetching.  So a row is two threads' here
// (key columns [0, 64) and [64, 128) of a tile), four warps a scheduler, and the code of 32 columns is a loop's body.
//
// A call with a cap that is not too high has one offset for all rows at first (`fixed` below).  In a loop over 32 columns
// the products come out of tensor memory, the polynomial for the largest of them is chosen, and they become weights,
// packed as bf16 over the first 32 of the thread's own 64 columns; sums of weights stay with the thread until the end.
// Where a row's sum shows that the offset was far from its scores, the block starts again, as a call without such a
// cap does.  There a tile takes two steps before that:
//   1. largest product of the half row.  The cap is monotonic and the bias a line along a tile's columns, so an upper
//      bound of the largest score follows; the offset of a softmax may lie above it by kLoose.  Tiles in which the
//      bias is no line (the row's own token or a zigzag seam inside), or too steep a one, go over their changed
//      scores instead.
//   2. the two threads of a row raise the row's bound, a word of shared memory, and take it as the offset, if it passes
//      the running one by 2^8.
//
// Bound, d = 128: a tile of 128 x 128 needs 1024 cycles of the tensor cores, which are busy half of the time; the
// multiply-add pipes are for 40 %, the issue slots for 52 %.  The rest are a tile's steps that wait for one another (a
// product, its weights, the next product), with two tiles in flight, which fill tensor memory (d = 64 leaves 128 columns,
// which would hold a third score tile).  Causal, 16,384 tokens of 32 heads of 128, softcap 50: 1.75 ms, 1252 TFLOP/s (65 %
// of the measured bf16 rate), 1.86 between other work; without the cap 1.54.  8192 tokens of 32 + 8 heads, softcap 30
// and a prefix 0.51 ms (0.45); 2 x 4096 tokens of 16 heads of 64, a bias, 4 striped shards 184 us (157).
// What led here, for the first: a row a thread 2.36 ms, half a row 2.14, one offset and 32 columns at a time 1.82 (1.88
// with the polynomials' constants from the parameters), heavy tiles first 1.72.  Choosing the polynomial afterwards
// and doing the few other tiles again took 1.79 for 1.82, but 0.59 for 0.56 where scores are larger next to their cap.
#pragma once

#include "ra_fwd.cuh"
#include "ra_score.cuh"

namespace ra {
namespace {

constexpr int kScoredThreads = 640;  // control, and two warpgroups for each query tile
// Register split as in the plain kernel: 640 threads launch with 96 each.
constexpr int kScoredLaunchRegs = 96, kScoredRegsLow = 64, kScoredRegsHigh = 104;
static_assert(128 * kScoredRegsLow + 512 * kScoredRegsHigh <= kScoredThreads * kScoredLaunchRegs,
              "register split exceeds the launch");

template <int D>
struct ScoredFwdLayout : FwdLayout<D> {
  using Base = FwdLayout<D>;
  static constexpr int kBound = Base::kMisc + 16;  // [2 tiles][128 rows], as to_ordered
  static constexpr int kCaps = (kBound + 2 * 128 * 4 + 7) / 8 * 8;  // constants
  static constexpr int kAlloc = kCaps + kCapTable + 1024;
  // the epilogue's row slots (16 warps x 32 rows of half a head, bf16) and sums reuse the operand buffers
  static_assert(16 * 32 * D + 2048 <= Base::kBar, "output slots exceed the operand buffers");
};

template <int D, bool VL, int SC>
__global__ void __launch_bounds__(kScoredThreads, 1)
    ring_scored_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const FwdParamsT<VL, SC> p) {
  using LY = ScoredFwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const int n_pairs = (p.L + kRowsPerCta - 1) / kRowsPerCta;
  const Start start = start_of<VL, true, kRowsPerCta>(p, n_pairs, p.r_only);
  const int b = start.head / p.H, h = start.head % p.H, r = start.r, i0 = start.i0;
  const uint32_t bar0 = sb + LY::kBar;
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + LY::kMisc + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + LY::kMisc);

  volatile int* again_flag = reinterpret_cast<volatile int*>(sp + LY::kMisc + 8);
  bool q_issued = false;  // by thread 0, the Q / K producer
  auto init_tile_barriers = [&](bool anew) {
    auto init = [&](int i, uint32_t count) {
      if (anew) mbar_inval(BAR(i));
      mbar_init(BAR(i), count);
    };
    for (int i = 0; i < kKStages; ++i) {
      init(B_K_EMPTY + i, 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      init(B_V_FULL + i, 1);
      init(B_V_EMPTY + i, 1);
    }
    for (int t = 0; t < kQTiles; ++t) {
      init(B_S_FULL + t, 1);
      init(B_P_FULL + t, 8);  // one elected arrival per softmax warp
    }
    init(B_O_DONE, 1);
    init(B_TEARDOWN, 1);
    fence_mbar_init();
  };
  if (threadIdx.x == 0) {
    mbar_init(BAR(B_Q_FULL), 1);
    *abort_flag = 0;
    *again_flag = 0;
    init_tile_barriers(false);
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if constexpr (!VL) after_previous_kernel();  // (varlen reads cu_seqlens through the read-only path)
  if (threadIdx.x == 0) {
    // the CTA's Q tiles depend on nothing the tile walk below computes: issued
    // first, their latency overlaps the CTA's set-up
    if (!(p.ctl.debug_flags & DBG_SKIP_Q_LOAD)) {
      const int prow0 = r * p.L + i0 - p.q_base;
      mbar_expect_tx(BAR(B_Q_FULL), kQTiles * LY::kTile);
      for (int t = 0; t < kQTiles; ++t)
        for (int c = 0; c < D / 64; ++c)
          if (in_bounds(tma_coords_ok(TmaExtent{D, p.q_rows, p.H, p.B}, c * 64, prow0 + t * kTileM, h, b), p.ctl, 1))
            tma_load_4d(sb + LY::kQ + t * LY::kTile + c * kBox, &tmQ, BAR(B_Q_FULL), c * 64, prow0 + t * kTileM, h,
                        b);
      q_issued = true;
    }
  }
  fill_cap_table(sp + LY::kCaps, p.sc);
  auto init_bounds = [&]() {
    if (threadIdx.x < 256) reinterpret_cast<volatile int*>(sp + LY::kBound)[threadIdx.x] = to_ordered(-INFINITY);
  };
  init_bounds();
  QRange cta;  // both query tiles together: decides which key tiles are visited
  const int pre = VL ? 0 : prefix_now(p, b);
  make_qrange(p, r, i0, kRowsPerCta, cta, pre);
  const int nkt = (p.L + kTileN - 1) / kTileN;
  int n_tiles = 0;
  walk_tiles(p, cta, nkt, [&](int, int) {
    ++n_tiles;
    return true;
  });

  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float slope2 = 0.f;
  if constexpr ((SC & SC_BIAS) != 0) slope2 = load_now(p.sc.slopes + h) * 1.4426950408889634f;
  // Capped scores lie within +-cap2, so where that is small enough one offset will do for nearly all rows: a weight is
  // 2^-101 to 2^61.  A bias only takes off, and nothing from the row's own token, which every row of a whole call sees.  A
  // row's sum tells afterwards how far its largest weight is from 1.  Within kSums values of 2^-60 to 2^80 have products
  // with it in fp32's range, and so have smaller weights as far as they count; else the block starts again, with
  // running offsets.  (With softcap 50: where a row's largest score lies below -17, or at the cap.  The 16,384 tokens above
  // take 1.73 ms, with every row at an end of the cap, so that all blocks start again, 5.5, and with running offsets from
  // the first on 2.2 and 2.9: scores near the cap are what caps are not meant for.)
  const bool fixed = (SC & SC_CAP) != 0 && p.sc.cap2 <= 81.f && ((SC & SC_BIAS) == 0 || (slope2 >= 0.f && p.step < 0));
  // Whether the block, all of whose threads come here with nothing in flight, starts again.
  auto again = [&]() -> bool {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!*again_flag || *abort_flag) return false;
    init_bounds();
    if (threadIdx.x == 0) init_tile_barriers(true);
    __syncthreads();
    return true;
  };
  if (warp < 4) {
    // ------------------------------------------------------------ control warpgroup
    regs_dec<kScoredRegsLow>();
    auto control = [&]() {
    if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ TMA producer (warp 0)
    if (warp == 0 && lane == 0 && n_tiles > 0) {
      // K(j) and V(j) land on one barrier (the V stage's), so that the MMA
      // thread waits once per key tile
      int issued[kVStages] = {};
      int j = 0;
      walk_tiles(p, cta, nkt, [&](int s, int kt) {
        const int sk = j % kKStages, sv = j % kVStages;
        // K's stage frees about two key tiles before V's: K goes first, its
        // bytes added to the V stage's phase without an arrival, once that
        // phase is the one of tile j (the phase of tile j - 2 has completed)
        if (j >= kKStages &&
            !wait_one<kWaitHint>(BAR(B_K_EMPTY + sk), (j / kKStages - 1) & 1, abort_flag, p.ctl, 1))
          return false;
        if (j >= kVStages &&
            !wait_one<kWaitHint>(BAR(B_V_FULL + sv), (j / kVStages - 1) & 1, abort_flag, p.ctl, 6))
          return false;
        const int hk = h / p.G;
        const int krow = s * p.L + kt * kTileN;
        const bool rows_ok = in_bounds(tma_coords_ok(TmaExtent{D, p.S, p.Hk, p.B}, 0, krow, hk, b), p.ctl, 2);
        mbar_add_tx(BAR(B_V_FULL + sv), LY::kTile);
        for (int c = 0; c < D / 64; ++c)
          if (rows_ok) tma_load_4d(sb + LY::kK + sk * LY::kTile + c * kBox, &tmK, BAR(B_V_FULL + sv), c * 64, krow, hk, b);
        if (j >= kVStages &&
            !wait_one<kWaitHint>(BAR(B_V_EMPTY + sv), (j / kVStages - 1) & 1, abort_flag, p.ctl, 10)) {
          // the phase then completes once K has landed, and the drain below waits for it
          mbar_arrive(BAR(B_V_FULL + sv));
          ++issued[sv];
          return false;
        }
        mbar_expect_tx(BAR(B_V_FULL + sv), LY::kTile);
        for (int c = 0; c < D / 64; ++c)
          if (rows_ok) tma_load_4d(sb + LY::kV + sv * LY::kTile + c * kBox, &tmV, BAR(B_V_FULL + sv), c * 64, krow, hk, b);
        ++issued[sv];
        ++j;
        return true;
      });
      for (int st = 0; st < kVStages; ++st)
        if (issued[st] && !drain_one(BAR(B_V_FULL + st), (issued[st] - 1) & 1, p.ctl, 21)) *abort_flag = 1;
    }
    if (threadIdx.x == 0 && q_issued) drain_one(BAR(B_Q_FULL), 0, p.ctl, 20);
    __syncwarp();
    } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_tiles > 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, kTileN, 0, 0);  // A = Q, B = K: both K-major
      constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, 0, 1);      // A = P (TMEM), B = V: MN-major
      bool ok = wait_one<kWaitHint>(BAR(B_Q_FULL), 0, abort_flag, p.ctl, 2);
      auto issue_s = [&](int t, int j) {
        // descriptors built once and stepped (low words only: this thread runs on few registers)
        constexpr uint32_t kHi = sdesc_sw128_hi(1024);
        const uint32_t lk = sdesc_sw128_lo(sb + LY::kK + (j % kKStages) * LY::kTile, 16);
        const uint32_t lq = sdesc_sw128_lo(sb + LY::kQ + t * LY::kTile, 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
          mma_bf16_ss(tmem + LY::kTmemS + t * 128, sdesc_words(lq + off, kHi), sdesc_words(lk + off, kHi), kIdS,
                      kk > 0 ? 1u : 0u);
        }
        mma_commit(BAR(B_S_FULL + t));
      };
      auto issue_pv = [&](int t, int i) -> bool {
        if (!wait_one<kWaitHint>(BAR(B_P_FULL + t), i & 1, abort_flag, p.ctl, 3)) return false;
        tc_fence_after();
        const uint32_t lv = sdesc_sw128_lo(sb + LY::kV + (i % kVStages) * LY::kTile, kBox);
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk) {
          // A = P: 16 keys = 8 packed columns, at 0 and 64 of the S_t tile; B = V: 16 key rows = 2048 bytes
          mma_bf16_ts(tmem + LY::kTmemO + t * 128, tmem + LY::kTmemS + t * 128 + (kk < 4 ? 8 * kk : 32 + 8 * kk),
                      sdesc_words(lv + kk * 128, sdesc_sw128_hi(1024)), kIdPV, (i > 0 || kk > 0) ? 1u : 0u);
        }
        if (t == kQTiles - 1 && i + kVStages < n_tiles) mma_commit(BAR(B_V_EMPTY + i % kVStages));
        return true;
      };
      int j = 0;
      if (ok) {
        tc_fence_after();
        walk_tiles(p, cta, nkt, [&](int, int) {
          for (int t = 0; t < kQTiles; ++t) {
            // PV_t(j-1) reads P_t from the S_t columns, so it goes first; S_t(j) then overwrites them
            if (j >= 1 && !issue_pv(t, j - 1)) {
              ok = false;
              return false;
            }
            if (t == 0) {
              if (!wait_one<kWaitHint>(BAR(B_V_FULL + j % kVStages), (j / kVStages) & 1, abort_flag, p.ctl, 5)) {
                ok = false;
                return false;
              }
              tc_fence_after();
            }
            issue_s(t, j);
          }
          if (j + kKStages < n_tiles) mma_commit(BAR(B_K_EMPTY + j % kKStages));
          ++j;
          return true;
        });
        if (ok && j >= 1)
          for (int t = 0; t < kQTiles && ok; ++t) ok = issue_pv(t, j - 1);
        if (ok) mma_commit(BAR(B_O_DONE));
      }
      // every issued MMA completes before the CTA frees TMEM, or starts again
      mma_commit(BAR(B_TEARDOWN));
      if (!drain_one(BAR(B_TEARDOWN), 0, p.ctl, 23) || (ok && !drain_one(BAR(B_O_DONE), 0, p.ctl, 22))) *abort_flag = 1;
    }
    __syncwarp();
    }
    };
    // (not a loop: what it keeps from one walk to the next is too much for these few registers, 3 % of the kernel's time)
    control();
    if (fixed && again()) control();
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    regs_inc<kScoredRegsHigh>();
    const int t = (warp - 4) >> 3;           // query tile
    const int half = ((warp - 4) >> 2) & 1;  // key columns [64 half, 64 half + 64)
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + LY::kTmemS + t * 128 + 64 * half;
    const uint32_t tO = tl + LY::kTmemO + t * 128 + half * (D / 2);
    const int i = i0 + t * kTileM + row;
    bool valid = i < p.L;
    const uint32_t bound = sb + LY::kBound + 4 * (t * 128 + row);  // of the row's scores so far
    const int pair_bar = 1 + t * 4 + (warp & 3);  // the two warps of 32 rows
    constexpr float kOffset = 20.f, kSums[2] = {0x1p-45f, 0x1p44f};  // of half a row
    const uint32_t cap_table = sb + LY::kCaps;
    QRange qt;
    RowWin win;
    int gq = 0;
    if constexpr (VL) {
      gq = make_row_win(p, r, min(i, p.L - 1), false, win);
    } else {
      make_qrange(p, r, i0 + t * kTileM, kTileM, qt, pre);
      gq = tok(p, r, valid ? i : max(qt.i_last, 0));
    }
    // offset of the weights, in log2 units, and the running sum of this half's
    float m_run = fixed ? fminf(p.sc.cap2, kOffset) : -INFINITY, l_run = 0.f;
    bool ok = true, running = !fixed;
    int j = 0;
    // allowed columns [c_lo, c_hi) of the thread's 64, as bits
    auto window = [&](int s, int kt, int& c_lo, int& c_hi) {
      c_lo = 0, c_hi = kTileN;
      if constexpr (VL)
        row_win_cols(p, win, s, kt * kTileN, kTileN, c_lo, c_hi);
      else if (!kv_tile_full(p, qt, s, kt))
        row_key_window(p, seeing_token<decltype(p)>(gq, pre), s, kt, c_lo, c_hi);
      c_lo = max(c_lo - 64 * half, 0), c_hi = min(c_hi - 64 * half, 64);
      return bit_window64(c_lo, c_hi);
    };
    if constexpr ((SC & SC_CAP) != 0) {
      if (fixed) {
        const uint64_t nm2 = f32x2(-m_run, -m_run);
        const Cap<SC, 0> most_often(cap_table);
        uint64_t acc[2] = {0, 0};
        walk_tiles(p, cta, nkt, [&](int s, int kt) {
          int c_lo, c_hi;
          const uint64_t mw = window(s, kt, c_lo, c_hi);
          const bool any_masked = __any_sync(0xffffffffu, c_lo > 0 || c_hi < 64);
          BiasLine bias = {};
          bool line = true;
          if constexpr ((SC & SC_BIAS) != 0) {
            bias = bias_line(tile_tokens(p, win, s, kt * kTileN + 64 * half), gq, c_lo, c_hi, slope2);
            line = __all_sync(0xffffffffu, bias.line);
            bias.off -= m_run;
          }
          if (!wait_warp<kWaitHint>(BAR(B_S_FULL + t), j & 1, abort_flag, p.ctl, 7)) {
            ok = false;
            return false;
          }
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t v[32], pk[16];
            tmem_ld32(tS + 32 * ch, v);
            const BiasLine part = bias.from(32 * ch);
            tmem_ld_wait(v);
            const int tier = tier_of(largest(v), p.sc, line && !any_masked);
            auto weights = [&](const auto& cap, auto li, auto mask) {
              const uint32_t m32 = (uint32_t)(mw >> (32 * ch));
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                const int c = 2 * u;
                uint64_t w;
                float x0, x1;
                f32x2_split(cap(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                with_bias<SC, decltype(li)::value, decltype(li)::value>(part, c, nm2), w),
                            x0, x1);
                float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                if constexpr (decltype(mask)::value != 0)
                  e0 = (m32 >> c) & 1u ? e0 : 0.f, e1 = (m32 >> (c + 1)) & 1u ? e1 : 0.f;
                acc[u & 1] = add_f32x2(acc[u & 1], f32x2(e0, e1));
                pk[u] = pack_bf16x2(e0, e1);
              }
              tmem_st16(tS + 16 * ch, pk);
            };
            if (tier == 0 && line && !any_masked)
              weights(most_often, Const<1>{}, Const<0>{});
            else if (any_masked)
              with_score_flags<SC>(max(tier, 2), line, [&](auto ti, auto li) {
                if constexpr (decltype(ti)::value >= 2) weights(Cap<SC, decltype(ti)::value>(cap_table), li, Const<1>{});
              });
            else
              with_score_flags<SC>(max(tier, 1), line, [&](auto ti, auto li) {
                if constexpr (decltype(ti)::value >= 1) weights(Cap<SC, decltype(ti)::value>(cap_table), li, Const<0>{});
              });
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_P_FULL + t));
          ++j;
          return true;
        });
        float s0, s1;
        f32x2_split(add_f32x2(acc[0], acc[1]), s0, s1);
        l_run = s0 + s1;
        // the halves' larger sum (0: the row sees nothing)
        raise_shared(bound, to_ordered(l_run));
        named_bar_sync(pair_bar, 64);
        const float l = from_ordered(load_shared(bound));
        if (valid && ok && l > 0.f && (l < kSums[0] || l > kSums[1])) *again_flag = 1;
        __syncwarp();
        running = again();
        if (running) m_run = -INFINITY, l_run = 0.f, j = 0;
      }
    }
    if (running) walk_tiles(p, cta, nkt, [&](int s, int kt) {
      int c_lo, c_hi;
      const uint64_t mw = window(s, kt, c_lo, c_hi);
      const bool masked = c_lo > 0 || c_hi < 64;
      BiasLine bias = {};
      bool line = true, exact = false;
      if constexpr ((SC & SC_BIAS) != 0) {
        bias = bias_line(tile_tokens(p, win, s, kt * kTileN + 64 * half), gq, c_lo, c_hi, slope2);
        line = __all_sync(0xffffffffu, bias.line);
        exact = !line || __any_sync(0xffffffffu, fabsf(bias.slp) * 64.f > kLoose);
      }
      if (!wait_warp<kWaitHint>(BAR(B_S_FULL + t), j & 1, abort_flag, p.ctl, 7)) {
        // the other warp of the pair may have seen the tile: it waits for this one once more at most, since its
        // next tile needs this one's weights
        named_bar_arrive(pair_bar, 64);
        ok = false;
        return false;
      }
      tc_fence_after();
      const bool any_masked = __any_sync(0xffffffffu, masked);
      uint32_t v[64];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v + 32));
      float size = 0.f, alpha = 1.f;
      if constexpr ((SC & SC_CAP) != 0) size = largest(v);
      const int tier = (SC & SC_CAP) ? tier_of(size, p.sc, line && !any_masked) : 0;
      {
        // the largest score, or a bound of it
        float mx = -INFINITY;
        bool loose = false;  // whether the largest magnitude will do
        if constexpr ((SC & SC_CAP) != 0) {
          mx = most<SC>(p.sc, bias, size, 64);
          const float rise = (SC & SC_BIAS) ? fabsf(bias.slp) * 64.f : 0.f;
          loose = !exact && __all_sync(0xffffffffu, 2.f * most<SC & SC_CAP>(p.sc, bias, size, 64) + rise <= kLoose);
        }
        if (loose) {
          if (c_lo >= c_hi) mx = -INFINITY;
        } else if (exact) {
          mx = -INFINITY;
          auto over = [&](auto li) {
            const Cap<SC, kTiers> cap(cap_table);
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              uint64_t w;
              float z0, z1;
              f32x2_split(cap(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                              with_bias<SC, decltype(li)::value, decltype(li)::value>(bias, c, 0), w),
                          z0, z1);
              mx = fmax3f(mx, (mw >> c) & 1ull ? z0 : -INFINITY, (mw >> (c + 1)) & 1ull ? z1 : -INFINITY);
            }
          };
          if (line)
            over(Const<1>{});
          else
            over(Const<0>{});
        } else {
          float mc[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mc[q] = -INFINITY;
          if (any_masked) {
#pragma unroll
            for (int c = 0; c < 64; ++c) mc[c & 3] = fmaxf(mc[c & 3], (mw >> c) & 1ull ? __uint_as_float(v[c]) : -INFINITY);
          } else {
#pragma unroll
            for (int c = 0; c < 64; c += 2)
              mc[(c >> 1) & 3] = fmax3f(mc[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
          }
          mx = most<SC>(p.sc, bias, fmax3f(mc[0], mc[1], fmaxf(mc[2], mc[3])), 64);
        }
        raise_shared(bound, to_ordered(mx));
        named_bar_sync(pair_bar, 64);
        mx = from_ordered(load_shared(bound));
        if (mx > -INFINITY) {
          if (m_run == -INFINITY) {
            m_run = mx;  // nothing accumulated yet for this row
          } else if (mx > m_run + 8.f) {
            alpha = fast_exp2(m_run - mx);
            m_run = mx;
          }
        }
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      const uint64_t nm2 = f32x2(-m_use, -m_use);
      bias.off -= m_use;
      uint64_t acc[2] = {0, 0};
      // weights of the 64 columns and their sums; mask: of those that the row sees
      auto weights = [&](auto ti, auto li, auto mask) {
        const Cap<SC, decltype(ti)::value> cap(cap_table);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const int c = 32 * ch + 2 * u;
            uint64_t w;
            float x0, x1;
            f32x2_split(cap(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                            with_bias<SC, decltype(li)::value, decltype(li)::value>(bias, c, nm2), w),
                        x0, x1);
            float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
            if constexpr (decltype(mask)::value != 0)
              e0 = (mw >> c) & 1ull ? e0 : 0.f, e1 = (mw >> (c + 1)) & 1ull ? e1 : 0.f;
            acc[u & 1] = add_f32x2(acc[u & 1], f32x2(e0, e1));
            pk[u] = pack_bf16x2(e0, e1);
          }
          tmem_st16(tS + 16 * ch, pk);
        }
      };
      if (any_masked)
        with_score_flags<SC>(max(tier, 2), line, [&](auto ti, auto li) {
          if constexpr (decltype(ti)::value >= 2 || (SC & SC_CAP) == 0) weights(ti, li, Const<1>{});
        });
      else
        with_score_flags<SC>(tier, line, [&](auto ti, auto li) { weights(ti, li, Const<0>{}); });
      float s0, s1;
      f32x2_split(add_f32x2(acc[0], acc[1]), s0, s1);
      l_run = l_run * alpha + (s0 + s1);
      // O_t is stable here (the commit behind S_FULL covers PV_t(j-1)) and PV_t(j)
      // waits for P_FULL, so the rescale fits between them; each half takes half of the head
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(tO + c * 32, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_P_FULL + t));
      ++j;
      return true;
    });

    const long long qpos = (long long)(r * p.L + i - p.q_base);  // row of q / out / lse
    if (valid && !in_bounds(qpos >= 0 && qpos < p.q_rows, p.ctl, 3)) valid = false;  // skip this row's stores
    // varlen computed in original order: out / lse rows of the caller's layout order
    const int* rmap = VL ? p.row_map : nullptr;
    const long long opos = rmap && valid ? (long long)__ldg(rmap + qpos) : qpos;
    float* lse_ptr = p.lse + (long long)b * p.l_sb + (long long)h * p.l_sh + opos * p.l_ss;
    const long long orow = (long long)b * p.o_sb + (long long)h * p.o_sh + opos * p.o_ss + half * (D / 2);
    if (n_tiles > 0) {
      if (ok && !wait_warp<kWaitHint>(BAR(B_O_DONE), 0, abort_flag, p.ctl, 9)) {
        named_bar_arrive(pair_bar, 64);
        ok = false;
      }
      if (ok) {
        tc_fence_after();
        fence_proxy_async_smem();
        // every product is done: the operand buffers are free.  The row's sum is the halves'
        float* sums = reinterpret_cast<float*>(sp + 16 * 32 * D) + t * 256 + row;
        sums[half * 128] = l_run;
        named_bar_sync(pair_bar, 64);
        l_run = sums[0] + sums[128];
        const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
        if constexpr (!VL) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
            if (valid) {
              if (p.out_f32) {
                float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow + c * 32);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  dst[k] = make_float4(__uint_as_float(o[4 * k]) * inv_l, __uint_as_float(o[4 * k + 1]) * inv_l,
                                       __uint_as_float(o[4 * k + 2]) * inv_l, __uint_as_float(o[4 * k + 3]) * inv_l);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow + c * 32);
#pragma unroll
                for (int k = 0; k < 4; ++k) dst[k] = scaled_bf16x8(o + 8 * k, inv_l);
              }
            }
          }
        } else {
          // through shared memory, as in the plain kernel (varlen results are bf16)
          constexpr int nch = D / 16, kSwz = nch < 8 ? nch - 1 : 7;  // 16-byte pieces of half a head
          uint8_t* slot = sp + (warp - 4) * (32 * D);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(slot + lane * nch * 16 + (((c * 4 + k) ^ (lane & kSwz)) << 4)) =
                  scaled_bf16x8(o + 8 * k, inv_l);
          }
          __syncwarp();
          constexpr int rows_per = 32 / nch;
          const int pc = lane % nch;
          const int i_w = i0 + t * kTileM + (warp & 3) * 32;  // local position of the warp's first row
#pragma unroll 1
          for (int R = lane / nch; R < 32; R += rows_per) {
            const uint4 val = *reinterpret_cast<const uint4*>(slot + R * nch * 16 + ((pc ^ (R & kSwz)) << 4));
            const long long q_row = (long long)(r * p.L + i_w + R - p.q_base);
            if (i_w + R < p.L && in_bounds(q_row >= 0 && q_row < p.q_rows, p.ctl, 4)) {
              const long long o_row = rmap ? (long long)__ldg(rmap + q_row) : q_row;
              const long long e = (long long)b * p.o_sb + (long long)h * p.o_sh + o_row * p.o_ss + half * (D / 2);
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + e + pc * 8) = val;
            }
          }
        }
        if (valid && half == 0) *lse_ptr = l_run > 0.f ? (m_run + log2f(l_run)) * 0.6931471805599453f : -INFINITY;
      }
    } else if (valid) {
      // no key tile at all (a single ring step can be empty): out = 0, lse = -inf
      if (p.out_f32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow);
        for (int k = 0; k < D / 8; ++k) dst[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow);
        for (int k = 0; k < D / 16; ++k) dst[k] = make_uint4(0, 0, 0, 0);
      }
      if (half == 0) *lse_ptr = -INFINITY;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int SC, int D, bool VL>
cudaError_t launch_fwd_sdv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdParams& p,
                           const ScoreParams& sc, cudaStream_t st) {
  FwdParamsT<VL, SC> pv;
  static_cast<FwdParams&>(pv) = p;
  pv.sc = sc;
  if constexpr (SC == SC_ON) {
    return launch_fwd_v<D, VL, SC>(tq, tk, tv, pv, st);
  } else {
    using LY = ScoredFwdLayout<D>;
    cudaError_t e = configure_kernel<ring_scored_fwd_kernel<D, VL, SC>>(kScoredLaunchRegs, LY::kAlloc);
    if (e != cudaSuccess) return e;
    const int n_pairs = (p.L + kRowsPerCta - 1) / kRowsPerCta;
    dim3 grid((unsigned)((p.r_only >= 0 ? 1 : p.N) * n_pairs), (unsigned)(p.B * p.H));
    if constexpr (!VL)
      return launch_early(ring_scored_fwd_kernel<D, VL, SC>, grid, kScoredThreads, LY::kAlloc, st, tq, tk, tv, pv);
    ring_scored_fwd_kernel<D, VL, SC><<<grid, kScoredThreads, LY::kAlloc, st>>>(tq, tk, tv, pv);
    return cudaGetLastError();
  }
}

}  // namespace

template <int SC>
cudaError_t launch_fwd_score(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const FwdParams& p, const ScoreParams& sc, cudaStream_t st) {
  if (D == 64)
    return p.cu ? launch_fwd_sdv<SC, 64, true>(tq, tk, tv, p, sc, st)
                : launch_fwd_sdv<SC, 64, false>(tq, tk, tv, p, sc, st);
  return p.cu ? launch_fwd_sdv<SC, 128, true>(tq, tk, tv, p, sc, st)
              : launch_fwd_sdv<SC, 128, false>(tq, tk, tv, p, sc, st);
}

}  // namespace ra
