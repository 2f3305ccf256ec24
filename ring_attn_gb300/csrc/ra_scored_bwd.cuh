// The ring backward with capped scores or a bias by distance.  Each ra_scored_bwd_*.cu makes it for one kind
// of change, so that they compile side by side.
//
// The plain backward's two kernels (ra_bwd.cuh: their tiles, their loads and their order of products) with scores
// changed as the forward does, P for dV, and P times the cap's derivative for dS, and with an exact D (a prefix alone
// takes the plain dK / dV kernel behind the dQ kernel here).  Two threads a row, as there: four, as in the
// forward with changed scores, measured 2 % to 20 % slower, since each waits for two products a tile, not for its
// own instructions.
//
// Bound, d = 128: a tile of 128 x 128 needs 2048 cycles of the tensor cores in either kernel (four products), which are
// busy 44 (dQ) and 54 % of the time; the multiply-add pipes are for 41 and 35 %, the issue slots for 46 and 39.  The rest are
// a tile's steps that wait for one another, with tensor memory full (d = 64: dK / dV leave 128 columns).  8192 tokens
// of 32 + 8 heads of 128, softcap 30 and a prefix: dK and dV 0.89 ms (plain scores 0.79), dQ 1.02 (0.57, with three
// products); 12 documents of 200 to 4000 tokens, 16 + 4 heads, a bias: 255 and 241 us (250, 185); 2 x 4096 tokens of
// 16 heads of 64, 4 striped shards, a bias: 220 and 234 us (222, 170).
#pragma once

#include "ra_bwd.cuh"
#include "ra_score.cuh"

namespace ra {
namespace {

// ======================================================================== dK / dV
template <int D, bool VL, int SC>
__global__ void __launch_bounds__(kThreads, 1)
    ring_scored_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const BwdParamsT<VL, SC> p) {
  using LY = DkdvLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // one key / value head; with grouped-query attention its G query heads share it
  const Start start = start_of<VL, false, kTileN>(p, p.n_ktiles, -1);
  const int b = start.head / p.Hk, hk = start.head % p.Hk, ks = start.r, kj0 = start.i0;
  const uint32_t bar0 = sb + LY::kBar;
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + LY::kMisc + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + LY::kMisc);
  if (threadIdx.x == 0) {
    mbar_init(BAR(E_KV_FULL), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(E_Q_FULL + i), 1);
      mbar_init(BAR(E_Q_EMPTY + i), 1);
      mbar_init(BAR(E_DO_EMPTY + i), 1);
    }
    mbar_init(BAR(E_S_FULL), 1);
    mbar_init(BAR(E_P_FULL), 8);
    mbar_init(BAR(E_DP_FULL), 1);
    mbar_init(BAR(E_DS_FULL), 8);
    mbar_init(BAR(E_KV_DONE), 1);
    mbar_init(BAR(E_TEARDOWN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmDO);
  }
  if constexpr (!VL) after_previous_kernel();
  if (threadIdx.x == 0) {
    // the key tile's K and V depend on nothing the walk below computes: issued
    // first, their latency overlaps the CTA's set-up
    const int krow = ks * p.L + kj0;
    mbar_expect_tx(BAR(E_KV_FULL), 2 * LY::kTile);
    for (int c = 0; c < D / 64; ++c)
      if (!(p.ctl.debug_flags & DBG_SKIP_KV_LOAD) &&
          in_bounds(tma_coords_ok(TmaExtent{D, p.S, p.Hk, p.B}, c * 64, krow, hk, b), p.ctl, 10)) {
        tma_load_4d(sb + LY::kK + c * kBox, &tmK, BAR(E_KV_FULL), c * 64, krow, hk, b);
        tma_load_4d(sb + LY::kV + c * kBox, &tmV, BAR(E_KV_FULL), c * 64, krow, hk, b);
      }
  }
  KRange k;
  const int pre = VL ? 0 : prefix_now(p, b);
  make_krange(p, ks, kj0, k, kTileN, pre);
  int n_tiles = 0;  // over all query heads of the group (every head meets the same tiles)
  walk_q_tiles<kTileM>(p, k, p.n_qtiles, [&](int, int) {
    ++n_tiles;
    return true;
  });
  n_tiles *= p.G;
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_dec<kDkdvRegsLow>();
    if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && n_tiles > 0) {
      int issued[2] = {0, 0};
      int i = 0;
      auto load = [&](int h, int r, int qt) {
        const int st = i & 1;
        const uint32_t par = ((i >> 1) - 1) & 1;
        const int qrow = r * p.L + qt * kTileM - p.q_base;
        const long long stat_bh = ((long long)b * p.H + h) * p.stat_N * p.stat_L;  // (b, h, first shard)
        // dV frees the dO stage two MMA groups before dK frees the Q stage: dO
        // goes first, onto the same barrier (its bytes added without an arrival)
        if (i >= 2 && !wait_one(BAR(E_DO_EMPTY + st), par, abort_flag, p.ctl, 39)) return false;
        const bool rows_ok = in_bounds(tma_coords_ok(TmaExtent{D, p.q_rows, p.H, p.B}, 0, qrow, h, b), p.ctl, 11);
        mbar_add_tx(BAR(E_Q_FULL + st), LY::kTile);
        for (int c = 0; c < D / 64; ++c)
          if (rows_ok)
            tma_load_4d(sb + LY::kDO + st * LY::kTile + c * kBox, &tmDO, BAR(E_Q_FULL + st), c * 64, qrow, h, b);
        if (i >= 2 && !wait_one(BAR(E_Q_EMPTY + st), par, abort_flag, p.ctl, 31)) {
          // the phase then completes once dO has landed, and the drain below waits for it
          mbar_arrive(BAR(E_Q_FULL + st));
          ++issued[st];
          return false;
        }
        // -lse2 / -D of the tile's 128 query rows: 512-byte aligned in the padded layout
        const long long e0 = stat_bh + (long long)(r - p.stat_r0) * p.stat_L + qt * kTileM;
        mbar_expect_tx(BAR(E_Q_FULL + st), LY::kTile + 2 * 512);
        for (int c = 0; c < D / 64; ++c)
          if (rows_ok)
            tma_load_4d(sb + LY::kQ + st * LY::kTile + c * kBox, &tmQ, BAR(E_Q_FULL + st), c * 64, qrow, h, b);
        if (in_bounds(stat_rows_ok(p, e0), p.ctl, 12)) {
          bulk_load(sb + LY::kStats + (st * 2 + 0) * 512, p.nlse2 + e0, 512, BAR(E_Q_FULL + st));
          bulk_load(sb + LY::kStats + (st * 2 + 1) * 512, p.nD + e0, 512, BAR(E_Q_FULL + st));
        }
        ++issued[st];
        ++i;
        return true;
      };
      // (one head per key head kept apart: the producer runs on few registers)
      if (p.G == 1)
        walk_q_tiles<kTileM>(p, k, p.n_qtiles, [&](int r, int qt) { return load(hk, r, qt); });
      else
        walk_group_q_tiles<kTileM>(p, k, p.n_qtiles, hk, load);
      for (int st = 0; st < 2; ++st)
        if (issued[st]) drain_one(BAR(E_Q_FULL + st), (issued[st] - 1) & 1, p.ctl, 41);
    }
    if (lane == 0) drain_one(BAR(E_KV_FULL), 0, p.ctl, 40);  // issued at entry
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_tiles > 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, kTileM, 0, 0);  // S^T, dP^T: K-major A and B
      constexpr uint32_t kIdKV = idesc_bf16_f32(128, D, 0, 1);      // dV, dK: TMEM A, MN-major B
      // X^T = A B^T over D: A (K or V) and B (Q or dO tile) K-major in shared memory
      auto issue_t = [&](uint32_t dcol, uint32_t a, uint32_t bq) {
        const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(bq, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
          mma_bf16_ss(tmem + dcol, sdesc_add(da, off), sdesc_add(db, off), kIdS, kk > 0 ? 1u : 0u);
        }
      };
      bool ok = wait_one(BAR(E_KV_FULL), 0, abort_flag, p.ctl, 32) &&
                wait_one(BAR(E_Q_FULL), 0, abort_flag, p.ctl, 33);
      if (ok) {
        tc_fence_after();
        issue_t(LY::kTmemS, sb + LY::kK, sb + LY::kQ);
        mma_commit(BAR(E_S_FULL));
        issue_t(LY::kTmemDP, sb + LY::kV, sb + LY::kDO);
        mma_commit(BAR(E_DP_FULL));
      }
      for (int i = 0; ok && i < n_tiles; ++i) {
        const int st = i & 1, st1 = (i + 1) & 1;
        const uint32_t par1 = ((i + 1) >> 1) & 1;
        // dV += P^T dO once P^T(i) is packed over the S^T columns
        if (!wait_one(BAR(E_P_FULL), i & 1, abort_flag, p.ctl, 45)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dob = sdesc_sw128(sb + LY::kDO + st * LY::kTile, kBox, 1024);
#pragma unroll
        for (int kk = 0; kk < kTileM / 16; ++kk)
          mma_bf16_ts(tmem + LY::kTmemDV, tmem + LY::kTmemS + pcol(kk), sdesc_add(dob, kk * 2048), kIdKV,
                      (i > 0 || kk > 0) ? 1u : 0u);
        if (i + 2 < n_tiles) mma_commit(BAR(E_DO_EMPTY + st));
        if (i + 1 < n_tiles) {
          // S^T(i+1) overwrites the P^T(i) the dV MMAs above read first
          if (!wait_one(BAR(E_Q_FULL + st1), par1, abort_flag, p.ctl, 33)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_t(LY::kTmemS, sb + LY::kK, sb + LY::kQ + st1 * LY::kTile);
          mma_commit(BAR(E_S_FULL));
        }
        // dK += dS^T Q once dS^T(i) is packed over the dP^T columns
        if (!wait_one(BAR(E_DS_FULL), i & 1, abort_flag, p.ctl, 35)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dqb = sdesc_sw128(sb + LY::kQ + st * LY::kTile, kBox, 1024);
#pragma unroll
        for (int kk = 0; kk < kTileM / 16; ++kk)
          mma_bf16_ts(tmem + LY::kTmemDK, tmem + LY::kTmemDP + pcol(kk), sdesc_add(dqb, kk * 2048), kIdKV,
                      (i > 0 || kk > 0) ? 1u : 0u);
        if (i + 2 < n_tiles) mma_commit(BAR(E_Q_EMPTY + st));
        if (i + 1 == n_tiles) {
          mma_commit(BAR(E_KV_DONE));
        } else {
          // dP^T(i+1) overwrites the dS^T(i) the dK MMAs above read first (dO(i+1)
          // landed with Q(i+1), waited for before S^T(i+1))
          issue_t(LY::kTmemDP, sb + LY::kV, sb + LY::kDO + st1 * LY::kTile);
          mma_commit(BAR(E_DP_FULL));
        }
      }
      mma_commit(BAR(E_TEARDOWN));
      drain_one(BAR(E_TEARDOWN), 0, p.ctl, 42);
    }
    __syncwarp();
    }
  } else {
    regs_inc<kDkdvRegsHigh>();
    // ------------------------------------------------------------ P^T and dS^T, half a key row per thread
    const int half = (warp - 4) >> 2;  // query columns [64 half, 64 half + 64)
    const int jr = ((warp - 4) & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int j = k.j0 + jr;
    const bool valid_k = j < p.L;
    // batched: tiles classified per key tile, masks per row on partial tiles;
    // varlen: every key row's query window, set up once
    RowWin win;
    int gk = 0;
    if constexpr (VL)
      gk = make_row_win(p, k.s, min(j, p.L - 1), true, win);
    else
      gk = tok(p, k.s, valid_k ? j : k.j_last);
    bool ok = true;
    int i = 0;
    float slope2 = 0.f;  // of the query head at hand
    auto tile = [&](int r, int qt) {
      const int st = i & 1;
      // padding query rows have -lse2 = -inf and -D = 0 (P = 0, dS = 0) without a mask
      int c_lo = 0, c_hi = kTileM;
      if constexpr (VL) {
        row_win_cols(p, win, r, qt * kTileM, kTileM, c_lo, c_hi);
        if (!valid_k) c_lo = c_hi = 0;
      } else if (!q_tile_full<kTileM>(p, k, r, qt)) {
        key_query_window<kTileM>(p, valid_k, seen_token<decltype(p)>(gk, pre), r, qt, c_lo, c_hi);
      }
      c_lo -= 64 * half;
      c_hi -= 64 * half;
      const bool masked = c_lo > 0 || c_hi < 64;
      const float4* ls4 = reinterpret_cast<const float4*>(sp + LY::kStats + (st * 2 + 0) * 512) + 16 * half;
      const float4* ds4 = reinterpret_cast<const float4*>(sp + LY::kStats + (st * 2 + 1) * 512) + 16 * half;
      // waiting on the stage barrier orders this thread's statistics reads after the copy landed
      if (!wait_warp(BAR(E_S_FULL), i & 1, abort_flag, p.ctl, 36) ||
          !wait_warp(BAR(E_Q_FULL + st), (i >> 1) & 1, abort_flag, p.ctl, 44)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      uint32_t v[64];
      tmem_ld64(tl + LY::kTmemS + 64 * half, v);
      uint32_t pp[32];  // P^T, bf16 pairs
      BiasLine bias = {};
      int tier = 0;
      bool line = true;
      if constexpr ((SC & SC_BIAS) != 0) {
        bias =
            bias_line(tile_tokens(p, win, r, qt * kTileM + 64 * half), gk, max(c_lo, 0), min(c_hi, 64), slope2);
        line = __all_sync(0xffffffffu, bias.line);
      }
      if constexpr ((SC & SC_CAP) != 0) tier = score_tier(v, p.sc, line);
      // v becomes P^T times the cap's derivative
      with_score_flags<SC>(tier, line, [&](auto ti, auto li) {
        const Cap<SC, decltype(ti)::value, true> cap(p.sc);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float4 l = ls4[c / 4];
          uint64_t w;
          float x0, x1;
          f32x2_split(cap(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                          with_bias<SC, decltype(li)::value, false>(bias, c, c % 4 ? f32x2(l.z, l.w) : f32x2(l.x, l.y)),
                          w),
                      x0, x1);
          x0 = fast_exp2(x0), x1 = fast_exp2(x1);
          pp[c / 2] = pack_bf16x2(x0, x1);
          if constexpr ((SC & SC_CAP) != 0)
            f32x2_split(mul_f32x2(f32x2(x0, x1), cap.derivative(w)), x0, x1);
          v[c] = __float_as_uint(x0), v[c + 1] = __float_as_uint(x1);
        }
      });
      if (masked) {
        const uint64_t mw = bit_window64(c_lo, c_hi);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const bool m0 = (mw >> (2 * c)) & 1ull, m1 = (mw >> (2 * c + 1)) & 1ull;
          pp[c] &= (m0 ? 0xffffu : 0u) | (m1 ? 0xffff0000u : 0u);
          v[2 * c] = m0 ? v[2 * c] : 0u, v[2 * c + 1] = m1 ? v[2 * c + 1] : 0u;
        }
      }
      // P^T packed over the first 32 of the thread's 64 S^T columns (column m:
      // queries 2m, 2m + 1), the A operand of dV += P^T dO; the MMA thread then
      // computes the next tile's S^T over it
      {
        const uint32_t ts = tl + LY::kTmemS + 64 * half;
        tmem_st16(ts, *reinterpret_cast<uint32_t(*)[16]>(pp));
        tmem_st16(ts + 16, *reinterpret_cast<uint32_t(*)[16]>(pp + 16));
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(E_P_FULL));
      if (!wait_warp(BAR(E_DP_FULL), i & 1, abort_flag, p.ctl, 37)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      // dS^T = P^T * (dP^T - D), 32 dP^T columns at a time, packed over the first
      // 32 of the thread's 64 dP^T columns (a packed half is stored once the
      // columns under it are read): the A operand of dK += dS^T Q
      const uint32_t tdp = tl + LY::kTmemDP + 64 * half;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t d[32];
        tmem_ld32(tdp + 32 * hh, d);
        tmem_ld_wait(d);
        uint32_t ps[16];
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          const float4 dd = ds4[8 * hh + c4];
          const int c = 32 * hh + 4 * c4;
          const float p0 = __uint_as_float(v[c]), p1 = __uint_as_float(v[c + 1]);
          const float p2 = __uint_as_float(v[c + 2]), p3 = __uint_as_float(v[c + 3]);
          // dS^T = P^T * (dP^T + (-D)), two lanes per instruction
          float s0, s1, s2, s3;
          f32x2_split(mul_f32x2(f32x2(p0, p1), add_f32x2(f32x2(__uint_as_float(d[4 * c4]), __uint_as_float(d[4 * c4 + 1])),
                                                         f32x2(dd.x, dd.y))),
                      s0, s1);
          f32x2_split(mul_f32x2(f32x2(p2, p3), add_f32x2(f32x2(__uint_as_float(d[4 * c4 + 2]),
                                                                __uint_as_float(d[4 * c4 + 3])),
                                                         f32x2(dd.z, dd.w))),
                      s2, s3);
          ps[2 * c4] = pack_bf16x2(s0, s1);
          ps[2 * c4 + 1] = pack_bf16x2(s2, s3);
        }
        tmem_st16(tdp + 16 * hh, ps);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(E_DS_FULL));
      ++i;
      return true;
    };
    // every query head of the group meets the same tiles; the walk does not depend on the head
    for (int g = 0; ok && g < p.G; ++g) {
      if constexpr ((SC & SC_BIAS) != 0) slope2 = load_now(p.sc.slopes + hk * p.G + g) * 1.4426950408889634f;
      walk_q_tiles<kTileM>(p, k, p.n_qtiles, tile);
    }
    // ---------------- epilogue: warpgroup 1 writes the dV rows, warpgroup 2 the dK rows
    const long long prow = (long long)k.s * p.L + j;
    const int* rmap = VL ? p.row_map : nullptr;  // varlen in original order: rows of the caller's layout
    __nv_bfloat16* base = half == 0 ? reinterpret_cast<__nv_bfloat16*>(p.dv) + (long long)b * p.v_sb +
                                          (long long)hk * p.v_sh
                                    : reinterpret_cast<__nv_bfloat16*>(p.dk) + (long long)b * p.k_sb +
                                          (long long)hk * p.k_sh;
    const long long pitch = half == 0 ? p.v_ss : p.k_ss;
    if (n_tiles > 0) {
      if (ok && wait_warp(BAR(E_KV_DONE), 0, abort_flag, p.ctl, 38)) {
        tc_fence_after();
        // every MMA is done: the operand buffers hold the warps' row slots
        fence_proxy_async_smem();
        const int j_w = j - lane;  // the warp's first key row
        const int nvalid = min(max(p.L - j_w, 0), 32);
        const long long row_w = (long long)k.s * p.L + j_w;  // the warp's first row of dk / dv
        if (in_bounds(nvalid == 0 || (row_w >= 0 && row_w + nvalid <= p.S), p.ctl, 14))
          store_rows_bf16<D / 32>(tl + (half == 0 ? LY::kTmemDV : LY::kTmemDK), half == 0 ? 1.f : p.scale,
                                  sp + (warp - 4) * (32 * D * 2), base, pitch, row_w, nvalid, rmap);
      }
    } else if (valid_k && in_bounds(prow >= 0 && prow < p.S, p.ctl, 15)) {
      __nv_bfloat16* dst = base + (rmap ? (long long)__ldg(rmap + prow) : prow) * pitch;
      for (int u = 0; u < D / 8; ++u) reinterpret_cast<uint4*>(dst)[u] = make_uint4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ======================================================================== dQ
// D = rowsum(dO * O) comes from the bf16 out, and O's rounding is an error of D that the sums over a row's keys do not
// average away: where a bias or a small cap leaves a row few keys, dP - D is small next to dP, and dQ and dK
// were off by up to 0.54 % (one head with a slope of 1).  Since the weights of a row sum to 1, the dQ pass gets the
// missing part for a multiply-add a score:
//   e = sum_j P_ij (dP_ij - D_i),  D_i + e is exact,  dQ_i = scale (sum_j dS_ij k_j - e sum_j P'_ij k_j)
// (P': P times the cap's derivative), for which it keeps a second product's sum.  It runs first and corrects the
// statistics for the dK / dV pass.  (A pass of its own for sum P dP, two products more, took 0.52 ms at 8192 tokens of
// 32 + 8 heads of 128, where this takes 0.31 ms.)
//
// That holds for a row whose keys are all here.  A call may also have a block of a row's keys, with out and lse of the
// whole row (a ring whose blocks are called one by one): its weights sum to less, and D stays as the given out has it,
// as in the plain backward.  kWholeRow is by how much a sum may miss 1: keys of that weight elsewhere put at most
// as much of dP - D into D, a quarter of what dS is rounded by, and lse's own rounding stays below it up to 2^11.  The
// sum of the weights costs dQ 1 to 2 % (d = 64: 4 %; added up while dP is awaited it cost 3.5 and 3 %).
//
// dS is rounded to bf16 as an operand, and since a row's dS nearly cancel in its sum, the rounding errors weigh more
// than they do in each: 0.182 % of dQ at softcap 30, 0.199 % at 15, where one rounding is 0.166 %.  Most of that is the sum
// of a row's errors times what its keys have in common, so that is taken off by P' K too: the sum of the rounded dS less
// the sum of dS joins e (as if P' summed to 1, which caps nearly leave).  With the rounding of dQ itself it is off by
// 0.22 and 0.23 %, 0.25 and 0.26 without.  It costs dQ 3 to 5 % (short rows of 64: 11 %).
//
// TMEM: S [0, 128), dP [128, 256).  d = 128: the sums of dS K and of P' K take the rest, so that Q and dO stay in shared
// memory; d = 64: as in the plain kernel, with the second sum behind the first.  P' is packed beside dS, over the
// second 32 of a thread's 64 dP columns.
constexpr float kWholeRow = 0x1p-10f;
template <int D>
struct ScoredDqLayout : DqLayout<D> {
  using Base = DqLayout<D>;
  static constexpr bool kQInTmem = D == 64;
  static constexpr int kSums = Base::kMisc + 16;  // 2 halves x 128 rows
  static constexpr int kAlloc = kSums + 1024 + 1024;
  static constexpr uint32_t kTmemDQ = kQInTmem ? 384 : 256, kTmemPK = kTmemDQ + D;
};

template <int D, bool VL, int SC>
__global__ void __launch_bounds__(kThreads, 1)
    ring_scored_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const BwdParamsT<VL, SC> p) {
  using LY = ScoredDqLayout<D>;
  constexpr int KS = LY::kKStages, VS = LY::kVStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Start start = start_of<VL, true, kTileM>(p, p.n_qtiles, p.r_only);
  const int b = start.head / p.H, h = start.head % p.H, r = start.r, i0 = start.i0;
  const int hk = h / p.G;  // the key / value head of query head h (grouped-query attention)
  const uint32_t bar0 = sb + LY::kBar;
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + LY::kMisc + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + LY::kMisc);
  if (threadIdx.x == 0) {
    mbar_init(BAR(F_QDO_FULL), 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(BAR(F_K_EMPTY + i), 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(BAR(F_V_FULL + i), 1);
      mbar_init(BAR(F_V_EMPTY + i), 1);
    }
    mbar_init(BAR(F_S_FULL), 1);
    mbar_init(BAR(F_S_READ), 8);
    mbar_init(BAR(F_DP_FULL), 1);
    mbar_init(BAR(F_DS_FULL), 8);
    mbar_init(BAR(F_QDO_TMEM), 8);
    mbar_init(BAR(F_DQ_DONE), 1);
    mbar_init(BAR(F_TEARDOWN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmDO);
  }
  if constexpr (!VL) after_previous_kernel();
  if (threadIdx.x == 0) {
    // the tile's Q and dO depend on nothing the tile walk below computes:
    // issued first, their latency overlaps the CTA's set-up
    const int qrow = r * p.L + i0 - p.q_base;
    mbar_expect_tx(BAR(F_QDO_FULL), 2 * LY::kTile);
    for (int c = 0; c < D / 64; ++c)
      if (!(p.ctl.debug_flags & DBG_SKIP_QDO_LOAD) &&
          in_bounds(tma_coords_ok(TmaExtent{D, p.q_rows, p.H, p.B}, c * 64, qrow, h, b), p.ctl, 16)) {
        tma_load_4d(sb + LY::kQ + c * kBox, &tmQ, BAR(F_QDO_FULL), c * 64, qrow, h, b);
        tma_load_4d(sb + LY::kDO + c * kBox, &tmDO, BAR(F_QDO_FULL), c * 64, qrow, h, b);
      }
  }
  QRange qr;
  const int pre = VL ? 0 : prefix_now(p, b);
  make_qrange(p, r, i0, kTileM, qr, pre);
  const int nkt = (p.L + kTileN - 1) / kTileN;
  int n_tiles = 0;
  walk_kv_tiles(p, qr, nkt, 0, p.N, [&](int, int) {
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

  if (warp < 4) regs_dec<kDkdvRegsLow>();
  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ TMA producers
    if (warp == 0 && lane == 0 && n_tiles > 0) {
      // K(j) and V(j) land on one barrier (the V stage's): the MMA thread
      // waits once per key tile
      int issued[2] = {0, 0};
      int j = 0;
      walk_kv_tiles(p, qr, nkt, 0, p.N, [&](int s, int kt) {
        const int sk = j % KS, sv = j % VS;
        if (j >= KS && !wait_one(BAR(F_K_EMPTY + sk), (j / KS - 1) & 1, abort_flag, p.ctl, 51)) return false;
        if (j >= VS && !wait_one(BAR(F_V_EMPTY + sv), (j / VS - 1) & 1, abort_flag, p.ctl, 52)) return false;
        mbar_expect_tx(BAR(F_V_FULL + sv), 2 * LY::kTile);
        for (int c = 0; c < D / 64; ++c)
          if (in_bounds(tma_coords_ok(TmaExtent{D, p.S, p.Hk, p.B}, c * 64, s * p.L + kt * kTileN, hk, b), p.ctl,
                        17)) {
            tma_load_4d(sb + LY::kK + sk * LY::kTile + c * kBox, &tmK, BAR(F_V_FULL + sv), c * 64,
                        s * p.L + kt * kTileN, hk, b);
            tma_load_4d(sb + LY::kV + sv * LY::kTile + c * kBox, &tmV, BAR(F_V_FULL + sv), c * 64,
                        s * p.L + kt * kTileN, hk, b);
          }
        ++issued[sv];
        ++j;
        return true;
      });
      for (int st = 0; st < VS; ++st)
        if (issued[st]) drain_one(BAR(F_V_FULL + st), (issued[st] - 1) & 1, p.ctl, 54);
    }
    if (threadIdx.x == 0) drain_one(BAR(F_QDO_FULL), 0, p.ctl, 53);  // issued at entry
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_tiles > 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, kTileN, 0, 0);  // S = Q K^T, dP = dO V^T: TMEM A, K-major B
      constexpr uint32_t kIdQ = idesc_bf16_f32(128, D, 0, 1);       // dQ += dS K: TMEM A, MN-major B
      bool ok = wait_one(BAR(LY::kQInTmem ? F_QDO_TMEM : F_QDO_FULL), 0, abort_flag, p.ctl, 55);
      // X = A B^T over D with A (Q or dO) packed in TMEM, 16 head-dim columns = 8 TMEM columns per step, or in
      // shared memory, K-major like B
      auto issue_t = [&](uint32_t dcol, uint32_t acol, uint32_t at, uint32_t bt) {
        const uint64_t da = sdesc_sw128(at, 16, 1024), db = sdesc_sw128(bt, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
          if constexpr (LY::kQInTmem)
            mma_bf16_ts(tmem + dcol, tmem + acol + 8 * kk, sdesc_add(db, off), kIdS, kk > 0 ? 1u : 0u);
          else
            mma_bf16_ss(tmem + dcol, sdesc_add(da, off), sdesc_add(db, off), kIdS, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_s = [&](int j) -> bool {
        const int ks = j % KS;
        if (!wait_one(BAR(F_V_FULL + j % VS), (j / VS) & 1, abort_flag, p.ctl, 56)) return false;
        if (j > 0 && !wait_one(BAR(F_S_READ), (j - 1) & 1, abort_flag, p.ctl, 57)) return false;
        tc_fence_after();
        issue_t(LY::kTmemS, LY::kTmemQ, sb + LY::kQ, sb + LY::kK + ks * LY::kTile);
        mma_commit(BAR(F_S_FULL));
        return true;
      };
      // dP(j) overwrites dS(j-1), which the dQ MMA issued before it has read
      auto issue_dp = [&](int j) -> bool {
        const int vs = j % VS;  // V(j) landed with K(j), waited for before S(j)
        issue_t(LY::kTmemDP, LY::kTmemDO, sb + LY::kDO, sb + LY::kV + vs * LY::kTile);
        mma_commit(BAR(F_DP_FULL));
        if (j + VS < n_tiles) mma_commit(BAR(F_V_EMPTY + vs));
        return true;
      };
      auto issue_dq = [&](int j) -> bool {
        if (!wait_one(BAR(F_DS_FULL), j & 1, abort_flag, p.ctl, 59)) return false;
        tc_fence_after();
        const uint64_t dkb = sdesc_sw128(sb + LY::kK + (j % KS) * LY::kTile, kBox, 1024);
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk) {
          // A = dS (16 keys = 8 packed columns of the dP region), B = K with 16 key rows per step
          mma_bf16_ts(tmem + LY::kTmemDQ, tmem + LY::kTmemDP + pcol(kk), sdesc_add(dkb, kk * 2048),
                      kIdQ, (j > 0 || kk > 0) ? 1u : 0u);
        }
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk)  // P' K
          mma_bf16_ts(tmem + LY::kTmemPK, tmem + LY::kTmemDP + pcol(kk) + 32, sdesc_add(dkb, kk * 2048), kIdQ,
                      (j > 0 || kk > 0) ? 1u : 0u);
        if (j + KS < n_tiles) mma_commit(BAR(F_K_EMPTY + j % KS));
        return true;
      };
      if (ok) {
        tc_fence_after();
        ok = issue_s(0) && issue_dp(0);
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (j + 1 < n_tiles) ok = issue_s(j + 1);
          ok = ok && issue_dq(j);
          if (ok && j + 1 < n_tiles) ok = issue_dp(j + 1);
        }
        if (ok) mma_commit(BAR(F_DQ_DONE));
      }
      mma_commit(BAR(F_TEARDOWN));
      drain_one(BAR(F_TEARDOWN), 0, p.ctl, 60);
    }
    __syncwarp();
  } else if (warp >= 4) {
    regs_inc<kDkdvRegsHigh>();
    // ------------------------------------------------------------ P and dS, half a query row per thread
    const int half = (warp - 4) >> 2;  // key columns [64 half, 64 half + 64)
    const int row = ((warp - 4) & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int i = i0 + row;
    const bool valid = i < p.L;
    // batched: tiles classified per query tile; varlen: every row's key window, set up once
    RowWin win;
    int gq = 0;
    if constexpr (VL)
      gq = make_row_win(p, r, min(i, p.L - 1), false, win);
    else
      gq = tok(p, r, valid ? i : max(qr.i_last, 0));
    // this row's statistics, negated (padding rows: -lse2 = -inf, -D = 0, so P = dS = 0)
    const long long srow = (((long long)b * p.H + h) * p.stat_N + (r - p.stat_r0)) * p.stat_L + i;
    const float nl = load_now(p.nlse2 + srow);
    const uint64_t nl2 = f32x2(nl, nl);
    const float nD = p.nD[srow];
    const uint64_t nD2 = f32x2(nD, nD);
    float slope2 = 0.f;
    if constexpr ((SC & SC_BIAS) != 0) slope2 = load_now(p.sc.slopes + h) * 1.4426950408889634f;
    // warpgroup 1 copies the row's Q, warpgroup 2 its dO, into tensor memory as
    // packed bf16 (column m: head-dim elements 2m, 2m + 1) for the S and dP MMAs
    bool ok = n_tiles == 0 || !LY::kQInTmem || wait_warp(BAR(F_QDO_FULL), 0, abort_flag, p.ctl, 64);
    if (LY::kQInTmem && ok && n_tiles > 0) {
      const uint8_t* src = sp + (half == 0 ? LY::kQ : LY::kDO);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          // 128-byte swizzle: 16-byte chunk q of row `row` sits at chunk q ^ (row & 7)
          const uint4 x = *reinterpret_cast<const uint4*>(src + c * kBox + row * 128 + ((q ^ (row & 7)) << 4));
          w[4 * q] = x.x;
          w[4 * q + 1] = x.y;
          w[4 * q + 2] = x.z;
          w[4 * q + 3] = x.w;
        }
        tmem_st32(tl + (half == 0 ? LY::kTmemQ : LY::kTmemDO) + 32 * c, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(F_QDO_TMEM));
    }
    // sums of P (dP - D), of P, of dS as rounded, and (cap; else the first) of dS
    uint64_t miss[2] = {0, 0}, weights = 0, rounded = 0, exact = 0;
    int j = 0;
    if (ok) walk_kv_tiles(p, qr, nkt, 0, p.N, [&](int s, int kt) {
      int c_lo = 0, c_hi = kTileN;
      if constexpr (VL)
        row_win_cols(p, win, s, kt * kTileN, kTileN, c_lo, c_hi);
      else if (!kv_tile_full(p, qr, s, kt))
        row_key_window(p, seeing_token<decltype(p)>(gq, pre), s, kt, c_lo, c_hi);
      c_lo -= 64 * half;
      c_hi -= 64 * half;
      const bool masked = c_lo > 0 || c_hi < 64;
      if (!wait_warp(BAR(F_S_FULL), j & 1, abort_flag, p.ctl, 61)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      uint32_t v[64];
      tmem_ld64(tl + LY::kTmemS + 64 * half, v);
      // S is in registers: the MMA thread may compute the next tile's S over it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(F_S_READ));
      BiasLine bias = {};
      int tier = 0;
      bool line = true;
      if constexpr ((SC & SC_BIAS) != 0) {
        bias = bias_line(tile_tokens(p, win, s, kt * kTileN + 64 * half), gq, max(c_lo, 0), min(c_hi, 64), slope2);
        line = __all_sync(0xffffffffu, bias.line);
        bias.off += nl;
      }
      if constexpr ((SC & SC_CAP) != 0) tier = score_tier(v, p.sc, line);
      uint32_t g[(SC & SC_CAP) != 0 ? 64 : 1];  // P times the cap's derivative
      with_score_flags<SC>(tier, line, [&](auto ti, auto li) {
        const Cap<SC, decltype(ti)::value, true> cap(p.sc);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          uint64_t w;
          float x0, x1;
          f32x2_split(cap(f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                          with_bias<SC, decltype(li)::value, decltype(li)::value>(bias, c, nl2), w),
                      x0, x1);
          x0 = fast_exp2(x0), x1 = fast_exp2(x1);
          v[c] = __float_as_uint(x0), v[c + 1] = __float_as_uint(x1);
          if constexpr ((SC & SC_CAP) != 0) {
            f32x2_split(mul_f32x2(f32x2(x0, x1), cap.derivative(w)), x0, x1);
            g[c] = __float_as_uint(x0), g[c + 1] = __float_as_uint(x1);
          }
        }
      });
      if (masked) {
        const uint64_t mw = bit_window64(c_lo, c_hi);
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          v[c] = ((mw >> c) & 1ull) ? v[c] : 0u;
          if constexpr ((SC & SC_CAP) != 0) g[c] = ((mw >> c) & 1ull) ? g[c] : 0u;
        }
      }
      uint32_t pp[32];  // P', packed while dP is on its way
#pragma unroll
      for (int m = 0; m < 32; ++m) {
        if constexpr ((SC & SC_CAP) != 0)
          pp[m] = pack_bf16x2(__uint_as_float(g[2 * m]), __uint_as_float(g[2 * m + 1]));
        else
          pp[m] = pack_bf16x2(__uint_as_float(v[2 * m]), __uint_as_float(v[2 * m + 1]));
      }
      if (!wait_warp(BAR(F_DP_FULL), j & 1, abort_flag, p.ctl, 62)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      // dS = P' * (dP - D), packed too (column m: keys 2m, 2m + 1): both over this thread's 64 dP columns once these
      // are read
      const uint32_t tdp = tl + LY::kTmemDP + 64 * half;
      uint32_t ds[32];
      uint64_t in_tile = 0;  // (single weights of a long row are too small next to 1)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t d[32];
        tmem_ld32(tdp + 32 * hh, d);
        tmem_ld_wait(d);
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int c = 32 * hh + 2 * u;
          const uint64_t pair = f32x2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
          const uint64_t diff = add_f32x2(f32x2(__uint_as_float(d[2 * u]), __uint_as_float(d[2 * u + 1])), nD2);
          miss[u & 1] = fma_f32x2(pair, diff, miss[u & 1]);
          in_tile = add_f32x2(in_tile, pair);
          uint64_t grad = pair;
          if constexpr ((SC & SC_CAP) != 0) grad = f32x2(__uint_as_float(g[c]), __uint_as_float(g[c + 1]));
          grad = mul_f32x2(grad, diff);
          if constexpr ((SC & SC_CAP) != 0) exact = add_f32x2(exact, grad);
          float s0, s1;
          f32x2_split(grad, s0, s1);
          ds[c / 2] = pack_bf16x2(s0, s1);
        }
      }
      weights = add_f32x2(weights, in_tile);
      tmem_st32(tdp, ds);
      tmem_st32(tdp + 32, pp);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(F_DS_FULL));
#pragma unroll
      for (int m = 0; m < 32; ++m)
        rounded = add_f32x2(rounded, f32x2(__uint_as_float(ds[m] << 16), __uint_as_float(ds[m] & 0xffff0000u)));
      ++j;
      return true;
    });
    // a row's sums over both halves (every warp of a pair comes here, whatever happened before)
    float* sums = reinterpret_cast<float*>(sp + LY::kSums) + row;
    auto of_row = [&](uint64_t x) -> float {
      float x0, x1;
      f32x2_split(x, x0, x1);
      sums[half * 128] = x0 + x1;
      named_bar_sync(1 + (warp & 3), 64);
      const float all = sums[0] + sums[128];
      named_bar_sync(1 + (warp & 3), 64);
      return all;
    };
    const float sum = of_row(add_f32x2(miss[0], miss[1]));
    const float missing = fabsf(of_row(weights) - 1.f) <= kWholeRow ? sum : 0.f;
    const float too_much = of_row(rounded) - ((SC & SC_CAP) != 0 ? of_row(exact) : sum);
    if (half == 0 && valid && ok) const_cast<float*>(p.nD)[srow] = nD - missing;
    // ---------------- epilogue: dQ = scale * (dS K - (missing + too_much) P' K), half the head dim per thread
    const int* rmap = VL ? p.row_map : nullptr;  // varlen in original order: rows of the caller's layout
    __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(p.dq) + (long long)b * p.q_sb + (long long)h * p.q_sh +
                          half * (D / 2);
    const long long qrow = (long long)r * p.L + i - p.q_base;
    if (n_tiles > 0) {
      if (ok && wait_warp(BAR(F_DQ_DONE), 0, abort_flag, p.ctl, 63)) {
        tc_fence_after();
        // every MMA is done: the operand buffers hold the warps' row slots
        fence_proxy_async_smem();
        const int i_w = i - lane;  // the warp's first query row
        const int nvalid = min(max(p.L - i_w, 0), 32);
        const long long row_w = (long long)r * p.L + i_w - p.q_base;  // the warp's first row of dq
        if (in_bounds(nvalid == 0 || (row_w >= 0 && row_w + nvalid <= p.q_rows), p.ctl, 18))
          store_rows_bf16<D / 64, true>(tl + LY::kTmemDQ + half * (D / 2), p.scale, sp + (warp - 4) * (32 * D), base,
                                        p.q_ss, row_w, nvalid, rmap, tl + LY::kTmemPK + half * (D / 2), missing + too_much);
      }
    } else if (valid && in_bounds(qrow < p.q_rows, p.ctl, 19)) {
      __nv_bfloat16* dst = base + (rmap ? (long long)__ldg(rmap + qrow) : qrow) * p.q_ss;
      for (int u = 0; u < D / 16; ++u) reinterpret_cast<uint4*>(dst)[u] = make_uint4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int SC, int D, bool VL>
cudaError_t launch_bwd_sdv(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                           const BwdParams& p, const ScoreParams& sc, int which, cudaStream_t st) {
  BwdParamsT<VL, SC> pv;
  static_cast<BwdParams&>(pv) = p;
  pv.sc = sc;
  // the register splits inside the kernels are only safe with the launch allocation they were sized for
  if (which == 1) {
    using LY = ScoredDqLayout<D>;
    cudaError_t e = configure_kernel<ring_scored_dq_kernel<D, VL, SC>>(kDkdvLaunchRegs, LY::kAlloc);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)((p.r_only >= 0 ? 1 : p.N) * p.n_qtiles), (unsigned)(p.B * p.H));
    if constexpr (!VL)
      return launch_early(ring_scored_dq_kernel<D, VL, SC>, grid, kThreads, LY::kAlloc, st, tq, tk, tv, tdo, pv);
    ring_scored_dq_kernel<D, VL, SC><<<grid, kThreads, LY::kAlloc, st>>>(tq, tk, tv, tdo, pv);
  } else if constexpr (SC == SC_ON) {
    return launch_dkdv_v<D, VL, SC>(tq, tk, tv, tdo, pv, st);
  } else {
    cudaError_t e = configure_kernel<ring_scored_dkdv_kernel<D, VL, SC>>(kDkdvLaunchRegs, DkdvLayout<D>::kAlloc);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(p.N * p.n_ktiles), (unsigned)(p.B * p.Hk));
    if constexpr (!VL)
      return launch_early(ring_scored_dkdv_kernel<D, VL, SC>, grid, kThreads, DkdvLayout<D>::kAlloc, st, tq, tk, tv, tdo, pv);
    ring_scored_dkdv_kernel<D, VL, SC><<<grid, kThreads, DkdvLayout<D>::kAlloc, st>>>(tq, tk, tv, tdo, pv);
  }
  return cudaGetLastError();
}

}  // namespace

template <int SC>
cudaError_t launch_bwd_score(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tdo, const BwdParams& p, const ScoreParams& sc, int which,
                             cudaStream_t st) {
  if (D == 64)
    return p.cu ? launch_bwd_sdv<SC, 64, true>(tq, tk, tv, tdo, p, sc, which, st)
                : launch_bwd_sdv<SC, 64, false>(tq, tk, tv, tdo, p, sc, which, st);
  return p.cu ? launch_bwd_sdv<SC, 128, true>(tq, tk, tv, tdo, p, sc, which, st)
              : launch_bwd_sdv<SC, 128, false>(tq, tk, tv, tdo, p, sc, which, st);
}

}  // namespace ra
