// What the scored kernels do to a tile's scores: the cap, and the bias by distance.
//
// A product s = q.k becomes, in log2 units (SC_CAP, SC_BIAS; a prefix changes masks only,
// ra_tiles.cuh),
//   y = cap2 tanh(s scale / softcap),  z = y - slope2 |i - j|,  P = 2^(z - max or lse),
// and a gradient with respect to z becomes one with respect to scale * s by the factor
// 1 - (y / cap2)^2.
//
// The cap.  tanh(u) = u (1 + w (c1 + w (c2 + w (c3 + w c4)))), w = u^2, on |u| <= 0.6: minimax
// coefficients, 2^-23.5 off relatively and 2^-22.4 as evaluated; the scales are folded into the
// coefficients, so that a score costs five multiply-adds, two lanes an instruction.  Beyond that
// tanh(u) = 1 - 2 / (1 + e^(2u)) with the hardware's exponential and reciprocal: right for
// every u (infinite ones too), off by about 2^-22 absolutely, and twice as many instructions of the
// special-function unit on top of the softmax's.  A warp takes the first way for the scores that it has in
// registers when none of them is beyond: caps are meant to be far above most scores.
//
// The bias.  In a tile the distance is a - st c for column c, or its negative, or (a tile
// that the row's own token, or the seam of a zigzag shard's two chunks, lies in) one line left
// and another right of column cb and the magnitude of that: the first two cost one multiply-add.
// Distances are fp32 numbers, exact up to 2^24.
#pragma once

#include "ra_tiles.cuh"

namespace ra {

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tokens of a tile's columns: t0 + st c left of column cb, t1 + st c from there on.
struct TileTokens {
  int t0, t1, st, cb;
};
constexpr int kNoSeam = 1 << 20;

// Columns: local positions [j0, ...) of shard s (win: the row's window, for varlen).
template <class P>
__device__ __forceinline__ TileTokens tile_tokens(const P& p, const RowWin& win, int s, int j0) {
  TileTokens x{s * p.L + j0, 0, 1, kNoSeam};
  if constexpr (P::kVarlen) {
    if (vz(p)) {
      const int o = j0 - win.base;
      x = TileTokens{win.first + s * win.c + o, win.first + (2 * p.N - 1 - s) * win.c + o - win.c, 1, win.c - o};
    }
  } else if (p.layout == LAYOUT_STRIPE) {
    x = TileTokens{j0 * p.N + s, 0, p.N, kNoSeam};
  } else if (p.layout == LAYOUT_ZIGZAG) {
    const int c = p.L >> 1;
    x = TileTokens{s * c + j0, (2 * p.N - 1 - s) * c + j0 - c, 1, c - j0};
  }
  return x;
}

// The bias of a row over a tile's columns, in log2 units.
struct BiasLine {
  float off, slp;         // off + slp c, where it is a line
  float a, b, st, neg;    // else neg * |(c < cb ? a : b) - st c|
  int cb;
  bool line;
};

// own: the row's token; [lo, hi): its columns that count.
__device__ __forceinline__ BiasLine bias_line(const TileTokens& x, int own, int lo, int hi, float slope2) {
  BiasLine r;
  const bool left = hi <= x.cb, right = lo >= x.cb;
  const int at = own - (left ? x.t0 : x.t1);  // distance at column c: at - st c
  const bool after = at - x.st * (hi - 1) >= 0, before = at - x.st * lo <= 0;
  r.line = lo >= hi || ((left || right) && (after || before));
  const float sg = after ? slope2 : -slope2;
  r.off = -sg * (float)at;
  r.slp = sg * (float)x.st;
  r.a = (float)(own - x.t0);
  r.b = (float)(own - x.t1);
  r.st = (float)x.st;
  r.neg = -slope2;
  r.cb = x.cb;
  return r;
}

// Constants of a tile's transformation, as the compiler keeps them in registers.
template <int SC>
struct ScoreTile {
  const ScoreParams& sc;
  BiasLine bias;

  // Two products s0, s1 of columns c, c + 1: y (capped) and z, pairs.  kSmall: |s| <= lim; kLine: bias.line.
  template <bool kSmall, bool kLine>
  __device__ __forceinline__ void operator()(int c, float s0, float s1, uint64_t& y, uint64_t& z) const {
    uint64_t b = 0;
    if constexpr ((SC & SC_BIAS) != 0) {
      float b0, b1;
      if constexpr (kLine) {
        b0 = fmaf((float)c, bias.slp, bias.off), b1 = fmaf((float)(c + 1), bias.slp, bias.off);
      } else {
        b0 = bias.neg * fabsf(fmaf(-(float)c, bias.st, c < bias.cb ? bias.a : bias.b));
        b1 = bias.neg * fabsf(fmaf(-(float)(c + 1), bias.st, c + 1 < bias.cb ? bias.a : bias.b));
      }
      b = f32x2(b0, b1);
    }
    const uint64_t s = f32x2(s0, s1);
    if constexpr ((SC & SC_CAP) == 0) {
      y = 0;  // (not asked for)
      z = (SC & SC_BIAS) ? fma_f32x2(s, f32x2(sc.c[0], sc.c[0]), b) : mul_f32x2(s, f32x2(sc.c[0], sc.c[0]));
    } else if constexpr (kSmall) {
      const uint64_t w = mul_f32x2(s, s);
      uint64_t h = fma_f32x2(w, f32x2(sc.c[4], sc.c[4]), f32x2(sc.c[3], sc.c[3]));
      h = fma_f32x2(w, h, f32x2(sc.c[2], sc.c[2]));
      h = fma_f32x2(w, h, f32x2(sc.c[1], sc.c[1]));
      h = fma_f32x2(w, h, f32x2(sc.c[0], sc.c[0]));
      y = mul_f32x2(s, h);
      z = (SC & SC_BIAS) ? fma_f32x2(s, h, b) : y;
    } else {
      float e0, e1;
      f32x2_split(mul_f32x2(s, f32x2(sc.e2, sc.e2)), e0, e1);
      const uint64_t r = f32x2(fast_rcp(fast_exp2(e0) + 1.f), fast_rcp(fast_exp2(e1) + 1.f));
      y = fma_f32x2(r, f32x2(-2.f * sc.cap2, -2.f * sc.cap2), f32x2(sc.cap2, sc.cap2));
      z = (SC & SC_BIAS) ? add_f32x2(y, b) : y;
    }
  }
};

template <bool B>
struct Flag {
  static constexpr bool value = B;
};
// f(small, line) with the flags as compile-time constants; both are the same in the whole warp.
template <int SC, class F>
__device__ __forceinline__ void with_score_flags(bool small, bool line, F&& f) {
  if (!(SC & SC_CAP) || small) {
    if (!(SC & SC_BIAS) || line)
      f(Flag<true>{}, Flag<true>{});
    else
      f(Flag<true>{}, Flag<false>{});
  } else {
    if (!(SC & SC_BIAS) || line)
      f(Flag<false>{}, Flag<true>{});
    else
      f(Flag<false>{}, Flag<false>{});
  }
}

// Whether no product of N is beyond the polynomial's range, for the whole warp.
template <int N>
__device__ __forceinline__ bool all_small(const uint32_t (&v)[N], float lim) {
  static_assert(N % 32 == 0, "chains of 16");
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    m[0] = fmax3f(m[0], fabsf(__uint_as_float(v[c])), fabsf(__uint_as_float(v[c + 1])));
    m[1] = fmax3f(m[1], fabsf(__uint_as_float(v[c + 2])), fabsf(__uint_as_float(v[c + 3])));
  }
  return !__any_sync(0xffffffffu, fmaxf(m[0], m[1]) > lim);
}

}  // namespace ra
