// What the scored kernels do to a tile's scores: the cap, and the bias by distance.
//
// A product s = q.k becomes, in log2 units (SC_CAP, SC_BIAS; a prefix changes masks only,
// ra_tiles.cuh),
//   y = cap2 tanh(s scale / softcap),  z = y - slope2 |i - j|,  P = 2^(z - max or lse),
// and a gradient with respect to z becomes one with respect to scale * s by the factor
// 1 - (y / cap2)^2.
//
// The cap.  tanh(u) = u (1 + w P(w)), w = u^2, with P of degree 2, 3 or 5 for |u| up to 0.4, 0.6 or 1: minimax
// coefficients, off relatively by 2^-23.1, 2^-23.5, 2^-24.1 (2^-22.4 as evaluated).  The scales are folded into
// the coefficients, so that a score costs five, six or eight multiply-adds where a plain one costs one, and
// they are what the kernels with a cap wait for: a multiply-add takes a cycle of its pipe for every 32
// scores, in pairs or not, the exponential four.  The derivative is 1 + w G(w) with G of degree 1, 2 or 4, off
// by 2^-14.1, 2^-15.4, 2^-16.7, next to the half step of bf16 (2^-8) that the gradient is rounded by as an operand.
// Beyond 1, tanh(u) = 1 - 2 / (1 + e^(2u)) with the hardware's exponential and reciprocal (4 and 8 cycles on top
// of the softmax's 4): right for every u, infinite ones too, off by about 2^-22 absolutely.  The backward takes e^(-2|u|)
// there, e, and the derivative as 4 e / (1 + e)^2, which keeps its bits where tanh is next to 1 (from the rounded tanh,
// 1 - tanh^2 is off by 4 % at |u| = 7 and by all of it at 9).
// A warp goes by the largest score that it has in registers: caps are meant to be far above most scores.
// (Coefficients have powers of scale / softcap up to the twelfth.  Where those leave fp32's range a polynomial holds
// up to a smaller u, or not at all: ScoreParams::lim.)
//
// The bias.  In a tile the distance is a - st c for column c, or its negative, or (a tile
// that the row's own token, or the seam of a zigzag shard's two chunks, lies in) one line left
// and another right of column cb and the magnitude of that: the first two cost one multiply-add.
// Distances are fp32 numbers, exact up to 2^24.
#pragma once

#include "ra_early.cuh"
#include "ra_tiles.cuh"

namespace ra {

// Eight fp32 numbers times mul, as bf16.
__device__ __forceinline__ uint4 scaled_bf16x8(const uint32_t* o, float mul) {
  auto two = [&](int i) { return pack_bf16x2(__uint_as_float(o[i]) * mul, __uint_as_float(o[i + 1]) * mul); };
  return make_uint4(two(0), two(2), two(4), two(6));
}

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

// A softmax's offset may be this much (log2 units) above the largest score: that one's products with values of 2^-60
// are then still normal numbers, and those of smaller weights as far as they count.  (So bounds are fp32 numbers wherever they are kept: those of steep
// biases are 2^14 and more, and with the bits of bf16 they would be off by that much themselves.)
constexpr float kLoose = 48.f;

// Numbers (no NaN) as integers in the same order, and a word of shared memory that is raised to the larger.
__device__ __forceinline__ int to_ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
__device__ __forceinline__ void raise_shared(uint32_t at, int x) {
  asm volatile("red.shared.max.s32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ int load_shared(uint32_t at) {
  int x;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

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
  // The same for columns counted from c0.
  __device__ __forceinline__ BiasLine from(int c0) const {
    const float f = (float)c0;
    return BiasLine{fmaf(f, slp, off), slp, fmaf(-f, st, a), fmaf(-f, st, b), st, neg, cb - c0, line};
  }
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

template <int N>
__device__ __forceinline__ uint64_t polynomial(uint64_t w, const uint64_t (&c)[N]) {
  uint64_t h = c[N - 1];
#pragma unroll
  for (int i = N - 2; i >= 0; --i) h = fma_f32x2(w, h, c[i]);
  return h;
}

// The constants of the caps, each twice for the two lanes of a packed instruction, in shared memory, for kernels
// short of registers: there the assembler makes pairs of kernel parameters anew next to their uses, two moves for a
// multiply-add of two scores, while pairs that are loaded stay (16,384 tokens capped: 1.82 ms, 1.88 without).
constexpr int kCapConsts = 20;
constexpr int kCapTable = 8 * kCapConsts;  // bytes
__device__ __forceinline__ void fill_cap_table(uint8_t* table, const ScoreParams& sc) {
  const int i = threadIdx.x;
  if (i >= kCapConsts) return;
  float x;
  if (i < 4)
    x = sc.t0[i];
  else if (i < 9)
    x = sc.t1[i - 4];
  else if (i < 16)
    x = sc.t2[i - 9];
  else
    x = i == 16 ? sc.e2 : i == 17 ? -2.f * sc.cap2 : i == 18 ? sc.cap2 : sc.c0;
  reinterpret_cast<float2*>(table)[i] = make_float2(x, x);
}
__device__ __forceinline__ uint64_t cap_const(uint32_t table, int i) {
  uint64_t v;
  asm volatile("ld.volatile.shared.b64 %0, [%1];" : "=l"(v) : "r"(table + 8 * i));
  return v;
}

// Scores without their bias: the cap, or the plain scale.  kTier: the polynomial that holds for all of the warp's
// products (kTiers: none).  kGrad: with the derivative.  It is made from the parameters or the table's address.
template <int SC, int kTier, bool kGrad = false>
struct Cap {
  static constexpr bool kCap = (SC & SC_CAP) != 0, kAny = kTier == kTiers;
  static constexpr int kT = !kCap ? 1 : kAny ? 3 : kTier == 0 ? 4 : kTier == 1 ? 5 : 7;
  static constexpr int kG = !kCap || !kGrad || kAny ? 1 : kTier == 0 ? 2 : kTier == 1 ? 3 : 5;
  uint64_t t[kT], g[kG];

  __device__ __forceinline__ explicit Cap(const ScoreParams& sc) {
    auto two = [](float x) { return f32x2(x, x); };
    if constexpr (!kCap) {
      t[0] = two(sc.c0);
    } else if constexpr (kAny) {
      t[0] = two(sc.e2), t[1] = two(-2.f * sc.cap2), t[2] = two(sc.cap2);
    } else {
#pragma unroll
      for (int i = 0; i < kT; ++i) t[i] = two(kTier == 0 ? sc.t0[i % 4] : kTier == 1 ? sc.t1[i % 5] : sc.t2[i % 7]);
#pragma unroll
      for (int i = 0; i < kG; ++i) g[i] = two(kTier == 0 ? sc.g0[i % 2] : kTier == 1 ? sc.g1[i % 3] : sc.g2[i % 5]);
    }
  }
  __device__ __forceinline__ explicit Cap(uint32_t table) {
    static_assert(!kGrad, "the derivative's coefficients are not in the table");
    constexpr int at = !kCap ? 19 : kAny ? 16 : kTier == 0 ? 0 : kTier == 1 ? 4 : 9;
#pragma unroll
    for (int i = 0; i < kT; ++i) t[i] = cap_const(table, at + i);
  }
  // Two products s: their scores + add, and w, from which their derivatives follow (kAny: the derivatives).
  __device__ __forceinline__ uint64_t operator()(uint64_t s, uint64_t add, uint64_t& w) const {
    if constexpr (!kCap) {
      w = 0;
      return fma_f32x2(s, t[0], add);
    } else if constexpr (!kAny) {
      w = mul_f32x2(s, s);
      return fma_f32x2(s, polynomial(w, t), add);
    } else if constexpr (kGrad) {
      float a0, a1, m0, m1;
      f32x2_split(mul_f32x2(s, t[0]), a0, a1);
      const float e0 = fast_exp2(-fabsf(a0)), e1 = fast_exp2(-fabsf(a1));
      const uint64_t e = f32x2(e0, e1), r = f32x2(fast_rcp(e0 + 1.f), fast_rcp(e1 + 1.f));
      const uint64_t r2 = add_f32x2(r, r);
      w = mul_f32x2(mul_f32x2(e, r2), r2);
      f32x2_split(fma_f32x2(r, t[1], t[2]), m0, m1);
      return add_f32x2(f32x2(copysignf(m0, a0), copysignf(m1, a1)), add);
    } else {
      float e0, e1;
      f32x2_split(mul_f32x2(s, t[0]), e0, e1);
      w = fma_f32x2(f32x2(fast_rcp(fast_exp2(e0) + 1.f), fast_rcp(fast_exp2(e1) + 1.f)), t[1], t[2]);  // the capped score
      return add_f32x2(w, add);
    }
  }
  __device__ __forceinline__ uint64_t derivative(uint64_t w) const {
    if constexpr (kAny)
      return w;
    else
      return fma_f32x2(w, polynomial(w, g), f32x2(1.f, 1.f));
  }
};

// What is added to the scores of columns c, c + 1 before the exponential: their bias and `add` (kLine: bias.line).
// kFolded: add is the same for all columns, and where kLine is, bias.off has it.
template <int SC, bool kLine, bool kFolded>
__device__ __forceinline__ uint64_t with_bias(const BiasLine& bias, int c, uint64_t add) {
  if constexpr ((SC & SC_BIAS) == 0) {
    return add;
  } else if constexpr (kLine) {
    const uint64_t b = f32x2(fmaf((float)c, bias.slp, bias.off), fmaf((float)(c + 1), bias.slp, bias.off));
    return kFolded ? b : add_f32x2(b, add);
  } else {
    float a0, a1;
    f32x2_split(add, a0, a1);
    return f32x2(fmaf(bias.neg, fabsf(fmaf(-(float)c, bias.st, c < bias.cb ? bias.a : bias.b)), a0),
                 fmaf(bias.neg, fabsf(fmaf(-(float)(c + 1), bias.st, c + 1 < bias.cb ? bias.a : bias.b)), a1));
  }
}

// The largest score of n columns whose bias is a line, or more by at most what that rises over them, from their largest
// product.
template <int SC>
__device__ __forceinline__ float most(const ScoreParams& sc, const BiasLine& bias, float s, int n) {
  if (s == -INFINITY) return s;
  float z = s * sc.c0;
  if constexpr ((SC & SC_CAP) != 0) z = fmaf(fast_rcp(fast_exp2(s * sc.e2) + 1.f), -2.f * sc.cap2, sc.cap2);
  return (SC & SC_BIAS) ? z + fmaxf(bias.off, fmaf((float)(n - 1), bias.slp, bias.off)) : z;
}

template <int N>
struct Const {
  static constexpr int value = N;
};
// f(tier, line) with both, which are the same in the whole warp, as compile-time constants.  Tiles without a line
// are few: one polynomial serves them (tier: not the least).
template <int SC, class F>
__device__ __forceinline__ void with_score_flags(int tier, bool line, F&& f) {
  if constexpr ((SC & SC_BIAS) != 0)
    if (!line) {
      if ((SC & SC_CAP) && tier == kTiers)
        f(Const<kTiers>{}, Const<0>{});
      else
        f(Const<2>{}, Const<0>{});
      return;
    }
  if (!(SC & SC_CAP) || tier == 0)
    f(Const<0>{}, Const<1>{});
  else if (tier == 1)
    f(Const<1>{}, Const<1>{});
  else if (tier == 2)
    f(Const<2>{}, Const<1>{});
  else
    f(Const<kTiers>{}, Const<1>{});
}

// The tile and the head of this block, of a grid of (shards' tiles, batch x heads): every head's heaviest tiles first,
// so that the light ones end the grid (a head after the other, the last heads' heavy tiles kept few SMs busy at the
// end: 16,384 tokens of 32 heads 1.82 ms, so 1.72; dK and dV of 8192 tokens of 32 + 8 heads 1.10 and 0.88).
// Causal calls of one sequence: late query tiles see more keys, early key tiles are seen by more queries (kLate).  In packed
// documents a tile weighs as much as its place in its document, which this does not look up: only the heads' order helps
// there (forward, dK / dV and dQ of 12 documents 211, 283 and 269 us, so 177, 256 and 239).
struct Start {
  int r, i0, head;  // shard, first row there, batch x heads
};
template <bool VL, bool kLate, int kRows, class P>
__device__ __forceinline__ Start start_of(const P& p, int n, int only) {  // n: tiles a shard
  const unsigned lin = blockIdx.y * gridDim.x + blockIdx.x;
  const int x = (int)(lin / gridDim.y), total = (int)gridDim.x, late = kLate ? x : total - 1 - x;
  Start s;
  s.head = (int)(lin % gridDim.y);
  int tile;
  if (!VL && p.causal && p.layout == LAYOUT_ZIGZAG && only < 0 && p.L % (2 * kRows) == 0) {
    zigzag_heavy_first(late, p.N, n / 2, s.r, tile);
  } else {
    const int o = p.causal && kLate ? total - 1 - x : x;
    const bool dealt = !VL && p.causal && p.layout == LAYOUT_STRIPE && only < 0;  // tile t of every shard: alike
    s.r = only >= 0 ? only : dealt ? o % p.N : o / n;
    tile = dealt ? o / p.N : o % n;
  }
  s.i0 = tile * kRows;
  return s;
}

// Batch i's prefix, as prefix_of gives it, behind after_previous_kernel.
template <class P>
__device__ __forceinline__ int prefix_now(const P& p, int i) {
  return p.sc.prefix && p.causal ? min(max(load_now(p.sc.prefix + i), 0), 1 << 30) : 0;
}

// The largest magnitude of N products (none that is NaN).
template <int N>
__device__ __forceinline__ float largest(const uint32_t (&v)[N]) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    m[0] = fmax3f(m[0], fabsf(__uint_as_float(v[c])), fabsf(__uint_as_float(v[c + 1])));
    m[1] = fmax3f(m[1], fabsf(__uint_as_float(v[c + 2])), fabsf(__uint_as_float(v[c + 3])));
  }
  return fmaxf(m[0], m[1]);
}
// The polynomial that holds for products of up to `size` in every lane: the least one, or (not `least`: code that has
// one polynomial for all) 2 or none.
__device__ __forceinline__ int tier_of(float size, const ScoreParams& sc, bool least = true) {
  // (not negative and no NaN: the bits are in the numbers' order)
  const float all = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
  if (!least) return all <= sc.lim[2] ? 2 : kTiers;
  return all <= sc.lim[0] ? 0 : all <= sc.lim[1] ? 1 : all <= sc.lim[2] ? 2 : kTiers;
}
template <int N>
__device__ __forceinline__ int score_tier(const uint32_t (&v)[N], const ScoreParams& sc, bool least) {
  return tier_of(largest(v), sc, least);
}

}  // namespace ra
