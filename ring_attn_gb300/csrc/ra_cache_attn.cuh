// Attention of few new tokens (decoding, verified proposals) over the paged 4-bit
// cache: out = softmax(scale q K^T) V with one pass over the keys.
//
// An item has up to R = 8 NT query rows; the blocks share the items' units as
// ra_cache_line.cuh says, in one wave.
//
// A block's W warps take a piece's tiles of 32 keys in turn.  Each streams its tiles
// through a ring of cp.async stages of its own and keeps its own running maximum,
// sum and O^T: no barrier in the loop.  Matrix products are warp-level m16n8k16 on fp16, which holds number *
// scale exactly, with keys (then head dims) as the 16 rows and 8 query rows as
// the columns, so a group of 8 heads wastes nothing:
//   S^T = K Q^T: a lane holds head dims [32 t, 32 t + 32) of rows g, g + 8, one
//     16-byte load each (g = lane / 4, t = lane % 4; the order of the contraction is
//     free as long as Q has the same).
//   O^T = V^T P^T: P^T is the transpose of the score fragment (movmatrix); a lane
//     holds 16 head dims of one scale group, for the keys 2t, 2t + 1, 2t + 8, 2t + 9.
// Both operands of a product have 16 bits; fp16 rather than bf16, because that holds number *
// scale and three more bits of p.  Queries are scaled per row by a power of two, the largest entry to
// [2^12, 2^13): entries down to 2^-26 of it are exact, those below 2^-36 of it count as 0, which
// is less than the rounding of the fp32 sums unless a key is 0 wherever its query is not
// small.  p is rounded to 11 bits (off by at most 2^-11 of it), for an fp32 out, too; the
// exponent's offset M keeps the largest p between 2^8 and 2^12, so p down to
// 2^-22 of it has all its fp16 bits; O is rescaled only when a score passes that.  Scores, M, sums
// and O are fp32, the exponential is the hardware's (2^-22).
//
// kScored: the call changes its scores (ra_cache_attn_scored.cu): the same kernel, with the cap and the
// bias applied to the scores of a tile as `mode` says, 8 or 16 numbers a lane, and rows that see their prefix.
//
// Bound: 0.5625 bytes per number from HBM, and close behind it the issue slots.  A tile of 32 keys
// and 8 query rows costs a warp about 630 instructions (d = 128: 140 conversions, 128 products with
// scales, 32 matrix products): over the whole kernel 50 to 53 % of the slots, start and end included,
// while it reads 3.7 TB/s (56 % of the measured copy rate; 64 ragged sequences).  One query of 32
// heads over 128K keys of 8: 151 MB in 42 us; 64 sequences of 200 to 16384 keys of 4 heads: 38 us, of
// which about 6 are the joining kernel's; with a cap 44, with a bias 40.
#pragma once

#include <algorithm>

#include "ra_cache_line.cuh"
#include "ra_score.cuh"

namespace ra {
namespace {

constexpr int kTilesPerUnit = kUnit / 32;
constexpr float kLift = 8.f;        // log2 of the largest p when M is set
constexpr float kSlack = 4.f;       // M is raised when a score is this much beyond
constexpr float kNone = -3.0e38f;   // M of a row that has seen no key

template <int D, int NT, int W>
struct Lay {
  static constexpr int kWarps = W;
  static constexpr int R = 8 * NT;
  static constexpr int kK = 0, kV = 32 * D / 2, kKs = 2 * kV, kVs = kKs + 32 * D / 16;
  static constexpr int kStage = kVs + 32 * D / 16;
  // the shared memory of an SM over its warps
  static constexpr int kStages = (W == 4 ? 3 : W == 12 ? 4 : 6) * (128 / D);
  static constexpr int kRing = kWarps * kStages * kStage;
  // A warp's results at an item's end: R rows of D floats (padded), M and sums.
  // With 8 rows they fit into the stage just consumed, so the next item's tiles
  // stay in flight; with more the ring is drained and reused.
  static constexpr int kOPitch = D + 4;
  static constexpr int kResult = R * (kOPitch + 2) * 4;
  static constexpr bool kFlow = kResult <= kStage;
  static constexpr int kAhead = kFlow ? kStages - 1 : 0;  // turns that the copies run ahead, into later pieces
  static constexpr int kResultPitch = kFlow ? kStages * kStage : kResult;  // from warp to warp
  // Queries at an item's start, R x D fp16, then R scales: with 8 rows in the
  // free stage of warp 0, else behind the ring.  So four blocks fit on an SM.
  static constexpr int kQ = kRing > kWarps * kResult ? kRing : kWarps * kResult;
  static constexpr int kBytes = kFlow ? kRing : kQ + R * D * 2 + R * 4;
};

// Cost in units: starting and finishing an item costs about as much as kItemCost.
// `whole`: every item is one place on the line, so none is shared.
template <int NT>
struct FewRows {
  static constexpr int R = 8 * NT, kItemCost = 3;
  static constexpr bool kOneTile = true, kPrefix = false;
  static __device__ __forceinline__ void cost(const CacheAttnArgs& g, LineSeq& s) {
    s.a = g.whole ? 1 : max(1, (s.len + kUnit - 1) / kUnit) + kItemCost;
  }
  // a turn of all warps, and 2 units (one leaves more to join: 28 rows of 3000 keys 20.4 us, 18.5 with two)
  static __device__ __forceinline__ int min_places(const CacheAttnArgs& g, int warps) {
    return g.whole ? 1 : max(2, warps / kTilesPerUnit);
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// zeros unless ok (nothing is read then)
__device__ __forceinline__ void cp16_or_0(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small_or_0(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(ok ? N : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// a where the mask has ones, else b
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(mask));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// N consecutive words
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "1, 2 or 4 words");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    v[0] = lds32(a);
}

// Where V's key row r (0..31) lies in a stage: the first keys 2t of a lane's pairs
// side by side, then the second ones (slot 4 (r & 1) + r / 2 of every 8 rows), and for
// 64-byte rows chunks swapped in pairs, so that the 16 lanes of a load phase meet all
// banks once.  The swap depends on r mod 8 only, so a lane's rows 8 apart lie 8 rows apart.
template <int D>
__device__ __forceinline__ uint32_t v_place(int r, int chunk) {  // r < 8
  const int slot = ((r & 1) << 2) | (r >> 1);
  return slot * (D / 2) + ((D == 128 ? chunk ^ (slot & 2) : chunk) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_offset(int r, int chunk) {
  return v_place<D>(r & 7, chunk) + (r & ~7) * (D / 2);
}

// Turns of a block's warps over the tiles of `units` units.
template <int W>
__device__ __forceinline__ int turns_of(int units) {
  return (units * kTilesPerUnit + W - 1) / W;
}

// The block's pieces in shared memory, some ahead of the one being worked on, so that the
// warps hold no place on the line in registers; ub = 0 ends the run.
struct BlockPiece {
  int seq, head, cu0, len, n_new, ua, ub, whole;
};
constexpr int kPieces = 8;
struct Pieces {
  volatile BlockPiece ring[kPieces];
  LinePos at;
  int end, quota;
  JoinNote note;
  int made;
  bool over;
};
// One thread: the next piece goes to the ring.
template <class Kind>
__device__ __forceinline__ void make_piece(const CacheAttnArgs& g, Pieces& p) {
  LinePos at = p.at;
  Piece x;
  const bool more = next_piece<Kind>(g, at, p.end, x);
  volatile BlockPiece& y = p.ring[p.made % kPieces];
  ++p.made;
  if (!more) {
    y.ua = y.ub = 0;
    p.over = true;
    return;
  }
  p.at = at;
  const int cu0 = g.s.cu[x.seq];
  JoinNote n = p.note;
  note_piece<Kind>(g, x, p.quota, cu0, n);
  p.note = n;
  y.seq = x.seq, y.head = x.head, y.cu0 = cu0, y.len = x.len, y.n_new = x.n_new;
  y.ua = x.ua, y.ub = x.ub, y.whole = x.ub - x.ua == x.units;
  if (g.s.lens[x.seq] > g.max_kv) record_error(g.ctl, DEV_BOUNDS, SITE_CACHE_LEN);
}

// A warp's copies: its tiles go to the ring slot by slot, their pages read two turns ahead.
template <int D, int NT, int W>
struct Stream {
  using L = Lay<D, NT, W>;
  const CacheAttnArgs& a;
  const Pieces& p;
  int index;                          // of the piece
  int turns, end_key;                 // turns to come of a piece, and the end of its keys
  const int* table;                   // the sequence's page table
  int pa, pb, k0;                     // pages of the warp's keys [k0, k0 + 16) and the 16 after them
  int na, nb;                         // the same a turn ahead
  const uint8_t *kc, *vc, *ks, *vs;   // the head's rows, this lane's part of the offset included
  int step_c;                         // bytes between this lane's code chunks in the cache (512 in a stage)
  uint32_t v_at;                      // this lane's first V chunk in a stage
  uint32_t to, end, slot0;            // ring slot, the ring's end and start

  __device__ __forceinline__ Stream(const CacheAttnArgs& args, const Pieces& pieces, uint32_t ring)
      : a(args), p(pieces), index(0), turns(0), end_key(0), pa(0), pb(0), k0(0), na(0), nb(0), to(ring),
        end(ring + L::kStages * L::kStage), slot0(ring) {
    constexpr int CPR = D / 32;
    step_c = (int)a.c.k.s_row * (32 / CPR);
    const int lane = threadIdx.x & 31;
    v_at = v_offset<D>(lane / CPR, lane % CPR);
  }
  __device__ __forceinline__ void piece(int i) {
    index = i;
    const volatile BlockPiece& x = p.ring[i % kPieces];
    const int lane = threadIdx.x & 31, head = x.head, ua = x.ua, ub = x.ub;
    turns = turns_of<W>(ub - ua);
    k0 = ua * kUnit + (threadIdx.x >> 5) * 32;
    end_key = min(x.len, ub * kUnit);
    constexpr int CPR = D / 32;  // 16-byte chunks per row
    const long long oc = head * a.c.k.s_head + (lane / CPR) * a.c.k.s_row + lane % CPR * 16;
    const long long os = head * a.c.ks.s_head + lane * a.c.ks.s_row;
    kc = a.c.k.data + oc, vc = a.c.v.data + oc;
    ks = a.c.ks.data + os, vs = a.c.vs.data + os;
    table = a.s.table + (long long)x.seq * a.s.table_stride;
    pages(k0, pa, pb);
    pages(k0 + 32 * W, na, nb);
  }
  __device__ __forceinline__ void pages(int k, int& p, int& q) {
    if (k < end_key) {
      p = table[k >> a.c.page_shift];
      if (a.c.page_shift == 4) q = k + 16 < end_key ? table[(k >> 4) + 1] : p;
    }
  }
  // Copies the warp's tile of a turn (nothing when none is left) and moves on, to the run's
  // next piece when `follow`.
  __device__ __forceinline__ void load(bool follow) {
    if (turns == 0 && follow && p.ring[(index + 1) % kPieces].ub > 0) piece(index + 1);
    if (turns > 0) {
      if (k0 < end_key) {
        const bool full = k0 + 32 <= end_key && (unsigned)pa < (unsigned)a.c.n_pages;
        if (full && a.c.page_shift > 4)
          copy_full();
        else if (full && (unsigned)pb < (unsigned)a.c.n_pages)
          copy_two();
        else
          copy_part();
      }
      k0 += 32 * W;
      --turns;
      pa = na, pb = nb;
      pages(k0 + 32 * W, na, nb);
    }
    cp_commit();
    to += L::kStage;
    if (to == end) to = slot0;
  }
  // 32 keys of one page
  __device__ __forceinline__ void copy_full() {
    const int lane = threadIdx.x & 31, row = k0 & ((1 << a.c.page_shift) - 1);
    constexpr int CPR = D / 32;
    const long long o = (long long)pa * a.c.k.s_page + row * (int)a.c.k.s_row;
    const uint8_t *k = kc + o, *v = vc + o;
    const uint32_t tk = to + L::kK + lane * 16, tv = to + L::kV + v_at;
    if (step_c == 512) {  // packed rows: every offset is a constant
#pragma unroll
      for (int j = 0; j < CPR; ++j) {
        cp16(tk + j * 512, k + j * 512);
        cp16(tv + j * 512, v + j * 512);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CPR; ++j) {
        cp16(tk + j * 512, k + (long long)j * step_c);
        cp16(tv + j * 512, v + (long long)j * step_c);
      }
    }
    const long long os = (long long)pa * a.c.ks.s_page + row * (int)a.c.ks.s_row;
    cp_small<D / 16>(to + L::kKs + lane * (D / 16), ks + os);
    cp_small<D / 16>(to + L::kVs + lane * (D / 16), vs + os);
  }
  // 32 keys of two pages of 16 tokens
  __device__ __forceinline__ void copy_two() {
    const int lane = threadIdx.x & 31;
    constexpr int CPR = D / 32;
    const uint32_t tk = to + L::kK + lane * 16, tv = to + L::kV + v_at;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long o = (long long)(h ? pb : pa) * a.c.k.s_page;
#pragma unroll
      for (int j = 0; j < CPR / 2; ++j) {
        cp16(tk + (h * (CPR / 2) + j) * 512, kc + o + (long long)j * step_c);
        cp16(tv + (h * (CPR / 2) + j) * 512, vc + o + (long long)j * step_c);
      }
    }
    const long long os = lane < 16 ? (long long)pa * a.c.ks.s_page
                                   : (long long)pb * a.c.ks.s_page - 16 * (int)a.c.ks.s_row;
    cp_small<D / 16>(to + L::kKs + lane * (D / 16), ks + os);
    cp_small<D / 16>(to + L::kVs + lane * (D / 16), vs + os);
  }
  // Fewer keys or a page that is none: the other rows are zeros.
  __device__ __forceinline__ void copy_part() {
    const int lane = threadIdx.x & 31, mask = (1 << a.c.page_shift) - 1;
    if (a.c.page_shift > 4) pb = pa;
    const bool oka = (unsigned)pa < (unsigned)a.c.n_pages, okb = (unsigned)pb < (unsigned)a.c.n_pages;
    if (!(oka && okb) && lane == 0) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_PAGE);
    constexpr int CPR = D / 32, RPJ = 32 / CPR;
#pragma unroll 1
    for (int j = 0; j <= CPR; ++j) {  // the last turn copies the scales
      const int r = j < CPR ? j * RPJ + lane / CPR : lane, ch = lane % CPR;
      const bool ok = k0 + r < end_key && (r < 16 ? oka : okb);
      const int page = ok ? (r < 16 ? pa : pb) : 0, row = (k0 + r) & mask;
      if (j < CPR) {
        const long long o = (long long)page * a.c.k.s_page + (row - lane / CPR) * (long long)a.c.k.s_row;
        cp16_or_0(to + L::kK + r * (D / 2) + ch * 16, kc + o, ok);
        cp16_or_0(to + L::kV + v_offset<D>(r, ch), vc + o, ok);
      } else {
        const long long o = (long long)page * a.c.ks.s_page + (row - lane) * (long long)a.c.ks.s_row;
        cp_small_or_0<D / 16>(to + L::kKs + lane * (D / 16), ks + o, ok);
        cp_small_or_0<D / 16>(to + L::kVs + lane * (D / 16), vs + o, ok);
      }
    }
  }
};

// Small blocks (4 warps) per SM: as many as the registers of a row tile allow without spills.
// (8 rows of d = 128 with three: 64 sequences of 4000 keys of 4 heads 41.5 us, with four 43.1;
// 16 rows with two: 40 sequences of 2000 keys of 8 heads 43 us, with three 46.)
constexpr int small_blocks(int d, int nt) { return nt == 1 ? (d == 64 ? 4 : 3) : 2; }

template <int D, int NT, int W, bool kScored>
__global__ void __launch_bounds__(32 * W, W == 4 ? small_blocks(D, NT) : 1) cache_attn_kernel(const CacheAttnArgs a) {
  using L = Lay<D, NT, W>;
  constexpr int kWarps = W, kThreads = 32 * W;
  constexpr int R = L::R, KS = D / 16;  // contraction steps of S, row tiles of O^T
  // the piece worked on and those planned ahead, of a turn at least each
  static_assert(kPieces >= 1 + (L::kAhead > 1 ? L::kAhead : 1), "the planner would overwrite a piece in use");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ LineShared<kWarps> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t sb = smem_u32(smem), ring = sb + warp * L::kStages * L::kStage;

  after_previous_kernel();
  using Kind = FewRows<NT>;
  __shared__ Pieces sp;
  __shared__ __align__(16) float2 row_bias[kScored ? R : 1];  // slope (log2 units) and own cache index of every row
  const bool planner = threadIdx.x == kThreads - 32;
  {
    LinePos at;
    int end_u, quota;
    if (!find_run<Kind, W>(a, at, end_u, quota, sh)) {
      if (planner) notes_of(a)[blockIdx.x] = empty_note();
      return;
    }
    if (planner) {
      sp.at = at, sp.end = end_u, sp.quota = quota;
      sp.note = empty_note();
      sp.made = 0;
      sp.over = false;
      make_piece<Kind>(a, sp);
      // the first copies may go beyond a short first piece
      if (L::kFlow)
        for (int ahead = turns_of<W>(sp.ring[0].ub - sp.ring[0].ua); ahead < L::kAhead && !sp.over;) {
          make_piece<Kind>(a, sp);
          ahead += turns_of<W>(sp.ring[sp.made - 1].ub - sp.ring[sp.made - 1].ua);
        }
    }
  }
  __syncthreads();
  Stream<D, NT, W> st(a, sp, ring);
  // this lane's V numbers of key 2t (key 2t + 1 lies 4 rows on)
  const uint32_t lane_v = L::kV + v_place<D>(2 * t, g * (D / 64) / 4) + (g * (D / 64) % 4) * 4;
  // a row's token: r / G for r < 32 (a product instead of a division)
  const uint32_t inv_g = (65536u + a.G - 1) / a.G;
  auto token_of_row = [inv_g](int r) { return (int)((r * inv_g) >> 16); };
  uint32_t slot = 0;
  for (int i = 0; sp.ring[i % kPieces].ub > 0; ++i) {
    // ---------------------------------------------------------------- the next item
    const volatile BlockPiece& w = sp.ring[i % kPieces];
    const int ua = w.ua, n_it = turns_of<W>(w.ub - ua), end_key = min(w.len, w.ub * kUnit);
    const int len = w.len, n_new = w.n_new, rows = n_new * a.G;
    const int pre = kScored ? cache_prefix(a, w.seq) : 0;
    if (!L::kFlow || i == 0) {  // a drained ring starts again
      slot = 0;
      st.to = ring;
      st.piece(i);
#pragma unroll 1
      for (int s = 0; s < L::kStages - 1; ++s) st.load(L::kFlow);
    }
    if (planner) {  // the pieces that the copies may reach during this one, and the one after it
      for (int k = i + 1, ahead = 0; k == i + 1 || ahead < L::kAhead; ++k) {
        if (k == sp.made && !sp.over) make_piece<Kind>(a, sp);
        const int n = sp.ring[k % kPieces].ub - sp.ring[k % kPieces].ua;
        if (n == 0) break;
        ahead += turns_of<W>(n);
      }
    }

    // ---------------------------------------------------------------- queries
    const int q_at = L::kFlow ? (int)(st.to - ring) : L::kQ;  // the slot that the next copies go to
    uint2* sq = reinterpret_cast<uint2*>(smem + q_at);  // a fragment's 32 lanes side by side
    float* sscale = reinterpret_cast<float*>(smem + q_at + R * D * 2);
    {
      constexpr int LPR = D / 8;  // lanes per row
      for (int r = threadIdx.x / LPR; r < R; r += kThreads / LPR) {
        const int c = threadIdx.x % LPR;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int tk = token_of_row(r), tok = w.cu0 + tk, hd = w.head * a.G + r - tk * a.G;
          q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.data) + (long long)tok * a.q.s_row +
                                              (long long)hd * a.q.s_head + 8 * c);
        }
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
        float x[8], m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(qw[i] << 16);
          x[2 * i + 1] = __uint_as_float(qw[i] & 0xffff0000u);
          m = fmaxf(m, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
        }
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // the row's largest entry goes to [2^12, 2^13)
        const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = pack_f16x2(x[2 * i] * up, x[2 * i + 1] * up);
        // head dims 8 c.. are lane t's of steps s and s + 1
        uint2* to = sq + ((r >> 3) * KS + c % (D / 32) * 2) * 32 + (r & 7) * 4 + c / (D / 32);
        to[0] = make_uint2(h[0], h[1]);
        to[32] = make_uint2(h[2], h[3]);
        if (c == 0) sscale[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e - 12) << 23);
        if (kScored && c == 0 && (a.mode & SC_BIAS)) {
          const int tk = token_of_row(r);
          const float slope = r < rows ? a.sc.slopes[w.head * a.G + r - tk * a.G] : 0.f;
          row_bias[r] = make_float2(slope * 1.4426950408889634f, __int_as_float(len - n_new + tk));
        }
      }
    }
    __syncthreads();
    // the fragments of Q^T: in registers, or read where they are used when there are many
    constexpr bool kQReg = NT == 1;
    uint32_t qb[kQReg ? NT : 1][KS][2];
    auto q_frag = [&](int n, int s) { return sq[(n * KS + s) * 32 + lane]; };
    float sc[kQReg ? NT : 1][2];
    int end[kQReg ? NT : 1][2], min_end = len;
    auto row_end = [&](int r) {  // keys that row r sees
      const int own = len - n_new + token_of_row(r) + 1;
      return a.causal && r < rows ? min(len, kScored ? max(own, pre) : own) : len;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (kQReg) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 v = q_frag(n, s);
          qb[n][s][0] = v.x, qb[n][s][1] = v.y;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) sc[n][x] = sscale[8 * n + 2 * t + x], end[n][x] = row_end(8 * n + 2 * t + x);
      }
    }
    auto row_scale = [&](int n) {
      if constexpr (kQReg)
        return make_float2(sc[n][0], sc[n][1]);
      else
        return *reinterpret_cast<const float2*>(sscale + 8 * n + 2 * t);
    };
    if (a.causal) min_end = min(len, kScored ? max(len - n_new + 1, pre) : len - n_new + 1);
    if (L::kFlow) __syncthreads();

    // ---------------------------------------------------------------- keys
    float o[NT][KS][4], M[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < KS; ++s) o[n][s][0] = o[n][s][1] = o[n][s][2] = o[n][s][3] = 0.f;
      M[n][0] = M[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
    }
    // Tiles of 16 keys whose scores are computed side by side: two read a query fragment
    // once and keep the matrix unit busier, where the registers hold them.
    constexpr int AT = NT <= 2 ? 2 : 1;
    uint32_t stg = 0;
    for (int it = 0; it < n_it; ++it) {
      cp_wait<L::kStages - 2>();
      __syncwarp();
      st.load(L::kFlow);
      const int k0 = ua * kUnit + (it * W + warp) * 32;
      stg = ring + slot * L::kStage;
      if (++slot == L::kStages) slot = 0;
      if (k0 >= end_key) continue;
      const uint32_t stv = stg + lane_v;
      // scores of 32 keys: rows g, g + 8 of two tiles
      float s[2][NT][4];
#pragma unroll
      for (int a0 = 0; a0 < 2; a0 += AT) {
        uint32_t ka[AT][D / 32], kb[AT][D / 32], sa[AT], sbq[AT];  // this lane's one (d = 64) or two scales of each row
#pragma unroll
        for (int i = 0; i < AT; ++i) {
#pragma unroll
          for (int n = 0; n < NT; ++n) s[a0 + i][n][0] = s[a0 + i][n][1] = s[a0 + i][n][2] = s[a0 + i][n][3] = 0.f;
          const int row = 16 * (a0 + i) + g;
          const uint32_t ra = stg + L::kK + row * (D / 2) + t * (D / 8), rs = stg + L::kKs + row * (D / 16) + t * (D / 64);
          lds_words(ra, ka[i]);
          lds_words(ra + 8 * (D / 2), kb[i]);
          if constexpr (D == 128) {
            sa[i] = e4m3x2_to_f16(lds16(rs));
            sbq[i] = e4m3x2_to_f16(lds16(rs + 8 * (D / 16)));
          } else {
            sa[i] = e4m3x2_to_f16(lds8(rs));
            sbq[i] = e4m3x2_to_f16(lds8(rs + 8 * (D / 16)));
          }
        }
#pragma unroll
        for (int wd = 0; wd < D / 32; ++wd) {
          uint32_t x[AT][4], y[AT][4];
#pragma unroll
          for (int i = 0; i < AT; ++i) {
            e2m1x8_to_f16(ka[i][wd], x[i]);
            e2m1x8_to_f16(kb[i][wd], y[i]);
            const uint32_t s_a = wd < 2 ? half_lo2(sa[i]) : half_hi2(sa[i]), s_b = wd < 2 ? half_lo2(sbq[i]) : half_hi2(sbq[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] = hmul2(x[i][k], s_a), y[i][k] = hmul2(y[i][k], s_b);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint2 q;
              if constexpr (kQReg)
                q = make_uint2(qb[n][2 * wd + v][0], qb[n][2 * wd + v][1]);
              else
                q = q_frag(n, 2 * wd + v);
#pragma unroll
              for (int i = 0; i < AT; ++i) {
                const uint32_t f[4] = {x[i][2 * v], y[i][2 * v], x[i][2 * v + 1], y[i][2 * v + 1]};
                mma16816(s[a0 + i][n], f, q.x, q.y);
              }
            }
        }
      }
      // log2 scores (rounded before M is taken off, so that the largest gives an
      // exact difference however large it is), masked; M is raised only when one
      // of them passes it by far
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 f = row_scale(n);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[mt][n][x] = __fmul_rn(s[mt][n][x], x & 1 ? f.y : f.x);
      }
      if constexpr (kScored) {
        if (a.mode & SC_CAP) {
          // 1 - 2 / (1 + e^(2u)), off by cap2 2^-22; above a cap of 128 that shows, and small scores take the polynomial
          auto change = [&](auto high) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float u = s[mt][n][x], w = u * u;
                  s[mt][n][x] = fmaf(fast_rcp(fast_exp2(u * a.sc.e2) + 1.f), -2.f * a.sc.cap2, a.sc.cap2);
                  if (decltype(high)::value && fabsf(u) <= a.sc.lim[0])
                    s[mt][n][x] = u * fmaf(w, fmaf(w, fmaf(w, a.sc.t0[3], a.sc.t0[2]), a.sc.t0[1]), a.sc.t0[0]);
                }
          };
          if (a.sc.cap2 <= 185.f)
            change(Const<0>{});
          else
            change(Const<1>{});
        }
        if (a.mode & SC_BIAS) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 b = *reinterpret_cast<const float4*>(row_bias + 8 * n + 2 * t);
            // distances from key k0 + g
            const float d[2] = {(float)(__float_as_int(b.y) - k0 - g), (float)(__float_as_int(b.w) - k0 - g)};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                s[mt][n][x] = fmaf(-(x & 1 ? b.z : b.x), fabsf(d[x & 1] - (float)(16 * mt + 8 * (x >> 1))), s[mt][n][x]);
          }
        }
      }
      if (k0 + 32 > min_end) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          int to[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (kQReg)
              to[x] = end[n][x];
            else
              to[x] = row_end(8 * n + 2 * t + x);
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (k0 + 16 * mt + g + 8 * (x >> 1) >= to[x & 1]) s[mt][n][x] = -INFINITY;
        }
      }
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[n][x] = fmaxf(fmax3f(s[0][n][x], s[0][n][x + 2], s[1][n][x]), s[1][n][x + 2]);
          over |= mx[n][x] > M[n][x] + (kLift + kSlack);
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float m = mx[n][x];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
            const float to = m > M[n][x] + kLift ? m - kLift : M[n][x];
            alpha[x] = fast_exp2(M[n][x] - to);
            M[n][x] = to;
            l[n][x] *= alpha[x];
          }
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[n][d][0] *= alpha[0], o[n][d][2] *= alpha[0];
            o[n][d][1] *= alpha[1], o[n][d][3] *= alpha[1];
          }
        }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            p[x] = fast_exp2(__fsub_rn(s[mt][n][x], M[n][x & 1]));
            l[n][x & 1] += p[x];
          }
          pb[mt][n][0] = transpose8x8(pack_f16x2(p[0], p[1]));
          pb[mt][n][1] = transpose8x8(pack_f16x2(p[2], p[3]));
        }
      // O^T += V^T P^T
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        constexpr int W = D / 64;  // words of a lane's D / 8 head dims
        uint32_t v[4][W], s2[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // keys 2t, 2t + 1, 2t + 8, 2t + 9
          lds_words(stv + (16 * mt + 8 * (k >> 1) + 4 * (k & 1)) * (D / 2), v[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t rs = stg + L::kVs + (16 * mt + 2 * t + 8 * k) * (D / 16) + g * W / 2;
          s2[k] = e4m3x2_to_f16(lds8(rs) | (lds8(rs + D / 16) << 8));
        }
#pragma unroll
        for (int wd = 0; wd < W; ++wd) {
          uint32_t f[4][4];  // [a register][pair of head dims]
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w0 = v[2 * k][wd], w1 = v[2 * k + 1][wd];
            e2m1x8_to_f16(select_bits(w0, w1 << 4, 0x0f0f0f0fu), f[2 * k]);
            e2m1x8_to_f16(select_bits(w0 >> 4, w1, 0x0f0f0f0fu), f[2 * k + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t fr[4] = {hmul2(f[0][i], s2[0]), hmul2(f[1][i], s2[0]), hmul2(f[2][i], s2[1]),
                                    hmul2(f[3][i], s2[1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][4 * wd + i], fr, pb[mt][n][0], pb[mt][n][1]);
          }
        }
      }
    }

    // ---------------------------------------------------------------- the warps' results
    if (!L::kFlow) {
      cp_wait<0>();
      __syncthreads();
    } else {
      __syncwarp();
    }
    // warp k's results: R rows of kOPitch floats, then M, then the sums
    const uint32_t res0 = L::kFlow ? stg - ring : 0;
    auto result = [&](int k) { return reinterpret_cast<float*>(smem + res0 + k * L::kResultPitch); };
    constexpr int kM = R * L::kOPitch, kL = kM + R;
    float* mine = result(warp);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = l[n][x];
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        const int r = 8 * n + 2 * t + x;
        if (g == 0) mine[kM + r] = M[n][x], mine[kL + r] = v;
#pragma unroll
        for (int d = 0; d < KS; ++d)  // head dims D / 8 g + 2 d, + 1 at place 16 d + 2 g
          *reinterpret_cast<float2*>(mine + r * L::kOPitch + 16 * d + 2 * g) =
              make_float2(o[n][d][x], o[n][d][x + 2]);
      }
    }
    __syncthreads();
    const bool whole = w.whole;
    const int cu0 = w.cu0, head = w.head;
    float* part = slot_of<R, D>(a, gridDim.x, blockIdx.x, ua == 0);
    for (int e = threadIdx.x; e < rows * (D / 2); e += kThreads) {
      const int r = e / (D / 2), d = e % (D / 2) * 2;
      const int from = (d % (D / 8)) / 2 * 16 + d / (D / 8) * 2;
      float m = result(0)[kM + r];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) m = fmaxf(m, result(k)[kM + r]);
      float lsum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float* res = result(k);
        const float f = fast_exp2(res[kM + r] - m);
        const float2 v = *reinterpret_cast<const float2*>(res + r * L::kOPitch + from);
        lsum += res[kL + r] * f;
        o0 += v.x * f, o1 += v.y * f;
      }
      if (!whole) {
        *reinterpret_cast<float2*>(part + r * D + d) = make_float2(o0, o1);
        if (d == 0) *reinterpret_cast<float2*>(part + R * D + 2 * r) = make_float2(m, lsum);
      } else {
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
        const int tk = token_of_row(r), tok = cu0 + tk, hd = head * a.G + r - tk * a.G;
        const long long to = (long long)tok * a.out.s_row + (long long)hd * a.out.s_head + d;
        if (a.out_f32)
          *reinterpret_cast<float2*>(static_cast<float*>(a.out.data) + to) = make_float2(o0 * inv, o1 * inv);
        else
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out.data) + to) = pack_bf16x2(o0 * inv, o1 * inv);
        if (d == 0) store_lse(a, tok, hd, m, lsum);
      }
    }
    __syncthreads();
  }
  if (planner) notes_of(a)[blockIdx.x] = sp.note;
}

// Warps of the block when there is one per SM.  With 8 rows, 12 warps with 4 stages each
// take 42 us for one query over 128K keys, 16 with 3 stages 49 us.
constexpr int big_warps(int nt) { return nt == 4 ? 8 : 12; }

template <int D, int NT, int W, bool kScored>
cudaError_t launch_w(const CacheAttnPlan& p, cudaStream_t st) {
  using L = Lay<D, NT, W>;
  const cudaError_t e = configure_kernel<cache_attn_kernel<D, NT, W, kScored>>(0, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_early(cache_attn_kernel<D, NT, W, kScored>, p.grid, 32 * W, L::kBytes, st, p.args);
}

template <bool kScored, int D, int NT>
cudaError_t launch(const CacheAttnPlan& p, cudaStream_t st) {
  return p.big ? launch_w<D, NT, big_warps(NT), kScored>(p, st) : launch_w<D, NT, 4, kScored>(p, st);
}
template <bool kScored>
cudaError_t launch_few(const CacheAttnPlan& p, cudaStream_t st) {
  const int nt = p.row_tiles;
  if (p.args.d == 64)
    return nt == 1   ? launch<kScored, 64, 1>(p, st)
           : nt == 2 ? launch<kScored, 64, 2>(p, st)
                     : launch<kScored, 64, 4>(p, st);
  return nt == 1   ? launch<kScored, 128, 1>(p, st)
         : nt == 2 ? launch<kScored, 128, 2>(p, st)
                   : launch<kScored, 128, 4>(p, st);
}

}  // namespace
}  // namespace ra
