// How the attention over the paged cache is shared out.
//
// An item is one key / value head of one sequence with R of its query rows (row r
// of the sequence is token r / G, head r % G of the group): a row tile.  Its keys
// are cut into units of 128.  All items lie one after the other on a line, each
// with a length that stands for its cost, and each block of the grid takes an
// equal run of the line: the units of an item go to the blocks in order.
// The lengths are read from device memory, so a captured launch follows them.
//
// A piece that holds all units of its item is written as the result.  The other
// pieces go to the workspace, two slots per block: slot 1 for a piece that holds
// its item's first unit (at most the last of the block), slot 0 for one that does not
// (at most the first).  A note per block says which slots it filled and where the
// item of slot 1 ends, so the kernel that joins the pieces, in block order, needs
// no plan of its own.
#pragma once

#include "ra_cache.cuh"

namespace ra {

constexpr int kUnit = 128;

// Numbers that lambdas take as compile-time constants.
template <int N>
struct Int {
  static constexpr int value = N;
};

// One sequence: its row tiles' costs are a + b * tile places.  `per` places stand for a
// unit (with line_shift, a place for 2^line_shift units, so that any line's length
// fits 32 bits), after kItemCost units' worth for starting and finishing the item.
struct LineSeq {
  int len, n_new, tiles, per;
  int a, b;
  int pre;  // tokens that every causal row sees (Kind::kPrefix, else 0)
  __device__ __forceinline__ int before(int tile) const { return a * tile + b * (tile * (tile - 1) / 2); }
};

// Kind: R, kItemCost, kOneTile (R holds all of a sequence's rows), kPrefix (calls may have prefixes), and for line_shift 0
// the cost rule `static void cost(args, LineSeq&)` and the least places that a block of a
// number of warps takes, `static int min_places(args, warps)`.
// Tokens of sequence i's prefix, which all of its causal rows see.
__device__ __forceinline__ int cache_prefix(const CacheAttnArgs& g, int i) {
  return g.sc.prefix && g.causal ? min(max(g.sc.prefix[i], 0), 1 << 30) : 0;
}
template <class Kind>
__device__ __forceinline__ LineSeq line_of(const CacheAttnArgs& g, int seq, int len, int n_new) {
  LineSeq s;
  s.pre = Kind::kPrefix ? cache_prefix(g, seq) : 0;
  s.n_new = n_new;
  s.len = len;
  s.tiles = Kind::kOneTile ? min(n_new, 1) : (int)(((long long)n_new * g.G + Kind::R - 1) / Kind::R);
  s.per = 1;
  s.b = 0;
  if (g.line_shift == 0)
    Kind::cost(g, s);
  else
    s.a = ((max(1, (len + kUnit - 1) / kUnit) + Kind::kItemCost - 1) >> g.line_shift) + 1;
  return s;
}
template <class Kind>
__device__ __forceinline__ LineSeq line_seq(const CacheAttnArgs& g, int i) {
  const int n_new = g.s.cu[i + 1] - g.s.cu[i];
  return line_of<Kind>(g, i, max(0, min(g.s.lens[i], g.max_kv)), n_new);
}
template <class Kind>
__device__ __forceinline__ int line_length(const CacheAttnArgs& g, const LineSeq& s) {
  return g.hk * (Kind::kOneTile ? s.a * s.tiles : s.before(s.tiles));
}

// Keys that the rows of a tile see, the last one's, in units (at least one: a row without
// keys is written too).
template <class Kind>
__device__ __forceinline__ int tile_units(const CacheAttnArgs& g, const LineSeq& s, int tile) {
  int end = s.len;
  if (g.causal && !Kind::kOneTile) {
    const int last = (int)min((long long)s.n_new - 1, ((long long)tile * Kind::R + Kind::R - 1) / g.G);
    end = min(end, Kind::kPrefix ? max(s.len - s.n_new + last + 1, s.pre) : s.len - s.n_new + last + 1);
  }
  return max(1, (end + kUnit - 1) / kUnit);
}

// The unit at place p of an item of `units` units (p = cost: the end).  The cost
// may be a few units off, so that it is linear: the last block takes the rest.
template <class Kind>
__device__ __forceinline__ int unit_at(const CacheAttnArgs& g, int p, int units, int cost, int per) {
  if (p >= cost) return units;
  const int u = (int)min((long long)units + Kind::kItemCost, (long long)(per == 1 ? p : p / per) << g.line_shift);
  return max(0, u - Kind::kItemCost);
}

// Sum of v over the warp's lower lanes and this one.
__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// Sum of v over the block (every thread gets it) and the sum over lower threads.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int& below, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = warp_scan(v);
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int pre = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    pre += w < warp ? sh[w] : 0;
    all += sh[w];
  }
  below = pre + x - v;
  return all;
}

// Shared memory of find_run.
template <int WARPS>
struct LineShared {
  int sums[WARPS], first, seq;
};

// A place on the line, and the item it lies in.
struct LinePos {
  int u, start;        // place, and the item's first place
  int seq, head, tile;
  int len, n_new;      // of the sequence
};

// The item of sequence `seq`, which begins at `first`, that holds at.u.
template <class Kind>
__device__ __forceinline__ void enter_item(const CacheAttnArgs& g, LinePos& at, int seq, int first) {
  const LineSeq s = line_seq<Kind>(g, seq);
  at.seq = seq;
  at.len = s.len;
  at.n_new = s.n_new;
  at.tile = 0;
  const int per = Kind::kOneTile ? s.a : s.before(s.tiles);
  int q = at.u - first;
  at.head = (int)((unsigned)q / (unsigned)per);
  at.start = first + at.head * per;
  if (!Kind::kOneTile) {
    q = at.u - at.start;
    int lo = 0, hi = s.tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.before(mid) <= q)
        lo = mid;
      else
        hi = mid - 1;
    }
    at.tile = lo;
    at.start += s.before(lo);
  }
}

// This block's run [at.u, end) of the line, found by the whole thread block.  False when it is empty.
template <class Kind, int WARPS>
__device__ __forceinline__ bool find_run(const CacheAttnArgs& g, LinePos& at, int& end, int& quota,
                                         LineShared<WARPS>& sh) {
  constexpr int T = 32 * WARPS;
  const int tid = threadIdx.x, lane = tid & 31, n = g.s.n_seqs;
  const bool one_warp = n <= 32, few = n <= T;  // one sequence per lane, per thread: read once
  const int mine = one_warp ? lane : tid;
  int v = 0, below = 0, all;
  if (few) {
    if (mine < n) v = line_length<Kind>(g, line_seq<Kind>(g, mine));
  } else {
    for (int i = tid; i < n; i += T) v += line_length<Kind>(g, line_seq<Kind>(g, i));
  }
  if (one_warp) {  // every warp by itself
    below = warp_scan(v);
    all = __shfl_sync(0xffffffffu, below, 31);
    below -= v;
  } else {
    all = block_scan<WARPS>(v, below, sh.sums);
  }
  quota = (int)(((unsigned)all + gridDim.x - 1) / gridDim.x);
  if (g.line_shift == 0) quota = max(quota, Kind::min_places(g, WARPS));
  at.u = (int)min((long long)all, (long long)blockIdx.x * quota);
  end = (int)min((long long)all, (long long)at.u + quota);
  if (at.u >= end) return false;
  int seq, first;
  if (one_warp) {
    seq = 31 - __clz(__ballot_sync(0xffffffffu, v > 0 && below <= at.u));
    first = __shfl_sync(0xffffffffu, below, seq);
  } else {
    if (few) {
      if (at.u >= below && at.u < below + v) sh.seq = tid, sh.first = below;
    } else {
      int base = 0;
      for (int i0 = 0; i0 < n && base <= at.u; i0 += T) {
        const int i = i0 + tid;
        v = i < n ? line_length<Kind>(g, line_seq<Kind>(g, i)) : 0;
        const int sum = block_scan<WARPS>(v, below, sh.sums);
        if (at.u >= base + below && at.u < base + below + v) sh.seq = i, sh.first = base + below;
        base += sum;
      }
    }
    __syncthreads();
    seq = sh.seq;
    first = sh.first;
  }
  enter_item<Kind>(g, at, seq, first);
  return true;
}

// An item and a range of its units.
struct Piece {
  int seq, head, tile, len, n_new, units, ua, ub;
  int start, cost;  // place of the item on the line
};

// The next piece of the run that ends at `end`, moving `at` behind it.  False at the run's end.
template <class Kind>
__device__ __forceinline__ bool next_piece(const CacheAttnArgs& g, LinePos& at, int end, Piece& x) {
  while (at.u < end) {
    LineSeq s = line_of<Kind>(g, at.seq, at.len, at.n_new);
    x.seq = at.seq;
    x.head = at.head;
    x.tile = at.tile;
    x.len = at.len;
    x.n_new = at.n_new;
    x.start = at.start;
    x.cost = s.a + s.b * at.tile;
    x.units = tile_units<Kind>(g, s, at.tile);
    const int p0 = at.u - at.start, p1 = min(x.cost, p0 + (end - at.u));
    x.ua = unit_at<Kind>(g, p0, x.units, x.cost, s.per);
    x.ub = unit_at<Kind>(g, p1, x.units, x.cost, s.per);
    at.u += p1 - p0;
    if (at.u < end) {  // to the next item
      at.start = at.u;
      if (++at.tile == s.tiles) {
        at.tile = 0;
        if (++at.head == g.hk) {
          at.head = 0;
          do {  // (the run ends before the sequences do)
            s = line_seq<Kind>(g, ++at.seq);
          } while (s.tiles == 0);
          at.len = s.len;
          at.n_new = s.n_new;
        }
      }
    }
    if (x.ua < x.ub) return true;
  }
  return false;
}

// What the joining kernel reads of a block: whether slot 0 is filled, and of the
// item in slot 1 (last < 0: none) the last block that shares it, its first row and
// the sequence's rows, first token row and head.
struct __align__(16) JoinNote {
  int slot0, last, row0, rows, cu0, head, pad[2];
};
template <class Kind>
__device__ __forceinline__ void note_piece(const CacheAttnArgs& g, const Piece& x, int quota, int cu0,
                                           JoinNote& n) {
  if (x.ub - x.ua == x.units) return;
  if (x.ua > 0) {
    n.slot0 = 1;
  } else {
    n.last = (x.start + x.cost - 1) / quota;
    n.row0 = x.tile * Kind::R;
    n.rows = x.n_new * g.G;
    n.cu0 = cu0;
    n.head = x.head;
  }
}
__device__ __forceinline__ JoinNote empty_note() { return JoinNote{0, -1, 0, 0, 0, 0, {0, 0}}; }
__device__ __forceinline__ JoinNote* notes_of(const CacheAttnArgs& g) { return static_cast<JoinNote*>(g.ws); }

// A workspace slot, behind the notes: R rows of D sums, then R (offset M, sum of weights) pairs; the
// weights are 2^(score - M) and rows without keys have a zero sum.
template <int R, int D>
__host__ __device__ constexpr long long slot_floats() {
  return (long long)R * (D + 2);
}
template <int R, int D>
__device__ __forceinline__ float* slot_of(const CacheAttnArgs& g, int grid, int block, bool begins) {
  return reinterpret_cast<float*>(notes_of(g) + grid) + ((long long)block * 2 + (begins ? 1 : 0)) * slot_floats<R, D>();
}
// The line_shift for a call: `items` items of at most `units` units.
inline int line_shift_for(long long items, long long units) {
  int shift = 0;
  while (items * ((units >> shift) + 2) >= (1LL << 30)) ++shift;
  return shift;
}
template <int R>
size_t line_ws_bytes(int grid, int d) {
  return (size_t)grid * (sizeof(JoinNote) + 2 * R * (d + 2) * sizeof(float));
}

__device__ __forceinline__ void store_lse(const CacheAttnArgs& g, int tok, int hd, float M, float sum) {
  g.lse[(long long)hd * g.l_sh + (long long)tok * g.l_ss] =
      sum > 0.f ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Joins the item in slot 1 of block blockIdx.x, if there is one: rows [8 blockIdx.y,
// 8 blockIdx.y + 8) of its tile, kJoinGroups warps each, which take the pieces in turn.
constexpr int kJoinGroups = 2;
template <int R, int D>
__global__ void __launch_bounds__(32 * 8 * kJoinGroups) cache_join_kernel(const CacheAttnArgs g) {
  constexpr int V = D / 32;
  __shared__ float so[8][D], sm[8][2];
  after_previous_kernel();
  const JoinNote* notes = notes_of(g);
  const JoinNote n = notes[blockIdx.x];
  if (n.last < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp >> 3;
  const int r = blockIdx.y * 8 + (warp & 7), row = n.row0 + r, grid = gridDim.x;
  const bool live = row < n.rows;
  float M = -INFINITY, sum = 0.f, o[V] = {};
  if (live) {
    // this group's pieces: every kJoinGroups-th block, 32 at a time, a lane each
    for (int base = blockIdx.x + group; base <= n.last; base += 32 * kJoinGroups) {
      const int c = base + lane * kJoinGroups;
      const bool begins = c == (int)blockIdx.x, there = begins || (c <= n.last && notes[c].slot0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (there) ml = *reinterpret_cast<const float2*>(slot_of<R, D>(g, grid, c, begins) + R * D + 2 * r);
      float mx = ml.x;
#pragma unroll
      for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      mx = fmaxf(mx, M);
      const float f0 = M == -INFINITY ? 0.f : fast_exp2(M - mx), f1 = there ? fast_exp2(ml.x - mx) : 0.f;
      float part = ml.y * f1;
#pragma unroll
      for (int k = 16; k; k >>= 1) part += __shfl_xor_sync(0xffffffffu, part, k);
      M = mx;
      sum = sum * f0 + part;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] *= f0;
      const unsigned all = __ballot_sync(0xffffffffu, there);
      const int cnt = 32 - __clz(all);  // pieces up to the last that is there
#pragma unroll 8
      for (int k = 0; k < cnt; ++k) {
        const float f = __shfl_sync(0xffffffffu, f1, k);
        const int ck = base + k * kJoinGroups;
        const float* q = slot_of<R, D>(g, grid, ck, ck == (int)blockIdx.x) + r * D + lane * V;
        if ((all >> k) & 1u) {
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 y = *reinterpret_cast<const float2*>(q + i);
            o[i] = fmaf(y.x, f, o[i]);
            o[i + 1] = fmaf(y.y, f, o[i + 1]);
          }
        }
      }
    }
    if (group == 1) {
      if (lane == 0) sm[warp & 7][0] = M, sm[warp & 7][1] = sum;
#pragma unroll
      for (int i = 0; i < V; ++i) so[warp & 7][lane * V + i] = o[i];
    }
  }
  __syncthreads();
  if (!live || group == 1) return;
  {
    const float m1 = sm[warp][0], mx = fmaxf(M, m1);  // (the first piece is group 0's: M is finite)
    const float f0 = fast_exp2(M - mx), f1 = fast_exp2(m1 - mx);
    M = mx;
    sum = sum * f0 + sm[warp][1] * f1;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * f0 + so[warp][lane * V + i] * f1;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = n.cu0 + row / g.G, hd = n.head * g.G + row % g.G;
  const long long to = (long long)tok * g.out.s_row + (long long)hd * g.out.s_head + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if (g.out_f32)
      *reinterpret_cast<float2*>(static_cast<float*>(g.out.data) + to + i) = make_float2(o[i] * inv, o[i + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(g.out.data) + to + i) =
          pack_bf16x2(o[i] * inv, o[i + 1] * inv);
  }
  if (lane == 0) store_lse(g, tok, hd, M, sum);
}

}  // namespace ra
