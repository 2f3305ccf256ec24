// Attention of few new tokens (decoding, verified proposals) over the paged 4-bit
// cache: out = softmax(scale q K^T) V with one pass over the keys.
//
// Work.  An item is one key / value head of one sequence with up to R = 8 NT of
// its query rows (row r is token r / G, head r % G of the group).  Its keys are cut
// into units of 128, all items' units form one line, and each of the grid's blocks
// takes an equal run of that line (lengths are read from device memory, so a
// captured launch follows them).  A run that holds an item whole writes its
// result; pieces of an item go to the workspace as (O, max, sum) and a second
// kernel joins them in block order, so results do not depend on timing.
//
// Each of the 4 warps streams its own 32 keys of a unit through a ring of
// cp.async stages and keeps its own running maximum, sum and O^T; no barrier in
// the loop.  Matrix products are warp-level m16n8k16 on fp16, which holds number *
// scale exactly, with keys (then head dims) as the 16 rows and 8 query rows as
// the columns, so a group of 8 heads wastes nothing:
//   S^T = K Q^T: a lane holds head dims [32 t, 32 t + 32) of rows g, g + 8, one
//     16-byte load each (g = lane / 4, t = lane % 4; the order of the contraction is
//     free as long as Q has the same).
//   O^T = V^T P^T: P^T is the transpose of the score fragment (movmatrix); a lane
//     holds 16 head dims of one scale group, for the keys 2t, 2t + 1, 2t + 8, 2t + 9.
// Queries are scaled per row by a power of two into fp16's normal range.  The
// exponent's offset M keeps the largest p between 2^8 and 2^12, so p down to
// 2^-22 of it has all its fp16 bits; O is rescaled only when a score passes that.
//
// Bound: 0.5625 bytes per number from HBM; the conversions cost about 1.3 lane
// instructions per number against the 3 that fit into its memory time.
#include "ra_cache.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 32 * kWarps;  // keys per unit
constexpr float kLift = 8.f;        // log2 of the largest p when M is set
constexpr float kSlack = 4.f;       // M is raised when a score is this much beyond
constexpr float kNone = -3.0e38f;   // M of a row that has seen no key

template <int D, int NT>
struct Lay {
  static constexpr int R = 8 * NT;
  static constexpr int kK = 0, kV = 32 * D / 2, kKs = 2 * kV, kVs = kKs + 32 * D / 16;
  static constexpr int kStage = kVs + 32 * D / 16;
  static constexpr int kStages = 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kOPitch = D + 4;                          // floats per row of a warp's O
  static constexpr int kMerge = kWarps * R * (kOPitch + 2) * 4;  // reuses the ring
  static constexpr int kQ = kRing > kMerge ? kRing : kMerge;     // R x D fp16, then R floats
  static constexpr int kBytes = kQ + R * D * 2 + R * 4;
};

// Keys of sequence i, its units per (head, row tile) and its row tiles.
struct SeqWork {
  int len, n_new, units, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const CacheAttnArgs& a, int i, int R) {
  SeqWork w;
  w.n_new = __ldg(a.s.cu + i + 1) - __ldg(a.s.cu + i);
  w.len = __ldg(a.s.lens + i);
  w.len = max(0, min(w.len, a.max_kv));
  w.tiles = (w.n_new * a.G + R - 1) / R;
  w.units = w.n_new > 0 ? max(1, (w.len + kUnit - 1) / kUnit) : 0;
  return w;
}
__device__ __forceinline__ long long total_units(const SeqWork& w, int hk) {
  return (long long)w.units * w.tiles * hk;
}

// Sum of v over the block (every thread gets it) and the sum over lower threads.
__device__ __forceinline__ long long block_scan(long long v, long long& below, long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  long long pre = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    pre += w < warp ? sh[w] : 0;
    all += sh[w];
  }
  below = pre + x - v;
  return all;
}

// All units of the call.
__device__ __forceinline__ long long count_units(const CacheAttnArgs& a, int R, long long* sh) {
  long long v = 0, below;
  for (int i = threadIdx.x; i < a.s.n_seqs; i += kThreads) v += total_units(seq_work(a, i, R), a.hk);
  return block_scan(v, below, sh);
}

// The sequence that holds unit u of the line and its first unit (block-wide; u < the total).
__device__ __forceinline__ int find_seq(const CacheAttnArgs& a, int R, long long u, long long& first, long long* sh) {
  __shared__ int s_seq;
  __shared__ long long s_first;
  long long base = 0;
  for (int i0 = 0; i0 < a.s.n_seqs; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const long long v = i < a.s.n_seqs ? total_units(seq_work(a, i, R), a.hk) : 0;
    long long below;
    const long long all = block_scan(v, below, sh);
    if (u >= base + below && u < base + below + v) s_seq = i, s_first = base + below;
    base += all;
    if (u < base) break;
  }
  __syncthreads();
  first = s_first;
  return s_seq;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, bool ok) {
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
// side by side, then the second ones, and for 64-byte rows chunks swapped in
// pairs, so that the 16 lanes of a load phase meet all banks once.
template <int D>
__device__ __forceinline__ uint32_t v_offset(int r, int chunk) {
  const int slot = (r & ~7) | ((r & 1) << 2) | ((r >> 1) & 3);
  return slot * (D / 2) + ((D == 128 ? chunk ^ (slot & 2) : chunk) << 4);
}

// One of a segment's keys tiles: its pages, prefetched, and its copies.
template <int D, int NT>
struct Stream {
  using L = Lay<D, NT>;
  const CacheAttnArgs& a;
  const int* table;
  int head, len, pa, pb;
  uint32_t ring;

  __device__ __forceinline__ Stream(const CacheAttnArgs& args, int seq, int h, int n, uint32_t r)
      : a(args), table(args.s.table + (long long)seq * args.s.table_stride), head(h), len(n), pa(0), pb(0), ring(r) {}

  __device__ __forceinline__ void pages(int k0) {
    if (k0 < len) {
      pa = __ldg(table + (k0 >> a.c.page_shift));
      pb = k0 + 16 < len ? __ldg(table + ((k0 + 16) >> a.c.page_shift)) : pa;
    }
  }
  __device__ __forceinline__ void load(int k0, int slot) {
    if (k0 < len) {
      const int lane = threadIdx.x & 31;
      const bool oka = (unsigned)pa < (unsigned)a.c.n_pages, okb = (unsigned)pb < (unsigned)a.c.n_pages;
      if (!(oka && okb) && lane == 0) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_PAGE);
      const int xa = oka ? pa : 0, xb = okb ? pb : 0, mask = (1 << a.c.page_shift) - 1;
      const uint32_t dst = ring + slot * L::kStage;
      constexpr int CPR = D / 32;  // 16-byte chunks per row
#pragma unroll
      for (int j = 0; j < CPR; ++j) {
        const int r = j * (32 / CPR) + lane / CPR, c = lane % CPR;
        const bool ok = k0 + r < len && (j < CPR / 2 ? oka : okb);
        const int pg = j < CPR / 2 ? xa : xb, row = (k0 + r) & mask;
        cp16(dst + L::kK + r * (D / 2) + c * 16, a.c.k.data + row_offset(a.c.k, pg, head, row) + c * 16, ok);
        cp16(dst + L::kV + v_offset<D>(r, c), a.c.v.data + row_offset(a.c.v, pg, head, row) + c * 16, ok);
      }
      const int pg = lane < 16 ? xa : xb, row = (k0 + lane) & mask;
      const bool ok = k0 + lane < len && (lane < 16 ? oka : okb);
      cp_small<D / 16>(dst + L::kKs + lane * (D / 16), a.c.ks.data + row_offset(a.c.ks, pg, head, row), ok);
      cp_small<D / 16>(dst + L::kVs + lane * (D / 16), a.c.vs.data + row_offset(a.c.vs, pg, head, row), ok);
    }
    cp_commit();
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) cache_attn_kernel(const CacheAttnArgs a) {
  using L = Lay<D, NT>;
  constexpr int R = L::R, KS = D / 16;  // contraction steps of S, row tiles of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long sh[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t sb = smem_u32(smem), ring = sb + warp * L::kStages * L::kStage;
  __half* sq = reinterpret_cast<__half*>(smem + L::kQ);
  float* sscale = reinterpret_cast<float*>(smem + L::kQ + R * D * 2);

  const long long all = count_units(a, R, sh);
  const long long quota = (all + gridDim.x - 1) / gridDim.x;
  long long u = blockIdx.x * quota;
  const long long u_end = min(all, u + quota);
  if (u >= u_end) return;
  long long first;
  int seq = find_seq(a, R, u, first, sh);
  SeqWork w = seq_work(a, seq, R);
  if (threadIdx.x == 0 && __ldg(a.s.lens + seq) > a.max_kv) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_LEN);

  while (u < u_end) {
    // ---------------------------------------------------------------- the next item
    while (u - first >= total_units(w, a.hk)) {
      first += total_units(w, a.hk);
      w = seq_work(a, ++seq, R);
      if (threadIdx.x == 0 && __ldg(a.s.lens + seq) > a.max_kv) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_LEN);
    }
    const int item = (int)((u - first) / w.units), ua = (int)((u - first) % w.units);
    const int ub = (int)min((long long)w.units, ua + (u_end - u));
    const int head = item / w.tiles, row0 = (item % w.tiles) * R;
    const int cu0 = __ldg(a.s.cu + seq), rows = min(R, w.n_new * a.G - row0);
    const int n_it = ub - ua, kbase = ua * kUnit + warp * 32;

    Stream<D, NT> st(a, seq, head, w.len, ring);
    st.pages(kbase);
#pragma unroll
    for (int s = 0; s < L::kStages - 1; ++s) {
      if (s < n_it)
        st.load(kbase + s * kUnit, s);
      else
        cp_commit();
      if (s + 1 < n_it) st.pages(kbase + (s + 1) * kUnit);
    }

    // ---------------------------------------------------------------- queries
    {
      constexpr int LPR = D / 8;  // lanes per row
      for (int r = threadIdx.x / LPR; r < R; r += kThreads / LPR) {
        const int c = threadIdx.x % LPR, rr = row0 + r;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int tok = cu0 + rr / a.G, hd = head * a.G + rr % a.G;
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
        *reinterpret_cast<uint4*>(sq + r * D + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0) sscale[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e - 12) << 23);
      }
    }
    __syncthreads();
    uint32_t qb[NT][KS][2];
    float sc[NT][2];
    int end[NT][2], min_end = w.len;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint2 v = *reinterpret_cast<const uint2*>(sq + (8 * n + g) * D + (D / 4) * t + 4 * s);
        qb[n][s][0] = v.x, qb[n][s][1] = v.y;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * n + 2 * t + x;
        sc[n][x] = sscale[r];
        end[n][x] = w.len;
        if (a.causal && r < rows) end[n][x] = min(w.len, w.len - w.n_new + (row0 + r) / a.G + 1);
      }
    }
    if (a.causal) min_end = min(w.len, w.len - w.n_new + row0 / a.G + 1);

    // ---------------------------------------------------------------- keys
    float o[NT][KS][4], M[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < KS; ++s) o[n][s][0] = o[n][s][1] = o[n][s][2] = o[n][s][3] = 0.f;
      M[n][0] = M[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
    }
    for (int it = 0; it < n_it; ++it) {
      cp_wait<L::kStages - 2>();
      __syncwarp();
      const int nx = it + L::kStages - 1;
      if (nx < n_it) {
        st.load(kbase + nx * kUnit, nx % L::kStages);
        if (nx + 1 < n_it) st.pages(kbase + (nx + 1) * kUnit);
      } else {
        cp_commit();
      }
      const int k0 = kbase + it * kUnit;
      if (k0 >= w.len) continue;
      const uint32_t stg = ring + (it % L::kStages) * L::kStage;
      // scores of 32 keys: rows g, g + 8 of two tiles
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
        uint32_t ka[D / 32], kb[D / 32];
        const uint32_t ra = stg + L::kK + (16 * mt + g) * (D / 2) + t * (D / 8);
        lds_words(ra, ka);
        lds_words(ra + 8 * (D / 2), kb);
        uint32_t sa, sbq;  // this lane's one (d = 64) or two scales of each row
        const uint32_t rs = stg + L::kKs + (16 * mt + g) * (D / 16) + t * (D / 64);
        if constexpr (D == 128) {
          sa = e4m3x2_to_f16(lds16(rs));
          sbq = e4m3x2_to_f16(lds16(rs + 8 * (D / 16)));
        } else {
          sa = e4m3x2_to_f16(lds8(rs));
          sbq = e4m3x2_to_f16(lds8(rs + 8 * (D / 16)));
        }
#pragma unroll
        for (int wd = 0; wd < D / 32; ++wd) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16(ka[wd], x);
          e2m1x8_to_f16(kb[wd], y);
          const uint32_t s_a = wd < 2 ? half_lo2(sa) : half_hi2(sa), s_b = wd < 2 ? half_lo2(sbq) : half_hi2(sbq);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = hmul2(x[i], s_a), y[i] = hmul2(y[i], s_b);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t f[4] = {x[2 * v], y[2 * v], x[2 * v + 1], y[2 * v + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[mt][n], f, qb[n][2 * wd + v][0], qb[n][2 * wd + v][1]);
          }
        }
      }
      // log2 scores, masked; M is raised only when one of them passes it by far
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[mt][n][x] *= sc[n][x & 1];
      if (k0 + 32 > min_end) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (k0 + 16 * mt + g + 8 * (x >> 1) >= end[n][x & 1]) s[mt][n][x] = -INFINITY;
      }
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[n][x] = fmaxf(fmaxf(s[0][n][x], s[0][n][x + 2]), fmaxf(s[1][n][x], s[1][n][x + 2]));
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
            p[x] = fast_exp2(s[mt][n][x] - M[n][x & 1]);
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
          const int r = 16 * mt + 2 * t + (k & 1) + 8 * (k >> 1);
          lds_words(stg + L::kV + v_offset<D>(r, g * W / 4) + (g * W % 4) * 4, v[k]);
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
            e2m1x8_to_f16((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), f[2 * k]);
            e2m1x8_to_f16(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), f[2 * k + 1]);
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
    cp_wait<0>();
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);           // [warp][row][kOPitch]
    float* sm = so + kWarps * R * L::kOPitch;             // [warp][row] M, then sums
    float* sl = sm + kWarps * R;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = l[n][x];
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        const int r = 8 * n + 2 * t + x;
        if (g == 0) sm[warp * R + r] = M[n][x], sl[warp * R + r] = v;
#pragma unroll
        for (int d = 0; d < KS; ++d)  // head dims D / 8 g + 2 d, + 1 at place 16 d + 2 g
          *reinterpret_cast<float2*>(so + (warp * R + r) * L::kOPitch + 16 * d + 2 * g) =
              make_float2(o[n][d][x], o[n][d][x + 2]);
      }
    }
    __syncthreads();
    const bool whole = ua == 0 && ub == w.units;
    float* part = static_cast<float*>(a.ws) + ((long long)blockIdx.x * 2 + (ua > 0 ? 0 : 1)) * R * (D + 2);
    for (int e = threadIdx.x; e < rows * (D / 2); e += kThreads) {
      const int r = e / (D / 2), d = e % (D / 2) * 2;
      const int at = (d % (D / 8)) / 2 * 16 + d / (D / 8) * 2;
      float m = sm[r];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) m = fmaxf(m, sm[k * R + r]);
      float lsum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float f = fast_exp2(sm[k * R + r] - m);
        const float2 v = *reinterpret_cast<const float2*>(so + (k * R + r) * L::kOPitch + at);
        lsum += sl[k * R + r] * f;
        o0 += v.x * f, o1 += v.y * f;
      }
      if (!whole) {
        *reinterpret_cast<float2*>(part + r * (D + 2) + 2 + d) = make_float2(o0, o1);
        if (d == 0) *reinterpret_cast<float2*>(part + r * (D + 2)) = make_float2(m, lsum);
      } else {
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
        const int rr = row0 + r, tok = cu0 + rr / a.G, hd = head * a.G + rr % a.G;
        const long long at_o = (long long)tok * a.out.s_row + (long long)hd * a.out.s_head + d;
        if (a.out_f32)
          *reinterpret_cast<float2*>(static_cast<float*>(a.out.data) + at_o) = make_float2(o0 * inv, o1 * inv);
        else
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out.data) + at_o) = pack_bf16x2(o0 * inv, o1 * inv);
        if (d == 0)
          a.lse[(long long)hd * a.l_sh + (long long)tok * a.l_ss] =
              lsum > 0.f ? (m + log2f(lsum)) * 0.6931471805599453f : -INFINITY;
      }
    }
    __syncthreads();
    u += n_it;
  }
}

// Joins the pieces of one query row of one item: the block in which the item
// begins left its piece in its slot 1, those that begin inside the item in slot 0.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) cache_join_kernel(const CacheAttnArgs a, int grid) {
  constexpr int R = 8 * NT;
  __shared__ long long sh[kWarps];
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = blockIdx.x, hd = blockIdx.y;
  const long long all = count_units(a, R, sh);
  const long long quota = (all + grid - 1) / grid;
  const int seq = segment_of_warp(a.s.cu, a.s.n_seqs, tok);
  long long v = 0, below;
  for (int i = threadIdx.x; i < seq; i += kThreads) v += total_units(seq_work(a, i, R), a.hk);
  const long long first = block_scan(v, below, sh);
  const SeqWork w = seq_work(a, seq, R);
  const int rr = (tok - __ldg(a.s.cu + seq)) * a.G + hd % a.G, r = rr % R;
  const long long u0 = first + ((long long)(hd / a.G) * w.tiles + rr / R) * w.units, u1 = u0 + w.units;
  const long long c0 = u0 / quota, c1 = (u1 - 1) / quota;
  if (c0 == c1) return;
  constexpr int V = D / 32;
  float m = kNone, lsum = 0.f, o[V] = {};
  for (long long c = c0 + warp; c <= c1; c += kWarps) {
    const float* part = static_cast<const float*>(a.ws) + ((c * 2 + (c == c0 ? 1 : 0)) * R + r) * (D + 2);
    const float2 ml = *reinterpret_cast<const float2*>(part);
    const float to = fmaxf(m, ml.x), f0 = fast_exp2(m - to), f1 = fast_exp2(ml.x - to);
    m = to;
    lsum = lsum * f0 + ml.y * f1;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(part + 2 + lane * V + i);
      o[i] = o[i] * f0 + x.x * f1;
      o[i + 1] = o[i + 1] * f0 + x.y * f1;
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = lsum;
#pragma unroll
  for (int i = 0; i < V; ++i) so[warp][lane * V + i] = o[i];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float mm = sm[0];
    for (int k = 1; k < kWarps; ++k) mm = fmaxf(mm, sm[k]);
    float ls = 0.f, x = 0.f;
    for (int k = 0; k < kWarps; ++k) {
      const float f = fast_exp2(sm[k] - mm);
      ls += sl[k] * f;
      x += so[k][d] * f;
    }
    x *= ls > 0.f ? 1.f / ls : 0.f;
    const long long at = (long long)tok * a.out.s_row + (long long)hd * a.out.s_head + d;
    if (a.out_f32)
      static_cast<float*>(a.out.data)[at] = x;
    else
      static_cast<__nv_bfloat16*>(a.out.data)[at] = __float2bfloat16(x);
    if (d == 0)
      a.lse[(long long)hd * a.l_sh + (long long)tok * a.l_ss] = ls > 0.f ? (mm + log2f(ls)) * 0.6931471805599453f : -INFINITY;
  }
}

// Blocks that fit on an SM (registers and shared memory), so the grid is one wave.
int blocks_per_sm(int nt) { return nt == 4 ? 2 : 3; }

// Query rows of an item in units of 8.
int row_tiles(long long rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int D, int NT>
cudaError_t launch(const CacheAttnArgs& a, cudaStream_t st) {
  using L = Lay<D, NT>;
  cudaError_t e = configure_kernel<cache_attn_kernel<D, NT>>(0, L::kBytes);
  if (e != cudaSuccess) return e;
  const int grid = num_sms() * blocks_per_sm(NT);
  cache_attn_kernel<D, NT><<<grid, kThreads, L::kBytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_join_kernel<D, NT><<<dim3((unsigned)a.s.total, (unsigned)a.h), kThreads, 0, st>>>(a, grid);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_ws_bytes(long long, int max_new, int h, int hk, int d, int) {
  const int nt = row_tiles((long long)max_new * (h / hk));
  return (size_t)num_sms() * blocks_per_sm(nt) * 2 * 8 * nt * (d + 2) * sizeof(float);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t st) {
  const int nt = row_tiles((long long)a.max_new * a.G);
  if (a.d == 64) return nt == 1 ? launch<64, 1>(a, st) : nt == 2 ? launch<64, 2>(a, st) : launch<64, 4>(a, st);
  return nt == 1 ? launch<128, 1>(a, st) : nt == 2 ? launch<128, 2>(a, st) : launch<128, 4>(a, st);
}

}  // namespace ra
