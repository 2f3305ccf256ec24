// Rotary positions: queries and keys turned by table rows that their positions name, on one
// axis or several; turned back for the backward.
//
// Bound by memory: every number is read and written once (4 bytes in bf16), and a token's table
// entries, 4 r bytes, serve all of its heads.  A warp takes 32 / (d / 16) rows of one head
// at a time, with their tokens' entries in registers, and goes through a range of heads, four in flight (two: 2 %
// slower, eight: 3 %; the first four asked for before the positions are looked up: 18 %, for the registers).
// 65,536 tokens of 32 + 8 heads of 128, three axes: 200 us, 6.9 TB/s (101 % of the measured copy rate); 9001 tokens
// of 16 + 16 heads of 64, turned back: 14.5 us a launch within a graph, 5.2 TB/s, and 17.3 as separate calls: 1126 blocks,
// of which 760 are resident at a time (95 registers: 20 warps an SM), a wave and a half.
#include "ra_cache.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kAhead = 4;  // heads whose rows a warp has in flight

// A lane's 8 numbers of a row.
struct Eight {
  float x[8];
};
__device__ __forceinline__ void load8(const __nv_bfloat16* p, uint4 (&w)[1]) {
  w[0] = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load8(const float* p, uint4 (&w)[2]) {
  w[0] = reinterpret_cast<const uint4*>(p)[0], w[1] = reinterpret_cast<const uint4*>(p)[1];
}
__device__ __forceinline__ Eight unpack(const uint4 (&w)[1]) {
  const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.x[2 * i] = __uint_as_float(u[i] << 16);
    e.x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return e;
}
__device__ __forceinline__ Eight unpack(const uint4 (&w)[2]) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    e.x[4 * i] = __uint_as_float(w[i].x), e.x[4 * i + 1] = __uint_as_float(w[i].y);
    e.x[4 * i + 2] = __uint_as_float(w[i].z), e.x[4 * i + 3] = __uint_as_float(w[i].w);
  }
  return e;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& e) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(e.x[0], e.x[1]), pack_bf16x2(e.x[2], e.x[3]),
                                            pack_bf16x2(e.x[4], e.x[5]), pack_bf16x2(e.x[6], e.x[7]));
}
__device__ __forceinline__ void store8(float* p, const Eight& e) {
  reinterpret_cast<float4*>(p)[0] = make_float4(e.x[0], e.x[1], e.x[2], e.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(e.x[4], e.x[5], e.x[6], e.x[7]);
}

// A lane's two chunks of 8 numbers: the two that turn together (l, l + r / 16) for pairs
// (i, i + r / 2), else neighbours (2 l, 2 l + 1); either way the lane's pairs are 8 l .. 8 l + 7.
template <class T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, int parts, int heads_per_part) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, W = sizeof(T) / 2;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  after_previous_kernel();
  const long long rows = (long long)a.b * a.s;
  const long long n_warps = (rows + RPW - 1) / RPW * parts;
  const int heads = a.h[0] + a.h[1], half = a.rot >> 4;
  const bool turn = HALVES ? l < half : 16 * l < a.rot;
  const int ca = 8 * (HALVES && turn ? l : 2 * l), cb = 8 * (HALVES && turn ? l + half : 2 * l + 1);
  const long long step = (long long)gridDim.x * kWarps;
  for (long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); gw < n_warps; gw += step) {
    const int part = (int)(gw % parts);
    const long long row = gw / parts * RPW + lane / LPR;
    bool live = row < rows;
    const int bi = live ? (int)(row / a.s) : 0, i = live ? (int)(row - (long long)bi * a.s) : 0;
    float cs[8], sn[8];
    if (live && turn) {
      const int* at = a.pos + bi * a.p_b + i * a.p_s;
      int tok = 0;
      if (!a.pos) {
        const int L = a.s / a.N;
        tok = token_of(a.layout, a.N, L, i / L, i % L);
      }
      auto place = [&](int pair) -> int {  // the pair's table row, or -1
        const int p = a.pos ? at[a.axis[pair] * a.p_axis] : tok;
        return (unsigned)p < (unsigned)a.max_pos ? p : -1;
      };
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int f = 8 * l + 4 * g;
        if (!((a.mixed >> (f >> 2)) & 1u)) {
          const int p = place(f);
          if (p < 0) {
            live = false;
          } else {
            const float4 c = *reinterpret_cast<const float4*>(a.cos_t + p * a.cos_stride + f);
            const float4 s = *reinterpret_cast<const float4*>(a.sin_t + p * a.sin_stride + f);
            cs[4 * g] = c.x, cs[4 * g + 1] = c.y, cs[4 * g + 2] = c.z, cs[4 * g + 3] = c.w;
            sn[4 * g] = s.x, sn[4 * g + 1] = s.y, sn[4 * g + 2] = s.z, sn[4 * g + 3] = s.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int p = place(f + k);
            if (p < 0) {
              live = false;
            } else {
              cs[4 * g + k] = a.cos_t[p * a.cos_stride + f + k];
              sn[4 * g + k] = a.sin_t[p * a.sin_stride + f + k];
            }
          }
        }
      }
      if (!live) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_POS);
      if (a.inverse)
#pragma unroll
        for (int k = 0; k < 8; ++k) sn[k] = -sn[k];
    }
    // a row is left out by all of its lanes
    const unsigned all = __ballot_sync(0xffffffffu, live), mine = ((1u << LPR) - 1u) << (lane / LPR * LPR);
    live = (all & mine) == mine;
    const int h1 = min(heads, (part + 1) * heads_per_part);
    for (int h0 = part * heads_per_part; h0 < h1; h0 += kAhead) {
      uint4 x[kAhead][W], y[kAhead][W];
      T* dst[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int h = h0 + k;
        if (live && h < h1) {
          const int w = h >= a.h[0], hh = w ? h - a.h[0] : h;
          const RopeRows &in = w ? a.in[1] : a.in[0], &out = w ? a.out[1] : a.out[0];
          const T* src = static_cast<const T*>(in.data) + bi * in.sb + hh * in.sh + i * in.ss;
          dst[k] = static_cast<T*>(out.data) + bi * out.sb + hh * out.sh + i * out.ss;
          load8(src + ca, x[k]);
          load8(src + cb, y[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!live || h0 + k >= h1) continue;
        Eight u = unpack(x[k]), v = unpack(y[k]);
        if (turn) {
          const Eight p = u, q = v;
          if (HALVES) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              u.x[j] = fmaf(p.x[j], cs[j], -q.x[j] * sn[j]);
              v.x[j] = fmaf(q.x[j], cs[j], p.x[j] * sn[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u.x[2 * j] = fmaf(p.x[2 * j], cs[j], -p.x[2 * j + 1] * sn[j]);
              u.x[2 * j + 1] = fmaf(p.x[2 * j + 1], cs[j], p.x[2 * j] * sn[j]);
              v.x[2 * j] = fmaf(q.x[2 * j], cs[j + 4], -q.x[2 * j + 1] * sn[j + 4]);
              v.x[2 * j + 1] = fmaf(q.x[2 * j + 1], cs[j + 4], q.x[2 * j] * sn[j + 4]);
            }
          }
        }
        store8(dst[k] + ca, u);
        store8(dst[k] + cb, v);
      }
    }
  }
}

template <class T, int D, bool HALVES>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16);
  const long long groups = ((long long)a.b * a.s + RPW - 1) / RPW;
  const int heads = a.h[0] + a.h[1], most = (heads + kAhead - 1) / kAhead;
  // few tokens: their heads go to several warps, up to 32 for every SM, of which 20 are resident (9001 tokens of 32 heads
  // of 64: 17.3 us, 18.5 with 16, 18.3 with 64)
  const long long want = (32LL * num_sms() + groups - 1) / groups;
  const int turns = (most + (int)(want < most ? want : most) - 1) / (int)(want < most ? want : most);
  const int parts = (most + turns - 1) / turns;
  const long long blocks = (groups * parts + kWarps - 1) / kWarps;
  const int grid = (int)(blocks < (1LL << 30) ? blocks : (1LL << 30));
  return launch_early(rope_kernel<T, D, HALVES>, dim3(grid), dim3(kThreads), 0, st, a, parts, turns * kAhead);
}
template <class T>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  const bool halves = a.style == 0;
  if (a.d == 64) return halves ? launch<T, 64, true>(a, st) : launch<T, 64, false>(a, st);
  return halves ? launch<T, 128, true>(a, st) : launch<T, 128, false>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  return a.f32 ? launch_t<float>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace ra
