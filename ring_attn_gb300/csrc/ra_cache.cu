// Appending to and reading from the paged 4-bit key / value cache.
//
// Both are bound by memory: a new token moves 4 d bytes per query head, 2 d per
// key and value head in and 0.5625 d out, a read token 0.5625 d in and 2 d out.
// A row (one head of one token) is handled by d / 8 lanes, 8 numbers (16 bytes
// of bf16, 4 bytes of codes) each, so two neighbouring lanes share a scale.
#include "ra_cache.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// q with its last bit set when something (`rest`, of magnitude below one unit
// in the last place) is missing from it: rounding to odd.
__device__ __forceinline__ float to_odd(float q, float rest) {
  int bits = __float_as_int(q);
  if (rest != 0.f && !(bits & 1)) bits += ((rest > 0.f) == (bits >= 0)) ? 1 : -1;
  return __int_as_float(bits);
}

// a * b + c * d to about 2^-47 as hi + lo (two exact products, an exact sum of
// the leading parts), rounded to odd: hi's last bit is set when bits are missing,
// so a later rounding to few bits, or a comparison with a number of few bits,
// comes out as for the exact value.
__device__ __forceinline__ float dot2_odd(float a, float b, float c, float d) {
  const float p = __fmul_rn(a, b), q = __fmul_rn(c, d);
  const float ep = __fmaf_rn(a, b, -p), eq = __fmaf_rn(c, d, -q);
  const float s = __fadd_rn(p, q);
  const float t = __fsub_rn(s, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t));
  const float lo = __fadd_rn(es, __fadd_rn(ep, eq));
  const float hi = __fadd_rn(s, lo);
  const float rest = __fadd_rn(__fsub_rn(s, hi), lo);
  // an infinite input gives the plain sum
  return fabsf(hi) <= 3.0e38f ? to_odd(hi, rest) : s;
}

// x / s rounded to odd (r: the reciprocal of s, rounded): one correction step
// brings the quotient within a unit of its last place, and the remainder's sign
// says on which side the exact one lies, so that the conversion to 4 or 8 bits
// rounds as for the exact quotient.
__device__ __forceinline__ float div_odd(float x, float s, float r) {
  const float q0 = __fmul_rn(x, r);
  const float q = __fmaf_rn(__fmaf_rn(-q0, s, x), r, q0);
  return fabsf(q0) < 1e30f ? to_odd(q, __fmaf_rn(-q, s, x)) : q0;
}

__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b16 %0, {t, 0};\n\t}\n"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r;
}

// The scale byte of a group of 16 numbers held 8 each by lanes 2i and 2i + 1,
// and the four code bytes of the caller's 8.
__device__ __forceinline__ void quantise8(const float (&x)[8], uint32_t& codes, uint32_t& scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fminf(m, 6.f * 448.f);
  const float q = div_odd(m, 6.f, 1.f / 6.f);
  scale = to_e4m3(q);
  if (scale == 0) scale = 1;  // 2^-9
  const float s = f16x2_to_f32(e4m3x2_to_f16(scale)).x;
  const float r = __frcp_rn(s);
  codes = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) codes |= to_e2m1x2(div_odd(x[i], s, r), div_odd(x[i + 1], s, r)) << (4 * i);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// One warp: `passes` times 32 / (d / 8) rows of one token.  Rows are the query
// heads, then the key heads, then the value heads.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(AppendArgs a, int warps_per_token, int passes) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long gw = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(gw / warps_per_token);
  if (t >= a.s.total) return;
  const int row0 = (int)(gw % warps_per_token) * passes * RPP;
  const int i = segment_of_warp(a.s.cu, a.s.n_seqs, t);
  const int n_end = __ldg(a.s.cu + i + 1);
  const int len = cache_len(a.s, i, a.s.max_tokens, a.ctl);
  const int tok = len - n_end + t;
  if (tok < 0) return;
  const int c = lane % LPR, half = a.rot >> 4;  // this lane's 8 numbers; chunks in half the rotated part
  float cs[8], sn[8];
  if (a.rot) {
    const int pos = a.positions ? __ldg(a.positions + t) : tok;
    if ((unsigned)pos >= (unsigned)a.max_pos) {
      if (lane == 0) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_POS);
      return;
    }
    const bool inter = a.style == 1;
    const int at = inter ? 4 * c : 8 * (c < half ? c : c - half);
    const bool turn = 8 * c < a.rot;
    const float4* pc = reinterpret_cast<const float4*>(a.cos_t + (long long)pos * a.cos_stride + at);
    const float4* ps = reinterpret_cast<const float4*>(a.sin_t + (long long)pos * a.sin_stride + at);
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 c0 = turn ? __ldg(pc) : one, s0 = turn ? __ldg(ps) : zero;
    const float4 c1 = turn && !inter ? __ldg(pc + 1) : one, s1 = turn && !inter ? __ldg(ps + 1) : zero;
    cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
    sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
  }
  const int page = cache_page(a.s, a.c, i, tok, a.ctl);
  if (page < 0) return;
  const int prow = tok & ((1 << a.c.page_shift) - 1);
  const int n_rows = a.h + 2 * a.hk;
  for (int p = 0; p < passes; ++p) {
    const int row = row0 + p * RPP + lane / LPR;
    const bool live = row < n_rows;
    const bool is_q = row < a.h, is_v = row >= a.h + a.hk;
    const int head = is_q ? row : is_v ? row - a.h - a.hk : row - a.h;
    const Rows3& src = is_q ? a.q : is_v ? a.v : a.k;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live)
      w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src.data) + (long long)t * src.s_row +
                                          (long long)head * src.s_head + 8 * c);
    float x[8];
    unpack8(w, x);
    if (a.rot) {
      const bool turn = !is_v && 8 * c < a.rot;
      if (a.style == 1) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float xa = x[2 * u], xb = x[2 * u + 1];
          if (turn) {
            x[2 * u] = dot2_odd(xa, cs[u], -xb, sn[u]);
            x[2 * u + 1] = dot2_odd(xb, cs[u], xa, sn[u]);
          }
        }
      } else {
        const bool first = c < half;
        const int from = lane - c + (turn ? (first ? c + half : c - half) : c);
        uint4 z;
        z.x = __shfl_sync(0xffffffffu, w.x, from);
        z.y = __shfl_sync(0xffffffffu, w.y, from);
        z.z = __shfl_sync(0xffffffffu, w.z, from);
        z.w = __shfl_sync(0xffffffffu, w.w, from);
        float y[8];
        unpack8(z, y);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (turn) x[u] = dot2_odd(x[u], cs[u], first ? -y[u] : y[u], sn[u]);
      }
    }
    uint32_t codes, scale;
    quantise8(x, codes, scale);
    if (!live) continue;
    if (is_q) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out.data) + (long long)t * a.q_out.s_row +
                                (long long)head * a.q_out.s_head + 8 * c) = pack8(x);
    } else {
      const CacheRows& cr = is_v ? a.c.v : a.c.k;
      const CacheRows& sr = is_v ? a.c.vs : a.c.ks;
      *reinterpret_cast<uint32_t*>(cr.data + row_offset(cr, page, head, prow) + 4 * c) = codes;
      if (!(c & 1)) sr.data[row_offset(sr, page, head, prow) + (c >> 1)] = (uint8_t)scale;
    }
  }
}

// One warp: 32 / (d / 8) rows at a time of one token; rows are the key heads, then the value heads.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(ReadArgs a) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.s.total) return;
  const int i = segment_of_warp(a.s.cu, a.s.n_seqs, t);
  const int len = cache_len(a.s, i, a.s.max_tokens, a.ctl);
  const int tok = len - __ldg(a.s.cu + i + 1) + t;
  if (tok < 0) return;
  const int page = cache_page(a.s, a.c, i, tok, a.ctl);
  if (page < 0) return;
  const int prow = tok & ((1 << a.c.page_shift) - 1);
  const int c = lane % LPR;
  for (int row = lane / LPR; row < 2 * a.hk; row += RPP) {
    const bool is_v = row >= a.hk;
    const int head = is_v ? row - a.hk : row;
    const CacheRows& cr = is_v ? a.c.v : a.c.k;
    const CacheRows& sr = is_v ? a.c.vs : a.c.ks;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(cr.data + row_offset(cr, page, head, prow) + 4 * c);
    const uint32_t s2 = half_lo2(e4m3x2_to_f16(sr.data[row_offset(sr, page, head, prow) + (c >> 1)]));
    uint32_t r[4];
    e2m1x8_to_f16(w, r);
    float x[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f = f16x2_to_f32(hmul2(r[u], s2));
      x[2 * u] = f.x, x[2 * u + 1] = f.y;
    }
    const Rows3& o = is_v ? a.v_out : a.k_out;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o.data) + (long long)t * o.s_row +
                              (long long)head * o.s_head + 8 * c) = pack8(x);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  const int rpp = 256 / a.d, need = (a.h + 2 * a.hk + rpp - 1) / rpp;  // passes for all rows of a token
  const int passes = 1;
  const int wpt = (need + passes - 1) / passes;
  const long long blocks = ((long long)a.s.total * wpt + kWarps - 1) / kWarps;
  if (a.d == 64)
    cache_append_kernel<64><<<(unsigned)blocks, kThreads, 0, st>>>(a, wpt, passes);
  else
    cache_append_kernel<128><<<(unsigned)blocks, kThreads, 0, st>>>(a, wpt, passes);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.s.total + kWarps - 1) / kWarps);
  if (a.d == 64)
    cache_read_kernel<64><<<blocks, kThreads, 0, st>>>(a);
  else
    cache_read_kernel<128><<<blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace ra
