// Appending to and reading from the paged 4-bit key / value cache.
//
// Both are bound by memory: a new token moves 4 d bytes per query head, 2 d per
// key and value head in and 0.5625 d out, a read token 0.5625 d in and 2 d out.
// One pass, a warp per token (or a part of one when tokens are few), no shared memory.
// 65,536 tokens of 32 + 2 x 8 heads of 128 are appended in 254 us (1.45 GB, 5.7 TB/s: 85 % of
// the measured copy rate; half the issue slots go to the rotation and its bounds),
// 131,072 tokens of 2 x 8 heads read in 104 us (0.69 GB, 6.6 TB/s: 99 %).
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

// x / s (r: the reciprocal of s, rounded): one correction step brings the quotient
// within half a unit of its last place.
__device__ __forceinline__ float near_quotient(float x, float s, float r) {
  const float q0 = __fmul_rn(x, r);
  return fabsf(q0) < 1e30f ? __fmaf_rn(__fmaf_rn(-q0, s, x), r, q0) : q0;
}
// x / s rounded to odd: the remainder's sign says on which side of the quotient
// the exact one lies, so that the conversion to 4 or 8 bits rounds as for that.
__device__ __forceinline__ float div_odd(float x, float s, float r) {
  const float q = near_quotient(x, s, r);
  return fabsf(q) < 1e30f ? to_odd(q, __fmaf_rn(-q, s, x)) : q;
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

__device__ __forceinline__ float max8(const float (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) m = fmax3f(m, fabsf(x[i]), fabsf(x[i + 1]));
  return m;
}
// The scale byte of a group whose largest magnitude is m, given as fp32 rounded to odd.
__device__ __forceinline__ uint32_t scale_of(float m) {
  const uint32_t s = to_e4m3(div_odd(fminf(m, 6.f * 448.f), 6.f, 1.f / 6.f));
  return s ? s : 1u;  // at least 2^-9
}
// Four code bytes of 8 numbers of a group with the given scale byte.  ODD: the
// numbers are rounded to odd; otherwise they are bf16, whose quotients by a scale
// lie on a border or at least 2^-9 of it away, so that the rounded quotient (one correction step,
// right to half a unit in the last place) is enough.
template <bool ODD>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], uint32_t scale) {
  const float s = f16x2_to_f32(e4m3x2_to_f16(scale)).x, r = __frcp_rn(s);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      q[k] = ODD ? div_odd(x[i + k], s, r) : near_quotient(x[i + k], s, r);
    }
    codes |= to_e2m1x2(q[0], q[1]) << (4 * i);
  }
  return codes;
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

// sure_scale and sure_codes: scale_of and codes_of for fp32 numbers known to within
// `off`, setting `unsure` where that leaves two answers.  exact: the numbers are bf16
// (not rotated; they often lie on borders), and the answers are final.
__device__ __forceinline__ uint32_t sure_scale(float m, float off, bool exact, bool& unsure) {
  // (m / 6 as a product: no bf16 m lies so near a border of e4m3 that it matters)
  const float q = fminf(m, 6.f * 448.f) * (1.f / 6.f), d = exact ? 0.f : fmaf(q, 0x1p-22f, off);
  const uint32_t lo = to_e4m3(q - d), hi = to_e4m3(q + d);
  unsure |= lo != hi;
  return hi ? hi : 1u;
}
__device__ __forceinline__ uint32_t sure_codes(const float (&x)[8], uint32_t scale, float off, bool exact, bool& unsure) {
  const float s = f16x2_to_f32(e4m3x2_to_f16(scale)).x, r = __frcp_rn(s);
  const float d = exact ? 0.f : fmaf(off, r, 0x1p-19f);  // quotients up to 8 in fp32 are off by less than the second part
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float q0 = near_quotient(x[i], s, r), q1 = near_quotient(x[i + 1], s, r);
    lo |= to_e2m1x2(q0 - d, q1 - d) << (4 * i);
    hi |= to_e2m1x2(q0 + d, q1 + d) << (4 * i);
  }
  unsure |= lo != hi;
  return hi;
}

// The two chunks x, y of a lane turned by its table entries; f(a, c, b, d) = a c + b d.
template <int STYLE, class F>
__device__ __forceinline__ void rotate16(const float (&x)[8], const float (&y)[8], const float (&cs)[8],
                                         const float (&sn)[8], bool turn, float (&u)[8], float (&v)[8], F f) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (STYLE == 1) {
#pragma unroll
      for (int j = k; j < 8; j += 4) {
        u[j] = turn ? f(x[j], cs[j], -y[j], sn[j]) : x[j];
        v[j] = turn ? f(y[j], cs[j], x[j], sn[j]) : y[j];
      }
    } else {
      u[2 * k] = turn ? f(x[2 * k], cs[k], -x[2 * k + 1], sn[k]) : x[2 * k];
      u[2 * k + 1] = turn ? f(x[2 * k + 1], cs[k], x[2 * k], sn[k]) : x[2 * k + 1];
      v[2 * k] = turn ? f(y[2 * k], cs[k + 4], -y[2 * k + 1], sn[k + 4]) : y[2 * k];
      v[2 * k + 1] = turn ? f(y[2 * k + 1], cs[k + 4], y[2 * k], sn[k + 4]) : y[2 * k + 1];
    }
  }
}
// Largest magnitudes of the scale groups of a lane's two chunks, which it has whole (own) or
// shares with its neighbour.
template <int STYLE>
__device__ __forceinline__ void group_max(const float (&u)[8], const float (&v)[8], bool own, float& ma, float& mb) {
  ma = max8(u), mb = max8(v);
  if (STYLE == 1) {
    const float oa = __shfl_xor_sync(0xffffffffu, ma, 1), ob = __shfl_xor_sync(0xffffffffu, mb, 1);
    ma = own ? fmaxf(ma, mb) : fmaxf(ma, oa);
    mb = own ? ma : fmaxf(mb, ob);
  } else {
    ma = mb = fmaxf(ma, mb);
  }
}

// A token's rows are the query heads, then the key heads, then the value heads. A
// row is handled by d / 16 lanes with two 16-byte chunks each: the two that turn
// together (l, l + r / 16) for pairs (i, i + r / 2), else neighbours (2l, 2l + 1).  Only
// keys ask for more than fp32 (see dot2_odd), and few of them take that way.  A warp takes `per_warp` passes of 32 / (d / 16)
// rows of one kind, with the token's table entries in registers.
template <int D, int STYLE>  // 0: no rotation, 1: halves, 2: interleaved
__global__ void __launch_bounds__(kThreads, 8) cache_append_kernel(const AppendArgs a, int warps_per_token, int per_warp) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  after_previous_kernel();
  const long long n_warps = (long long)a.s.total * warps_per_token;
  for (long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); gw < n_warps; gw += (long long)gridDim.x * kWarps) {
    const int t = (int)(gw / warps_per_token), part = (int)(gw % warps_per_token);
    const int i = sequence_of(a.s, t);
    const int tok = cache_index(a.s, i, t, a.ctl);
    if (tok < 0) continue;
    const int half = a.rot >> 4;  // chunks in half the rotated part
    const bool turn = STYLE == 1 ? l < half : STYLE == 2 ? 16 * l < a.rot : false;
    const int ca = STYLE == 1 && turn ? l : 2 * l, cb = STYLE == 1 && turn ? l + half : 2 * l + 1;
    const bool own = cb == ca + 1 && !(ca & 1);  // both chunks are one scale group
    float cs[8], sn[8];
    if (STYLE) {
      const int pos = a.positions ? a.positions[t] : tok;
      if ((unsigned)pos >= (unsigned)a.max_pos) {
        if (lane == 0) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_POS);
        continue;
      }
      const float4* pc = reinterpret_cast<const float4*>(a.cos_t + (long long)pos * a.cos_stride + 8 * l);
      const float4* ps = reinterpret_cast<const float4*>(a.sin_t + (long long)pos * a.sin_stride + 8 * l);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 c = turn ? pc[k] : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 s = turn ? ps[k] : make_float4(0.f, 0.f, 0.f, 0.f);
        cs[4 * k] = c.x, cs[4 * k + 1] = c.y, cs[4 * k + 2] = c.z, cs[4 * k + 3] = c.w;
        sn[4 * k] = s.x, sn[4 * k + 1] = s.y, sn[4 * k + 2] = s.z, sn[4 * k + 3] = s.w;
      }
    }
    const int at_table = a.s.table[(long long)i * a.s.table_stride + (tok >> a.c.page_shift)];  // used below
    const int nq = (a.h + RPP - 1) / RPP, nk = (a.hk + RPP - 1) / RPP;
    const int p_end = min(nq + 2 * nk, (part + 1) * per_warp);
    int p = part * per_warp;

    // queries
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.data) + (long long)t * a.q.s_row;
    __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(a.q_out.data) + (long long)t * a.q_out.s_row;
#pragma unroll 2
    for (; p < min(nq, p_end); ++p) {
      const int head = p * RPP + sub;
      if (head >= a.h) continue;
      const __nv_bfloat16* src = q + head * a.q.s_head;
      __nv_bfloat16* dst = qo + head * a.q_out.s_head;
      const uint4 wa = *reinterpret_cast<const uint4*>(src + 8 * ca), wb = *reinterpret_cast<const uint4*>(src + 8 * cb);
      if (STYLE == 0) {
        *reinterpret_cast<uint4*>(dst + 8 * ca) = wa;
        *reinterpret_cast<uint4*>(dst + 8 * cb) = wb;
        continue;
      }
      float x[8], y[8], u[8], v[8];
      unpack8(wa, x);
      unpack8(wb, y);
      rotate16<STYLE>(x, y, cs, sn, true, u, v, [](float p, float c, float q, float d) { return fmaf(p, c, q * d); });
      *reinterpret_cast<uint4*>(dst + 8 * ca) = turn ? pack8(u) : wa;
      *reinterpret_cast<uint4*>(dst + 8 * cb) = turn ? pack8(v) : wb;
    }
    if (p >= p_end) continue;
    const int page = check_page(a.c, at_table, a.ctl), prow = tok & ((1 << a.c.page_shift) - 1);
    if (page < 0) continue;
    // keys
    for (; p < min(nq + nk, p_end); ++p) {
      const int head = (p - nq) * RPP + sub;
      const bool live = head < a.hk;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.k.data) + (long long)t * a.k.s_row + head * a.k.s_head;
      uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
      if (live) wa = *reinterpret_cast<const uint4*>(src + 8 * ca), wb = *reinterpret_cast<const uint4*>(src + 8 * cb);
      float x[8], y[8], u[8], v[8];
      unpack8(wa, x);
      unpack8(wb, y);
      uint32_t sa, sbb, xa, xb;
      if (STYLE == 0) {
        sa = sbb = scale_of(fmaxf(max8(x), max8(y)));
        xa = codes_of<false>(x, sa), xb = codes_of<false>(y, sa);
      } else {
        // The fp32 rotation, with bounds: where the scale or a code would come out
        // otherwise for numbers a little off (about one row in a few hundred) the
        // warp takes the exact way below.
        float in = fmaxf(max8(x), max8(y)) * fmaxf(1.f, fmaxf(max8(cs), max8(sn)));
        in = fmaxf(in, __shfl_xor_sync(0xffffffffu, in, 1));
        bool unsure = !(in < 1e30f);
        rotate16<STYLE>(x, y, cs, sn, turn, u, v, [](float p, float c, float q, float d) { return fmaf(p, c, q * d); });
        // two products of size up to `in` and their sum: off by at most 3 * 2^-24 of it
        const float off = in * 0x1p-22f;
        float ma, mb;
        group_max<STYLE>(u, v, own, ma, mb);
        sa = sure_scale(ma, off, !turn, unsure), sbb = STYLE == 1 ? sure_scale(mb, off, !turn, unsure) : sa;
        xa = sure_codes(u, sa, off, !turn, unsure), xb = sure_codes(v, sbb, off, !turn, unsure);
        if (__any_sync(0xffffffffu, unsure && live)) {
          rotate16<STYLE>(x, y, cs, sn, turn, u, v, dot2_odd);
          group_max<STYLE>(u, v, own, ma, mb);
          sa = scale_of(ma), sbb = STYLE == 1 ? scale_of(mb) : sa;
          xa = codes_of<true>(u, sa), xb = codes_of<true>(v, sbb);
        }
      }
      if (!live) continue;
      uint8_t* row = a.c.k.data + row_offset(a.c.k, page, head, prow);
      uint8_t* srow = a.c.ks.data + row_offset(a.c.ks, page, head, prow);
      if (own) {
        *reinterpret_cast<uint2*>(row + 4 * ca) = make_uint2(xa, xb);
        srow[ca >> 1] = (uint8_t)sa;
      } else {
        *reinterpret_cast<uint32_t*>(row + 4 * ca) = xa;
        *reinterpret_cast<uint32_t*>(row + 4 * cb) = xb;
        if (!(l & 1)) srow[ca >> 1] = (uint8_t)sa, srow[cb >> 1] = (uint8_t)sbb;
      }
    }
    // values: a lane's neighbouring chunks are one group
    for (; p < p_end; ++p) {
      const int head = (p - nq - nk) * RPP + sub;
      if (head >= a.hk) continue;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v.data) +
                                                        (long long)t * a.v.s_row + head * a.v.s_head + 16 * l);
      const uint4 wa = src[0], wb = src[1];
      float x[8], y[8];
      unpack8(wa, x);
      unpack8(wb, y);
      const uint32_t sc = scale_of(fmaxf(max8(x), max8(y)));
      *reinterpret_cast<uint2*>(a.c.v.data + row_offset(a.c.v, page, head, prow) + 8 * l) =
          make_uint2(codes_of<false>(x, sc), codes_of<false>(y, sc));
      a.c.vs.data[row_offset(a.c.vs, page, head, prow) + l] = (uint8_t)sc;
    }
  }
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A lane turns one scale group (8 code bytes) into 16 bf16 numbers, d / 16 lanes a
// row; a warp takes `per_warp` passes over the rows of one token, first the key
// heads, then the value heads, kUnroll passes' loads in flight.
// WIDE: rows of the outputs start on 32-byte boundaries, so a lane stores at once.
constexpr int kReadUnroll = 4;
template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a, int warps_per_token, int per_warp) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  after_previous_kernel();
  const long long n_warps = (long long)a.s.total * warps_per_token;
  for (long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); gw < n_warps; gw += (long long)gridDim.x * kWarps) {
    const int t = (int)(gw / warps_per_token), part = (int)(gw % warps_per_token);
    const int i = sequence_of(a.s, t);
    const int tok = cache_index(a.s, i, t, a.ctl);
    if (tok < 0) continue;
    const int page = cache_page(a.s, a.c, i, tok, a.ctl);
    if (page < 0) continue;
    const int prow = tok & ((1 << a.c.page_shift) - 1);
    const long long oc = (long long)page * a.c.k.s_page + prow * (int)a.c.k.s_row + 8 * l;
    const long long os = (long long)page * a.c.ks.s_page + prow * (int)a.c.ks.s_row + l;
    const int end = min(2 * a.hk, (part + 1) * per_warp * RPP);
    for (int row0 = part * per_warp * RPP + sub; row0 < end; row0 += kReadUnroll * RPP) {
      uint2 w[kReadUnroll];
      uint32_t sc[kReadUnroll];
#pragma unroll
      for (int k = 0; k < kReadUnroll; ++k) {
        const int row = row0 + k * RPP;
        if (row < end) {
          const bool is_v = row >= a.hk;
          const int head = is_v ? row - a.hk : row;
          w[k] = *(reinterpret_cast<const uint2*>((is_v ? a.c.v.data : a.c.k.data) + oc + head * a.c.k.s_head));
          sc[k] = (is_v ? a.c.vs.data : a.c.ks.data)[os + head * a.c.ks.s_head];
        }
      }
#pragma unroll
      for (int k = 0; k < kReadUnroll; ++k) {
        const int row = row0 + k * RPP;
        if (row < end) {
          const bool is_v = row >= a.hk;
          const int head = is_v ? row - a.hk : row;
          const uint32_t s2 = half_lo2(e4m3x2_to_f16(sc[k]));
          uint32_t r[4], o[8];
          e2m1x8_to_f16(w[k].x, r);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 f = f16x2_to_f32(hmul2(r[u], s2));
            o[u] = pack_bf16x2(f.x, f.y);
          }
          e2m1x8_to_f16(w[k].y, r);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 f = f16x2_to_f32(hmul2(r[u], s2));
            o[4 + u] = pack_bf16x2(f.x, f.y);
          }
          const Rows3& to = is_v ? a.v_out : a.k_out;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(to.data) + (long long)t * to.s_row + head * to.s_head + 16 * l;
          if (WIDE) {
            store32(dst, o);
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
  }
}

}  // namespace

// A warp takes a whole token, or fewer of its passes while that leaves SMs without warps.
struct Share {
  int warps_per_token, per_warp;
  unsigned grid;
};
static Share share_of(long long tokens, int passes) {
  const long long want = (long long)num_sms() * 16;
  int per_warp = passes;
  while (per_warp > 1 && tokens * ((passes + per_warp - 1) / per_warp) < want) per_warp = (per_warp + 1) / 2;
  const int wpt = (passes + per_warp - 1) / per_warp;
  const long long blocks = (tokens * wpt + kWarps - 1) / kWarps;
  return Share{wpt, per_warp, (unsigned)(blocks < (1LL << 30) ? blocks : (1LL << 30))};
}

template <int D>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  constexpr int RPP = 512 / D;  // rows per pass
  const int passes = (a.h + RPP - 1) / RPP + 2 * ((a.hk + RPP - 1) / RPP);
  const Share s = share_of(a.s.total, passes);
  if (!a.rot)
    return launch_early(cache_append_kernel<D, 0>, s.grid, kThreads, 0, st, a, s.warps_per_token, s.per_warp);
  if (a.style == 0)
    return launch_early(cache_append_kernel<D, 1>, s.grid, kThreads, 0, st, a, s.warps_per_token, s.per_warp);
  return launch_early(cache_append_kernel<D, 2>, s.grid, kThreads, 0, st, a, s.warps_per_token, s.per_warp);
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_append<64>(a, st) : launch_append<128>(a, st);
}

template <int D>
cudaError_t launch_read(const ReadArgs& a, cudaStream_t st) {
  constexpr int RPP = 512 / D;
  const int passes = (2 * a.hk + RPP - 1) / RPP;
  const Share s = share_of(a.s.total, passes);
  auto wide = [](const Rows3& r) {
    return reinterpret_cast<uintptr_t>(r.data) % 32 == 0 && r.s_row % 16 == 0 && r.s_head % 16 == 0;
  };
  if (wide(a.k_out) && wide(a.v_out))
    return launch_early(cache_read_kernel<D, true>, s.grid, kThreads, 0, st, a, s.warps_per_token, s.per_warp);
  return launch_early(cache_read_kernel<D, false>, s.grid, kThreads, 0, st, a, s.warps_per_token, s.per_warp);
}

cudaError_t launch_cache_read(const ReadArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch_read<64>(a, st) : launch_read<128>(a, st);
}

}  // namespace ra
