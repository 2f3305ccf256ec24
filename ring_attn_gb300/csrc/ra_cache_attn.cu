// Attention of new tokens over the paged 4-bit cache, the plain way: one warp per
// query row walks the sequence's keys 32 at a time (a key per lane for the scores,
// d / 32 head dims per lane for the values), with a running maximum and sum.
#include "ra_cache.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) cache_attn_simple_kernel(CacheAttnArgs a) {
  __shared__ float sq[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, head = blockIdx.y * kWarps + warp;
  if (head >= a.h) return;
  const int hk = head / a.G;
  const int i = segment_of_warp(a.s.cu, a.s.n_seqs, t);
  const int len = cache_len(a.s, i, a.max_kv, a.ctl);
  const int end = a.causal ? min(len, len - __ldg(a.s.cu + i + 1) + t + 1) : len;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.data) + (long long)t * a.q.s_row +
                           (long long)head * a.q.s_head;
  for (int c = lane; c < D; c += 32) sq[warp][c] = __bfloat162float(q[c]) * a.scale_log2;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  for (int k0 = 0; k0 < end; k0 += 32) {
    const int tok = k0 + lane;
    int page = -1;
    float s = -INFINITY;
    if (tok < end) page = cache_page(a.s, a.c, i, tok, a.ctl);
    const int prow = tok & ((1 << a.c.page_shift) - 1);
    if (page >= 0) {
      const uint8_t* kr = a.c.k.data + row_offset(a.c.k, page, hk, prow);
      const uint8_t* sr = a.c.ks.data + row_offset(a.c.ks, page, hk, prow);
      s = 0.f;
      for (int w = 0; w < D / 8; ++w) {
        uint32_t r[4];
        e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(kr + 4 * w), r);
        const float sc = f16x2_to_f32(e4m3x2_to_f16(sr[w >> 1])).x;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 f = f16x2_to_f32(r[u]);
          s += f.x * sc * sq[warp][8 * w + 2 * u] + f.y * sc * sq[warp][8 * w + 2 * u + 1];
        }
      }
    }
    float mx = s;
    for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float m_new = fmaxf(m, mx), mu = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m - mu), p = exp2f(s - mu);
    l = l * alpha + p;
    m = m_new;
    for (int c = 0; c < D / 32; ++c) o[c] *= alpha;
    for (int j = 0; j < 32; ++j) {
      const int pg = __shfl_sync(0xffffffffu, page, j);
      const float pj = __shfl_sync(0xffffffffu, p, j);
      if (pg < 0) continue;
      const int pr = (k0 + j) & ((1 << a.c.page_shift) - 1);
      const uint8_t* vr = a.c.v.data + row_offset(a.c.v, pg, hk, pr);
      const uint8_t* sr = a.c.vs.data + row_offset(a.c.vs, pg, hk, pr);
      uint32_t r[4];
      e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(vr + ((lane * (D / 64)) & ~3)), r);
      const float sc = f16x2_to_f32(e4m3x2_to_f16(sr[lane * (D / 32) / 16])).x;
#pragma unroll
      for (int c = 0; c < D / 32; c += 2) {
        const int at = (lane * (D / 32) + c) % 8 / 2;
        const float2 f = f16x2_to_f32(at == 0 ? r[0] : at == 1 ? r[1] : at == 2 ? r[2] : r[3]);
        o[c] += pj * sc * f.x;
        o[c + 1] += pj * sc * f.y;
      }
    }
  }
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const long long at = (long long)t * a.out.s_row + (long long)head * a.out.s_head + lane * (D / 32);
  for (int c = 0; c < D / 32; ++c) {
    if (a.out_f32)
      static_cast<float*>(a.out.data)[at + c] = o[c] * inv;
    else
      static_cast<__nv_bfloat16*>(a.out.data)[at + c] = __float2bfloat16(o[c] * inv);
  }
  if (lane == 0)
    a.lse[(long long)head * a.l_sh + (long long)t * a.l_ss] =
        l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t cache_attn_ws_bytes(long long, int, int, int, int, int) { return 256; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.s.total, (unsigned)((a.h + kWarps - 1) / kWarps));
  if (a.d == 64)
    cache_attn_simple_kernel<64><<<grid, 32 * kWarps, 0, st>>>(a);
  else
    cache_attn_simple_kernel<128><<<grid, 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace ra
