// Chunks over the paged cache with plain scores, and what joins the pieces of any (the kernel: ra_cache_chunk.cuh).
#include "ra_cache_chunk.cuh"

namespace ra {
namespace {

// Joins the item in slot 1 of block blockIdx.x, if there is one: rows [32 blockIdx.y, + 32)
// of its 256, a row per lane and D / 8 head dims per warp, over the few pieces that
// an item has here.  (A slot holds four head dims of all rows together.)
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const CacheAttnArgs g) {
  constexpr int V = D / 8, kAtOnce = 4;
  after_previous_kernel();
  const JoinNote* notes = notes_of(g);
  const JoinNote n = notes[blockIdx.x];
  if (n.last < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grid = gridDim.x;
  const int r = blockIdx.y * 32 + lane, row = n.row0 + r;
  if (n.row0 + (int)blockIdx.y * 32 >= n.rows) return;
  float M = kNone, sum = 0.f, o[V] = {};
  for (int base = blockIdx.x; base <= n.last; base += 32) {
    const int c = base + lane;
    unsigned there = __ballot_sync(0xffffffffu, c == (int)blockIdx.x || (c <= n.last && notes[c].slot0));
    while (there) {  // kAtOnce pieces' loads in flight
      float2 ml[kAtOnce];
      float4 x[kAtOnce][V / 4];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        ml[k] = make_float2(kNone, 0.f);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) x[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there) {
          const int b = base + __ffs(there) - 1;
          there &= there - 1;
          const float* slot = slot_of<256, D>(g, grid, b, b == (int)blockIdx.x);
          ml[k] = *reinterpret_cast<const float2*>(slot + 256 * D + 2 * r);  // (rows behind the sequence's: unused)
#pragma unroll
          for (int i = 0; i < V / 4; ++i) x[k][i] = reinterpret_cast<const float4*>(slot)[(warp * (V / 4) + i) * 256 + r];
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float to = fmaxf(M, ml[k].x), f0 = fast_exp2(M - to), f1 = fast_exp2(ml[k].x - to);
        M = to;
        sum = sum * f0 + ml[k].y * f1;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          o[4 * i] = o[4 * i] * f0 + x[k][i].x * f1;
          o[4 * i + 1] = o[4 * i + 1] * f0 + x[k][i].y * f1;
          o[4 * i + 2] = o[4 * i + 2] * f0 + x[k][i].z * f1;
          o[4 * i + 3] = o[4 * i + 3] * f0 + x[k][i].w * f1;
        }
      }
    }
  }
  if (row >= n.rows) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = n.cu0 + row / g.G, hd = n.head * g.G + row % g.G;
  const long long to = (long long)tok * g.out.s_row + (long long)hd * g.out.s_head + warp * V;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] *= inv;
  if (g.out_f32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(g.out.data) + to);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out.data) + to);
#pragma unroll
    for (int i = 0; i < V / 8; ++i)
      dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                          pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
  }
  if (warp == 0) store_lse(g, tok, hd, M, sum);
}

}  // namespace

size_t cache_chunk_ws_bytes(int d) { return line_ws_bytes<256>(num_sms(), d); }

void plan_cache_chunk(CacheAttnPlan& p) {
  CacheAttnArgs& a = p.args;
  p.grid = num_sms();
  p.joins = true;
  // the causal cost of an item is at most G (units + kItemCost) + 2 + 2 tiles places
  const long long units = (a.max_kv + kUnit - 1) / kUnit + ManyRows<0>::kItemCost;
  const long long places = a.causal ? a.G * units + 2 + 2 * (((long long)a.max_new * a.G + 255) / 256) : units;
  a.line_shift = a.items * (places + 2) < (1LL << 30) ? 0 : std::max(1, line_shift_for(a.items, units));
}

cudaError_t launch_cache_chunk(const CacheAttnPlan& p, cudaStream_t st) {
  return p.args.d == 64 ? launch_chunk<64, 0>(p, st) : launch_chunk<128, 0>(p, st);
}

cudaError_t launch_chunk_join(const CacheAttnPlan& p, cudaStream_t st) {
  return launch_early(p.args.d == 64 ? chunk_join_kernel<64> : chunk_join_kernel<128>, dim3(p.grid, 8), 256, 0, st, p.args);
}

}  // namespace ra
