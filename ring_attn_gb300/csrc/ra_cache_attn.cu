// How attention over the paged cache is planned and launched (the kernel for few query rows: ra_cache_attn.cuh).
#include "ra_cache_attn.cuh"

namespace ra {
namespace {

// From how many query rows per key / value head on the tensor-core kernel takes over: with 32
// this one is faster (64 items of 10,000 keys: 57 us against 68, d = 64: 38 against 53; 8 items of
// 3000 keys: 19 and 21), with more it would read the cache twice, and that one takes the same 68 us.
bool many_rows(int max_new, int G) { return (long long)max_new * G > 32; }

// Query rows of an item in units of 8.
int row_tiles(long long rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int D, int NT>
cudaError_t launch_join(const CacheAttnPlan& p, cudaStream_t st) {
  constexpr int R = 8 * NT;
  return launch_early(cache_join_kernel<R, D>, dim3(p.grid, (std::min(p.args.max_new * p.args.G, R) + 7) / 8),
                      256 * kJoinGroups, 0, st, p.args);
}

}  // namespace

// Bytes for calls of up to max_new tokens a sequence: a call of fewer may run as a kind that
// has smaller slots but more blocks (d = 64: 8 rows in four blocks an SM, 16 in two).
size_t cache_attn_ws_bytes(long long, int max_new, int h, int hk, int d, int) {
  auto few = [d](int nt) {
    const int grid = num_sms() * small_blocks(d, nt);
    return nt == 1 ? line_ws_bytes<8>(grid, d) : nt == 2 ? line_ws_bytes<16>(grid, d) : line_ws_bytes<32>(grid, d);
  };
  const bool many = many_rows(max_new, h / hk);
  const int up_to = many ? 4 : row_tiles((long long)max_new * (h / hk));
  size_t n = many ? cache_chunk_ws_bytes(d) : 0;
  for (int nt = 1; nt <= up_to; nt *= 2) n = std::max(n, few(nt));
  return n;
}

long long cache_attn_items(const int* cu_host, int n_seqs, int max_new, int G, int hk) {
  const int R = many_rows(max_new, G) ? 256 : 8 * row_tiles((long long)max_new * G);
  long long tiles = 0;
  for (int i = 0; i < n_seqs; ++i) tiles += ((long long)(cu_host[i + 1] - cu_host[i]) * G + R - 1) / R;
  return tiles * hk;
}

// Items short enough for one block (2048 keys: about 7 us, as long as a second kernel takes)
// and no more than SMs: a big block for each, nothing to join.  Very few items of 8 rows:
// big blocks too, so that an item has fewer pieces to join (8 items of 30,000 keys of d = 128:
// 22.6 us, with small blocks 23.6; d = 64: 18.5 and 20.6; 16 items: 30.4 and 28.7).  Else small
// blocks, whose starts and ends overlap (64 items of 10,000 keys: 31 us, with big blocks
// 35; 12 rows: 38 and 44; 28 rows: 56 and 64).
CacheAttnPlan plan_cache_attn(const CacheAttnArgs& a) {
  CacheAttnPlan p = {a, many_rows(a.max_new, a.G) ? 0 : row_tiles((long long)a.max_new * a.G), 0, false, false};
  if (p.row_tiles == 0) {
    plan_cache_chunk(p);
    return p;
  }
  constexpr int kItemCost = FewRows<1>::kItemCost;  // (whatever the rows)
  const int units = (a.max_kv + kUnit - 1) / kUnit, sms = num_sms();
  const bool whole = a.items <= sms && units <= 16;
  p.big = whole || (p.row_tiles == 1 && a.items * 10 <= sms);
  p.joins = !whole;
  const long long line = a.items * (whole ? 1 : units + kItemCost);  // at most
  p.grid = (int)std::min(line, (long long)sms * (p.big ? 1 : small_blocks(a.d, p.row_tiles)));
  p.args.whole = whole;
  p.args.line_shift = line_shift_for(a.items, units + kItemCost);
  return p;
}

cudaError_t launch_cache_attn(const CacheAttnPlan& p, cudaStream_t st) {
  if (p.row_tiles == 0) {
    switch (p.args.mode) {
      case SC_ON: return launch_cache_chunk_score<SC_ON>(p, st);
      case SC_ON | SC_CAP: return launch_cache_chunk_score<SC_ON | SC_CAP>(p, st);
      case SC_ON | SC_BIAS: return launch_cache_chunk_score<SC_ON | SC_BIAS>(p, st);
      case SC_ON | SC_CAP | SC_BIAS: return launch_cache_chunk_score<SC_ON | SC_CAP | SC_BIAS>(p, st);
      default: return launch_cache_chunk(p, st);
    }
  }
  return p.args.mode ? launch_cache_attn_scored(p, st) : launch_few<false>(p, st);
}

cudaError_t launch_cache_join(const CacheAttnPlan& p, cudaStream_t st) {
  const int nt = p.row_tiles;
  if (nt == 0) return launch_chunk_join(p, st);
  if (p.args.d == 64) return nt == 1 ? launch_join<64, 1>(p, st) : nt == 2 ? launch_join<64, 2>(p, st) : launch_join<64, 4>(p, st);
  return nt == 1 ? launch_join<128, 1>(p, st) : nt == 2 ? launch_join<128, 2>(p, st) : launch_join<128, 4>(p, st);
}

}  // namespace ra
