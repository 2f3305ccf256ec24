// Attention of many new tokens (chunks of prompts) over the paged 4-bit cache, on
// the tensor cores.
//
// An item is 256 query rows (two tiles of 128) of one key / value head; the blocks,
// one per SM, share the items' units as ra_cache_line.cuh says.  Per unit of 128
// keys a tile needs S = Q K^T and O += P V, 4 * 128 * 128 * d flops, for which keys
// and values are converted once per unit and block:
//   warp 0       MMA issuer (one thread): PV0(j-1), S0(j), PV1(j-1), S1(j), so one
//                tile's products run while the other's softmax does.  S_t in
//                tensor-memory columns [128 t, 128 t + 128), O_t from 256 + 128 t.
//                A sequence's only tile is worked on as two twins instead, which take
//                its units in turn and are added up at the end.
//   warp 1       allocates / frees tensor memory.
//   warp 2       one thread walks the block's pieces of the line and hands them to the
//                others in shared memory, a few ahead (so that no other role holds a
//                place on the line in registers).  Warp 3 is idle.
//   warps 4-7    one key row per thread: its 4-bit codes and scales go from global
//                memory through registers to fp16 rows in the 128-byte swizzle that
//                the MMA reads, K two stages, V three.  About 340 instructions a
//                thread and unit, a tenth of the unit's issue slots.
//   warps 8-15   a query row per thread: queries scaled per row by a power of two into
//                fp16's normal range and stored for the MMA; scores from tensor
//                memory, running offset M (O is rescaled when a score passes it by
//                far), P as fp16 over the score columns; the epilogue.
// Bound: tensor throughput, and with it shared memory: of a unit's 2048 tensor cycles
// (256 rows, d = 128) operand reads take 1536 and the converted tiles' stores 512.
// 2048 tokens of 32 heads at the end of 65,536 keys of 8 heads: 1.53 ms, 1413 TFLOP/s
// (73 % of the measured bf16 rate); 1.41 ms without the conversions, 1.19 without softmax.
// fp16 operands hold number * scale exactly; queries and p are rounded to fp16 and the rest is
// fp32, as in ra_cache_attn.cu, whose comment says what that costs.
#include <algorithm>

#include "ra_cache_line.cuh"

namespace ra {
namespace {

constexpr int kBox = 128 * 128;  // 128 rows x 64 fp16
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKStages = 2, kVStages = 3;  // V is needed up to two units longer (twin tiles)
constexpr uint32_t kWaitHint = 2000;
constexpr float kLift = 8.f, kSlack = 4.f;  // largest p between 2^8 and 2^12
constexpr float kNone = -3.0e38f;           // M of a row that has seen no key
// Registers per thread of the control, conversion and softmax warpgroups.
constexpr int kLaunchRegs = 128, kRegsCtl = 72, kRegsConv = 88, kRegsSoft = 176;
static_assert(128 * (kRegsCtl + kRegsConv + 2 * kRegsSoft) <= kThreads * kLaunchRegs, "register split exceeds the launch");

// G places per unit, so that the causal growth of 256 / G keys per tile is whole.
struct ManyRows {
  static constexpr int R = 256, kItemCost = 4;
  static constexpr bool kOneTile = false;
  static __device__ __forceinline__ void cost(const CacheAttnArgs& g, LineSeq& s) {
    s.per = g.causal ? g.G : 1;
    const int seen = g.causal ? max(0, s.len - s.n_new) : s.len;  // by every row
    s.a = s.per * ((seen + kUnit - 1) / kUnit + kItemCost) + 2;
    s.b = g.causal ? 2 : 0;
  }
  // (fewer leave more pieces to join: one item of 160 rows and 20,000 keys 38.9 us with 2, 34.4 with 3, 33.0
  // with 4; four items of 240 rows and 2500 keys 25.0, 25.6 and 26.8)
  static __device__ __forceinline__ int min_places(const CacheAttnArgs& g, int) { return 3 * (g.causal ? g.G : 1); }
};

// A piece as the roles need it; n = 0: the run's end.
struct Item {
  int ua, n;                 // first unit, units
  int head, row0, rows;      // first query row of the item, rows of the sequence
  int seq, cu0, len, n_new;
  int whole;                 // the piece is the whole item
};
constexpr int kItems = 4;

enum Bar {
  B_Q_FULL = 0,    // per query tile
  B_KV_FULL = 2,   // kKStages; K and V of a unit complete on one barrier, so the issuer waits once
  B_K_EMPTY = 4,   // kKStages
  B_V_EMPTY = 6,   // kVStages
  B_S_FULL = 9,    // per query tile
  B_P_FULL = 11,
  B_O_DONE = 13,      // once an item: its products have ended, and the second warpgroup has come to it
  B_TEARDOWN = 14,
  B_ITEM_FULL = 15,   // kItems
  B_ITEM_EMPTY = 19,
  B_TWIN_STATE = 23,  // the second twin's M and sums are in shared memory
  B_TWIN_DONE = 24,   // the first has read the second's O
  kNumBars = 25
};
template <int D>
struct Lay {
  static constexpr int kTile = D / 64 * kBox;
  static constexpr int kQ = 0, kK = 2 * kTile, kV = kK + kKStages * kTile, kBar = kV + kVStages * kTile;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kItem = kMisc + 16;
  static constexpr int kTwin = kItem + kItems * (int)sizeof(Item);  // 128 rows' M and sums
  static constexpr int kAlloc = kTwin + 128 * 8 + 1024;  // slack to align the base to 1024 bytes
};
constexpr int kReaders = 13;  // of an item: the issuer, 4 conversion and 8 softmax warps

// kind::f16 with fp16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// A key row's codes and scales.
template <int D>
struct RawRow {
  uint4 code[D / 32];
  uint32_t scale[D / 64];
  __device__ __forceinline__ void load(const uint8_t* c, const uint8_t* s, bool ok) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      code[i] = ok ? reinterpret_cast<const uint4*>(c)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) scale[i] = ok ? reinterpret_cast<const uint32_t*>(s)[i] : 0u;
  }
  // Row `r` of a tile at `tile`.
  __device__ __forceinline__ void store(uint32_t tile, int r) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      const uint32_t two = e4m3x2_to_f16(scale[i >> 1] >> (16 * (i & 1)));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        e2m1x8_to_f16(w[k], x);
        const uint32_t s = k < 2 ? half_lo2(two) : half_hi2(two);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = hmul2(x[j], s);
        const int chunk = 4 * i + k;  // 16 bytes of the row
        sts128(tile + (chunk >> 3) * kBox + sw128_offset(r, chunk & 7), x);
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_chunk_kernel(const CacheAttnArgs a) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  uint8_t* sp = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = sb + L::kBar;
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kMisc + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + L::kMisc);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kVStages; ++i) mbar_init(BAR(B_V_EMPTY + i), 1);
    mbar_init(BAR(B_TWIN_STATE), 4);
    mbar_init(BAR(B_TWIN_DONE), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_Q_FULL + i), 4);
      mbar_init(BAR(B_KV_FULL + i), 4);
      mbar_init(BAR(B_K_EMPTY + i), 1);
      mbar_init(BAR(B_S_FULL + i), 1);
      mbar_init(BAR(B_P_FULL + i), 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(BAR(B_ITEM_FULL + i), 1);
      mbar_init(BAR(B_ITEM_EMPTY + i), kReaders);
    }
    mbar_init(BAR(B_O_DONE), 5);
    mbar_init(BAR(B_TEARDOWN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  after_previous_kernel();
  // (in the twins' place: an SM's shared memory is all taken)
  LineShared<kWarps>& sh = *reinterpret_cast<LineShared<kWarps>*>(sp + L::kTwin);
  static_assert(sizeof(LineShared<kWarps>) <= 128 * 8, "the plan's shared memory");
  LinePos at;
  int end_u, quota;
  JoinNote note = empty_note();
  if (!find_run<ManyRows, kWarps>(a, at, end_u, quota, sh)) {
    if (threadIdx.x == 0) notes_of(a)[blockIdx.x] = note;
    return;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile Item* items = reinterpret_cast<volatile Item*>(sp + L::kItem);
  // Query tiles of an item.  A sequence's only one, over several units, is worked on by
  // both softmax warpgroups, which take its units in turn (twins), each with its own O:
  // 64 rows of 16 sequences of 8000 keys and 8 key / value heads take 99 us, 123 without.
  // Not the last one of many rows: changing between the two ways costs more than it gives
  // (320 rows of 8 sequences of 8000 keys: 129 us, 155 with).
  auto tiles_of = [](const volatile Item& x) { return x.rows - x.row0 > 128 ? 2 : 1; };
  auto is_twin = [](const volatile Item& x) { return x.n > 1 && x.rows <= 128; };
  volatile float2* twin_state = reinterpret_cast<volatile float2*>(sp + L::kTwin);

  if (warp < 4) {
    regs_dec<kRegsCtl>();
    if (warp == 0) {
      // -------------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t kIdS = idesc_f16_f32(128, kUnit, 0), kIdPV = idesc_f16_f32(128, D, 1);
        constexpr uint32_t kHi = sdesc_sw128_hi(1024);
        bool ok = true;
        uint32_t k_at = 0, v_at = 0;    // stages of the next unit's S and PV, times kTile
        uint32_t par_kv = 0, n_all = 0;
        uint32_t par_q = 0, par_p = 0;  // phases of the query tiles' barriers, bit t (t is known at compile time)
        // S_t of the next unit, from query tile `qt`
        auto issue_s = [&](auto tile, auto qtile) {
          constexpr int t = decltype(tile)::value, qt = decltype(qtile)::value;
          const uint32_t lk = sdesc_sw128_lo(sb + L::kK + k_at, 16);
          const uint32_t lq = sdesc_sw128_lo(sb + L::kQ + qt * L::kTile, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tmem + t * 128, sdesc_words(lq + off, kHi), sdesc_words(lk + off, kHi), kIdS, kk > 0 ? 1u : 0u);
          }
          mma_commit(BAR(B_S_FULL + t));
        };
        auto issue_pv = [&](auto tile, uint32_t first) -> bool {
          constexpr int t = decltype(tile)::value;
          if (!wait_one<kWaitHint>(BAR(B_P_FULL + t), (par_p >> t) & 1, abort_flag, a.ctl, 33)) return false;
          par_p ^= 1u << t;
          tc_fence_after();
          const uint32_t lv = sdesc_sw128_lo(sb + L::kV + v_at, kBox);
#pragma unroll
          for (int kk = 0; kk < kUnit / 16; ++kk)
            mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, sdesc_words(lv + kk * 128, kHi), kIdPV,
                        kk > 0 ? 1u : first ^ 1u);
          return true;
        };
        auto wait_kv = [&]() -> bool {
          return wait_one<kWaitHint>(BAR(B_KV_FULL) + (k_at ? 8u : 0u), par_kv, abort_flag, a.ctl, 35);
        };
        auto wait_q = [&](auto tile) -> bool {
          constexpr int t = decltype(tile)::value;
          if (!wait_one<kWaitHint>(BAR(B_Q_FULL + t), (par_q >> t) & 1, abort_flag, a.ctl, 36)) return false;
          par_q ^= 1u << t;
          return true;
        };
        auto v_done = [&]() {
          mma_commit(BAR(B_V_EMPTY) + 8u * (v_at / L::kTile));
          v_at = v_at == (kVStages - 1) * L::kTile ? 0u : v_at + L::kTile;
        };
        auto k_done = [&]() {
          mma_commit(BAR(B_K_EMPTY) + (k_at ? 8u : 0u));
          if (k_at) par_kv ^= 1u;
          k_at ^= L::kTile;
          ++n_all;
        };
        // PV_t(j-1) reads P_t from the S_t columns, so it goes before S_t(j)
        auto turn = [&](auto tile, int j, int n) -> bool {
          constexpr int t = decltype(tile)::value;
          if (j >= 1 && !issue_pv(tile, j == 1)) return false;
          if (j == n) return true;
          if (t == 0 && !wait_kv()) return false;
          if (j == 0 && !wait_q(tile)) return false;
          tc_fence_after();
          issue_s(tile, tile);
          return true;
        };
        // one query tile, two S and O: unit j is tile j % 2's
        auto twin_turn = [&](auto tile, int j, int n) -> bool {
          if (j >= 2) {
            if (!issue_pv(tile, j < 4)) return false;
            v_done();
          }
          if (j >= n) return true;
          if (!wait_kv() || (j == 0 && !wait_q(Int<0>{}))) return false;
          tc_fence_after();
          issue_s(tile, Int<0>{});
          k_done();
          return true;
        };
        for (int i = 0; ok; ++i) {
          if (!wait_one<kWaitHint>(BAR(B_ITEM_FULL + i % kItems), (i / kItems) & 1, abort_flag, a.ctl, 45)) {
            ok = false;
            break;
          }
          const int nt = tiles_of(items[i % kItems]), n = items[i % kItems].n;
          const bool twin = is_twin(items[i % kItems]);
          mbar_arrive(BAR(B_ITEM_EMPTY + i % kItems));
          if (n == 0) break;
          if (twin) {
            for (int j = 0; ok && j < n + 2; j += 2)
              ok = twin_turn(Int<0>{}, j, n) && (j + 1 >= n + 2 || twin_turn(Int<1>{}, j + 1, n));
          } else {
            for (int j = 0; ok && j <= n; ++j) {
              ok = turn(Int<0>{}, j, n) && (nt == 1 || turn(Int<1>{}, j, n));
              if (ok && j >= 1) v_done();
              if (ok && j < n) k_done();
            }
          }
          if (ok) mma_commit(BAR(B_O_DONE));
        }
        // every issued MMA, and every arrival it makes, completes before the block ends
        mma_commit(BAR(B_TEARDOWN));
        drain_one(BAR(B_TEARDOWN), 0, a.ctl, 37);
        for (uint32_t s = 0; ok && s < kVStages; ++s) {
          const uint32_t ck = (n_all + kKStages - 1 - s) / kKStages, cv = (n_all + kVStages - 1 - s) / kVStages;
          if (s < kKStages && ck) drain_one(BAR(B_K_EMPTY + s), (ck - 1) & 1, a.ctl, 38);
          if (cv) drain_one(BAR(B_V_EMPTY + s), (cv - 1) & 1, a.ctl, 39);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // -------------------------------------------------------------- planner
      if (lane == 0) {
        Piece x;
        int seen = -1;
        for (int i = 0;; ++i) {
          const bool more = next_piece<ManyRows>(a, at, end_u, x);
          const int cu0 = more ? a.s.cu[x.seq] : 0;
          if (more) {
            if (x.seq != seen && a.s.lens[x.seq] > a.max_kv) record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_LEN);
            seen = x.seq;
            note_piece<ManyRows>(a, x, quota, cu0, note);
          }
          if (i >= kItems && !wait_one<kWaitHint>(BAR(B_ITEM_EMPTY + i % kItems), (i / kItems - 1) & 1, abort_flag,
                                                  a.ctl, 46))
            break;
          volatile Item& y = items[i % kItems];
          y.ua = x.ua, y.n = more ? x.ub - x.ua : 0;
          y.head = x.head, y.row0 = x.tile * 256, y.rows = x.n_new * a.G;
          y.seq = x.seq, y.cu0 = cu0, y.len = x.len, y.n_new = x.n_new;
          y.whole = x.ub - x.ua == x.units;
          mbar_arrive(BAR(B_ITEM_FULL + i % kItems));
          if (!more) break;
        }
        notes_of(a)[blockIdx.x] = note;
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- keys and values to fp16
    regs_dec<kRegsConv>();
    const int r = threadIdx.x - 128;
    uint32_t n = 0, sv = 0, pv = 1;  // units converted; V's stage and the parity of its last release
    bool ok = true;
    const int mask = (1 << a.c.page_shift) - 1;
    for (int i = 0; ok; ++i) {
      if (!wait_warp<kWaitHint>(BAR(B_ITEM_FULL + i % kItems), (i / kItems) & 1, abort_flag, a.ctl, 47)) break;
      const volatile Item& x = items[i % kItems];
      const int len = x.len, u0 = x.ua, u1 = u0 + x.n;
      const int* table = a.s.table + (long long)x.seq * a.s.table_stride;
      const long long hc = x.head * a.c.k.s_head, hs = x.head * a.c.ks.s_head;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_ITEM_EMPTY + i % kItems));
      if (u0 == u1) break;
      RawRow<D> k, v;
      long long oc = 0, os = 0;
      bool live = false;
      int page = 0;
      auto page_of = [&](int u) {  // read a unit ahead
        const int key = u * kUnit + r;
        live = key < len;
        page = live ? table[key >> a.c.page_shift] : 0;
      };
      auto place = [&](int u) {
        if (live && (unsigned)page >= (unsigned)a.c.n_pages) {
          record_error(a.ctl, DEV_BOUNDS, SITE_CACHE_PAGE);
          live = false;
        }
        const int row = (u * kUnit + r) & mask;
        oc = live ? (long long)page * a.c.k.s_page + row * (int)a.c.k.s_row + hc : 0;
        os = live ? (long long)page * a.c.ks.s_page + row * (int)a.c.ks.s_row + hs : 0;
      };
      page_of(u0);
      place(u0);
      bool ok_row = live;
      k.load(a.c.k.data + oc, a.c.ks.data + os, ok_row);
      v.load(a.c.v.data + oc, a.c.vs.data + os, ok_row);
      if (u0 + 1 < u1) page_of(u0 + 1);
      for (int u = u0; u < u1; ++u, ++n) {
        const uint32_t s = n % kKStages;
        const bool more = u + 1 < u1;
        if (n >= kKStages &&
            !wait_warp<kWaitHint>(BAR(B_K_EMPTY + s), (n / kKStages - 1) & 1, abort_flag, a.ctl, 40)) {
          ok = false;
          break;
        }
        k.store(sb + L::kK + s * L::kTile, r);
        if (more) {
          place(u + 1);
          ok_row = live;
          k.load(a.c.k.data + oc, a.c.ks.data + os, ok_row);
        }
        if (n >= kVStages && !wait_warp<kWaitHint>(BAR(B_V_EMPTY + sv), pv, abort_flag, a.ctl, 41)) {
          ok = false;
          break;
        }
        v.store(sb + L::kV + sv * L::kTile, r);
        if (++sv == kVStages) sv = 0, pv ^= 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_KV_FULL + s));
        if (more) {
          v.load(a.c.v.data + oc, a.c.vs.data + os, ok_row);
          if (u + 2 < u1) page_of(u + 2);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax, a row per thread
    regs_inc<kRegsSoft>();
    const int t = (warp - 8) >> 2, r = (threadIdx.x - 256) & 127;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + t * 128, tO = tl + 256 + t * 128;
    uint32_t n_s = 0, n_o = 0, n_twin = 0;  // score tiles, results and twin items seen
    bool ok = true;
    float sc = 0.f;             // of this thread's row of the item at hand
    int end_row = 0;
    // Item i's query row to shared memory, sc and end_row for it; false when the wait
    // gives up.  The tile's last S has been computed when this is called.
    auto take_item = [&](int i) -> bool {
      if (!wait_warp<kWaitHint>(BAR(B_ITEM_FULL + i % kItems), (i / kItems) & 1, abort_flag, a.ctl, 48)) return false;
      const volatile Item& x = items[i % kItems];
      const bool twin = is_twin(x);
      if (x.n == 0 || (t >= tiles_of(x) && !twin)) return true;
      const int row = x.row0 + (twin ? r : t * 128 + r), tok = row / a.G;
      uint32_t q[D / 2];
      end_row = 0;
      if (row < x.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.data) +
                                                          (long long)(x.cu0 + tok) * a.q.s_row +
                                                          (long long)(x.head * a.G + row % a.G) * a.q.s_head);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint4 w = src[k];
          q[4 * k] = w.x, q[4 * k + 1] = w.y, q[4 * k + 2] = w.z, q[4 * k + 3] = w.w;
        }
        end_row = a.causal ? min(x.len, x.len - x.n_new + tok + 1) : x.len;
      } else {
#pragma unroll
        for (int k = 0; k < D / 2; ++k) q[k] = 0;
      }
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < D / 2; ++k)
        m = fmax3f(m, fabsf(__uint_as_float(q[k] << 16)), fabsf(__uint_as_float(q[k] & 0xffff0000u)));
      // the row's largest entry goes to [2^12, 2^13)
      const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
      // not 0 (tiny scales, rows of zeros), so that a masked score, -infinity, stays one; scores
      // are below 2^33 before it, so below 2^-90 under the least
      sc = fmaxf(a.scale_log2 * __uint_as_float((uint32_t)(127 + e - 12) << 23), 0x1p-126f);
      if (twin && t == 1) return true;  // the first twin stores the row
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = pack_f16x2(__uint_as_float(q[4 * c + k] << 16) * up, __uint_as_float(q[4 * c + k] & 0xffff0000u) * up);
        sts128(sb + L::kQ + t * L::kTile + (c >> 3) * kBox + sw128_offset(r, c & 7), h);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_Q_FULL + t));
      return true;
    };
    ok = take_item(0);
    for (int i = 0; ok; ++i) {
      const volatile Item& x = items[i % kItems];
      const bool twin = is_twin(x);
      const int row = x.row0 + (twin ? r : t * 128 + r), u0 = x.ua, u1 = u0 + x.n;
      if (u0 == u1) break;
      // Items of one tile go on without the second warpgroup.  Its arrival keeps the phase from
      // ending twice before it has looked (the first one's products are in every item).
      if (t == 1 && lane == 0) mbar_arrive(BAR(B_O_DONE));
      if (t >= tiles_of(x) && !twin) {  // not this warpgroup's, but its phase passes
        ok = take_item(i + 1) && wait_warp<kWaitHint>(BAR(B_O_DONE), n_o & 1, abort_flag, a.ctl, 44);
        ++n_o;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_ITEM_EMPTY + i % kItems));
        continue;
      }
      const bool valid = row < x.rows;
      float M = kNone, l_run = 0.f;
      const int step = twin ? 2 : 1;
      for (int u = twin ? u0 + t : u0; u < u1; u += step, ++n_s) {
        const int c_hi = end_row - u * kUnit;
        if (!wait_warp<kWaitHint>(BAR(B_S_FULL + t), n_s & 1, abort_flag, a.ctl, 42)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[kUnit];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(v + 0));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v + 0));
        tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(v + 64));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(v + 96));
        float mc[4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          if (hh == 1) {
            tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v + 64));
            tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(v + 96));
          }
          if (c_hi < kUnit) {
            const uint64_t mw = bit_window64(0, c_hi - 64 * hh);
#pragma unroll
            for (int k = 0; k < 64; ++k)
              v[64 * hh + k] = ((mw >> k) & 1ull) ? v[64 * hh + k] : __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c0 = 64 * hh + 16 * q;
            float m = hh == 0 ? __uint_as_float(v[c0]) : fmaxf(mc[q], __uint_as_float(v[c0]));
#pragma unroll
            for (int c = c0 + 1; c < c0 + 15; c += 2) m = fmax3f(m, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
            mc[q] = fmaxf(m, __uint_as_float(v[c0 + 15]));
          }
        }
        const float mx = __fmul_rn(fmax3f(mc[0], mc[1], fmaxf(mc[2], mc[3])), sc);
        float alpha = 1.f;
        if (mx > M + (kLift + kSlack)) {
          alpha = fast_exp2(M - (mx - kLift));
          M = mx - kLift;
        }
        const uint64_t sc2 = f32x2(sc, sc), nm2 = f32x2(-M, -M);
        uint64_t acc[4] = {0, 0, 0, 0};
        // Offsets so large that the product's rounding shows next to them: the
        // products are rounded first, so that the largest score gives an exact difference.
        const bool far = __any_sync(0xffffffffu, fabsf(M) > 65536.f && M > kNone);
        auto weights = [&](auto rounded) {
#pragma unroll
          for (int c32 = 0; c32 < kUnit / 32; ++c32) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int c = c32 * 32 + 2 * k;
              float x0 = __uint_as_float(v[c]), x1 = __uint_as_float(v[c + 1]);
              if constexpr (decltype(rounded)::value)
                x0 = __fsub_rn(__fmul_rn(x0, sc), M), x1 = __fsub_rn(__fmul_rn(x1, sc), M);
              else
                f32x2_split(fma_f32x2(f32x2(x0, x1), sc2, nm2), x0, x1);
              const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              acc[k & 3] = add_f32x2(acc[k & 3], f32x2(e0, e1));
              pk[k] = pack_f16x2(e0, e1);
            }
            tmem_st16(tS + c32 * 16, pk);
          }
        };
        if (far)
          weights(Int<1>{});
        else
          weights(Int<0>{});
        float s0, s1;
        f32x2_split(add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3])), s0, s1);
        l_run = l_run * alpha + (s0 + s1);
        // O_t is stable here: the commit behind S_FULL covers PV_t of the unit before
        if (u >= u0 + step && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_P_FULL + t));
      }
      // The next item's queries first, so that its products start behind this one's
      // (behind a twin item's only when they have ended: both tiles read its queries).
      if (!ok || !(twin || take_item(i + 1)) ||
          !wait_warp<kWaitHint>(BAR(B_O_DONE), n_o & 1, abort_flag, a.ctl, 43)) {
        ok = false;
        break;
      }
      ++n_o;
      tc_fence_after();
      float f_own = 1.f, f_other = 0.f;
      if (twin) {
        if (t == 1) {  // hands its state over and waits until its O has been read
          twin_state[r].x = M;
          twin_state[r].y = l_run;
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_TWIN_STATE));
          ok = take_item(i + 1) && wait_warp<kWaitHint>(BAR(B_TWIN_DONE), n_twin & 1, abort_flag, a.ctl, 49);
          ++n_twin;
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_ITEM_EMPTY + i % kItems));
          continue;
        }
        if (!take_item(i + 1) || !wait_warp<kWaitHint>(BAR(B_TWIN_STATE), n_twin & 1, abort_flag, a.ctl, 50)) {
          ok = false;
          break;
        }
        ++n_twin;
        const float m1 = twin_state[r].x, l1 = twin_state[r].y, m = fmaxf(M, m1);
        f_own = fast_exp2(M - m), f_other = fast_exp2(m1 - m);
        l_run = l_run * f_own + l1 * f_other;
        M = m;
      }
      const bool whole = x.whole;
      const int cu0 = x.cu0, head = x.head;
      const float inv = whole ? (l_run > 0.f ? 1.f / l_run : 0.f) : 1.f;
      f_own *= inv, f_other *= inv;
      float* part = slot_of<256, D>(a, gridDim.x, blockIdx.x, u0 == 0);
      const int pr = t * 128 + r;
      const int tok = cu0 + row / a.G, hd = head * a.G + row % a.G;
      const long long to = valid ? (long long)tok * a.out.s_row + (long long)hd * a.out.s_head : 0;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f_own);
        if (twin) {
          uint32_t y[32];
          tmem_ld32(tO + 128 + c * 32, y);
          tmem_ld_wait(y);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(fmaf(__uint_as_float(y[k]), f_other, __uint_as_float(o[k])));
        }
        if (!valid) {
        } else if (!whole) {
          // four head dims of all rows together, so that a warp stores 512 bytes at once
          uint4* dst = reinterpret_cast<uint4*>(part) + (c * 8) * 256 + pr;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[256 * k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else if (a.out_f32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(a.out.data) + to + c * 32);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out.data) + to + c * 32);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t* p = o + 8 * k;
            auto f = [&](int i) { return pack_bf16x2(__uint_as_float(p[i]), __uint_as_float(p[i + 1])); };
            dst[k] = make_uint4(f(0), f(2), f(4), f(6));
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      if (twin) {
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_TWIN_DONE));
      }
      if (valid) {
        if (whole)
          store_lse(a, tok, hd, M, l_run);
        else
          *reinterpret_cast<float2*>(part + 256 * D + 2 * pr) = make_float2(M, l_run);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_ITEM_EMPTY + i % kItems));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

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

template <int D>
cudaError_t launch(const CacheAttnPlan& p, cudaStream_t st) {
  const cudaError_t e = configure_kernel<cache_chunk_kernel<D>>(kLaunchRegs, Lay<D>::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_early(cache_chunk_kernel<D>, p.grid, kThreads, Lay<D>::kAlloc, st, p.args);
}

}  // namespace

size_t cache_chunk_ws_bytes(int d) { return line_ws_bytes<256>(num_sms(), d); }

void plan_cache_chunk(CacheAttnPlan& p) {
  CacheAttnArgs& a = p.args;
  p.grid = num_sms();
  p.joins = true;
  // the causal cost of an item is at most G (units + kItemCost) + 2 + 2 tiles places
  const long long units = (a.max_kv + kUnit - 1) / kUnit + ManyRows::kItemCost;
  const long long places = a.causal ? a.G * units + 2 + 2 * (((long long)a.max_new * a.G + 255) / 256) : units;
  a.line_shift = a.items * (places + 2) < (1LL << 30) ? 0 : std::max(1, line_shift_for(a.items, units));
}

cudaError_t launch_cache_chunk(const CacheAttnPlan& p, cudaStream_t st) {
  return p.args.d == 64 ? launch<64>(p, st) : launch<128>(p, st);
}

cudaError_t launch_chunk_join(const CacheAttnPlan& p, cudaStream_t st) {
  return launch_early(p.args.d == 64 ? chunk_join_kernel<64> : chunk_join_kernel<128>, dim3(p.grid, 8), 256, 0, st, p.args);
}

}  // namespace ra
