// The paged 4-bit key / value cache as its kernels see it: where a token's row
// lies, what its bits stand for, and how a group of 16 numbers is quantised.
#pragma once

#include <cuda_fp16.h>

#include "ra_cache_args.h"

namespace ra {

// The cache's kernels are launched so that their blocks may be set up while the
// stream's previous kernel still runs (programmatic dependent launch): every kernel
// calls after_previous_kernel before it touches memory, which waits until that
// kernel has ended and its writes are visible, and only then allows the same to
// the next one, so no more than two kernels overlap.  Global memory is read by
// plain loads, which stay behind the wait (loads through the read-only path need
// not).  Saves about 2 us a launch for single tokens.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Sites of device-side errors in the low byte of check_device_error's info.
enum : int { SITE_CACHE_LEN = 0x61, SITE_CACHE_PAGE = 0x62, SITE_CACHE_POS = 0x63 };

// Sequence whose new tokens row t is one of; t is the same in every lane of a full
// warp, which probes 32 entries of cu a round.
__device__ __forceinline__ int sequence_of(const CacheSeqs& s, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = s.n_seqs - 1;
  while (lo < hi) {
    const int step = (hi - lo + 32) >> 5, at = lo + lane * step;
    const bool le = at <= hi && s.cu[at] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le) | 1u;
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Cache index of row t, one of sequence i's new tokens, or -1 when it has no place: before the
// cache's start (padding; a negative length counts as 0, so that the index is exact), or
// past the page table (recorded).  It follows from the length as it is: one cut to the
// table would move the tokens onto others' places.
__device__ __forceinline__ int cache_index(const CacheSeqs& s, int i, int t, const DevCtl& ctl) {
  const int tok = max(s.lens[i], 0) - s.cu[i + 1] + t;
  if (tok >= s.max_tokens) {
    record_error(ctl, DEV_BOUNDS, SITE_CACHE_LEN);
    return -1;
  }
  return tok;
}

// A page number of the table, or -1 (recorded) when there is no such page.
__device__ __forceinline__ int check_page(const CacheView& c, int pg, const DevCtl& ctl) {
  if ((unsigned)pg >= (unsigned)c.n_pages) {
    record_error(ctl, DEV_BOUNDS, SITE_CACHE_PAGE);
    return -1;
  }
  return pg;
}
// Physical page of token `tok` of sequence i (0 <= tok < max_pages * page), or -1.
__device__ __forceinline__ int cache_page(const CacheSeqs& s, const CacheView& c, int i, int tok, const DevCtl& ctl) {
  return check_page(c, s.table[(long long)i * s.table_stride + (tok >> c.page_shift)], ctl);
}

__device__ __forceinline__ long long row_offset(const CacheRows& r, int page, int head, int row) {
  return (long long)page * r.s_page + (long long)head * r.s_head + (long long)row * r.s_row;
}

// Eight 4-bit numbers of a word as fp16 pairs (0,1) (2,3) (4,5) (6,7).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two e4m3 scales (the low byte in the low half) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  const uint16_t t = (uint16_t)two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(t));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half_lo2(uint32_t a) { return __byte_perm(a, a, 0x1010); }
__device__ __forceinline__ uint32_t half_hi2(uint32_t a) { return __byte_perm(a, a, 0x3232); }

}  // namespace ra
