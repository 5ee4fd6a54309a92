// kv.cuh -- the 8-bit paged key/value cache: page layout, the arguments of its
// kernels, which pages and keys a query sees, and the e4m3 conversions.
//
// A page holds PTL_KV_PAGE = 64 consecutive tokens of one sequence, 64 KB of
// e4m3 codes: [2][8 heads][64][64] bytes, first the keys as [token][dim], then
// the values as [dim][token].  Keys and values both lie along the axis that
// their product sums over (the dims of Q K^T, the tokens of P V), so one 4 KB
// tile is one plain copy, and 16 consecutive bytes of a row are 16 consecutive
// steps of the contraction: no transposition when the pages are read, which
// happens for every token served; it is paid once, in the append.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace ptl {

constexpr int KV_PAGE = PTL_KV_PAGE;        // tokens of a page
constexpr int KV_TILE = KV_PAGE * DH;       // bytes of one side of one head of a page
constexpr int KV_SIDE = H * KV_TILE;        // bytes of the keys (or the values) of a page
constexpr int KV_PAGE_BYTES = 2 * KV_SIDE;  // 65536
constexpr int KV_MIN_EXP = -100;            // smallest scale 2^-100
// Users with at most this many new tokens take attn_paged.cu's kernel, which
// reads the pages once for each 8 of them; the tcgen05 kernel reads them once
// for 256, but works on 128 rows whether or not they are there.  Of 60 users
// over 2,000 tokens each: 8, 16 and 32 new ones 47, 61 and 98 us in the first, 33
// take 94 in the second.  The fp32 build has the first kernel only, which holds
// queries and weights in two halves each; the second has them in one.
constexpr int PAGED_FEW = 32;
constexpr int PAGED_FEW_STEPS = 1000, PAGED_FEW_NEW = 1024;
constexpr int PAGED_TC_MAX_CTAS = 148;
constexpr int PAGED_MAX_CTAS = 2 * 148;     // bound on the paged attention's grid (its workspace holds two parts per block)
constexpr int KV_MAX_USERS = 1 << 30;       // a thread's range of users stays below 2^31
constexpr int KV_MAX_PAGES = (1 << 25) - 1;  // pages of a sequence: positions stay below 2^31

struct KvAppendArgs {
  const void* qkv;
  const int32_t *cu, *table, *past;
  uint8_t* codes;
  float* scales;
  int32_t* err;
  int num_pages, max_pages, U, T;
};

struct PagedArgs {
  const void* qkv;
  void* out;
  const int32_t *cu, *table, *past;
  const uint8_t* codes;
  const float* scales;
  int32_t* err;
  int32_t* counters;  // [CTA][head] parts of a split unit done so far
  float* partial;     // [2 CTA + which][head] unfinished sums of split units
  int num_pages, max_pages, U, T, window, sinks;
  int few;            // users with more new tokens are the tcgen05 kernel's, unless paged_all_few
};

// One user's place in a call, checked: n new tokens behind `past` kept ones.
// Returns the ptl_status that the user's offsets or positions break, or 0.
__device__ __forceinline__ int kv_check_user(const int32_t* cu, const int32_t* past, int u, int U, int T,
                                             int max_pages, int& n, int& p) {
  const int c0 = cu[u], c1 = cu[u + 1];
  p = past[u];
  n = c1 - c0;
  if ((u == 0 && c0 != 0) || c0 < 0 || c1 < c0 || c1 > T || (u == U - 1 && c1 != T)) return PTL_ERR_BAD_OFFSETS;
  if (p < 0 || int64_t(p) + n > int64_t(max_pages) * KV_PAGE) return PTL_ERR_BAD_PAGE;
  return 0;
}

// The pages that queries at positions p0 .. p1 of a sequence read: `sinks`
// pages from the first one on, then the pages `first` .. last.
struct PageSpan {
  int sinks, first, count;
  __device__ __forceinline__ int page(int k) const { return k < sinks ? k : first + k - sinks; }
  // of the first page of the span that is not below `page`
  __device__ __forceinline__ int place(int page) const {
    return page < sinks ? page : page < first ? sinks : page - first + sinks;
  }
};
__device__ __forceinline__ PageSpan page_span(int p0, int p1, int window, int sinks) {
  PageSpan s{0, 0, (p1 >> 6) + 1};
  if (window > 0 && p0 >= window) {
    s.first = (p0 - window + 1) >> 6;
    const int sp = (sinks >> 6) + ((sinks & 63) != 0);
    s.sinks = sp < s.first ? sp : s.first;
    s.count = s.sinks + (p1 >> 6) - s.first + 1;
  }
  return s;
}

// Cost of a user's units in the tcgen05 kernel: a page of a two-tile unit counts
// 2, one of a one-tile unit 1 (measured 0.92 and 0.51 us), and a unit's first page
// PTC_UNIT more, what beginning and ending a unit costs (31 prompts of 1,419
// tokens: 229, 214, 208 and 208 us with 4, 8, 12 and 16).
constexpr int PTC_QB = 256;  // queries of a unit, two tiles of 128
constexpr int PTC_UNIT = 12;
__device__ __forceinline__ int64_t paged_tc_user_cost(const PagedArgs& a, int n, int past) {
  int64_t s = 0;
  for (int q0 = 0; q0 < n; q0 += PTC_QB)
    s += H * (PTC_UNIT + (int64_t(page_span(past + q0, past + min(q0 + PTC_QB, n) - 1, a.window, a.sinks).count)
                          << (n - q0 > 128 ? 1 : 0)));
  return s;
}
// The same user's (8 queries, page) steps in the other kernel, about: as if all
// groups saw what the middle one sees.  A user with more than PAGED_FEW_NEW new tokens
// counts as too many for a whole call: one thread counts a user's groups one by
// one (a sum over all users stays below 2^63).
__device__ __forceinline__ int64_t paged_few_steps(const PagedArgs& a, int n, int past) {
  if (n > PAGED_FEW_NEW) return int64_t(1) << 40;
  const int mid = past + (n >> 1);
  return int64_t((n + 7) >> 3) * page_span(mid, mid, a.window, a.sinks).count;
}
// Does attn_paged.cu's kernel take the users with many new tokens as well?
// (Decided by both kernels from the same sums over those users.)  The tcgen05
// kernel needs 25 us to begin and end, which a call with few steps does not earn
// back.  First kernel / tcgen05 kernel, us: one user's 100 new tokens 20 / 25, 300
// 26 / 43, 900 44 / 52; 60 users' 100 each 38 / 50, 40 over 500 48 / 58; 20 users'
// 64 over 500 40 / 40; the other way, 20 users' 300 each 54 / 50, 500 of two over
// 2,000 68 / 52, 33 of 30 over 4,000 112 / 93, 900 of ten 144 / 67.
__device__ __forceinline__ bool paged_all_few(int64_t few_steps, int64_t tc_cost) {
  return few_steps < PAGED_FEW_STEPS + (tc_cost >> 2);
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Bit b: does the query at position `pos` see token 64 * page + b (base = 64 *
// page)?  Tokens up to itself, and with a window only the last `window` of
// them and the first `sinks` of the sequence.
__device__ __forceinline__ uint64_t page_visible(int pos, int base, int window, int sinks) {
  const int hi = pos - base;
  if (hi < 0) return 0;
  uint64_t m = hi >= 63 ? ~0ull : (2ull << hi) - 1;
  if (window > 0) {
    const int lo = hi - window + 1;
    const uint64_t in = lo <= 0 ? ~0ull : lo >= 64 ? 0ull : ~0ull << lo;
    const int s = sinks - base;
    m &= in | (s <= 0 ? 0ull : s >= 64 ? ~0ull : (1ull << s) - 1);
  }
  return m;
}
// Does every query at positions p0 .. p1 see all 64 tokens from base on?
__device__ __forceinline__ bool page_all_visible(int p0, int p1, int base, int window, int sinks) {
  return base + 63 <= p0 && (window <= 0 || p1 - base < window || base + 63 < sinks);
}

// Two e4m3 codes to two halves (exact: e4m3 is a subset of fp16; 0x7F and
// 0xFF become NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
// Two numbers to halves, lo in the low bits.
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 0x80 in each byte that holds a NaN code
__device__ __forceinline__ uint32_t e4m3_nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

}  // namespace ptl
