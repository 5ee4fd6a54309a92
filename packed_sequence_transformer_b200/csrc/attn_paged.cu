// attn_paged.cu -- attention of new tokens over the 8-bit paged cache, for few
// new tokens per user: bound by reading the pages.
//
// A unit of work is a group of up to QG = 8 consecutive new tokens of one user;
// it walks the pages that its queries see (page_span), and the (unit, page)
// steps of the whole call, laid end to end, are cut into equal ranges, one per
// block, so that one long history is spread over all SMs and many short ones
// share them evenly.  A block has one warp per head; the warps never meet.
// A warp streams its head's 4 KB key and value tiles through a ring of its own
// (plain bulk copies, about 190 KB in flight per SM) and
// computes, per page, on the tensor cores:
//   S[token][query] = K Q^T, 64 x 8, codes converted to fp16 (exact) straight
//     from 16-byte reads of the tile: a lane's 16 bytes are 16 consecutive
//     dims, taken as the k positions of four m16n8k16 steps (the order of a
//     contraction is free, Q is laid out to match);
//   p = 2^(S - m + 15) with the running maximum m of each query;
//   O[dim][query] += V P, where P reaches the operand layout by one 8 x 8
//     transposition per 8 tokens; tokens are dealt to the rows of S in the
//     order in which the value tile's 16-byte reads deliver them.
// The scale of the keys goes into the exponent's factor, that of the values
// onto the page's product, which is summed apart and added to O in fp32: one
// rounding per page, no drift over long histories.
// Q is brought to fp16 by a power of two per row (its largest element into
// [2^13, 2^14)): exact down to 2^-27 of that element.  P is fp16 (2^-12) in
// the bf16 build; in the fp32 build Q and P are each the sum of two halves,
// 22 bits, and the products run twice.
//
// A unit that ends up in several blocks leaves its parts (O, m, l) in the
// workspace; the last of the blocks to arrive, counted per (unit, head), adds
// them in block order, so the result does not depend on who was last.
//
// What bounds it (device time, cold L2): reading the pages, at 90% of the rate of a
// plain copy when there are enough (250 users, one token each over 8,000: 2.05 GB in
// 346 us); with a window of 1,000 the same users take 61 us (258 MB, 65%): 60 to 1,000
// such users take 18 us and their bytes at 5.2 TB/s, for their units have 17 pages
// where the long ones, read at 5.9 TB/s, have 125; one user's token over 1,000: 11 us,
// two launches, a page or two and one exchange of parts.  8 new tokens of each of 60
// users over 2,000 take 47 us, 9 or 16 take 60, 32 take 98: each further group of 8
// reads and converts the pages again.  The fp32 build: 27 us for 5 new tokens of 60
// users over 700 (44 MB, 25%), its products twice as many on half the warps; made for
// few new tokens, it takes many as well: 376 us for 100 of each of 60 users over 2,000,
// 1.06 ms for 31 prompts of 1,419 (their exponentials alone 56 us).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kv.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace ptl {
using namespace sm100;

constexpr int PA_THREADS = 32 * H;
constexpr int PA_QG = 8;        // queries of a unit
// Blocks that share a unit of k pages, at most about PA_PARTS sqrt(k): a step
// takes the blocks 1.3 us each and a part the one that adds them up 0.15 us (one
// query) to 0.6 us (eight), and the sum k / parts * step + parts * part is least
// near there.  One user over 8,000: one query 28 us, with 128 parts 46; eight
// queries 50 us, with 128 parts 153.
constexpr float PA_PARTS_ONE = 4.f, PA_PARTS = 1.5f;
// The largest weight of a query is 2^PA_TOP, so that fp16 holds weights down to
// 2^-39 of it (with 1 for the largest, all below 2^-25 were lost, however many).
constexpr float PA_TOP = 15.f, PA_DOWN = 1.f / 32768.f;
// 4 KB tiles in a warp's ring, about 190 KB an SM: two blocks of the bf16 build,
// one of the fp32 build, whose two-part operands need the registers of both
// (with two blocks it spilled: 36 us instead of 27 for 5 new tokens of 60 users
// over 700).
template <int SPLIT>
constexpr int PA_STAGES = SPLIT == 1 ? 3 : 6;
template <int SPLIT>
constexpr int PA_BLOCKS = SPLIT == 1 ? 2 : 1;
constexpr int PA_PART = PA_QG * (DH + 2);  // floats of one head's part: O, then (m, l) per query

__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), halves
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transposes an 8 x 8 matrix of halves held as (row lane / 4, columns 2 (lane % 4) and + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_rest2(float lo, float hi, uint32_t first) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&first));
  return pack_half2(lo - f.x, hi - f.y);
}

template <int N>
struct Count {
  static constexpr int value = N;
};

// A position in the call's (unit, page) steps.
struct PagedWalk {
  int u, q0, n, past, k;
  int few;        // users with at most this many new tokens count
  int64_t start;  // step of the unit's first page
  PageSpan span;
  __device__ __forceinline__ void load(const PagedArgs& a) {
    n = a.cu[u + 1] - a.cu[u];
    past = a.past[u];
  }
  __device__ __forceinline__ void see(const PagedArgs& a) {
    span = page_span(past + q0, past + min(q0 + PA_QG, n) - 1, a.window, a.sinks);
  }
  __device__ __forceinline__ int entry(const PagedArgs& a) const {
    return a.table[int64_t(u) * a.max_pages + span.page(k)];
  }
  // the next step; only called while one is left
  __device__ __forceinline__ void next(const PagedArgs& a) {
    if (++k < span.count) return;
    k = 0;
    start += span.count;
    q0 += PA_QG;
    if (q0 >= n) {
      q0 = 0;
      do {
        ++u;
        load(a);
      } while (n == 0 || n > few);
    }
    see(a);
  }
};

// Steps of one user.
__device__ __forceinline__ int64_t paged_user_steps(const PagedArgs& a, int n, int past, int few) {
  int64_t s = 0;
  if (n > few) return 0;
  for (int q0 = 0; q0 < n; q0 += PA_QG)
    s += page_span(past + q0, past + min(q0 + PA_QG, n) - 1, a.window, a.sinks).count;
  return s;
}

template <typename T, int SPLIT>
__global__ void __launch_bounds__(PA_THREADS, PA_BLOCKS<SPLIT>) attn_paged_kernel(const PagedArgs a) {
  constexpr int STAGES = PA_STAGES<SPLIT>;
  extern __shared__ __align__(128) uint8_t ring_all[];
  __shared__ uint64_t s_bar[H][STAGES];
  __shared__ int64_t s_scan[H], s_many[2][H];
  __shared__ int s_longest[H];
  __shared__ int s_first[3];
  __shared__ PagedWalk s_walk[H][2];
  __shared__ int64_t s_start;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = warp, g = lane >> 2, t = lane & 3;
  uint64_t* bar = s_bar[warp];
  uint8_t* ring = ring_all + warp * STAGES * KV_TILE;
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  pdl_trigger();

  // every block counts the call's steps by itself: a sum per thread, a scan; and
  // once more if users with many new tokens turn out to be this kernel's as well
  const int per = (a.U + PA_THREADS - 1) / PA_THREADS;
  const int u_lo = min(tid * per, a.U), u_hi = min(u_lo + per, a.U);
  int few = a.few;
  int longest;  // pages of the longest unit, twice, and 1 if its user has several queries
  int64_t mine, base, W;
#pragma unroll 1
  while (true) {
    int64_t many_steps = 0, many_cost = 0;
    int bad = 0;
    mine = 0;
    longest = 0;
#pragma unroll 1
    for (int u = u_lo; u < u_hi; ++u) {
      int n, p;
      const int e = kv_check_user(a.cu, a.past, u, a.U, a.T, a.max_pages, n, p);
      bad |= e == 0 ? 0 : e == PTL_ERR_BAD_OFFSETS ? 1 : 2;
      if (e != 0 || n == 0) continue;
      if (n <= few) {
        mine += paged_user_steps(a, n, p, few);
        longest = max(longest, 2 * page_span(p + (n - 1) / PA_QG * PA_QG, p + n - 1, a.window, a.sinks).count + (n > 1));
      } else {
        many_steps += paged_few_steps(a, n, p);
        many_cost += paged_tc_user_cost(a, n, p);
      }
    }
    if (__syncthreads_or(bad)) {  // every block sees the same offsets: nothing is written
      const int offsets = __syncthreads_or(bad & 1);
      pdl_wait();
      if (blockIdx.x == 0 && tid == 0) set_error(a.err, offsets ? PTL_ERR_BAD_OFFSETS : PTL_ERR_BAD_PAGE);
      return;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (a.T > few) {
      many_steps = warp_sum(many_steps);
      many_cost = warp_sum(many_cost);
    }
    if (lane == 31) {
      s_scan[warp] = incl;
      s_longest[warp] = longest;
      s_many[0][warp] = many_steps;
      s_many[1][warp] = many_cost;
    }
    __syncthreads();
    base = incl - mine;
    W = many_steps = many_cost = 0;
#pragma unroll
    for (int w = 0; w < H; ++w) {
      if (w < warp) base += s_scan[w];
      W += s_scan[w];
      longest = max(longest, s_longest[w]);
      many_steps += s_many[0][w];
      many_cost += s_many[1][w];
    }
    if (many_steps == 0 || !paged_all_few(many_steps, many_cost)) break;
    few = INT32_MAX;
  }
  // this block's steps [A, B), in so few blocks that no unit falls into too many
  int64_t G = W < int64_t(gridDim.x) ? W : int64_t(gridDim.x);
  const int64_t pages = longest >> 1, parts = int(sqrtf(float(pages)) * ((longest & 1) ? PA_PARTS : PA_PARTS_ONE));
  if (G * pages > parts * W) G = parts * W / pages;
  if (int64_t(blockIdx.x) >= G) {
    pdl_wait();
    return;
  }
  // (a 64-bit division costs a small call a noticeable part of its time)
  int64_t A, B;
  if (W < (1 << 22)) {
    A = uint32_t(blockIdx.x * uint32_t(W)) / uint32_t(G);
    B = uint32_t((blockIdx.x + 1) * uint32_t(W)) / uint32_t(G);
  } else {
    A = blockIdx.x * W / G;
    B = (blockIdx.x + 1) * W / G;
  }
  if (A >= base && A < base + mine) {
    int64_t left = A - base;
    for (int u = u_lo; u < u_hi; ++u) {
      const int n = a.cu[u + 1] - a.cu[u], p = a.past[u];
      const int64_t s = paged_user_steps(a, n, p, few);
      if (left >= s) {
        left -= s;
        continue;
      }
      for (int q0 = 0; q0 < n; q0 += PA_QG) {
        const int cnt = page_span(p + q0, p + min(q0 + PA_QG, n) - 1, a.window, a.sinks).count;
        if (left < cnt) {
          s_first[0] = u;
          s_first[1] = q0;
          s_first[2] = int(left);
          s_start = A - left;
          break;
        }
        left -= cnt;
      }
      break;
    }
  }
  __syncthreads();

  // The step being computed and the step whose tiles are loaded next live in
  // shared memory (a warp's own; lane 0 moves them on): the loop needs the
  // registers.
  PagedWalk& cw = s_walk[warp][0];
  PagedWalk& iw = s_walk[warp][1];
  if (lane == 0) {
    cw.few = few;
    cw.u = s_first[0];
    cw.q0 = s_first[1];
    cw.k = s_first[2];
    cw.start = s_start;
    cw.load(a);
    cw.see(a);
    iw = cw;
  }
  __syncwarp();
  const int64_t steps = B - A;

  // tiles are loaded in the order K0 V0 K1 V1 ..., by lane 0; a stage's phase
  // flips each time round
  int64_t sent = 0, used = 0;
  int st_i = 0, st_c = 0, ph_c = 0;
  int id = 0, id_next = lane == 0 ? iw.entry(a) : 0;
  // Scales of the pages under way, the current one's among them at most 4 (a
  // ring of 2 n tiles is at most n pages ahead): page i's in lane i % 4.
  static_assert(STAGES / 2 + 1 <= 4, "lanes for the scales");
  float ks_ahead = 0.f, vs_ahead = 0.f;
  auto issue = [&]() {
    if (sent >= 2 * steps) return;
    const bool key = (sent & 1) == 0;
    if (key) {
      if (lane == 0) {
        id = id_next;
        if (id < 0 || id >= a.num_pages) {  // reported; page 0 stands in, the output is undefined
          pdl_wait();
          set_error(a.err, PTL_ERR_BAD_PAGE);
          id = 0;
        }
        if ((sent >> 1) + 1 < steps) {
          iw.next(a);
          id_next = iw.entry(a);
        }
      }
      const int page = __shfl_sync(0xffffffffu, id, 0);
      if (lane == int((sent >> 1) & 3)) {
        const float* sc = a.scales + int64_t(page) * 2 * H + head;
        ks_ahead = __ldg(sc);
        vs_ahead = __ldg(sc + H);
      }
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar[st_i], KV_TILE);
      bulk_load(ring + st_i * KV_TILE, a.codes + int64_t(id) * KV_PAGE_BYTES + (key ? 0 : KV_SIDE) + head * KV_TILE,
                KV_TILE, &bar[st_i]);
    }
    ++sent;
    if (++st_i == STAGES) st_i = 0;
  };
  for (int i = 0; i < STAGES; ++i) issue();

  uint32_t qf[SPLIT][4][2];
  float cf[2];  // factor of this lane's two queries: softmax scale, log2 e, the row's power of two
  float m[2], l[2], o[4][4];
  bool ok = true;
  for (int64_t i = 0; i < steps && ok; ++i) {
    if (i == 0 || cw.k == 0) {
      // a new unit (or this block's part of one): Q in the order of the key tile's reads
      const int row = cw.q0 + g;
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
      if (row < cw.n) {
        constexpr int VEC = 16 / sizeof(T);
        const T* src = static_cast<const T*>(a.qkv) + int64_t(a.cu[cw.u] + row) * QKV_N + head * DH + 16 * t;
#pragma unroll
        for (int k = 0; k < 16 / VEC; ++k) {
          const uint4 r = __ldg(reinterpret_cast<const uint4*>(src + k * VEC));
          const T* v = reinterpret_cast<const T*>(&r);
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[k * VEC + e] = to_f32<T>(v[e]);
        }
      }
      uint32_t mx = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = max(mx, __float_as_uint(x[e]) & 0x7FFFFFFFu);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int up = min(13 - (int(mx >> 23) - 127), 126);  // the largest element into [2^13, 2^14)
      const float f = __uint_as_float(uint32_t(up + 127) << 23);
      const float c = __uint_as_float(uint32_t(127 - up) << 23) * (0.125f * 1.4426950408889634f);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float lo = x[4 * kk + 2 * b] * f, hi = x[4 * kk + 2 * b + 1] * f;
          qf[0][kk][b] = pack_half2(lo, hi);
          if constexpr (SPLIT == 2) qf[1][kk][b] = pack_rest2(lo, hi, qf[0][kk][b]);
        }
      cf[0] = __shfl_sync(0xffffffffu, c, 8 * t);
      cf[1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    }
    const float ks = __shfl_sync(0xffffffffu, ks_ahead, int(i & 3));
    const float vs = __shfl_sync(0xffffffffu, vs_ahead, int(i & 3)) * PA_DOWN;

    // S = K Q^T: row r of tile mt is token 16 (r / 2 % 4) + 4 mt + 2 (r / 8) + r % 2
    if (!mbar_wait(&bar[st_c], ph_c)) {
      ok = false;
      break;
    }
    float s[4][4];
    {
      const uint8_t* kt = ring + st_c * KV_TILE + (16 * (g >> 1) + (g & 1)) * DH + 16 * t;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const uint4 r0 = *reinterpret_cast<const uint4*>(kt + 4 * mt * DH);
        const uint4 r1 = *reinterpret_cast<const uint4*>(kt + (4 * mt + 2) * DH);
        const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t a0 = e4m3x2_to_half2(w0[kk]), a1 = e4m3x2_to_half2(w1[kk]);
          const uint32_t a2 = e4m3x2_to_half2(w0[kk] >> 16), a3 = e4m3x2_to_half2(w1[kk] >> 16);
#pragma unroll
          for (int sp = 0; sp < SPLIT; ++sp) mma_f16(s[mt], a0, a1, a2, a3, qf[sp][kk][0], qf[sp][kk][1]);
        }
      }
    }
    ++used;
    __syncwarp();  // the tile is read: its stage takes the next one
    issue();
    if (++st_c == STAGES) {
      st_c = 0;
      ph_c ^= 1;
    }

    // the page's keys, the queries' positions
    const int kbase = cw.span.page(cw.k) * KV_PAGE;
    const int p0 = cw.past + cw.q0;
    const bool whole = page_all_visible(p0, cw.past + min(cw.q0 + PA_QG, cw.n) - 1, kbase, a.window, a.sinks);
    const float k0 = cf[0] * ks, k1 = cf[1] * ks;
    uint64_t see[2] = {~0ull, ~0ull};
    if (!whole) {
      see[0] = page_visible(p0 + 2 * t, kbase, a.window, a.sinks);
      see[1] = page_visible(p0 + 2 * t + 1, kbase, a.window, a.sinks);
      const int sh = 16 * (g >> 1) + (g & 1);
      const uint64_t b0 = see[0] >> sh, b1 = see[1] >> sh;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int b = 4 * mt + 2 * r;
          s[mt][2 * r] = ((b0 >> b) & 1) ? s[mt][2 * r] * k0 : -INFINITY;
          s[mt][2 * r + 1] = ((b1 >> b) & 1) ? s[mt][2 * r + 1] * k1 : -INFINITY;
        }
    } else {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[mt][2 * r] *= k0;
          s[mt][2 * r + 1] *= k1;
        }
    }
    float alpha[2], mu[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float mx = s[0][q];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(s[mt][q], s[mt][2 + q]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float mn = fmaxf(m[q], mx);
      alpha[q] = mn == -INFINITY ? 0.f : ex2_approx(m[q] - mn);
      mu[q] = mn == -INFINITY ? 0.f : mn - PA_TOP;  // nothing seen yet: every p is 2^-inf = 0
      m[q] = mn;
      l[q] *= alpha[q];
    }
    uint32_t pf[SPLIT][4][2];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0v = ex2_approx(s[mt][2 * r] - mu[0]), p1v = ex2_approx(s[mt][2 * r + 1] - mu[1]);
        l[0] += p0v;
        l[1] += p1v;
        const uint32_t h = pack_half2(p0v, p1v);
        pf[0][mt][r] = transpose8(h);
        if constexpr (SPLIT == 2) pf[1][mt][r] = transpose8(pack_rest2(p0v, p1v, h));
      }

    // O += V P
    if (!mbar_wait(&bar[st_c], ph_c)) {
      ok = false;
      break;
    }
    {
      const uint8_t* vt = ring + st_c * KV_TILE + g * KV_PAGE + 16 * t;
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) {
        uint4 r0 = *reinterpret_cast<const uint4*>(vt + 16 * dt * KV_PAGE);
        uint4 r1 = *reinterpret_cast<const uint4*>(vt + (16 * dt + 8) * KV_PAGE);
        uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
        uint64_t nan0 = 0, nan1 = 0;
        if (!whole) {
          // values that some query does not see may be anything, NaN codes
          // among them: those are taken out and given back to the queries
          // that do see them
          uint32_t n0 = 0, n1 = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b0 = e4m3_nan_bytes(w0[e]), b1 = e4m3_nan_bytes(w1[e]);
            w0[e] &= ~((b0 >> 7) * 0xFFu);
            w1[e] &= ~((b1 >> 7) * 0xFFu);
            // bits 0 .. 3 of a nibble: the word's bytes
            n0 |= (((b0 >> 7) * 0x10204080u >> 28) & 0xFu) << (4 * e);
            n1 |= (((b1 >> 7) * 0x10204080u >> 28) & 0xFu) << (4 * e);
          }
          if (__any_sync(0xffffffffu, (n0 | n1) != 0u)) {
            nan0 = uint64_t(n0) << (16 * t);
            nan1 = uint64_t(n1) << (16 * t);
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
              nan0 |= __shfl_xor_sync(0xffffffffu, nan0, off);
              nan1 |= __shfl_xor_sync(0xffffffffu, nan1, off);
            }
          }
        }
        float op[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          const uint32_t a0 = e4m3x2_to_half2(w0[mt]), a1 = e4m3x2_to_half2(w1[mt]);
          const uint32_t a2 = e4m3x2_to_half2(w0[mt] >> 16), a3 = e4m3x2_to_half2(w1[mt] >> 16);
#pragma unroll
          for (int sp = 0; sp < SPLIT; ++sp) mma_f16(op, a0, a1, a2, a3, pf[sp][mt][0], pf[sp][mt][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[dt][e] = fmaf(o[dt][e], alpha[e & 1], vs * op[e]);
          if (((e < 2 ? nan0 : nan1) & see[e & 1]) != 0) o[dt][e] = __uint_as_float(0x7FC00000u);
        }
      }
    }
    ++used;
    __syncwarp();
    issue();
    if (++st_c == STAGES) {
      st_c = 0;
      ph_c ^= 1;
    }

    const bool unit_end = cw.k == cw.span.count - 1;
    if (unit_end || i == steps - 1) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], 4);
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], 8);
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], 16);
      }
      const int nq = min(PA_QG, cw.n - cw.q0);
      T* dst = static_cast<T*>(a.out) + int64_t(a.cu[cw.u] + cw.q0) * D + head * DH;
      if (unit_end && cw.start >= A) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (2 * t + q >= nq) continue;
          const float inv = 1.0f / (l[q] * PA_DOWN);
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            dst[(2 * t + q) * D + 16 * d + g] = from_f32<T>(o[d][q] * inv);
            dst[(2 * t + q) * D + 16 * d + 8 + g] = from_f32<T>(o[d][2 + q] * inv);
          }
        }
      } else {
        // the blocks c0 .. c1 hold the unit; block c starts at step c W / G
        const int64_t end = cw.start + cw.span.count;
        const int c0 = int(((cw.start + 1) * G - 1) / W), c1 = int((end * G - 1) / W);
        auto part = [&](int c) { return a.partial + (int64_t(2 * c + (c == c0 ? 1 : 0)) * H + head) * PA_PART; };
        float* mp = part(blockIdx.x);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (2 * t + q >= nq) continue;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            mp[(2 * t + q) * DH + 16 * d + g] = o[d][q];
            mp[(2 * t + q) * DH + 16 * d + 8 + g] = o[d][2 + q];
          }
          if (g == 0) *reinterpret_cast<float2*>(mp + PA_QG * DH + 2 * (2 * t + q)) = make_float2(m[q], l[q]);
        }
        __threadfence();
        __syncwarp();
        pdl_wait();  // the counters are zero
        int done = 0;
        if (lane == 0) done = atomicAdd(a.counters + c0 * H + head, 1);
        done = __shfl_sync(0xffffffffu, done, 0);
        if (done == c1 - c0) {  // the last part: add them up, in block order
          __threadfence();
          // four lanes a query: maximum and sum over all parts
          const int q4 = lane >> 2;
          float M = -INFINITY, L = 0.f;
#pragma unroll 4
          for (int c = c0 + (lane & 3); c <= c1; c += 4) {
            if (q4 < nq) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(c) + PA_QG * DH + 2 * q4));
              const float mn = fmaxf(M, ml.x);
              if (mn != -INFINITY) L = ex2_approx(M - mn) * L + ex2_approx(ml.x - mn) * ml.y;
              M = mn;
            }
          }
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) {
            const float Mo = __shfl_xor_sync(0xffffffffu, M, off), Lo = __shfl_xor_sync(0xffffffffu, L, off);
            const float mn = fmaxf(M, Mo);
            if (mn != -INFINITY) L = ex2_approx(M - mn) * L + ex2_approx(Mo - mn) * Lo;
            M = mn;
          }
          if (M == -INFINITY) M = 0.f;
          const float inv = 1.0f / (L * PA_DOWN);
          // 16 lanes hold a row, the two halves of the warp take parts in turn
          const int half = lane >> 4, d4 = lane & 15;
          auto add_up = [&](auto rows, auto depth, int q0) {
            constexpr int NQ = decltype(rows)::value, UN = decltype(depth)::value;
            float4 acc[NQ];
            float Mq[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
              Mq[q] = __shfl_sync(0xffffffffu, M, 4 * min(q0 + q, PA_QG - 1));
            }
#pragma unroll UN
            for (int c = c0 + half; c <= c1; c += 2) {
              const float* pc = part(c);
#pragma unroll
              for (int q = 0; q < NQ; ++q) {
                if (q0 + q >= nq) continue;
                const float we = ex2_approx(__ldcg(pc + PA_QG * DH + 2 * (q0 + q)) - Mq[q]);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(pc + (q0 + q) * DH) + d4);
                acc[q].x = fmaf(we, v.x, acc[q].x);
                acc[q].y = fmaf(we, v.y, acc[q].y);
                acc[q].z = fmaf(we, v.z, acc[q].z);
                acc[q].w = fmaf(we, v.w, acc[q].w);
              }
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              const float iq = __shfl_sync(0xffffffffu, inv, 4 * min(q0 + q, PA_QG - 1));
              float o4[4] = {acc[q].x, acc[q].y, acc[q].z, acc[q].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) o4[e] = (o4[e] + __shfl_xor_sync(0xffffffffu, o4[e], 16)) * iq;
              if (half == 0 && q0 + q < nq) {
                T* d = dst + (q0 + q) * D + 4 * d4;
                if constexpr (sizeof(T) == 2)
                  *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(o4[0], o4[1]), pack_bf16x2(o4[2], o4[3]));
                else
                  *reinterpret_cast<float4*>(d) = make_float4(o4[0], o4[1], o4[2], o4[3]);
              }
            }
          };
          if (nq == 1)
            add_up(Count<1>{}, Count<8>{}, 0);
          else
            for (int q0 = 0; q0 < nq; q0 += 4) add_up(Count<4>{}, Count<2>{}, q0);
        }
      }
    }
    __syncwarp();
    if (lane == 0 && i + 1 < steps) cw.next(a);
    __syncwarp();
  }
  pdl_wait();
  if (!ok) {
    set_error(a.err, PTL_ERR_TIMEOUT);
    // this warp's own copies must not land after the block has left
    for (; used < sent; ++used) {
      mbar_wait(&bar[st_c], ph_c);
      if (++st_c == STAGES) {
        st_c = 0;
        ph_c ^= 1;
      }
    }
  }
}

template <int SPLIT>
static int paged_grid() {
  const int g = PA_BLOCKS<SPLIT> * num_sms();
  return g < PAGED_MAX_CTAS ? g : PAGED_MAX_CTAS;
}

template <typename T, int SPLIT>
static int launch_paged_t(const PagedArgs& a, cudaStream_t st) {
  constexpr int smem = H * PA_STAGES<SPLIT> * KV_TILE;
  static PerDevice configured;
  if (configured.get([] {
        return cudaFuncSetAttribute(attn_paged_kernel<T, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem) == cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return -1;
  if (launch_k(attn_paged_kernel<T, SPLIT>, dim3(paged_grid<SPLIT>()), dim3(PA_THREADS), smem, st, a) != 0) return -1;
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

size_t paged_partial_bytes() {
  const size_t few = sizeof(float) * 2 * PAGED_MAX_CTAS * H * PA_PART;
  return few > paged_tc_partial_bytes() ? few : paged_tc_partial_bytes();  // one launch after the other
}

int launch_attn_paged(PagedArgs a, ptl_dtype dt, cudaStream_t st) {
  a.few = dt == PTL_BF16 ? PAGED_FEW : INT32_MAX;
  const int r = dt == PTL_BF16 ? launch_paged_t<__nv_bfloat16, 1>(a, st) : launch_paged_t<float, 2>(a, st);
  if (r != 0 || dt != PTL_BF16 || a.T <= PAGED_FEW) return r;
  // A call too small for the other kernel, whatever its lengths are
  // (paged_all_few): at most T / 33 users have more than PAGED_FEW = 32 new tokens
  // and one unfinished group each, and no query sees more pages than the table or
  // the window has.  The launch that finds nothing to do costs 3 us (60 users, one
  // token each: 15 us with it, 12 without).
  int64_t pages = a.max_pages;
  if (a.window > 0) {
    const int64_t seen = (a.window - 1) / KV_PAGE + 2 + (int64_t(a.sinks) + KV_PAGE - 1) / KV_PAGE;
    if (seen < pages) pages = seen;
  }
  if (a.T <= PAGED_FEW_NEW && (a.T / 8 + a.T / (PAGED_FEW + 1) + 1) * pages < PAGED_FEW_STEPS) return r;
  return launch_attn_paged_tc(a, st);
}

}  // namespace ptl
