// attn_paged_tc.cu -- attention of new tokens over the 8-bit paged cache on
// tcgen05, for users with many new tokens (bf16 build).
//
// A unit of work is (user, 256-query block, head): one or two tiles of 128
// queries that share the pages their queries see.  The (unit, page) costs of
// the whole call, laid end to end, are cut into equal ranges, one per SM, as in
// attn_paged.cu; a unit that ends up in several blocks leaves parts that the
// last block adds in block order.
//
//   warps 0..15   four softmax groups: thread r of a group owns query row r of
//                 a tile (TMEM lane r).  In a two-tile unit two groups share a
//                 tile and take its pages in turn, in a one-tile unit all four
//                 do; each has scores, weights and sums of its own, which are
//                 added at the unit's end.  So each scheduler has four warps
//                 whose waits and exponentials interleave: with two groups, each
//                 with a tile to itself, 256 queries over each of 16
//                 histories of 8,000 took 201 us where four took 160.
//   warps 16..19  converters, two pairs: a pair takes every second page, brings
//                 it into shared memory with asynchronous copies, two pages of
//                 its own ahead, and turns it into fp16 in the 128-byte-swizzled
//                 layout of the MMA operands (exact; both sides are stored along
//                 the contraction, so both are K-major); at a unit's start also
//                 its queries, brought to fp16 by a power of two per row.  The
//                 first one also walks the block's units and lays down what
//                 the roles need of each (PagedPart) in a ring in shared
//                 memory, so that no other spends registers on it.
//   warps 20..23  MMA issuers, one thread per group: per page S = Q K^T
//                 (128 x 64), then O += P V with P from TMEM, where it has
//                 taken S's place.  The whole warp walks along and one lane
//                 issues: with the other lanes parted from it a page's eight
//                 products took 788 cycles instead of 543.
//
// What bounds it: the groups' chains from a page's scores to its weights, its
// product and the next scores.  A round of the four groups takes about 3,400
// cycles, of which the exponentials fill 2,048 and the products 1,250; with the
// conversions, the exponentials, the maximum or three quarters of the products
// left out it is at most 7% shorter each, with all of the softmax left out 50%.
// Measured (device time, cold L2): 16 users with 256 new tokens over 16,000: 244 us,
// 554 TFLOP/s; 100 of each of 60 users over 2,000: 100 us; 31 users' prompts of 1,419
// tokens (44,000 in all): 208 us; a call that only begins and ends, 25 us.
//
// Exponent: t = s q_row k_page + log2(v_page), w = 2^(t - m): the value scale,
// a power of two, rides in the exponent, so that O accumulates over pages in
// TMEM.  m comes from the maximum of the pages before; only when a page exceeds
// that by 2^4 is m raised and O rescaled in place.  The normaliser counts scores
// without value scales: l = sum 2^(s - n) has a reference n of its own, the
// largest score (raised like m), so that l lies between about 1 and 2^4 times the
// number of keys whatever the scales are (relative to m, 131 pages of zero values
// took it beyond fp32).  A page adds its w times 2^(m - log2(v_page) - n); where
// its w would fall below what fp32 holds, which weighs nothing in O but may weigh
// all in l, they are taken relative to the page's own maximum.  At last
// out = O / l 2^(m - n).
// Values that are NaN codes in a page that some query does not see wholly are
// taken out by the converters and given back, per row, to the queries that see
// them.  Every wait is bounded.
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

constexpr int PTC_GROUPS = 4;
constexpr int PTC_CONV0 = 4 * PTC_GROUPS, PTC_ISSUE0 = PTC_CONV0 + 4;  // first converter and issuer warp
constexpr int PTC_THREADS = 32 * (PTC_ISSUE0 + PTC_GROUPS);
constexpr int PTC_PARTS = 16;   // units in the plan's ring: converters ask for pages up to 4 units ahead
// 24 warps, 80 registers each at launch, dealt out anew (6 * 80 = 4 * 88 + 88 +
// 40): with 80 everywhere the loops spill more, and a spilled register costs a trip
// to L2 here, for shared memory takes nearly all of L1 (168 us instead of 160
// for 256 queries over each of 16 histories of 8,000 tokens).  What is left spilled is
// 12 bytes of stores and 24 of loads.
constexpr int PTC_REGS = 88, PTC_REGS_ISSUE = 40;
// Converted pages (keys and values of one head).  An even number: a stage then
// belongs to one converter pair, whose order keeps its phases apart (a barrier's
// parity cannot tell a phase from the one after next).
constexpr int PTC_STAGES = 6;
constexpr int PTC_RAW = 2;      // raw pages of each converter pair
constexpr int PTC_OPERAND = 64 * 128;  // bytes of 64 rows of 64 halves
constexpr int PTC_STAGE = 2 * PTC_OPERAND;
constexpr int PTC_QTILE = 128 * 128;
constexpr int PTC_RAW_BYTES = 2 * KV_TILE;
constexpr int PTC_SMEM = 4 * PTC_QTILE + PTC_STAGES * PTC_STAGE + 2 * PTC_RAW * PTC_RAW_BYTES + 1024;
constexpr int PTC_PART = 128 * (DH + 4);  // floats of one tile's part: O, then (m, n, l, 0) per row
// A tile's reference m lies 2^PTC_TOP below the largest exponent it was taken
// from, and is taken anew when a page exceeds that by 2^PTC_RAISE: weights reach
// 2^15 at most, and fp16 holds them to 2^-35 of the largest (with weights of 1
// for the largest, what lay 2^-25 below it was lost, as much as 2^20 tokens of it).
constexpr float PTC_TOP = 11.f, PTC_RAISE = 4.f;
// n, and the m of several groups, of a row that has seen nothing: below any score,
// and differences of two are numbers (a test for -inf at each of them cost 5% of a
// call's time).
constexpr float PTC_NONE = -3e38f;

__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// 16 consecutive 32-bit columns of the thread's TMEM lane, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// mbar_wait that looks at the clock only now and then (an issuer's wait is on
// the path from a page's weights to its next scores).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// The same for a whole warp: all lanes leave together, so that a limit that runs
// out never parts a warp.
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (int i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63) == 0 && __any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
}

// One unit and the pages of it that this block has.  Costs (paged_tc_user_cost),
// not pages, are laid end to end.  A page belongs to the block that its first
// cost falls into, and blocks have at least PTC_UNIT + 2 costs each, so every
// block between a unit's first and last has a page of it.
struct PagedTcUnit {
  int u, q0, head, n, past, k0, k1;
  bool two;
  int64_t start;  // the unit's first cost
  PageSpan span;
  __device__ __forceinline__ void user(const PagedArgs& a) {
    n = a.cu[u + 1] - a.cu[u];
    past = a.past[u];
  }
  __device__ __forceinline__ int64_t cost() const { return PTC_UNIT + (int64_t(span.count) << int(two)); }
  // where the last page's cost begins
  __device__ __forceinline__ int64_t last_page() const { return span.count == 1 ? start : start + cost() - (1 << int(two)); }
  __device__ __forceinline__ void see(const PagedArgs& a, int64_t A, int64_t B) {
    two = n - q0 > 128;
    span = page_span(past + q0, past + min(q0 + PTC_QB, n) - 1, a.window, a.sinks);
    mine(A, B);
  }
  // how many of the unit's pages begin before cost x
  __device__ __forceinline__ int before(int64_t x) const {
    if (x <= start) return 0;
    const int64_t r = two ? 1 : 0, k = (x - start - PTC_UNIT + r) >> r;
    return k < 1 ? 1 : k > span.count ? span.count : int(k);
  }
  __device__ __forceinline__ void mine(int64_t A, int64_t B) {
    k0 = before(A);
    k1 = before(B);
  }
  // the next unit; false when it starts at or behind B
  __device__ __forceinline__ bool next(const PagedArgs& a, int64_t A, int64_t B) {
    start += cost();
    if (start >= B) return false;
    if (++head < H) {
      mine(A, B);
      return true;
    }
    head = 0;
    q0 += PTC_QB;
    if (q0 >= n) {
      q0 = 0;
      do {
        ++u;
        user(a);
      } while (n <= a.few);
    }
    see(a, A, B);
    return true;
  }
};

// A query tile in a part [k0, k1) of a unit's pages: the tile sees the part's
// pages j (from k0 on) below `sink_end` and in [lo, hi), and wholly those whose
// numbers pass `whole`.
struct PagedTcTile {
  int rows, p0;  // its rows, position of the first
  int sink_end, lo, hi;
  int whole_hi, whole_lo, whole_sinks;
  __device__ __forceinline__ void set(const PagedArgs& a, const PagedTcUnit& w, int tile) {
    rows = min(128, w.n - w.q0 - 128 * tile);
    p0 = w.past + w.q0 + 128 * tile;
    const int p1 = p0 + rows - 1;
    whole_hi = (p0 - 63) >> 6;                                    // base + 63 <= p0
    whole_lo = a.window > 0 && p1 >= a.window ? ((p1 - a.window) >> 6) + 1 : 0;  // p1 - base < window
    whole_sinks = a.sinks >> 6;                                   // base + 63 < sinks
    // pages below `sinks`, and from `first` on to p1's, as places in the part
    const int sinks = (a.sinks >> 6) + ((a.sinks & 63) != 0);
    const int first = a.window > 0 && p0 >= a.window ? (p0 - a.window + 1) >> 6 : 0;
    hi = max(0, min(w.span.place(p1 >> 6) + 1, w.k1) - w.k0);
    sink_end = max(0, min(w.span.place(sinks) - w.k0, hi));
    lo = max(w.span.place(first) - w.k0, sink_end);
  }
  __device__ __forceinline__ bool whole(int page) const {
    return page <= whole_hi && (page >= whole_lo || page < whole_sinks);
  }
};
// A group takes pages j with (j & turns) == turn that its tile sees: in a
// two-tile unit every second, in a one-tile unit every fourth.
struct PagedTcShare {
  int turn, turns;
  // (a tile's first group, which also adds the sums up, comes last)
  __device__ __forceinline__ PagedTcShare(bool two, int g) : turn((g + (two ? 1 : 3)) & (two ? 1 : 3)), turns(two ? 1 : 3) {}
  __device__ __forceinline__ int below(int x) const { return (x + turns - turn) >> (turns == 1 ? 1 : 2); }  // j < x
  __device__ __forceinline__ int pages(const PagedTcTile& t) const {
    return below(t.sink_end) + max(0, below(t.hi) - below(t.lo));
  }
};
// What the roles need of a unit and this block's part of it.
struct PagedPart {
  int64_t list;      // entry of the page table where the sequence's pages begin
  int last;          // 1: no further unit (and nothing else is set)
  int head, row0, rows;  // head, first row of qkv, rows of the unit
  int two;           // two tiles
  int k0, pages;     // places in the span
  int sinks, first;  // the span: place k is page k below `sinks`, then first + k - sinks
  int c0, c1;        // the blocks that hold the unit
  PagedTcTile tile[2];
};

__global__ void __launch_bounds__(PTC_THREADS, 1) attn_paged_tc_kernel(const PagedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                                  // [slot][tile]
  uint8_t* sKV = sQ + 4 * PTC_QTILE;                   // [stage][keys, values]
  uint8_t* sRaw = sKV + PTC_STAGES * PTC_STAGE;        // [converter pair][raw stage]
  __shared__ uint64_t q_full[2], q_empty[2], kv_full[PTC_STAGES], kv_empty[PTC_STAGES];
  __shared__ uint64_t s_full[PTC_GROUPS], p_full[PTC_GROUPS], o_full[PTC_GROUPS], o_empty[PTC_GROUPS];
  // (who adds group 3's sums up depends on the unit's kind: a barrier for each,
  // so that each waits for every phase of the one that it looks at)
  __shared__ uint64_t x_full[2][PTC_GROUPS], x_empty[PTC_GROUPS], group_bar[PTC_GROUPS];
  __shared__ float s_rawscale[2][PTC_RAW][2];
  // [stage] key scale, value scale's log2, page number * 4 with bits 0 and 1:
  // tile 0's and 1's queries all see all of it
  __shared__ __align__(16) float4 s_meta[PTC_STAGES];
  __shared__ __align__(8) uint2 s_hasnan[PTC_STAGES];      // [stage] each warp of the pair took out NaN values
  __shared__ __align__(8) uint16_t s_nan[PTC_STAGES][64][4];  // which tokens of row d
  __shared__ int s_stage[PTC_GROUPS];                      // the stage of the group's page
  __shared__ float s_c[2][PTC_QB];                         // [slot][row] exponent's factor
  __shared__ float s_xm[PTC_GROUPS][128], s_xn[PTC_GROUPS][128], s_xl[PTC_GROUPS][128];  // m, n, l handed over
  __shared__ uint64_t s_xnan[PTC_GROUPS][128];
  __shared__ float s_wm[PTC_GROUPS][128];   // of the rows whose parts are added: m, and 1 / l, 2^(m - n)
  __shared__ float2 s_wl[PTC_GROUPS][128];
  __shared__ int64_t s_scan[PTC_THREADS / 32], s_few[PTC_THREADS / 32];
  __shared__ int64_t s_start;
  __shared__ int s_first[3];
  __shared__ int s_done[PTC_GROUPS];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(16) PagedPart s_part[PTC_PARTS];
  __shared__ PagedTcUnit s_walk;
  __shared__ uint64_t u_full[PTC_PARTS], u_empty[PTC_PARTS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&q_empty[i], PTC_GROUPS + 128 * PTC_GROUPS);
    }
    for (int i = 0; i < PTC_GROUPS; ++i) {
      mbar_init(&s_full[i], 2);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 128);
      mbar_init(&x_full[0][i], 128);
      mbar_init(&x_full[1][i], 128);
      mbar_init(&x_empty[i], 128);
      mbar_init(&group_bar[i], 128);
    }
    for (int i = 0; i < PTC_PARTS; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 4 + PTC_GROUPS + 128 * PTC_GROUPS);
    }
    for (int i = 0; i < PTC_STAGES; ++i) {
      mbar_init(&kv_full[i], 64);
      mbar_init(&kv_empty[i], 2);  // a page's group of each tile, or its one group twice
    }
    fence_mbar_init();
  }
  pdl_trigger();

  // the call's costs, counted by every block (see attn_paged.cu)
  const int per = (a.U + PTC_THREADS - 1) / PTC_THREADS;
  const int u_lo = min(tid * per, a.U), u_hi = min(u_lo + per, a.U);
  int64_t mine = 0, few_steps = 0;
  int bad = 0;
  for (int u = u_lo; u < u_hi; ++u) {
    int n, p;
    if (kv_check_user(a.cu, a.past, u, a.U, a.T, a.max_pages, n, p) != 0)
      bad = 1;
    else if (n > a.few) {
      mine += paged_tc_user_cost(a, n, p);
      few_steps += paged_few_steps(a, n, p);
    }
  }
  if (__syncthreads_or(bad)) {  // attn_paged_kernel reports it
    pdl_wait();
    return;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  few_steps = warp_sum(few_steps);
  if (lane == 31) {
    s_scan[warp] = incl;
    s_few[warp] = few_steps;
  }
  __syncthreads();
  int64_t base = incl - mine, W = 0;
  few_steps = 0;
#pragma unroll
  for (int w = 0; w < PTC_THREADS / 32; ++w) {
    if (w < warp) base += s_scan[w];
    W += s_scan[w];
    few_steps += s_few[w];
  }
  const int64_t G = min(int64_t(gridDim.x), max(W / (PTC_UNIT + 2), int64_t(1)));
  if (int64_t(blockIdx.x) >= G || W == 0 || paged_all_few(few_steps, W)) {
    pdl_wait();
    return;
  }
  const int64_t A = blockIdx.x * W / G, B = (blockIdx.x + 1) * W / G;
  if (A >= base && A < base + mine) {
    int64_t left = A - base;
    for (int u = u_lo; u < u_hi; ++u) {
      const int n = a.cu[u + 1] - a.cu[u], p = a.past[u];
      const int64_t s = n > a.few ? paged_tc_user_cost(a, n, p) : 0;
      if (left >= s) {
        left -= s;
        continue;
      }
      for (int q0 = 0; q0 < n; q0 += PTC_QB) {
        const int64_t c = PTC_UNIT + (int64_t(page_span(p + q0, p + min(q0 + PTC_QB, n) - 1, a.window, a.sinks).count)
                                      << (n - q0 > 128 ? 1 : 0));
        if (left < H * c) {
          s_first[0] = u;
          s_first[1] = q0;
          s_first[2] = int(left / c);
          s_start = A - left % c;
          break;
        }
        left -= H * c;
      }
      break;
    }
  }
  if (warp == PTC_ISSUE0) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // TMEM columns of group g, from 128 g on: S 0..63 (then P, pairs of halves,
  // in 0..31), O 64..127
  bool ok = true;

  if (warp >= PTC_CONV0 && warp < PTC_ISSUE0) {
    // ------------------------------------------------------------ converters
    regs_more<PTC_REGS>();
    const int cw = warp - PTC_CONV0;
    const int pair = cw >> 1, ct = tid & 63;  // thread of the pair
    uint8_t* raw = sRaw + pair * PTC_RAW * PTC_RAW_BYTES + ct * 16;
    // of this block's pages the pair has number `pair`, `pair` + 2, ...,
    // requested PTC_RAW ahead, across units
    int iu = -1, ik = pair, iend = 0, isinks = 0, ifirst = 0, ihead = 0, id_next = 0, raw_i = 0, raw_c = 0;
    const int32_t* ilist = nullptr;
    bool more = true;
    // lays down unit number iu (the first converter's first lane; it asks for
    // pages further ahead than any other role looks)
    auto plan = [&](int slot) {
      PagedTcUnit& w = s_walk;
      bool go = true;
      if (iu == 0) {
        w.u = s_first[0];
        w.q0 = s_first[1];
        w.head = s_first[2];
        w.start = s_start;
        w.user(a);
        w.see(a, A, B);
      } else {
        go = w.next(a, A, B);
      }
      while (go && w.k0 >= w.k1) go = w.next(a, A, B);  // no page of it is this block's
      if (!wait_bar(&u_empty[slot], ((iu / PTC_PARTS) & 1) ^ 1)) return;  // (the wait for it reports)
      PagedPart& p = s_part[slot];
      p.last = !go;
      if (go) {
        p.list = int64_t(w.u) * a.max_pages;
        p.head = w.head;
        p.row0 = a.cu[w.u] + w.q0;
        p.rows = min(PTC_QB, w.n - w.q0);
        p.two = w.two;
        p.k0 = w.k0;
        p.pages = w.k1 - w.k0;
        p.sinks = w.span.sinks;
        p.first = w.span.first;
        // block k starts at cost k W / G
        p.c0 = int(((w.start + 1) * G - 1) / W);
        p.c1 = int(((w.last_page() + 1) * G - 1) / W);
        p.tile[0].set(a, w, 0);
        p.tile[1].set(a, w, w.two ? 1 : 0);
      }
      mbar_arrive(&u_full[slot]);
    };
    auto settle = [&]() {  // to the pair's next page
      while (ik >= iend) {
        ik -= iend;  // pages of the next unit to pass over
        ++iu;
        const int slot = iu % PTC_PARTS;
        if (cw == 0) {
          if (lane == 0) plan(slot);
          __syncwarp();
        }
        ok = ok && warp_wait_bar(&u_full[slot], (iu / PTC_PARTS) & 1);
        const PagedPart& p = s_part[slot];
        if (!ok || p.last) {
          more = false;
          return;
        }
        isinks = p.sinks;
        ifirst = p.first;
        ihead = p.head;
        ilist = a.table + p.list;
        // the unit's queries into L2 while its first pages are on their way
        const int row = 32 * cw + lane;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.qkv) + int64_t(p.row0 + row) * QKV_N + ihead * DH;
        if (row < p.rows) prefetch_l2(q);
        if (row + 128 < p.rows) prefetch_l2(q + 128 * QKV_N);
        ik += p.k0;
        iend = p.k0 + p.pages;
      }
      id_next = ilist[ik < isinks ? ik : ifirst + ik - isinks];
    };
    settle();
    auto issue = [&]() {
      if (more) {
        int id = id_next;
        if (id < 0 || id >= a.num_pages) {  // reported; page 0 stands in, the output is undefined
          pdl_wait();
          if (lane == 0) set_error(a.err, PTL_ERR_BAD_PAGE);
          id = 0;
        }
        const uint8_t* src = a.codes + int64_t(id) * KV_PAGE_BYTES + ihead * KV_TILE + ct * 16;
        uint8_t* dst = raw + raw_i * PTC_RAW_BYTES;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          cp_async16(dst + 1024 * p, src + 1024 * p);
          cp_async16(dst + KV_TILE + 1024 * p, src + KV_SIDE + 1024 * p);
        }
        if (ct == 0) {
          cp_async4(&s_rawscale[pair][raw_i][0], a.scales + int64_t(id) * 2 * H + ihead);
          cp_async4(&s_rawscale[pair][raw_i][1], a.scales + int64_t(id) * 2 * H + H + ihead);
        }
        ik += 2;
        settle();
        if (++raw_i == PTC_RAW) raw_i = 0;
      }
      cp_async_commit();  // an empty group at the end keeps the count
    };
    for (int i = 0; i < PTC_RAW; ++i) issue();
    // the thread's 16 codes of a row: rows 16 p + ct / 4, quarter ct % 4
    const int rr = ct >> 2, q = ct & 3;
    const uint32_t swz0 = rr * 128 + 16 * ((2 * q) ^ (rr & 7)), swz1 = rr * 128 + 16 * ((2 * q + 1) ^ (rr & 7));
    int st = pair, ph = 1;  // stage of the pair's page and its phase
    int j = pair;           // the next page of the unit that is the pair's
    for (int unit = 0; ok; ++unit) {
      const int us = unit % PTC_PARTS, slot = unit & 1;
      const PagedPart& u = s_part[us];
      if (!warp_wait_bar(&u_full[us], (unit / PTC_PARTS) & 1)) {
        ok = false;
        break;
      }
      if (u.last) break;
      if (!warp_wait_bar(&q_empty[slot], ((unit >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
#pragma unroll 1
      for (int i = 0; i < (u.two ? 2 : 1); ++i) {
        const int row = 128 * i + 32 * cw + lane;  // of the unit; tile i
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.qkv) +
                                                          int64_t(u.row0 + row) * QKV_N + u.head * DH);
        uint4 x[8];
        const bool has = row < u.rows;
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = has ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t e[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int b = 0; b < 4; ++b) mx = max(mx, max(e[b] & 0x7FFFu, (e[b] >> 16) & 0x7FFFu));
        }
        const int up = min(13 - (int(mx >> 7) - 127), 126);  // the largest element into [2^13, 2^14)
        const float f = __uint_as_float(uint32_t(up + 127) << 23);
        s_c[slot][row] = __uint_as_float(uint32_t(127 - up) << 23) * (0.125f * 1.4426950408889634f);
        const uint32_t dst = smem_u32(sQ + 2 * slot * PTC_QTILE + row * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t e[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          uint32_t h[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            h[b] = pack_half2(__uint_as_float(e[b] << 16) * f, __uint_as_float(e[b] & 0xFFFF0000u) * f);
          st_shared_v4(dst + 16 * (c ^ (row & 7)), h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[slot]);
      for (; j < u.pages; j += 2) {
        if (!warp_wait_bar(&kv_empty[st], ph)) {
          ok = false;
          break;
        }
        cp_async_wait<PTC_RAW - 1>();
        uint8_t* src = raw + raw_c * PTC_RAW_BYTES;
        const int k = u.k0 + j, page = k < u.sinks ? k : u.first + k - u.sinks;
        const int whole = int(u.tile[0].whole(page)) | int(u.tile[1].whole(page)) << 1;
        if (ct == 0) {
          const float ks = s_rawscale[pair][raw_c][0], vs = s_rawscale[pair][raw_c][1];
          s_meta[st] = make_float4(ks, __log2f(vs), __int_as_float(page << 2 | whole), 0.f);
        }
        bool nan_any = false;
        if (whole != 3) {
#pragma unroll 1
          for (int p = 0; p < 4; ++p) {  // values
            uint4* at = reinterpret_cast<uint4*>(src + KV_TILE + 1024 * p);
            uint4 v = *at;
            uint32_t* e = reinterpret_cast<uint32_t*>(&v);
            uint32_t nan = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t m = e4m3_nan_bytes(e[b]);
              e[b] &= ~((m >> 7) * 0xFFu);
              nan |= (((m >> 7) * 0x10204080u >> 28) & 0xFu) << (4 * b);
            }
            s_nan[st][16 * p + rr][q] = uint16_t(nan);
            nan_any |= nan != 0;
            *at = v;
          }
          nan_any = __any_sync(0xffffffffu, nan_any);
        }
        const uint32_t dst = smem_u32(sKV + st * PTC_STAGE);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // keys, values
          uint4 v[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) v[p] = *reinterpret_cast<const uint4*>(src + half * KV_TILE + 1024 * p);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t to = dst + half * PTC_OPERAND + 2048 * p;
            st_shared_v4(to + swz0, e4m3x2_to_half2(v[p].x), e4m3x2_to_half2(v[p].x >> 16), e4m3x2_to_half2(v[p].y),
                         e4m3x2_to_half2(v[p].y >> 16));
            st_shared_v4(to + swz1, e4m3x2_to_half2(v[p].z), e4m3x2_to_half2(v[p].z >> 16), e4m3x2_to_half2(v[p].w),
                         e4m3x2_to_half2(v[p].w >> 16));
          }
        }
        if (lane == 0) reinterpret_cast<uint32_t*>(&s_hasnan[st])[cw & 1] = nan_any;
        fence_proxy_async_smem();
        mbar_arrive(&kv_full[st]);
        if (++raw_c == PTC_RAW) raw_c = 0;
        issue();
        st += 2;
        if (st >= PTC_STAGES) {
          st -= PTC_STAGES;
          ph ^= 1;
        }
      }
      j -= u.pages;
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[us]);
    }
    cp_async_wait<0>();
  } else if (warp >= PTC_ISSUE0) {
    // ----------------------------------------------------------- MMA issuers
    regs_fewer<PTC_REGS_ISSUE>();
    // The whole warp walks along (the values it derives are then uniform, and
    // the descriptors can stay in uniform registers), one lane issues.
    const auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int g = uniform(warp - PTC_ISSUE0);
    const uint32_t tS = uniform(tmem) + 128 * g, tO = tS + 64;
    const uint64_t desc_q = umma_desc_sw128(smem_u32(sQ), 1024), desc_kv = umma_desc_sw128(smem_u32(sKV), 1024);
    constexpr uint32_t idesc = umma_idesc_f16(128, 64);
    const bool leader = elect_one();
    int base = 0, base_ph = 0, n = 0;  // stage and phase of the unit's first page; pages of this group
    int opened = 0;                    // units of this group with a page
    for (int unit = 0; ok; ++unit) {
      const int us = unit % PTC_PARTS, slot = unit & 1;
      const PagedPart& u = s_part[us];
      if (!warp_wait_bar(&u_full[us], (unit / PTC_PARTS) & 1)) {
        ok = false;
        break;
      }
      if (uniform(u.last)) break;
      const bool two = uniform(u.two);
      const int tile = two ? g >> 1 : 0, pages = uniform(u.pages);
      const int sink_end = uniform(u.tile[tile].sink_end), lo = uniform(u.tile[tile].lo), hi = uniform(u.tile[tile].hi);
      const PagedTcShare share(two, g);
      __syncwarp();
      if (leader) mbar_arrive(&u_empty[us]);
      bool first = true;
      ok = warp_wait_bar(&q_full[slot], (unit >> 1) & 1);
      const uint64_t dq = desc_q + uint64_t((2 * slot + tile) * (PTC_QTILE >> 4));
      int st = base + share.turn, ph = base_ph;
      for (int j = share.turn; ok && j < pages; j += share.turns + 1) {
        if (st >= PTC_STAGES) {
          st -= PTC_STAGES;
          ph ^= 1;
        }
        // (the stage's page before this one is full already: it belongs to the
        // same pair and, in this unit, comes before the group's last page)
        if (!warp_wait_bar(&kv_full[st], ph)) {
          ok = false;
          break;
        }
        if (j < sink_end || (j >= lo && j < hi)) {
          tc_fence_after();
          const uint64_t dk = desc_kv + uint64_t(st * (PTC_STAGE >> 4)), dv = dk + (PTC_OPERAND >> 4);
          if (leader) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_bf16_ss(tS, dq + uint64_t(2 * i), dk + uint64_t(2 * i), idesc, i != 0);
            umma_commit(&s_full[g]);  // (the products before it are then done too)
            s_stage[g] = st;
            mbar_arrive(&s_full[g]);
          }
          if ((first && !warp_wait_bar(&o_empty[g], (opened & 1) ^ 1)) || !warp_wait_bar(&p_full[g], n & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_bf16_ts(tO, tS + 8 * i, dv + uint64_t(2 * i), idesc, i != 0 || !first);
            umma_commit(&kv_empty[st]);
          }
          first = false;
          ++n;
        } else if (leader) {
          mbar_arrive(&kv_empty[st]);
        }
        if (!two && leader) mbar_arrive(&kv_empty[st]);
        st += share.turns + 1;
      }
      if (!ok) break;
      base += pages % PTC_STAGES;
      base_ph ^= (pages / PTC_STAGES) & 1;
      if (base >= PTC_STAGES) {
        base -= PTC_STAGES;
        base_ph ^= 1;
      }
      if (leader) umma_commit(&q_empty[slot]);
      if (!first) {
        if (leader) umma_commit(&o_full[g]);
        ++opened;
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    regs_more<PTC_REGS>();
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lane_off = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + 128 * g + lane_off, tO = tS + 64;
    int singles = 0, n = 0, opened = 0, met = 0;
    // the group's 128 threads meet (a bounded wait, like every other)
    auto meet = [&]() {
      mbar_arrive(&group_bar[g]);
      ok = ok && warp_wait_bar(&group_bar[g], met & 1);
      ++met;
      return ok;
    };
    for (int unit = 0; ok; ++unit) {
      const int us = unit % PTC_PARTS, slot = unit & 1;
      if (!warp_wait_bar(&u_full[us], (unit / PTC_PARTS) & 1)) {
        ok = false;
        break;
      }
      const PagedPart& u = s_part[us];
      if (u.last) break;
      if (!warp_wait_bar(&q_full[slot], (unit >> 1) & 1)) {
        ok = false;
        break;
      }
      const bool two = u.two;
      const int tile = two ? g >> 1 : 0, rows = u.tile[tile].rows;
      const int pages = PagedTcShare(two, g).pages(u.tile[tile]);
      const int p0r = r < rows ? u.tile[tile].p0 + r : -1;  // this row's position (-1: sees nothing)
      const float c = s_c[slot][128 * tile + r];
      mbar_arrive(&q_empty[slot]);
      singles += !two;
      float m = -INFINITY, nm = PTC_NONE, l = 0.f;
      uint64_t nans = 0;  // dims of this row that saw a NaN value
#pragma unroll 1
      for (int i = 0; i < pages; ++i) {
        if (!warp_wait_bar(&s_full[g], n & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        ++n;
        const int st = s_stage[g];
        const float4 mt = s_meta[st];
        // the exponent's factor and offset; the factor not below the smallest
        // normal number: a masked -inf times 0 would be NaN
        const float ck = fmaxf(c * mt.x, 1.17549435e-38f);
        const int pw = __float_as_int(mt.z);
        const bool whole = (pw >> tile) & 1;
        uint64_t see = ~0ull;
        if (!whole) see = page_visible(p0r, (pw >> 2) * KV_PAGE, a.window, a.sinks);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t x[32];
          tmem_ld32(tS + 32 * h, x);
          tmem_ld_wait_regs(x);
          if (!whole) {
            const uint32_t bits = uint32_t(see >> (32 * h));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((bits >> e) & 1u)) x[e] = 0xFF800000u;  // -inf
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 1] = fmax3(mx[(e >> 1) & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        }
        const float score = fmaxf(mx[0], mx[1]) * ck, top = score + mt.y;
        if (i == 0) {
          m = top - PTC_TOP;
        } else if (__any_sync(0xffffffffu, top > m + (PTC_TOP + PTC_RAISE))) {
          // (the scores' arrival says that the products before are done)
          const float mn = fmaxf(m, top - PTC_TOP), d = mn == -INFINITY ? 0.f : m - mn;
          const float alpha = ex2_approx(d);
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * h, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(tO + 16 * h, o);
          }
          m = mn;
        }
        float off = mt.y - (m == -INFINITY ? 0.f : m);
        if (top < m - 64.f && top != -INFINITY)  // nothing in O: weights of 2^-26 and less, which are 0 in fp16
          off = mt.y - top - 26.f;
        const uint64_t ck2 = f2_pack(ck, ck), off2 = f2_pack(off, off);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t x[32];
          tmem_ld32(tS + 32 * h, x);
          tmem_ld_wait_regs(x);
          if (!whole) {
            const uint32_t bits = uint32_t(see >> (32 * h));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((bits >> e) & 1u)) x[e] = 0xFF800000u;  // -inf
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t y = f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), ck2, off2);
            float w0, w1;
            f2_unpack(y, w0, w1);
            w0 = ex2_approx(w0);
            w1 = ex2_approx(w1);
            sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2_pack(w0, w1));
            pk[e >> 1] = pack_half2(w0, w1);
          }
          tmem_st16(tS + 16 * h, pk);  // over scores that have been read
        }
        const uint2 has = s_hasnan[st];
        if (has.x | has.y) {
#pragma unroll 1
          for (int d = 0; d < 64; ++d)
            if (*reinterpret_cast<const uint64_t*>(&s_nan[st][d][0]) & see) nans |= 1ull << d;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[g]);
        // The normaliser, beside the page's product.  (The factor is at most 2^69
        // where the row sees a key of the page; the bound is for the others, whose
        // weights are 0.)
        if (score > nm + PTC_RAISE) {
          l *= ex2_approx(nm - score);
          nm = score;
        }
        float a0, a1, a2, a3;
        f2_unpack(sum[0], a0, a1);
        f2_unpack(sum[1], a2, a3);
        l = fmaf((a0 + a1) + (a2 + a3), ex2_approx(fminf(-off - nm, 80.f)), l);
      }
      if (!ok) break;

      // The unit's end (or this block's part of it): the groups that shared a
      // tile hand their sums to its first group.
      auto handed = [&](int d) { return d == 2 ? singles - 1 : unit; };  // earlier times that group d handed over
      if (pages > 0) {
        if (!warp_wait_bar(&o_full[g], opened & 1)) {
          ok = false;
          break;
        }
        ++opened;
        tc_fence_after();
      }
      if (two ? (g & 1) != 0 : g != 0) {
        mbar_arrive(&u_empty[us]);
        if (!warp_wait_bar(&x_empty[g], (handed(g) & 1) ^ 1)) {
          ok = false;
          break;
        }
        s_xm[g][r] = m;
        s_xn[g][r] = nm;
        s_xl[g][r] = pages > 0 ? l : -1.f;  // -1: no page, no O
        s_xnan[g][r] = nans;
        tc_fence_before();
        mbar_arrive(&x_full[two][g]);
        continue;
      }
      const int donors = two ? 1 : 3, row_base = u.row0 + 128 * tile, c0 = u.c0, c1 = u.c1;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + int64_t(row_base) * D + u.head * DH;
      mbar_arrive(&u_empty[us]);
      float M = fmaxf(m, PTC_NONE), N = nm;
#pragma unroll 1
      for (int d = 1; d <= donors; ++d) {
        if (!warp_wait_bar(&x_full[two][g + d], (two ? unit - singles : singles - 1) & 1)) {
          ok = false;
          break;
        }
        M = fmaxf(M, s_xm[g + d][r]);
        N = fmaxf(N, s_xn[g + d][r]);
      }
      if (!ok) break;
      tc_fence_after();
      // each group's weight takes the place of its maximum
      s_xm[g][r] = ex2_approx(m - M);
      s_xl[g][r] = pages > 0 ? l : -1.f;
      l *= ex2_approx(nm - N);
#pragma unroll 1
      for (int d = 1; d <= donors; ++d) {
        const float ld = s_xl[g + d][r];
        s_xm[g + d][r] = ex2_approx(s_xm[g + d][r] - M);
        if (ld != -1.f) l = fmaf(ld, ex2_approx(s_xn[g + d][r] - N), l);
        nans |= s_xnan[g + d][r];
      }
      if (c0 != c1) pdl_wait();  // the counters are zero, the parts' room is free
      auto part = [&](int i) { return a.partial + (int64_t(2 * i + (i == c0 ? 1 : 0)) * 2 + tile) * PTC_PART; };
      float* mp = part(blockIdx.x);
      // (two factors: 2^(M - N) is as small as 2^-115 where all values are, and
      // l may be large besides)
      const float inv = 1.0f / l, by = ex2_approx(M - N);
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {  // 16 dims at a time
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 1
        for (int d = 0; d <= donors; ++d) {
          if (s_xl[g + d][r] == -1.f) continue;  // (all rows or none)
          const float wd = s_xm[g + d][r];
          uint32_t x[16];
          tmem_ld16(tO + 128 * d + 16 * h, x);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(wd, __uint_as_float(x[e]), o[e]);
        }
        if (nans) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((nans >> (16 * h + e)) & 1) o[e] = __uint_as_float(0x7FC00000u);
        }
        if (r < rows) {
          if (c0 == c1) {
            uint4* dst = reinterpret_cast<uint4*>(out + int64_t(r) * D + 16 * h);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = o[e] * inv * by;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              dst[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                  pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              __stcg(reinterpret_cast<float4*>(mp + r * DH + 16 * h) + k,
                     make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
          }
        }
      }
      tc_fence_before();
      if (pages > 0) mbar_arrive(&o_empty[g]);
#pragma unroll 1
      for (int d = 1; d <= donors; ++d) {
        if (s_xl[g + d][r] != -1.f) mbar_arrive(&o_empty[g + d]);
        mbar_arrive(&x_empty[g + d]);
      }
      if (c0 == c1) continue;
      if (r < rows) __stcg(reinterpret_cast<float4*>(mp + 128 * DH) + r, make_float4(M, N, l, 0.f));
      __threadfence();
      if (!meet()) break;
      if (r == 0) s_done[g] = atomicAdd(a.counters + PAGED_MAX_CTAS * H + 2 * c0 + tile, 1);
      if (!meet()) break;
      if (s_done[g] != c1 - c0) continue;
      // The last part: add them up, in block order.  Thread r finds row r's
      // maximum and sum, then holds 4 dims of each 8th row.
      __threadfence();
      M = N = PTC_NONE;
      float L = 0.f;
      if (r < rows) {
#pragma unroll 4
        for (int i = c0; i <= c1; ++i) {
          const float4 p = __ldcg(reinterpret_cast<const float4*>(part(i) + 128 * DH) + r);
          const float nn = fmaxf(N, p.y);
          L = L * ex2_approx(N - nn) + p.z * ex2_approx(p.y - nn);
          N = nn;
          M = fmaxf(M, p.x);
        }
      }
      s_wm[g][r] = M;
      s_wl[g][r] = make_float2(1.0f / L, ex2_approx(M - N));
      if (!meet()) break;
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {  // 32 rows at a time
        const int first = 32 * h + (r >> 4);
        float4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int i = c0; i <= c1; ++i) {
          const float* pi = part(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = first + 8 * j;
            if (row >= rows) continue;
            const float we = ex2_approx(__ldcg(pi + 128 * DH + 4 * row) - s_wm[g][row]);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(pi + row * DH) + (r & 15));
            acc[j].x = fmaf(we, v.x, acc[j].x);
            acc[j].y = fmaf(we, v.y, acc[j].y);
            acc[j].z = fmaf(we, v.z, acc[j].z);
            acc[j].w = fmaf(we, v.w, acc[j].w);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = first + 8 * j;
          if (row >= rows) continue;
          const float2 f = s_wl[g][row];
          *reinterpret_cast<uint2*>(out + int64_t(row) * D + 4 * (r & 15)) =
              make_uint2(pack_bf16x2(acc[j].x * f.x * f.y, acc[j].y * f.x * f.y),
                         pack_bf16x2(acc[j].z * f.x * f.y, acc[j].w * f.x * f.y));
        }
      }
      if (!meet()) break;  // before another unit's rows take the places of these
    }
  }
  pdl_wait();
  if (!ok) set_error(a.err, PTL_ERR_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == PTC_ISSUE0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t paged_tc_partial_bytes() { return sizeof(float) * 2 * PAGED_TC_MAX_CTAS * 2 * PTC_PART; }

int launch_attn_paged_tc(const PagedArgs& a, cudaStream_t st) {
  static PerDevice configured;
  if (configured.get([] {
        return cudaFuncSetAttribute(attn_paged_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PTC_SMEM) ==
                       cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return -1;
  const int sms = num_sms();
  const int grid = sms < PAGED_TC_MAX_CTAS ? sms : PAGED_TC_MAX_CTAS;
  if (launch_k(attn_paged_tc_kernel, dim3(grid), dim3(PTC_THREADS), PTC_SMEM, st, a) != 0) return -1;
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace ptl
