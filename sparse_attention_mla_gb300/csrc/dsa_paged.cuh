// dsa_paged.cuh -- what the kernels over a paged cache share: uniform values and short
// bounded waits for their roles' loops, and cutting a line of tiles into equal ranges,
// one per CTA, from lengths that only the device knows.
#pragma once
#include "dsa_device.cuh"

namespace dsa {

// A value that is the same in all lanes, in a register of the whole warp.  The loops that issue MMAs run on such
// counters: only then are the MMAs' descriptors kept in registers of the warp.  An MMA (M = 64, N = 64) alone on the SM
// is then issued every 33 cycles, which is what it takes, instead of every 60 to 80; next to the other roles of the
// attention over the paged cache every 45.
__device__ __forceinline__ int warp_value(int v) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)v); }

// Four MMAs on consecutive 16-element steps of K (the descriptors step by SA and SB), issued by one elected lane: the
// election and the predicate of the first one (add to D or overwrite it) once for all four.  The issuing warps' pace is
// the pace at which their instructions arrive next to the other roles' code.
template <int SA, int SB>
__device__ __forceinline__ void mma4_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add_first) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, %6;\n\tadd.s64 a3, %1, %7;\n\t"
      "add.s64 b1, %2, %8;\n\tadd.s64 b2, %2, %9;\n\tadd.s64 b3, %2, %10;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(add_first), "n"(SA), "n"(2 * SA), "n"(3 * SA), "n"(SB), "n"(2 * SB), "n"(3 * SB)
      : "memory");
}

// TMA by one elected lane of a warp whose operands are the warp's (see warp_value): issued lane by lane, with operands of
// their own, the same copies take several times as long.
__device__ __forceinline__ void tma_load_2d_w(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d_w(const CUtensorMap* map, int32_t c0, int32_t c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}" ::"l"(map), "r"(c0), "r"(c1)
      : "memory");
}

// The bounded wait of dsa_device.cuh, in fewer instructions: a wait that runs out only sets *abort, and the CTA records
// it when it leaves.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, long long limit) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!*abort) {
    if (clock64() - t0 >= limit) { *abort = DSA_ERR_TIMEOUT; break; }
    if (mbar_try_wait(bar, parity)) return true;
  }
  return false;
}

// This CTA's tiles [w0, w1) of the line of W tiles, cut into C ranges.
struct TileRange {
  long long W, C, w0, w1;
};

// Whole CTA of NT threads.  Unit u (of U) has tiles_of(u) tiles; the units' tiles lie end to end.  visit(range, u,
// lo, n) is called by one thread for every unit [lo, lo + n) up to the range's end that has tiles.  `scratch`: NT / 32
// words of shared memory.  A pass for the sum and one for the prefix sums; up to NT units are looked at only once.
// Loops and not unrolled code: this runs once, before anything else, and at the time it takes to fetch it.
template <int NT, class F, class V>
__device__ __forceinline__ TileRange split_line(int U, const F& tiles_of, long long* scratch, const V& visit) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  TileRange r{0, 0, 0, 0};
  long long mine = 0, before = 0, total = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
#pragma unroll 1
    for (int u0 = 0; u0 < U; u0 += NT) {
      const int u = u0 + tid;
      if (pass == 0 || U > NT) {
        mine = u < U ? tiles_of(u) : 0;
        // sums over the CTA: inside the warps, then over the warps' totals
        long long inc = mine, x = 0;
#pragma unroll 1
        for (int level = 0; level < 2; ++level) {
#pragma unroll 1
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, level ? x : inc, o);
            if (lane >= o) { if (level) x += y; else inc += y; }
          }
          if (level == 0) {
            if (lane == 31) scratch[warp] = inc;
            __syncthreads();
            x = lane < NW ? scratch[lane] : 0;
            __syncthreads();
          }
        }
        total = __shfl_sync(0xffffffffu, x, 31);
        before = __shfl_sync(0xffffffffu, x, (warp + 31) & 31);
        before = inc - mine + (warp ? before : 0);
      }
      if (pass == 1 && mine > 0 && base + before < r.w1) visit(r, u, base + before, mine);
      base += total;
    }
    if (pass == 0) {
      r.W = base;
      r.C = min((long long)gridDim.x, r.W);
      if ((long long)blockIdx.x >= r.C) return r;
      // floor(W c / C) and floor(W (c + 1) / C), with one wide division
      const unsigned c = blockIdx.x, C = (unsigned)r.C;
      const long long each = r.W / r.C;
      const unsigned rest = (unsigned)(r.W - each * r.C);
      r.w0 = each * c + rest * c / C;
      r.w1 = each * (c + 1) + rest * (c + 1) / C;
    }
  }
  return r;
}

// Last i in [0, n) with a[i] <= v (a non-decreasing, a[0] <= v), by a whole warp: 32 probes at a time.
__device__ __forceinline__ int warp_last_le(const int32_t* __restrict__ a, int n, int v) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(a + at) <= v);
    lo += (31 - __clz(le | 1u)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace dsa
