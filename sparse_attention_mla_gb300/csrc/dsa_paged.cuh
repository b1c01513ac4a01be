// dsa_paged.cuh -- what the kernels over a paged cache share: cutting a line of
// tiles into equal ranges, one per CTA, from lengths that only the device knows.
#pragma once
#include "dsa_device.cuh"

namespace dsa {

// This CTA's tiles [w0, w1) of the line of W tiles, cut into C ranges.
struct TileRange {
  long long W, C, w0, w1;
};

// Whole CTA of NT threads.  Unit u (of U) has tiles_of(u) tiles; the units' tiles lie end to end.  visit(range, u,
// lo, n) is called by one thread for every unit [lo, lo + n) up to the range's end that has tiles.  `scratch`: NT / 32
// words of shared memory.  Two passes over the units (sum, then prefix sums): the lengths come from L2.
template <int NT, class F, class V>
__device__ __forceinline__ TileRange split_line(int U, const F& tiles_of, long long* scratch, const V& visit) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long sum = 0;
  for (int u = tid; u < U; u += NT) sum += tiles_of(u);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scratch[warp] = sum;
  __syncthreads();
  TileRange r;
  r.W = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) r.W += scratch[w];
  __syncthreads();
  r.C = min((long long)gridDim.x, r.W);
  const long long c = blockIdx.x;
  r.w0 = c < r.C ? r.W * c / r.C : 0;
  r.w1 = c < r.C ? r.W * (c + 1) / r.C : 0;
  if (r.w1 <= r.w0) return r;
  long long base = 0;
  for (int u0 = 0; u0 < U && base < r.w1; u0 += NT) {
    const int u = u0 + tid;
    const long long mine = u < U ? tiles_of(u) : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long before = base, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const long long v = scratch[w];
      if (w < warp) before += v;
      total += v;
    }
    if (mine > 0) visit(r, u, before + inc - mine, mine);
    base += total;
    __syncthreads();
  }
  return r;
}

}  // namespace dsa
