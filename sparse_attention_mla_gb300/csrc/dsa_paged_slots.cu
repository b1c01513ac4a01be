// dsa_paged_slots.cu -- pages and cache rows of a step's new tokens.
//
// Request b holds s_b tokens in ceil(s_b / P) pages and gets n_b more.  Its
// fresh pages (ceil((s_b + n_b) / P) - ceil(s_b / P) of them) come from the free
// list in request order; token j of the request sits at position s_b + j, in row
// table[b, pos / P] * P + pos % P of the cache.
//
// One launch.  Both exclusive sums over the requests (tokens and fresh pages)
// are needed by every token, and a batch has at most a few thousand requests, so
// each CTA forms both sums itself in shared memory (a few kilobytes from L2)
// instead of waiting for a kernel before it; then a token finds its request by a
// binary search there.  What bounds a decode step is one launch's latency; a
// step with prompts writes 8 bytes per token.  Measured: 256 requests of one token
// 3.8 us, 48 prompts of 110,000 tokens together 4.2 us.
#include "dsa_device.cuh"
#include "dsa_host.h"

namespace dsa {
namespace slots {

constexpr int kThreads = 256;
constexpr int kMaxRequests = 8192;  // two int32 sums per request in 64 KiB of shared memory
constexpr int kMaxBlocks = 304;     // two CTAs per SM

// Last i in [0, n) with a[i] <= v (a non-decreasing, a[0] <= v).
__device__ __forceinline__ int last_le(const int* a, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ long long ceil_div(long long a, int p) { return (a + p - 1) / p; }

__global__ void __launch_bounds__(kThreads)
    paged_slots_kernel(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ new_lens, int B, int N, int P,
                       int max_pages, const int32_t* __restrict__ free_pages, int F, int32_t* block_table,
                       int32_t* __restrict__ seq_lens_out, int32_t* __restrict__ cu_new, int32_t* __restrict__ slot_map,
                       int32_t* __restrict__ positions, int32_t* __restrict__ pages_taken, int* __restrict__ err) {
  extern __shared__ int sh[];
  int* cu = sh;             // [B + 1] new tokens of the requests before
  int* base = sh + B + 1;   // [B + 1] fresh pages of the requests before
  __shared__ long long wsum[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long tok = 0, pag = 0;  // running totals (64-bit: a bad length may not wrap into a good total)
  bool bad = false;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    long long n = 0, f = 0;
    if (b < B) {
      const long long s = __ldg(seq_lens + b);
      n = new_lens ? __ldg(new_lens + b) : 1;
      const bool fits = s >= 0 && n >= 0 && s + n <= 0x7fffffffll && ceil_div(s + n, P) <= max_pages;
      if (!fits) { bad = true; n = 0; }
      f = fits ? ceil_div(s + n, P) - ceil_div(s, P) : 0;
    }
    long long in = n, ifr = f;  // inclusive sums over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, in, o), c = __shfl_up_sync(0xffffffffu, ifr, o);
      if (lane >= o) { in += a; ifr += c; }
    }
    if (lane == 31) { wsum[0][warp] = in; wsum[1][warp] = ifr; }
    __syncthreads();
    long long before = tok, pbefore = pag;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long a = wsum[0][w], c = wsum[1][w];
      if (w < warp) { before += a; pbefore += c; }
      tok += a;
      pag += c;
    }
    if (tok > N || pag > F) bad = true;  // (the stored sums below are used only when nothing is bad)
    if (b < B) {
      cu[b] = (int)(before + in - n);
      base[b] = (int)(pbefore + ifr - f);
    }
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) { cu[B] = (int)tok; base[B] = (int)pag; }
  __syncthreads();
  const unsigned g0 = blockIdx.x * kThreads + tid, gstep = gridDim.x * kThreads;  // (unsigned: N may be 2^31 - 1)
  if (bad) {  // all or nothing: no request gets a token
    for (unsigned t = g0; t < (unsigned)N; t += gstep) { slot_map[t] = -1; positions[t] = -1; }
    for (unsigned b = g0; b <= (unsigned)B; b += gstep) {
      cu_new[b] = 0;
      if (b < (unsigned)B) seq_lens_out[b] = __ldg(seq_lens + b);
    }
    if (g0 == 0) { *pages_taken = 0; record_error(err, DSA_ERR_CAPACITY); }
    return;
  }
  const int total = cu[B], fresh = base[B];
  for (unsigned t = g0; t < (unsigned)N; t += gstep) {
    int slot = -1, pos = -1;
    if (t < (unsigned)total) {
      const int b = last_le(cu, B, (int)t);  // (skips requests without new tokens)
      const int s = __ldg(seq_lens + b);
      pos = s + ((int)t - cu[b]);
      const int pi = pos / P, first = (int)ceil_div(s, P);
      // a fresh page is read from the free list: its table entry may still be being written by another CTA
      const int page = pi >= first ? __ldg(free_pages + base[b] + (pi - first))
                                   : block_table[(size_t)b * max_pages + pi];
      const long long row = (long long)page * P + (pos - pi * P);
      if (page >= 0 && row <= 0x7fffffffll) slot = (int)row;
      else record_error(err, DSA_ERR_DEVICE_INDEX);
    }
    slot_map[t] = slot;
    positions[t] = pos;
  }
  for (unsigned i = g0; i < (unsigned)fresh; i += gstep) {
    const int b = last_le(base, B, (int)i);
    const int col = (int)ceil_div(__ldg(seq_lens + b), P) + ((int)i - base[b]);
    block_table[(size_t)b * max_pages + col] = __ldg(free_pages + i);
  }
  for (unsigned b = g0; b <= (unsigned)B; b += gstep) {
    cu_new[b] = cu[b];
    if (b < (unsigned)B) seq_lens_out[b] = __ldg(seq_lens + b) + (cu[b + 1] - cu[b]);
  }
  if (g0 == 0) *pages_taken = fresh;
}

// Whether two arrays of int32 share memory.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + 4 * nb && y < x + 4 * na;
}

}  // namespace slots
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_paged_slots(const int32_t* seq_lens, const int32_t* new_lens, int32_t B, int32_t N,
                                        int32_t page_size, int32_t max_pages, const int32_t* free_pages, int32_t F,
                                        int32_t* block_table, int32_t* seq_lens_out, int32_t* cu_new,
                                        int32_t* slot_map, int32_t* positions, int32_t* pages_taken, void* workspace,
                                        size_t workspace_bytes, dsa_stream_t stream) {
  const char* who = "dsa_paged_slots";
  if (B < 0 || B > slots::kMaxRequests || N < 0 || page_size < 1 || max_pages < 0 || F < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT,
                "%s: need 0 <= B <= %d, N >= 0, page_size >= 1, max_pages >= 0, F >= 0 (got %d, %d, %d, %d, %d)", who,
                slots::kMaxRequests, B, N, page_size, max_pages, F);
  if (!cu_new || !pages_taken || (B > 0 && (!seq_lens || !seq_lens_out)) || (N > 0 && (!slot_map || !positions)) ||
      (B > 0 && max_pages > 0 && !block_table) || (F > 0 && !free_pages))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  const void* ins[3] = {seq_lens, new_lens, free_pages};
  const size_t nin[3] = {(size_t)B, new_lens ? (size_t)B : 0, (size_t)F};
  const void* outs[6] = {block_table, seq_lens_out, cu_new, slot_map, positions, pages_taken};
  const size_t nout[6] = {(size_t)B * max_pages, (size_t)B, (size_t)B + 1, (size_t)N, (size_t)N, 1};
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 3; ++i)
      if (slots::overlap(outs[o], nout[o], ins[i], nin[i]))
        return fail(DSA_ERR_INVALID_ARGUMENT, "%s: an output shares memory with an input", who);
    for (int p = 0; p < o; ++p)
      if (slots::overlap(outs[o], nout[o], outs[p], nout[p]))
        return fail(DSA_ERR_INVALID_ARGUMENT, "%s: two outputs share memory", who);
  }
  dsa_status_t st = check_workspace(workspace, workspace_bytes, kErrorWordBytes, who);
  if (st != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  const int smem = 2 * (B + 1) * (int)sizeof(int);
  if ((st = configure_kernel_smem(reinterpret_cast<const void*>(slots::paged_slots_kernel),
                                  2 * (slots::kMaxRequests + 1) * (int)sizeof(int),
                                  "configuring paged_slots_kernel")) != DSA_OK)
    return st;
  const int64_t items = N > B + 1 ? N : B + 1;
  const int64_t want = (items + slots::kThreads - 1) / slots::kThreads;
  const int blocks = (int)(want < slots::kMaxBlocks ? want : slots::kMaxBlocks);
  slots::paged_slots_kernel<<<blocks, slots::kThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(
      seq_lens, new_lens, B, N, page_size, max_pages, free_pages, F, block_table, seq_lens_out, cu_new, slot_map,
      positions, pages_taken, reinterpret_cast<int*>(workspace));
  st = cuda_check(cudaGetLastError(), "launching paged_slots_kernel");
  return st == DSA_OK ? ok() : st;
}
