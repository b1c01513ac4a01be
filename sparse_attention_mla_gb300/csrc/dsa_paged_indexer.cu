// dsa_paged_indexer.cu -- top-k selection of new tokens over paged index keys (sm_103a).
//
// score(t, p) = sum_h w[t,h] max(0, <q_idx[t,h,:], k_p>) over the positions p that
// token t sees; the K best (ties to the lower position), ascending.  The floor is
// one read of every visible key (256 bytes); 64 heads of one token are 64 flops a
// byte, a quarter of what the tensor core could do meanwhile.
//
// Two kernels.  The first writes the scores (fp32, 4 bytes for 256 read): as in
// the attention over the paged cache, all requests' tiles of 128 keys are laid end
// to end and cut into equal ranges, one CTA per SM, so one long request fills the
// card; keys are on the MMA's M axis, the (token, head) pairs of up to 256 / heads
// tokens of a request on N, and a TMEM lane is a key, whose thread sums its heads.
// The second finds each token's K best with a cluster of 1 to 8 CTAs per token (by
// the longest length there can be): the scores, as integers of the same order, stay
// in registers; histograms of 11 bits, starting below the bits that all scores
// share, narrow the K-th down, summed over the cluster through distributed shared
// memory; then one ordered compaction.  Every step is exact and without order
// effects, so equal calls give equal lists.
#include <cooperative_groups.h>

#include <cmath>

#include "dsa_host.h"
#include "dsa_paged.cuh"

namespace dsa {
namespace pidx {

namespace cg = cooperative_groups;

constexpr int kD = 128;          // index width
constexpr int kTile = 128;       // keys per tile (MMA M)
constexpr int kCols = 256;       // (token, head) columns of a group (MMA N)
constexpr int kRing = 4;
constexpr int kThreads = 32 * 14;  // MMA, 8 epilogue, 4 gather, 1 query warp
constexpr int kMaxCtas = 160;

constexpr int Q_CHUNK = kCols * 128, K_CHUNK = kTile * 128;
constexpr int OFF_Q = 0, OFF_K = 2 * Q_CHUNK, OFF_W = OFF_K + kRing * 2 * K_CHUNK, OFF_MISC = OFF_W + 2 * kCols * 4;
constexpr int SMEM = OFF_MISC + 512 + 1024;
constexpr int M_K = 0, M_KF = 32, M_S = 64, M_SF = 80, M_Q = 96, M_SEG = 104, M_FIN = 112, M_TMEM = 120, M_ABORT = 124,
              M_PLAN = 128, M_SCRATCH = 192;

struct Params {
  const __nv_bfloat16* q;
  const __nv_bfloat16* cache;
  const float* w;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int N, B, Hi, num_pages, P, max_pages, max_len;
  float* scores;      // [N][stride]
  long long stride;
  int* err;
  long long wait_limit;
};

// max(x, 0) that keeps a NaN
__device__ __forceinline__ float relu(uint32_t x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(__uint_as_float(x)));
  return r;
}

struct Request {
  int n0, n, len, keys;  // first token, tokens, length, positions looked at
};
__device__ __forceinline__ Request request_of(const Params& p, int b) {
  Request r;
  const int lo = p.cu_q ? min(max(__ldg(p.cu_q + b), 0), p.N) : b;
  const int hi = p.cu_q ? min(max(__ldg(p.cu_q + b + 1), lo), p.N) : b + 1;
  r.n0 = lo;
  r.n = hi - lo;
  r.len = max(__ldg(p.seq_lens + b), 0);
  r.keys = (int)min((long long)min(r.len, p.max_len), (long long)p.max_pages * p.P);
  return r;
}

struct Plan {
  long long w0, w1, first;
  int u0, pad;
};

struct Seg {
  int t0, t1, tok, nt, b, keys;
};

template <int G>
struct Walk {
  const Params& p;
  int u, g, t, groups, tiles;
  long long left;
  Request rq;
  __device__ __forceinline__ void load() {
    rq = request_of(p, u);
    groups = (rq.n + G - 1) / G;
    tiles = (rq.keys + kTile - 1) / kTile;
    if (tiles == 0) groups = 0;
  }
  __device__ __forceinline__ Walk(const Params& p_, const Plan& pl) : p(p_) {
    left = pl.w1 - pl.w0;
    u = pl.u0;
    load();
    g = tiles > 0 ? (int)(pl.first / tiles) : 0;
    t = tiles > 0 ? (int)(pl.first - (long long)g * tiles) : 0;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (left <= 0) return false;
    while (g >= groups) {
      ++u;
      load();
      g = t = 0;
    }
    s.tok = rq.n0 + g * G;
    s.nt = min(G, rq.n - g * G);
    s.b = u;
    s.keys = rq.keys;
    s.t0 = t;
    s.t1 = (int)min((long long)tiles, t + left);
    left -= s.t1 - s.t0;
    t = s.t1;
    if (t >= tiles) { ++g; t = 0; }
    return true;
  }
};

// HP: heads per token, rounded up to 8, 16, 32 or 64 (the rest are zero rows)
template <int HP>
__global__ void __launch_bounds__(kThreads, 1) paged_score_kernel(const Params p) {
  constexpr int G = kCols / HP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem + OFF_Q), sK = smem_u32(smem + OFF_K);
  uint8_t* misc = smem + OFF_MISC;
  const uint32_t mb = smem_u32(misc);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + M_ABORT);
  Plan* s_plan = reinterpret_cast<Plan*>(misc + M_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(mb + M_K + 8 * s, 128);
      mbar_init(mb + M_KF + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(mb + M_S + 8 * b, 1);
      mbar_init(mb + M_SF + 8 * b, 4);
    }
    mbar_init(mb + M_Q, 32);
    mbar_init(mb + M_SEG, 1);
    mbar_init(mb + M_FIN, 1);
    *s_abort = 0;
    s_plan->u0 = 0;
    s_plan->first = 0;
    fence_mbar_init();
  }
  auto tiles_of = [&](int u) -> long long {
    const Request r = request_of(p, u);
    return (long long)((r.n + G - 1) / G) * ((r.keys + kTile - 1) / kTile);
  };
  auto visit = [&](const TileRange& r, int u, long long lo, long long n) {
    if (lo <= r.w0 && r.w0 < lo + n) {
      s_plan->u0 = u;
      s_plan->first = r.w0 - lo;
    }
  };
  __syncthreads();
  const TileRange rg = split_line<kThreads>(p.B, tiles_of, reinterpret_cast<long long*>(misc + M_SCRATCH), visit);
  if (threadIdx.x == 0) {
    s_plan->w0 = rg.w0;
    s_plan->w1 = rg.w1;
  }
  __syncthreads();
  const Plan plan = *s_plan;
  if (plan.w1 <= plan.w0) return;
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  __syncthreads();
  const uint32_t tmem = *s_tmem;
  Walk<G> walk(p, plan);
  Seg sg;
  int i = 0, seg = 0;

  if (warp == 0) {
    // ======================= MMA issuer =======================
    bool stop = false;
    while (!stop && walk.next(sg)) {
      const uint32_t id = idesc_bf16(kTile, (sg.nt * HP + 15) & ~15, false, false);
      if (!warp_all(mbar_wait(mb + M_Q, seg & 1, s_abort, p.err, p.wait_limit))) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % kRing, sb = i & 1;
        if (i >= 2 && !warp_all(mbar_wait(mb + M_SF + 8 * sb, ((i >> 1) - 1) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        if (!warp_all(mbar_wait(mb + M_K + 8 * sl, (i / kRing) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint64_t a = sdesc_sw128(sK + (sl * 2 + c) * K_CHUNK, 16, 1024), b = sdesc_sw128(sQ + c * Q_CHUNK, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_w(tmem + sb * kCols, a + (uint64_t)(k * 2), b + (uint64_t)(k * 2), id, (c | k) ? 1u : 0u);
        }
        mma_commit_w(mb + M_KF + 8 * sl);
        mma_commit_w(mb + M_S + 8 * sb);
      }
      mma_commit_w(mb + M_SEG);
      ++seg;
    }
    mma_commit_w(mb + M_FIN);
    volatile int dummy = 0;
    mbar_wait(mb + M_FIN, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 13) {
    // ======================= queries of a segment, once the products of the one before are done =======================
    while (walk.next(sg)) {
      if (seg > 0 && !mbar_wait(mb + M_SEG, (seg - 1) & 1, s_abort, p.err, p.wait_limit)) break;
      const int rows = ((sg.nt * HP + 15) & ~15);
      for (int x = lane; x < rows * 16; x += 32) {
        const int n = x >> 4, u = x & 15, tok = n / HP, h = n - tok * HP;
        const bool ok = tok < sg.nt && h < p.Hi;
        cp_async16(sQ + (u >> 3) * Q_CHUNK + sw128_off(n, u & 7),
                   p.q + (ok ? ((size_t)(sg.tok + tok) * p.Hi + h) * kD + u * 8 : 0), ok ? 16u : 0u);
      }
      cp_async_arrive(mb + M_Q);
      ++seg;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 9) {
    // ======================= gather: warp g copies rows 32 g .. of a tile, two rows at a time =======================
    const int gw = warp - 9;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      const int32_t* tab = p.table + (size_t)sg.b * p.max_pages;
      if (gw == 0 && lane == 0 && sg.keys < __ldg(p.seq_lens + sg.b)) record_error(p.err, DSA_ERR_DEVICE_INDEX);
      auto page_at = [&](int t) -> int {  // page of this lane's row of tile t; -1 past the end
        const int pos = t * kTile + gw * 32 + lane;
        return (t < sg.t1 && pos < sg.keys) ? __ldg(tab + (unsigned)pos / (unsigned)p.P) : -1;
      };
      int page = page_at(sg.t0);
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % kRing;
        const int pos = t * kTile + gw * 32 + lane;
        long long row = -1;
        if (pos < sg.keys) {
          if (page >= 0 && page < p.num_pages) row = (long long)page * p.P + (unsigned)pos % (unsigned)p.P;
          else record_error(p.err, DSA_ERR_DEVICE_INDEX);
        }
        page = page_at(t + 1);
        if (i >= kRing && !warp_all(mbar_wait(mb + M_KF + 8 * sl, ((i / kRing) - 1) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        const int u = lane & 15;
        const uint32_t dst = sK + (sl * 2 + (u >> 3)) * K_CHUNK;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int rr = 2 * e + (lane >> 4);
          const long long src = __shfl_sync(0xffffffffu, row, rr);
          cp_async16(dst + sw128_off(gw * 32 + rr, u & 7), p.cache + (src >= 0 ? (size_t)src * kD + u * 8 : 0),
                     src >= 0 ? 16u : 0u);
        }
        cp_async_arrive(mb + M_K + 8 * sl);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ======================= scores: two groups of four warps take alternate tiles; a thread is a key =======================
    const int grp = (warp - 1) >> 2, qd = warp & 3;
    float* s_w = reinterpret_cast<float*>(smem + OFF_W) + grp * kCols;
    bool stop = false;
    while (walk.next(sg)) {
      const int cols = sg.nt * HP;
      // the weights of the segment before have been read; all four warps leave together after a failed wait
      if (named_bar_or(1 + grp, 128, stop)) break;
      for (int x = ((warp - 1) & 3) * 32 + lane; x < cols; x += 128) {
        const int tok = x / HP, h = x - tok * HP;
        s_w[x] = h < p.Hi ? __ldg(p.w + (size_t)(sg.tok + tok) * p.Hi + h) : 0.f;
      }
      named_bar(1 + grp, 128);
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        if ((i & 1) != grp) continue;
        if (!warp_all(mbar_wait(mb + M_S + 8 * grp, (i >> 1) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        tc_fence_after();
        const int pos = t * kTile + qd * 32 + lane;
        float* out = p.scores + (size_t)sg.tok * p.stride + pos;
        const bool in = pos < sg.keys;
        float acc = 0.f;
        for (int c0 = 0; c0 < cols; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(tmem_addr(tmem + grp * kCols + c0, qd * 32, 0), v);
          tmem_ld_wait();
          const float4* w4 = reinterpret_cast<const float4*>(s_w + c0);
          if constexpr (HP >= 32) {
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 w = w4[j];
              a0 = fmaf(w.x, relu(v[4 * j]), a0);
              a1 = fmaf(w.y, relu(v[4 * j + 1]), a1);
              a2 = fmaf(w.z, relu(v[4 * j + 2]), a2);
              a3 = fmaf(w.w, relu(v[4 * j + 3]), a3);
            }
            acc += (a0 + a1) + (a2 + a3);
            if ((c0 + 32) % HP == 0) {
              if (in) out[(size_t)(c0 / HP) * p.stride] = acc;
              acc = 0.f;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32 / HP; ++k) {
              float a = 0.f;
#pragma unroll
              for (int j = 0; j < HP / 4; ++j) {
                const float4 w = w4[k * (HP / 4) + j];
                const int o = k * HP + 4 * j;
                a = fmaf(w.x, relu(v[o]), a);
                a = fmaf(w.y, relu(v[o + 1]), a);
                a = fmaf(w.z, relu(v[o + 2]), a);
                a = fmaf(w.w, relu(v[o + 3]), a);
              }
              if (in && c0 / HP + k < sg.nt) out[(size_t)(c0 / HP + k) * p.stride] = a;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + M_SF + 8 * grp);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------------------------------------------
constexpr int kSel = 1024;   // threads per CTA
constexpr int kPer = 16;     // scores per thread and round
constexpr int kRound = kSel * kPer;
constexpr int kBins = 2048;

// Integers in the order of the scores; 0 is no score.  -0 and +0 are one value, NaN is above all.
__device__ __forceinline__ uint32_t order_of(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum of v over the CTA's threads, and the total.  `sh`: 33 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sh, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();  // sh may still be in use
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint32_t mine = sh[lane];
    uint32_t s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    sh[lane] = s - mine;
    if (lane == 31) sh[32] = s;
  }
  __syncthreads();
  total = sh[32];
  return sh[warp] + inc - v;
}

template <int CS>
__global__ void __launch_bounds__(kSel, 1)
    paged_select_kernel(const float* __restrict__ scores, long long stride, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ cu_q, int N, int B, int K, int max_keys, int32_t* __restrict__ topk_idx,
                        int32_t* __restrict__ topk_len) {
  __shared__ uint32_t hist[kBins], tot[kBins];
  __shared__ uint32_t sh[33];
  __shared__ uint32_t box[2 * CS];       // min / max, later above / tied counts, of every CTA of the cluster
  __shared__ uint32_t pick[4];
  const int n = blockIdx.x / CS, rank = blockIdx.x % CS, tid = threadIdx.x;
  // the token's request and what it sees (the same in the whole cluster)
  int b = n, lo_tok = n, hi_tok = n + 1;
  if (cu_q) {
    if (n < __ldg(cu_q) || n >= __ldg(cu_q + B)) return;
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(cu_q + mid) <= n) lo = mid; else hi = mid;
    }
    b = lo;
    lo_tok = __ldg(cu_q + b);
    hi_tok = __ldg(cu_q + b + 1);
  }
  const int len = max(__ldg(seq_lens + b), 0);
  const int v = max(0, min(len - (hi_tok - lo_tok) + (n - lo_tok) + 1, max_keys));
  int32_t* out = topk_idx + (size_t)n * K;
  const int kept = min(v, K);
  if (topk_len != nullptr && rank == 0 && tid == 0) topk_len[n] = kept;
  for (int j = rank * kSel + tid; j < K; j += CS * kSel)
    if (j >= kept || v <= K) out[j] = j < kept ? j : -1;
  if (v <= K) return;

  cg::cluster_group cl = cg::this_cluster();
  if constexpr (CS > 1) cl.sync();  // every CTA of the cluster runs before its shared memory is written from outside
  // this CTA's piece of the row, a multiple of 4 so that the 16-byte loads stay aligned
  const int piece = ((v + CS - 1) / CS + 3) & ~3;
  const int begin = min(v, rank * piece), end = min(v, begin + piece);
  const int rounds = (end - begin + kRound - 1) / kRound;
  const float* row = scores + (size_t)n * stride;
  uint32_t key[kPer];
  auto load = [&](int r) {
    const int p0 = begin + r * kRound + tid * kPer;
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const int q = p0 + j;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < end) f = *reinterpret_cast<const float4*>(row + q);  // (the row's stride is a multiple of 4)
      key[j] = q < end ? order_of(f.x) : 0u;
      key[j + 1] = q + 1 < end ? order_of(f.y) : 0u;
      key[j + 2] = q + 2 < end ? order_of(f.z) : 0u;
      key[j + 3] = q + 3 < end ? order_of(f.w) : 0u;
    }
  };
#pragma unroll
  for (int j = 0; j < kPer; ++j) key[j] = 0u;
  if (rounds == 1) load(0);

  // smallest and largest: the bits above the highest one where they differ are shared by all
  uint32_t mn = 0xffffffffu, mx = 0u;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (key[j]) mn = min(mn, key[j]);
      mx = max(mx, key[j]);
    }
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (tid == 0) { pick[0] = 0xffffffffu; pick[1] = 0u; }
  __syncthreads();
  if ((tid & 31) == 0) { atomicMin(&pick[0], mn); atomicMax(&pick[1], mx); }
  __syncthreads();
  if (tid < CS) {
    uint32_t* to = cl.map_shared_rank(box, tid);
    to[2 * rank] = pick[0];
    to[2 * rank + 1] = pick[1];
  }
  cl.sync();
#pragma unroll
  for (int c = 0; c < CS; ++c) { mn = min(mn, box[2 * c]); mx = max(mx, box[2 * c + 1]); }

  // narrow the K-th largest down: `prefix` holds its bits from `bit` upwards, `need` how many of the scores that
  // share them are still to be taken
  int bit = mn == mx ? 0 : 32 - __clz(mn ^ mx);
  uint32_t prefix = bit == 32 ? 0u : (mx >> bit) << bit;
  int need = K;
  bool all = false;  // every score that shares the prefix is taken
  while (bit > 0 && !all) {
    const int shift = max(0, bit - 11);
    const uint32_t mask = (1u << (bit - shift)) - 1u;
    for (int x = tid; x < kBins; x += kSel) hist[x] = 0u;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t d = key[j] ^ prefix;
        if (key[j] && (bit == 32 || (d >> bit) == 0u)) atomicAdd(&hist[(key[j] >> shift) & mask], 1u);
      }
    }
    if constexpr (CS > 1) {
      cl.sync();
      // this CTA adds a slice of the bins over the cluster and gives the sums to all
      constexpr int kSlice = kBins / CS;
      for (int x = tid; x < kSlice; x += kSel) {
        const int at = rank * kSlice + x;
        uint32_t s = 0u;
#pragma unroll
        for (int c = 0; c < CS; ++c) s += cl.map_shared_rank(hist, c)[at];
#pragma unroll
        for (int c = 0; c < CS; ++c) cl.map_shared_rank(tot, c)[at] = s;
      }
      cl.sync();
    } else {
      __syncthreads();
    }
    const uint32_t* h = CS > 1 ? tot : hist;
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
    const uint32_t h1 = h[kBins - 1 - 2 * tid], h0 = h[kBins - 2 - 2 * tid];
    uint32_t total;
    const uint32_t above = block_scan(h1 + h0, sh, total);
    if (above < (uint32_t)need && above + h1 >= (uint32_t)need) {
      pick[0] = kBins - 1 - 2 * tid;
      pick[1] = above;
      pick[2] = h1;
    } else if (above + h1 < (uint32_t)need && above + h1 + h0 >= (uint32_t)need) {
      pick[0] = kBins - 2 - 2 * tid;
      pick[1] = above + h1;
      pick[2] = h0;
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    need -= (int)pick[1];
    all = (int)pick[2] == need;
    bit = shift;
    __syncthreads();
  }
  // taken: above the prefix's class, and the first `need` of the class in order of position
  auto is_above = [&](uint32_t k) { return bit == 32 ? false : (k >> bit) > (prefix >> bit); };
  auto is_tied = [&](uint32_t k) { return k != 0u && (bit == 32 || (k >> bit) == (prefix >> bit)); };
  uint32_t ca = 0, ct = 0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      ca += is_above(key[j]) ? 1u : 0u;
      ct += is_tied(key[j]) ? 1u : 0u;
    }
  }
  if (tid == 0) { pick[0] = 0u; pick[1] = 0u; }
  __syncthreads();
  ca = __reduce_add_sync(0xffffffffu, ca);
  ct = __reduce_add_sync(0xffffffffu, ct);
  if ((tid & 31) == 0) { atomicAdd(&pick[0], ca); atomicAdd(&pick[1], ct); }
  __syncthreads();
  uint32_t at = 0, tied = 0;  // entries of this row, and of its tied ones, before this CTA's piece
  if constexpr (CS > 1) {
    cl.sync();  // (box has been read by all)
    if (tid < CS) {
      uint32_t* to = cl.map_shared_rank(box, tid);
      to[2 * rank] = pick[0];
      to[2 * rank + 1] = pick[1];
    }
    cl.sync();  // (also: no CTA leaves while another still reads or writes its shared memory)
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      if (c < rank) {
        const uint32_t a = box[2 * c], e = box[2 * c + 1];
        at += a + (tied >= (uint32_t)need ? 0u : min(e, (uint32_t)need - tied));
        tied += e;
      }
    }
  }
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    uint32_t a = 0, e = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      a += is_above(key[j]) ? 1u : 0u;
      e += is_tied(key[j]) ? 1u : 0u;
    }
    uint32_t ta, te;
    const uint32_t sa = block_scan(a, sh, ta), se = block_scan(e, sh, te);
    uint32_t my_tied = tied + se;
    uint32_t o = at + sa + (min(my_tied, (uint32_t)need) - min(tied, (uint32_t)need));
    const int p0 = begin + r * kRound + tid * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      bool take = is_above(key[j]);
      if (is_tied(key[j])) {
        take = my_tied < (uint32_t)need;
        ++my_tied;
      }
      if (take) out[o++] = p0 + j;
    }
    at += ta + (min(tied + te, (uint32_t)need) - min(tied, (uint32_t)need));
    tied += te;
  }
}

inline long long stride_of(long long max_len) { return (max_len + 3) / 4 * 4; }

// CTAs per token: a round of 16 scores a thread covers a piece while the row is up to 131072 long; twice that
// many CTAs while they all fit the card at once.
inline int cluster_of(int N, long long max_len) {
  int cs = 1;
  while (cs < 8 && (long long)cs * kRound < max_len) cs *= 2;
  while (cs < 8 && (long long)cs * 4096 < max_len && (long long)N * cs * 2 <= 152) cs *= 2;
  return cs;
}

template <int HP>
dsa_status_t launch_scores(const Params& p, int ctas, cudaStream_t s) {
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_score_kernel<HP>), SMEM,
                                          "configuring paged_score_kernel");
  if (st != DSA_OK) return st;
  paged_score_kernel<HP><<<ctas, kThreads, SMEM, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching paged_score_kernel");
}

template <int CS>
dsa_status_t launch_select(const Params& p, int K, int max_keys, int32_t* idx, int32_t* len, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.N * CS);
  cfg.blockDim = dim3(kSel);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, paged_select_kernel<CS>, (const float*)p.scores, p.stride, p.seq_lens, p.cu_q,
                                       p.N, p.B, K, max_keys, idx, len),
                    "launching paged_select_kernel");
}

}  // namespace pidx
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_paged_indexer_topk_workspace_size(int32_t N, int32_t max_len) {
  if (N < 0 || max_len < 0) return kErrorWordBytes;
  return kErrorWordBytes + (size_t)N * pidx::stride_of(max_len) * sizeof(float);
}

extern "C" dsa_status_t dsa_paged_indexer_topk(const dsa_bf16_t* q_idx, const dsa_bf16_t* k_cache, const float* head_weights,
                                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                                               int32_t N, int32_t B, int32_t Hi, int32_t Di, int32_t K, int32_t num_pages,
                                               int32_t page_size, int32_t max_pages, int32_t max_len, int32_t* topk_idx,
                                               int32_t* topk_len, void* workspace, size_t workspace_bytes,
                                               dsa_stream_t stream) {
  const char* who = "dsa_paged_indexer_topk";
  if (N < 0 || B < 0 || num_pages < 0 || page_size < 1 || max_pages < 0 || max_len < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT,
                "%s: need N, B, num_pages, max_pages, max_len >= 0, page_size >= 1 (got %d, %d, %d, %d, %d, %d)", who, N, B,
                num_pages, max_pages, max_len, page_size);
  if (Hi < 1 || Hi > 64 || Di != pidx::kD)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: need Hi in [1, 64] and Di = 128 (got %d, %d)", who, Hi, Di);
  if (K < 1 || K > 2048) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: K must be in [1, 2048] (got %d)", who, K);
  if ((int64_t)N * 8 > 0x7fffffffll) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: N is too large (%d)", who, N);
  if (!cu_q && N != B)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: without cu_q every request has one token (N = %d, B = %d)", who, N, B);
  if (N > 0 && (!q_idx || !head_weights || !topk_idx)) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if (B > 0 && (!seq_lens || (max_pages > 0 && !block_table) || (num_pages > 0 && !k_cache)))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if (!aligned16(q_idx) || !aligned16(k_cache))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: q_idx and k_cache must be 16-byte aligned", who);
  dsa_status_t st = check_workspace(workspace, workspace_bytes, dsa_paged_indexer_topk_workspace_size(N, max_len), who);
  if (st != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (N == 0 || B == 0) return ok();
  int dev = 0, sms = 0;
  if ((st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) != DSA_OK) return st;
  if ((st = cuda_check(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "the SM count")) != DSA_OK) return st;
  const int ctas = sms < pidx::kMaxCtas ? sms : pidx::kMaxCtas;
  pidx::Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q_idx);
  p.cache = reinterpret_cast<const __nv_bfloat16*>(k_cache);
  p.w = head_weights;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.N = N;
  p.B = B;
  p.Hi = Hi;
  p.num_pages = num_pages;
  p.P = page_size;
  p.max_pages = max_pages;
  p.max_len = max_len;
  p.stride = pidx::stride_of(max_len);
  p.err = reinterpret_cast<int*>(workspace);
  p.scores = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kErrorWordBytes);
  p.wait_limit = wait_limit_cycles();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (Hi <= 8) st = pidx::launch_scores<8>(p, ctas, s);
  else if (Hi <= 16) st = pidx::launch_scores<16>(p, ctas, s);
  else if (Hi <= 32) st = pidx::launch_scores<32>(p, ctas, s);
  else st = pidx::launch_scores<64>(p, ctas, s);
  if (st != DSA_OK) return st;
  const int64_t table_len = (int64_t)max_pages * page_size;
  const int max_keys = (int)(table_len < max_len ? table_len : max_len);
  switch (pidx::cluster_of(N, max_keys)) {
    case 1: st = pidx::launch_select<1>(p, K, max_keys, topk_idx, topk_len, s); break;
    case 2: st = pidx::launch_select<2>(p, K, max_keys, topk_idx, topk_len, s); break;
    case 4: st = pidx::launch_select<4>(p, K, max_keys, topk_idx, topk_len, s); break;
    default: st = pidx::launch_select<8>(p, K, max_keys, topk_idx, topk_len, s); break;
  }
  return st == DSA_OK ? ok() : st;
}
