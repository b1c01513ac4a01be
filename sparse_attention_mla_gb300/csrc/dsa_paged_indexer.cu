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
// A ring of four tiles (128 KB) keeps DRAM busy, filled by TMA where pages allow it,
// else by cp.async.  The second kernel finds each token's K best with a cluster of 1
// to 8 CTAs per token (by the longest length there can be): the scores, as integers
// of the same order, stay in registers; histograms of 11 bits, starting below the
// bits that all scores share, narrow the K-th down, every CTA adding up all CTAs'
// bins through distributed shared memory (one cluster barrier a histogram); then
// one ordered compaction.  What bounds it is that chain of barriers, not its work;
// it is launched early and looks its request up while the scores are being made.
// Measured: one request of 65536 keys 19 us (two starts and the selection's chain),
// 678,000 keys of 32 requests 48 us, of which the scores are 36 (4.8 TB/s).
// Every step is exact and without order effects, so equal calls give equal lists.
#include <cooperative_groups.h>

#include <climits>
#include <cmath>

#include "dsa_host.h"
#include "dsa_paged.cuh"

namespace dsa {
namespace pidx {

namespace cg = cooperative_groups;

constexpr int kD = 128;          // index width
constexpr int kTile = 128;       // keys per tile (MMA M)
constexpr int kCols = 256;       // (token, head) columns of a group (MMA N)
constexpr int kRing = 4;         // tiles, one gather warp each
constexpr int kThreads = 32 * 15;  // MMA, 8 scores, 4 gather, 1 query, 1 announcing warp
constexpr int kReaders = 14;
constexpr int kSegs = 8;
constexpr int kMaxCtas = 160;

// tiles that the end of a group counts as when the tiles are dealt out: the next group's queries are waited for (100
// requests of 4000: 25.0 us, 27.4 when it counts for nothing; 32 of up to 32k: 48 and 49.6)
constexpr int kEnd = 3;
constexpr int kMaxLen = 1 << 30;  // (positions are counted past a row's end by up to a round of the selection)
constexpr int Q_CHUNK = kCols * 128, K_CHUNK = kTile * 128;
constexpr int OFF_Q = 0, OFF_K = 2 * Q_CHUNK, OFF_W = OFF_K + kRing * 2 * K_CHUNK, OFF_MISC = OFF_W + 2 * kCols * 4;
constexpr int SMEM = OFF_MISC + 1024 + 1024;
constexpr int M_K = 0, M_KF = 32, M_S = 64, M_SF = 80, M_Q = 96, M_SEG = 104, M_FIN = 112, M_TMEM = 120, M_ABORT = 124,
              M_PLAN = 128, M_SCRATCH = 192, M_ANN = 320, M_READ = M_ANN + 8 * kSegs, M_RING = M_READ + 8 * kSegs;
static_assert(M_RING + 32 * kSegs <= 1024 && M_SCRATCH + 8 * (kThreads / 32) <= M_ANN, "misc layout");

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
  int box;  // rows of a TMA box (32 or a smaller page), 0: every row by cp.async
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
  long long w0, w1;
  int u, g, t;  // request, group and tile of the first tile
  int skip;     // what lies before it: the end of a group
};

// A run of tiles [t0, t0 + n) of one group of a request's tokens, as announced (two int4).
struct Seg {
  int t0, n, tok, nt, b, keys;
  int last;  // the CTA's last run
};

__device__ __noinline__ bool read_announcement(uint32_t misc, const int4* ring, int k, volatile int* abort, long long limit,
                                               Seg& s) {
  const int at = k % kSegs;
  if (!__all_sync(0xffffffffu, wait_for(misc + M_ANN + 8 * at, (k / kSegs) & 1, abort, limit))) return false;
  const int4 a = ring[2 * at], c = ring[2 * at + 1];
  s = Seg{a.x, a.y, a.z, a.w, c.x, c.y, c.z};
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(misc + M_READ + 8 * at);
  return true;
}

template <int G>
__device__ __forceinline__ void announce(const Params& p, const Plan& pl, uint32_t misc, int4* ring, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  long long left = pl.w1 - pl.w0 - pl.skip;
  int u = pl.u, g = pl.g, t = pl.t;
  Request rq = request_of(p, u);
  bool cut = false;
#pragma unroll 1
  for (int k = 0; left > 0; ++k) {
    int tiles = (rq.keys + kTile - 1) / kTile;
#pragma unroll 1
    while (tiles == 0 || g * G >= rq.n) {  // (requests are skipped only while tiles are left)
      rq = request_of(p, ++u);
      tiles = (rq.keys + kTile - 1) / kTile;
      g = t = 0;
    }
    cut |= rq.keys < rq.len;
    const int n = (int)min((long long)(tiles - t), left), at = k % kSegs;
    left -= n + (t + n >= tiles ? kEnd : 0);
    if (k >= kSegs && !warp_all(wait_for(misc + M_READ + 8 * at, (k / kSegs - 1) & 1, abort, p.wait_limit))) break;
    if (lane == 0) {
      ring[2 * at] = make_int4(t, n, rq.n0 + g * G, min(G, rq.n - g * G));
      ring[2 * at + 1] = make_int4(u, rq.keys, left <= 0, 0);
      mbar_arrive(misc + M_ANN + 8 * at);
    }
    t += n;
    if (t >= tiles) { ++g; t = 0; }
  }
  if (cut && lane == 0) record_error(p.err, DSA_ERR_DEVICE_INDEX);  // longer than max_len or the table
}

// HP: heads per token, rounded up to 8, 16, 32 or 64 (the rest are zero rows)
template <int HP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_score_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map) {
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
      mbar_init(mb + M_K + 8 * s, 1);
      mbar_init(mb + M_KF + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(mb + M_S + 8 * b, 1);
      mbar_init(mb + M_SF + 8 * b, 4);
    }
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(mb + M_ANN + 8 * k, 1);
      mbar_init(mb + M_READ + 8 * k, kReaders);
    }
    mbar_init(mb + M_Q, 1);
    mbar_init(mb + M_SEG, 1);
    mbar_init(mb + M_FIN, 1);
    *s_abort = 0;
    fence_mbar_init();
    if (p.box > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
  }
  auto tiles_of = [&](int u) -> long long {
    const Request r = request_of(p, u);
    return r.keys > 0 ? (long long)((r.n + G - 1) / G) * ((r.keys + kTile - 1) / kTile + kEnd) : 0;
  };
  auto visit = [&](const TileRange& r, int u, long long lo, long long n) {
    if (lo <= r.w0 && r.w0 < lo + n) {
      const int tiles = (request_of(p, u).keys + kTile - 1) / kTile;
      const int span = tiles + kEnd;
      int g = (int)((r.w0 - lo) / span), t = (int)((r.w0 - lo) - (long long)g * span);
      s_plan->skip = 0;
      if (t >= tiles) {
        s_plan->skip = span - t;
        ++g;
        t = 0;
      }
      s_plan->u = u;
      s_plan->g = g;
      s_plan->t = t;
    }
  };
  const TileRange rg = split_line<kThreads>(p.B, tiles_of, reinterpret_cast<long long*>(misc + M_SCRATCH), visit);
  if (threadIdx.x == 0) {
    s_plan->w0 = rg.w0;
    s_plan->w1 = rg.w1;
  }
  __syncthreads();
  const Plan plan = *s_plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the selection waits for this kernel's end itself)
  if (plan.w1 <= plan.w0 || plan.w1 - plan.w0 <= plan.skip) return;
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  uint32_t tmem = 0;
  if (warp <= 8) {  // the others neither need it nor wait for it
    named_bar(3, 288);
    tmem = (uint32_t)warp_value((int)*s_tmem);
  }
  int4* ring = reinterpret_cast<int4*>(misc + M_RING);
  auto read_seg = [&](int k, Seg& s) -> bool { return read_announcement(mb, ring, k, s_abort, p.wait_limit, s); };
  Seg sg;

  if (warp == 0) {
    // ======================= MMA issuer =======================
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last);
      if (!warp_all(wait_for(mb + M_Q, seg & 1, s_abort, p.wait_limit))) break;
      // what the loop needs in registers of the warp (a call does not keep them)
      const int n = warp_value(sg.n);
      const uint32_t id = idesc_bf16(kTile, (warp_value(sg.nt) * HP + 15) & ~15, false, false);
      const uint32_t d0 = (uint32_t)warp_value((int)tmem), q0 = (uint32_t)warp_value((int)sQ), k0 = (uint32_t)warp_value((int)sK);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i) {
        const int sl = i % kRing, sb = i & 1;
        if (i >= 2 && !warp_all(wait_for(mb + M_SF + 8 * sb, ((i >> 1) - 1) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        if (!warp_all(wait_for(mb + M_K + 8 * sl, (i / kRing) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint64_t a = sdesc_sw128(k0 + (sl * 2 + c) * K_CHUNK, 16, 1024), b = sdesc_sw128(q0 + c * Q_CHUNK, 16, 1024);
          mma4_w<2, 2>(d0 + sb * kCols, a, b, id, c);
        }
        mma_commit_w(mb + M_KF + 8 * sl);
        mma_commit_w(mb + M_S + 8 * sb);
      }
      if (stop) break;
      mma_commit_w(mb + M_SEG);
    }
    mma_commit_w(mb + M_FIN);
    volatile int dummy = 0;
    mbar_wait(mb + M_FIN, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 14) {
    announce<G>(p, plan, mb, ring, s_abort);
  } else if (warp == 13) {
    // ======================= queries of a segment, once the products of the one before are done =======================
    for (int seg = 0, last = 0; !last; ++seg) {
      if (!warp_all(read_seg(seg, sg))) break;
      last = sg.last;
      if (seg > 0 && !warp_all(wait_for(mb + M_SEG, (seg - 1) & 1, s_abort, p.wait_limit))) break;
      const int rows = ((sg.nt * HP + 15) & ~15);
#pragma unroll 4
      for (int x = lane; x < rows * 16; x += 32) {
        const int n = x >> 4, u = x & 15, tok = n / HP, h = n - tok * HP;
        const bool ok = tok < sg.nt && h < p.Hi;
        cp_async16(sQ + (u >> 3) * Q_CHUNK + sw128_off(n, u & 7),
                   p.q + (ok ? ((size_t)(sg.tok + tok) * p.Hi + h) * kD + u * 8 : 0), ok ? 16u : 0u);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_Q);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 9) {
    // ======================= gather: a warp owns a slot of the ring and fills it with every fourth tile =======================
    // A lane looks four rows up, a tile of the slot ahead.  32 rows that are all there come by TMA in whole boxes; others by
    // cp.async, zero-filled where there is no key.
    const int sl = warp - 9;
    int seg = 0, base = 0, end = 0;
    int n_tiles = INT_MAX;  // this CTA's tiles, known once one past them has been looked for
    bool bad = false, stop = false;
    int page[4], at[4];  // of the rows 32 k + lane: page, place in it (-1: no key)
    auto look_up = [&](int i) {
      if (i >= n_tiles) return;
#pragma unroll 1
      while (i >= end) {
        if (seg > 0 && sg.last) { n_tiles = end; return; }
        if (!read_seg(seg, sg)) { stop = true; return; }
        ++seg;
        base = end;
        end += sg.n;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pos = (sg.t0 + i - base) * kTile + 32 * k + lane;
        at[k] = page[k] = -1;
        if (pos < sg.keys) {
          const unsigned q = (unsigned)pos / (unsigned)p.P;
          at[k] = pos - (int)q * p.P;
          page[k] = __ldg(p.table + (size_t)sg.b * p.max_pages + q);
        }
      }
    };
    look_up(sl);
    const uint32_t land = (uint32_t)warp_value((int)(sK + sl * 2 * K_CHUNK)), land_bar = (uint32_t)warp_value((int)(mb + M_K + 8 * sl));
    int armed = -1;  // the slot's last tile
#pragma unroll 1
    for (int i = sl; i < n_tiles && !stop; i += kRing) {
      long long row[4];
      unsigned whole = 0;  // bit k: rows 32 k .. are all there
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool ok = page[k] >= 0 && page[k] < p.num_pages && at[k] >= 0;
        bad |= at[k] >= 0 && !ok;
        row[k] = ok ? (long long)page[k] * p.P + at[k] : -1;
        if (p.box > 0 && __all_sync(0xffffffffu, ok)) whole |= 1u << k;
      }
      if (i >= kRing && !warp_all(wait_for(mb + M_KF + 8 * sl, ((i / kRing) - 1) & 1, s_abort, p.wait_limit))) break;
      const uint32_t bar = mb + M_K + 8 * sl;
      if (lane == 0 && whole)
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(__popc(whole) * 8192) : "memory");
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (whole & (1u << k)) {
#pragma unroll 1
          for (int at0 = 0; at0 < 32; at0 += p.box) {
            const int src = warp_value((int)__shfl_sync(0xffffffffu, row[k], at0));
            tma_load_2d_w(land + (32 * k + at0) * 128, &map, 0, src, land_bar);
            tma_load_2d_w(land + (32 * k + at0) * 128 + K_CHUNK, &map, 64, src, land_bar);
          }
        } else {
          const int u = lane & 15;
          const uint32_t dst = sK + (sl * 2 + (u >> 3)) * K_CHUNK;
#pragma unroll 4
          for (int e = 0; e < 16; ++e) {
            const int rr = 2 * e + (lane >> 4);
            const long long src = __shfl_sync(0xffffffffu, row[k], rr);
            cp_async16(dst + sw128_off(32 * k + rr, u & 7), p.cache + (src >= 0 ? (size_t)src * kD + u * 8 : 0),
                       src >= 0 ? 16u : 0u);
          }
        }
      }
      look_up(i + kRing);
      if (whole != 15u) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();  // the copies -> visible to the tensor core
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar);
      armed = i;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    volatile int dummy = 0;  // nothing lands after the CTA has left
    if (armed >= 0) mbar_wait(mb + M_K + 8 * sl, (armed / kRing) & 1, &dummy, p.err);
    if (bad) record_error(p.err, DSA_ERR_DEVICE_INDEX);
  } else {
    // ======================= scores: two groups of four warps take alternate tiles; a thread is a key =======================
    const int grp = (warp - 1) >> 2, qd = warp & 3;
    float* s_w = reinterpret_cast<float*>(smem + OFF_W) + grp * kCols;
    bool stop = false;
    int i = 0;
    for (int seg = 0; seg == 0 || !sg.last; ++seg) {
      if (!stop && !read_seg(seg, sg)) stop = true;
      // the weights of the segment before have been read; all four warps leave together after a failed wait
      if (named_bar_or(1 + grp, 128, stop)) break;
      const int cols = sg.nt * HP;
      for (int x = ((warp - 1) & 3) * 32 + lane; x < cols; x += 128) {
        const int tok = x / HP, h = x - tok * HP;
        s_w[x] = h < p.Hi ? __ldg(p.w + (size_t)(sg.tok + tok) * p.Hi + h) : 0.f;
      }
      named_bar(1 + grp, 128);
      const int t_end = sg.t0 + sg.n;
      for (int t = sg.t0; t < t_end; ++t, ++i) {
        if ((i & 1) != grp || stop) continue;
        if (!warp_all(wait_for(mb + M_S + 8 * grp, (i >> 1) & 1, s_abort, p.wait_limit))) { stop = true; continue; }
        tc_fence_after();
        const int pos = t * kTile + qd * 32 + lane;
        float* out = p.scores + (size_t)sg.tok * p.stride + pos;
        const bool in = pos < sg.keys;
        float acc = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(tmem_addr(tmem + grp * kCols + c0, qd * 32, 0), v);
          tmem_ld_wait();
          // the padding's products are left out, not weighed by 0: with an infinite key they are NaN
          const int real = p.Hi - (c0 & (HP - 1));  // of each token's columns in this chunk
          if (real < (HP < 32 ? HP : 32)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((j & (HP - 1)) >= real) v[j] = 0u;
          }
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
    if (lane == 0 && *s_abort) record_error(p.err, DSA_ERR_TIMEOUT);
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

// Exclusive sum of v over the CTA's threads (T: 32 or 64 bits), and the total.  `sh`: 32 words of T that no other scan
// in flight uses.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* sh, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  T s = sh[lane];  // every warp sums the warps' totals itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  return (warp ? before : 0) + inc - v;
}

template <int CS>
__global__ void __launch_bounds__(kSel, 1)
    paged_select_kernel(const float* scores, long long stride, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ cu_q, int N, int B, int K, int max_keys, int32_t* __restrict__ topk_idx,
                        int32_t* __restrict__ topk_len) {
  __shared__ uint32_t hist[2][kBins];
  __shared__ unsigned long long sh[2][32];
  __shared__ uint32_t box[2], pick[6];  // this CTA's smallest and largest; the bin of the K-th
  const int n = blockIdx.x / CS, rank = blockIdx.x % CS, tid = threadIdx.x;
  // the token's request and what it sees (the same in the whole cluster)
  int b = n, lo_tok = n, hi_tok = n + 1;
  if (cu_q) {
    if (n < __ldg(cu_q) || n >= __ldg(cu_q + B)) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // (this kernel does not end before the one with the scores)
      return;
    }
    b = warp_last_le(cu_q, B, n);
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
  if (v <= K) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  cg::cluster_group cl = cg::this_cluster();
  // this CTA's piece of the row, a multiple of 4 so that the 16-byte loads stay aligned
  const int piece = ((v + CS - 1) / CS + 3) & ~3;
  const int begin = min(v, rank * piece), end = min(v, begin + piece);
  // scores of a thread and round, four at a time: a short piece is spread over all threads
  const int per = min(kPer, (piece + 4 * kSel - 1) / (4 * kSel) * 4), round = per * kSel;
  const int rounds = (end - begin + round - 1) / round;
  const float* row = scores + (size_t)n * stride;
  uint32_t key[kPer];
  auto load = [&](int r) {
    const int p0 = begin + r * round + tid * per;
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      if (j >= per) continue;
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
  if (tid == 0) { box[0] = 0xffffffffu; box[1] = 0u; }
  hist[0][tid] = hist[0][tid + kSel] = 0u;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores (made during this kernel: no constant data)
  if (rounds == 1) load(0);

  // smallest and largest: the bits above the highest one where they differ are shared by all
  uint32_t mn = 0xffffffffu, mx = 0u;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j / 4 * 4 >= per) continue;
      if (key[j]) mn = min(mn, key[j]);
      mx = max(mx, key[j]);
    }
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) { atomicMin(&box[0], mn); atomicMax(&box[1], mx); }
  if constexpr (CS > 1) {
    cl.sync();
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      const uint32_t* q = cl.map_shared_rank(box, c);
      mn = min(mn, q[0]);
      mx = max(mx, q[1]);
    }
  } else {
    __syncthreads();
    mn = box[0];
    mx = box[1];
  }

  // narrow the K-th largest down: `prefix` holds its bits from `bit` upwards, `need` how many of the scores that
  // share them are still to be taken
  int bit = mn == mx ? 0 : 32 - __clz(mn ^ mx);
  uint32_t prefix = bit == 32 ? 0u : (mx >> bit) << bit;
  int need = K;
  uint32_t at = 0, tied = (uint32_t)begin;  // entries of the row, and of its tied scores, before this CTA's piece
  bool all = false;                         // every score that shares the prefix is taken
  for (int pass = 0; bit > 0 && !all; ++pass) {
    const int shift = max(0, bit - 11);
    const uint32_t span = bit == 32 ? 0xffffffffu : (1u << bit) - 1u;
    uint32_t* h = hist[pass & 1];
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (j / 4 * 4 >= per) continue;
        const uint32_t d = key[j] - prefix;  // (below 2^bit: the prefix is shared)
        if (key[j] && d <= span) atomicAdd(&h[d >> shift], 1u);
      }
    }
    if constexpr (CS > 1) cl.sync(); else __syncthreads();
    // the next histogram's bins (read by no CTA since the barrier before this one)
    hist[(pass + 1) & 1][tid] = hist[(pass + 1) & 1][tid + kSel] = 0u;
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t, summed over the cluster (low words) and over
    // the CTAs before this one (high words)
    unsigned long long h1 = 0, h0 = 0;
#pragma unroll
    for (int c = 0; c < CS; ++c) {
      const uint32_t* q = CS > 1 ? cl.map_shared_rank(h, c) : h;
      const uint2 x = *reinterpret_cast<const uint2*>(q + kBins - 2 - 2 * tid);
      const unsigned long long w = c < rank ? 0x100000001ull : 1ull;
      h1 += w * x.y;
      h0 += w * x.x;
    }
    unsigned long long total;
    const unsigned long long above = block_scan(h1 + h0, sh[pass & 1], total), mid = above + h1;
    const uint32_t a0 = (uint32_t)above, a1 = (uint32_t)mid, a2 = (uint32_t)(mid + h0);
    const bool first = a0 < (uint32_t)need && a1 >= (uint32_t)need;
    if (first || (a1 < (uint32_t)need && a2 >= (uint32_t)need)) {
      const unsigned long long up = first ? above : mid, in = first ? h1 : h0;
      pick[0] = kBins - (first ? 1 : 2) - 2 * tid;
      pick[1] = (uint32_t)up;
      pick[2] = (uint32_t)(up >> 32);
      pick[3] = (uint32_t)in;
      pick[4] = (uint32_t)(in >> 32);
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    need -= (int)pick[1];
    at += pick[2];
    tied = pick[4];
    all = (int)pick[3] == need;
    bit = shift;
    __syncthreads();
  }
  // (no CTA leaves while another may still read its shared memory; the last such reads are behind us)
  if constexpr (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // taken: above the prefix's class, and the first `need` of the class in order of position (few of a thread's scores:
  // one bit each, and the bits that are set are walked)
  at += min(tied, (uint32_t)need);
  const uint32_t low = max(prefix, 1u), top = prefix + ((1u << bit) - 1u);  // (bit < 32: a histogram or equal scores)
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    uint32_t above = 0, same = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j / 4 * 4 >= per) continue;
      above |= key[j] > top ? 1u << j : 0u;
      same |= key[j] >= low ? 1u << j : 0u;
    }
    same &= ~above;
    uint32_t sum;  // above, and tied from bit 16 (a round holds 16384)
    if (r) __syncthreads();
    const uint32_t before = block_scan((uint32_t)__popc(above) + ((uint32_t)__popc(same) << 16),
                                       reinterpret_cast<uint32_t*>(sh[0]) + 32 * (r & 1), sum);
    uint32_t my_tied = tied + (before >> 16);
    uint32_t o = at + (before & 0xffffu) + (min(my_tied, (uint32_t)need) - min(tied, (uint32_t)need));
    const int p0 = begin + r * round + tid * per;
    for (uint32_t left = above | same; left != 0u; left &= left - 1u) {
      const int j = __ffs(left) - 1;
      const bool tie = (same >> j) & 1u, take = !tie || my_tied < (uint32_t)need;
      my_tied += tie ? 1u : 0u;
      if (take) out[o] = p0 + j;
      o += take ? 1u : 0u;
    }
    at += (sum & 0xffffu) + (min(tied + (sum >> 16), (uint32_t)need) - min(tied, (uint32_t)need));
    tied += sum >> 16;
  }
  if constexpr (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

inline long long stride_of(long long max_len) { return (max_len + 3) / 4 * 4; }

// CTAs per token: as many as hold the row in one round, up to 8; and up to 4 while a piece is longer than 8192 and all
// CTAs fit the card at once (8 x 32768: 25.0 us with 4, 26.8 with 2; 1 x 65536: 20.7 with 4, 21.7 with 8, whose cluster
// barriers cost more than the shorter pieces save).
inline int cluster_of(int N, long long max_len) {
  int cs = 1;
  while (cs < 8 && (long long)cs * kRound < max_len) cs *= 2;
  while (cs < 4 && (long long)cs * 8192 < max_len && (long long)N * cs * 2 <= 152) cs *= 2;
  return cs;
}

template <int HP>
dsa_status_t launch_scores(const Params& p, const CUtensorMap& map, int ctas, cudaStream_t s) {
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_score_kernel<HP>), SMEM,
                                          "configuring paged_score_kernel");
  if (st != DSA_OK) return st;
  paged_score_kernel<HP><<<ctas, kThreads, SMEM, s>>>(p, map);
  return cuda_check(cudaGetLastError(), "launching paged_score_kernel");
}

template <int CS>
dsa_status_t launch_select(const Params& p, int K, int max_keys, int32_t* idx, int32_t* len, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.N * CS);
  cfg.blockDim = dim3(kSel);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CS;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CS > 1 ? 2 : 1;
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
  if (max_len > pidx::kMaxLen) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: max_len must be at most 2^30 (got %d)", who, max_len);
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
  // rows that follow one another in the cache, 32 or a whole page of them at a time
  CUtensorMap map{};
  if (num_pages > 0 && (page_size % 32 == 0 || 32 % page_size == 0) && page_size >= 8 &&
      (int64_t)num_pages * page_size <= 0x7fffffffll) {
    p.box = page_size < 32 ? page_size : 32;
    if ((st = make_map_2d_bf16(&map, k_cache, (uint64_t)num_pages * page_size, Di, Di, 64, p.box)) != DSA_OK) return st;
  }
  if (Hi <= 8) st = pidx::launch_scores<8>(p, map, ctas, s);
  else if (Hi <= 16) st = pidx::launch_scores<16>(p, map, ctas, s);
  else if (Hi <= 32) st = pidx::launch_scores<32>(p, map, ctas, s);
  else st = pidx::launch_scores<64>(p, map, ctas, s);
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
