// dsa_paged_mla.cu -- attention of new tokens over a paged latent cache (sm_103a).
//
// For new token j of request b (n_b of them, at the end of seq_lens[b] tokens) and
// head h:  z_p = scale <q, kv_p> over the positions p it sees (its own and all
// before, or the ones of its list),  lse = ln sum e^{z_p},
// out = sum e^{z_p - lse} kv_p[0:512].  One latent row serves all heads, so the
// floor is one read of every visible row; at 64 heads the tensor core needs about
// three quarters of the time that DRAM needs for a tile, at 128 it is the bound.
//
// Split: the (token, head) rows of a request that share its cache are packed into
// groups of NH = 16 or 64 MMA columns; a group's positions are cut into tiles of 64,
// and the tiles of all groups, laid end to end, are cut into equal ranges, one per
// CTA (one CTA per SM).  Every CTA finds its range from the lengths on the device
// (a sum over the requests), so no plan is made on the host and a captured step
// follows the lengths.  A group inside one range is finished there; the pieces of
// a group over several CTAs go to the workspace as (max, sum, unnormalised O) in
// fp32 and a second kernel joins them in a fixed order.
//
// A tile: S^T[key, row] = KV Q^T (M = 64 keys), an online softmax with a lazily
// raised maximum, O^T[channel, row] += V^T P^T (M = 128 channels), P as bf16 hi + lo
// side by side on the N axis, so that O keeps about fp32 accuracy (P in bf16 alone
// would add as much error as the output's own rounding).  Rows are copied by 16-byte
// cp.async, which takes any page size and order and zero-fills what is masked (no
// stale page, NaN included, reaches a product).
//
// Warps: 0 issues S^T, 1-8 softmax and epilogue, 9-12 copy tiles into a ring, 13
// issues P.V.  At width 576 and NH = 64 the ring's two tiles, Q and P need all the
// shared memory: P^T lies over the tile's last chunk (positions, read only by S^T)
// and an 8 KiB block that the two tiles share.
#include <cmath>

#include "dsa_host.h"
#include "dsa_paged.cuh"

namespace dsa {
namespace pmla {

constexpr int kTile = 64;
constexpr int kDv = 512;
constexpr int kWorkers = 256;
constexpr int kGather = 128;
constexpr int kThreads = 32 + kWorkers + kGather + 32;
constexpr int kRowsPer = kTile / (kGather / 8);  // tile rows per gather thread
constexpr int kMaxCtas = 160;
constexpr float kRaise = 8.0f;  // log2 units: the running maximum is raised only past this
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int DQK, int NH>
struct Smem {
  static constexpr int NCH = DQK / 64;
  static constexpr int CHUNK = kTile * 128;
  static constexpr int Q_CHUNK = NH * 128;
  // P over the ring only where nothing else fits
  static constexpr bool OVERLAY = NH == 64 && DQK == 576;
  static constexpr int R = (NH == 64 || DQK == 576) ? 2 : 3;
  static constexpr int NS = NH == 64 ? 1 : 2;  // S^T buffers in TMEM
  static constexpr int P_BLOCK = 2 * NH * 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = (NCH * Q_CHUNK + 1023) / 1024 * 1024;
  static constexpr int RING = OVERLAY ? 2 * NCH * CHUNK + CHUNK : R * NCH * CHUNK;
  static constexpr int OFF_P = OFF_KV + RING;
  static constexpr int OFF_MISC = OFF_P + (OVERLAY ? 0 : 2 * P_BLOCK);
  static constexpr int MISC = 2048;
  static constexpr int TOTAL = OFF_MISC + MISC + 1024;  // + alignment slack
  static_assert(TOTAL <= 232448, "shared memory budget");
  static_assert(NH == 64 || 4 * 2 * NH + NS * NH <= 256, "TMEM budget");
  // Overlay: [tile 0: chunks 0-7][its chunk 8][shared block][chunk 8 of tile 1][tile 1: chunks 0-7]
  __device__ static constexpr uint32_t chunk(uint32_t kv, int slot, int c) {
    if (!OVERLAY) return kv + (uint32_t)(slot * NCH + c) * CHUNK;
    if (c == 8) return kv + (uint32_t)(slot ? 10 : 8) * CHUNK;
    return kv + (uint32_t)(slot ? 11 + c : c) * CHUNK;
  }
  // P of tile i: hi rows, then (NH * 128 bytes on) lo rows
  __device__ static constexpr uint32_t p(uint32_t kv, int i) {
    if (OVERLAY) return kv + (uint32_t)((i & 1) ? 9 : 8) * CHUNK;
    return kv + (uint32_t)RING + (uint32_t)(i & 1) * P_BLOCK;
  }
  static constexpr int TM_COLS = NH == 64 ? 512 : 256;
  static constexpr int TM_O = NS * NH;  // first column of O^T
  // first column of channel tile m; at NH = 64 the last one adds hi and lo in the same 64 columns
  __device__ static constexpr int o_col(int m) { return TM_O + m * 2 * NH; }
};

// misc (bytes)
constexpr int M_KV = 0, M_PV = 24, M_S = 48, M_SF = 64, M_P = 80, M_Q = 96, M_FIN = 104;  // [3][3][2][2][2][1][2]
constexpr int M_TMEM = 120, M_ABORT = 124, M_PLAN = 128;  // plan: 64 bytes
constexpr int M_VALID = 192;                  // uint8 [3][64]
constexpr int M_STAT = 384, M_FAC = 640;      // float [64] each
constexpr int M_RED = 896;                    // float [4][64]
static_assert(M_RED + 1024 <= 2048, "misc layout");

struct Params {
  const __nv_bfloat16* q;
  const __nv_bfloat16* cache;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const int32_t* topk_idx;
  const int32_t* topk_len;
  int N, B, H, K, num_pages, P, max_pages;
  int G, HB;  // tokens per group, head blocks
  float sl2e;
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  int4* records;   // [kMaxCtas]: (first row, rows, first head, last CTA) of the group that a CTA opens; rows 0: none
  float* stats;    // [2 * kMaxCtas][2][64]
  float* partial;  // [2 * kMaxCtas][64][512]
  long long wait_limit;
};

struct Unit {
  int groups, tiles;  // groups of MMA columns, tiles of each
  int n0, n;          // first token, tokens
};

// A unit is a request (all its tokens see the same cache) or, with lists, one token.
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit r;
  if (p.topk_idx != nullptr) {
    const int end = p.cu_q ? min(max(__ldg(p.cu_q + p.B), 0), p.N) : p.N;
    r.n0 = u;
    r.n = u < end ? 1 : 0;
    int len = p.K;
    if (p.topk_len) len = min(max(__ldg(p.topk_len + u), 0), p.K);
    r.tiles = max(1, (len + kTile - 1) / kTile);
  } else {
    const int lo = p.cu_q ? min(max(__ldg(p.cu_q + u), 0), p.N) : u;
    const int hi = p.cu_q ? min(max(__ldg(p.cu_q + u + 1), lo), p.N) : u + 1;
    r.n0 = lo;
    r.n = hi - lo;
    const long long most = (long long)p.max_pages * p.P;
    const int len = (int)min((long long)max(__ldg(p.seq_lens + u), 0), most);
    r.tiles = max(1, (int)(((long long)len + kTile - 1) / kTile));
  }
  r.groups = (r.n + p.G - 1) / p.G * p.HB;
  return r;
}

// The CTA's range of tiles and where it starts (in shared memory, written by make_plan).
struct Plan {
  long long w0, w1;      // this CTA's tiles of the whole line
  int u0, pad;           // unit that holds tile w0
  long long first;       // w0 minus the unit's first tile
};

// A run of tiles [t0, t1) of one group.
struct Seg {
  int t0, t1, T;
  int row0, rows;   // rows (token, head) of q, out and lse
  int head0;        // head of the first row
  int b;            // request
  int seen0;        // positions that the group's first token sees
  int keys;         // positions looked at by any token (dense), or entries of the list
  int tok;          // first token
};

struct Walk {
  const Params& p;
  int u, g, t;
  long long left;
  Unit un;
  __device__ __forceinline__ Walk(const Params& p_, const Plan& pl) : p(p_) {
    left = pl.w1 - pl.w0;
    u = pl.u0;
    g = t = 0;
    if (left > 0) {
      un = unit_of(p, u);
      g = (int)(pl.first / un.tiles);
      t = (int)(pl.first - (long long)g * un.tiles);
    }
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (left <= 0) return false;
    while (g >= un.groups) {  // (units are skipped only while tiles are left, so u stays in range)
      un = unit_of(p, ++u);
      g = t = 0;
    }
    const int tb = g / p.HB, hb = g - tb * p.HB;
    const int n0 = un.n0 + tb * p.G, nt = min(p.G, un.n - tb * p.G);
    s.tok = n0;
    s.head0 = hb * 64;
    s.row0 = n0 * p.H + s.head0;
    s.rows = p.HB > 1 ? min(64, p.H - s.head0) : nt * p.H;
    s.T = un.tiles;
    s.t0 = t;
    s.t1 = (int)min((long long)un.tiles, t + left);
    left -= s.t1 - s.t0;
    if (p.topk_idx == nullptr) {
      s.b = u;
      const int len = max(__ldg(p.seq_lens + u), 0);
      s.keys = (int)min((long long)len, (long long)p.max_pages * p.P);
      s.seen0 = max(__ldg(p.seq_lens + u), 0) - un.n + tb * p.G + 1;  // may be <= 0: sees nothing
    } else {
      int b = n0, lo_tok = n0, hi_tok = n0 + 1;
      if (p.cu_q) {
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.cu_q + mid) <= n0) lo = mid; else hi = mid;
        }
        b = lo;
        lo_tok = __ldg(p.cu_q + b);
        hi_tok = __ldg(p.cu_q + b + 1);
      }
      s.b = b;
      s.seen0 = max(__ldg(p.seq_lens + b), 0) - (hi_tok - lo_tok) + (n0 - lo_tok) + 1;
      s.keys = p.topk_len ? min(max(__ldg(p.topk_len + n0), 0), p.K) : p.K;
    }
    t = s.t1;
    if (t >= un.tiles) { ++g; t = 0; }
    return true;
  }
};

// Whole CTA: this CTA's share of the tiles, the unit it starts in, and the record of the group that it opens and
// does not finish.
__device__ __forceinline__ void make_plan(const Params& p, Plan* plan, long long* scratch) {
  if (threadIdx.x == 0) p.records[blockIdx.x] = make_int4(0, 0, 0, 0);
  auto tiles_of = [&](int u) -> long long {
    const Unit x = unit_of(p, u);
    return (long long)x.groups * x.tiles;
  };
  auto visit = [&](const TileRange& r, int u, long long lo, long long n) {
    if (lo <= r.w0 && r.w0 < lo + n) {
      plan->u0 = u;
      plan->first = r.w0 - lo;
    }
    if (lo <= r.w1 - 1 && r.w1 - 1 < lo + n) {  // the range's last tile
      const Unit x = unit_of(p, u);
      const long long off = r.w1 - 1 - lo;
      const int g = (int)(off / x.tiles), tl = (int)(off - (long long)g * x.tiles);
      const long long opened = r.w1 - 1 - tl;  // the group's first tile
      if (tl + 1 < x.tiles && opened >= r.w0) {
        const int tb = g / p.HB, hb = g - tb * p.HB;
        const int n0 = x.n0 + tb * p.G, nt = min(p.G, x.n - tb * p.G);
        const int last = (int)(((opened + x.tiles) * r.C - 1) / r.W);  // the CTA of its last tile
        p.records[blockIdx.x] =
            make_int4(n0 * p.H + hb * 64, p.HB > 1 ? min(64, p.H - hb * 64) : nt * p.H, hb * 64, last);
      }
    }
  };
  const TileRange r = split_line<kThreads>(p.topk_idx ? p.N : p.B, tiles_of, scratch, visit);
  if (threadIdx.x == 0) {
    plan->w0 = r.w0;
    plan->w1 = r.w1;
  }
  __syncthreads();
}

// 16 TMEM lanes x 64 bits, N times: thread t of the warp gets lane base + (t >> 2) + 8 (t & 1) and the columns
// c + 2j + ((t >> 1) & 1), j = 0..N-1.
template <int N>
__device__ __forceinline__ void tmem_ld16x64b(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.16x64b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  } else {
    static_assert(N == 16, "columns per thread");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x64b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
  }
}
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(a, r); else tmem_ld32(a, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t a, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st8(a, r); else tmem_st32(a, r);
}

template <int DQK, int NH>
__global__ void __launch_bounds__(kThreads, 1) paged_mla_kernel(const Params p) {
  using L = Smem<DQK, NH>;
  constexpr int NCH = L::NCH, R = L::R, NS = L::NS;
  constexpr int NHH = NH / 2, NQ = NHH / 2;  // rows per softmax half, per thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem + L::OFF_Q), sKV = smem_u32(smem + L::OFF_KV);
  uint8_t* misc = smem + L::OFF_MISC;
  const uint32_t mb = smem_u32(misc);
  const uint32_t bar_kv = mb + M_KV, bar_pv = mb + M_PV, bar_s = mb + M_S, bar_sf = mb + M_SF, bar_p = mb + M_P,
                 bar_q = mb + M_Q, bar_fin = mb + M_FIN;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + M_ABORT);
  Plan* s_plan = reinterpret_cast<Plan*>(misc + M_PLAN);
  volatile uint8_t* s_valid = misc + M_VALID;
  float* s_stat = reinterpret_cast<float*>(misc + M_STAT);
  float* s_fac = reinterpret_cast<float*>(misc + M_FAC);
  float* s_red = reinterpret_cast<float*>(misc + M_RED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(bar_kv + 8 * s, kGather + kGather / 8);  // every copying thread's landings, every row flag's writer
      mbar_init(bar_pv + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_s + 8 * b, 1);
      mbar_init(bar_sf + 8 * b, 8);
      mbar_init(bar_p + 8 * b, 8);
      mbar_init(bar_fin + 8 * b, 1);
    }
    mbar_init(bar_q, kWorkers);
    *s_abort = 0;
    fence_mbar_init();
  }
  make_plan(p, s_plan, reinterpret_cast<long long*>(s_red));
  const Plan plan = *s_plan;
  if (plan.w1 <= plan.w0) return;  // (the whole CTA)
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), L::TM_COLS);
    tmem_relinquish();
  }
  __syncthreads();
  const uint32_t tmem = *s_tmem;

  if (warp == 0) {
    // ======================= S^T issuer =======================
    constexpr uint32_t kIdS = idesc_bf16(kTile, NH, false, false);
    Walk walk(p, plan);
    Seg sg;
    int i = 0, seg = 0;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      if (!warp_all(mbar_wait(bar_q, seg & 1, s_abort, p.err, p.wait_limit))) break;
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % R, sb = i % NS;
        if (i >= NS && !warp_all(mbar_wait(bar_sf + 8 * sb, ((i / NS) - 1) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        if (!warp_all(mbar_wait(bar_kv + 8 * sl, (i / R) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t b00 = sdesc_sw128(sQ, 16, 1024);
#pragma unroll 1
        for (int c = 0; c < NCH; ++c) {
          const uint64_t a0 = sdesc_sw128(L::chunk(sKV, sl, c), 16, 1024);
          const uint64_t b0 = b00 + (uint64_t)((c * L::Q_CHUNK) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_w(tmem + sb * NH, a0 + (uint64_t)(k * 2), b0 + (uint64_t)(k * 2), kIdS, (c | k) ? 1u : 0u);
        }
        mma_commit_w(bar_s + 8 * sb);
      }
      ++seg;
    }
    mma_commit_w(bar_fin);
    volatile int dummy = 0;
    mbar_wait(bar_fin, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 13) {
    // ======================= P.V issuer =======================
    Walk walk(p, plan);
    Seg sg;
    int i = 0;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % R;
        if (!warp_all(mbar_wait(bar_p + 8 * (i & 1), (i >> 1) & 1, s_abort, p.err, p.wait_limit))) { stop = true; break; }
        tc_fence_after();
        const uint64_t va = sdesc_sw128(L::chunk(sKV, sl, 0), L::CHUNK, 1024);
        constexpr uint64_t kPair = (2 * L::CHUNK) >> 4;
        const uint32_t sP = L::p(sKV, i);
        if constexpr (NH == 64) {  // P^T rows are keys (MN-major), hi and lo blocks of 64 rows' columns 8 KiB apart
          constexpr uint32_t kId2 = idesc_bf16(128, 128, true, true), kId1 = idesc_bf16(128, 64, true, true);
          const uint64_t pb = sdesc_sw128(sP, 8192, 1024);
#pragma unroll
          for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_w(tmem + L::o_col(m), va + m * kPair + (uint64_t)(k * 128), pb + (uint64_t)(k * 128), kId2,
                       (t > sg.t0 || k > 0) ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss_w(tmem + L::o_col(3), va + 3 * kPair + (uint64_t)((k & 3) * 128),
                     pb + (uint64_t)((k >> 2) * 512 + (k & 3) * 128), kId1, (t > sg.t0 || k > 0) ? 1u : 0u);
        } else {  // P^T rows are [hi rows | lo rows], keys along K
          constexpr uint32_t kId = idesc_bf16(128, 2 * NH, true, false);
          const uint64_t pb = sdesc_sw128(sP, 16, 1024);
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_w(tmem + L::o_col(m), va + m * kPair + (uint64_t)(k * 128), pb + (uint64_t)(k * 2), kId,
                       (t > sg.t0 || k > 0) ? 1u : 0u);
        }
        mma_commit_w(bar_pv + 8 * sl);
      }
    }
    mma_commit_w(bar_fin + 8);
    volatile int dummy = 0;
    mbar_wait(bar_fin + 8, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp >= 9) {
    // ======================= gather: tiles into the ring =======================
    const int gt = threadIdx.x - 32 - kWorkers, uc = gt & 7;
    Walk walk(p, plan);
    Seg sg;
    int i = 0;
    bool stop = false;
    while (!stop && walk.next(sg)) {
      const int32_t* tab = p.table + (size_t)sg.b * p.max_pages;
      if (p.topk_idx == nullptr && gt == 0 && sg.keys < __ldg(p.seq_lens + sg.b)) record_error(p.err, DSA_ERR_DEVICE_INDEX);
      const int32_t* list = p.topk_idx ? p.topk_idx + (size_t)sg.tok * p.K : nullptr;
      // position of tile row r, or -1; then its cache row
      auto load_pos = [&](int t, int (&pos)[kRowsPer]) {
#pragma unroll
        for (int e = 0; e < kRowsPer; ++e) {
          const int j = t * kTile + (gt >> 3) + (kGather / 8) * e;
          int x = -1;
          if (t < sg.t1 && j < sg.keys) {
            x = j;
            if (list) {
              x = __ldg(list + j);
              if (x < -1 || (x >= 0 && (x >= sg.seen0 || x >= (long long)p.max_pages * p.P))) {
                record_error(p.err, DSA_ERR_DEVICE_INDEX);
                x = -1;
              }
            }
          }
          pos[e] = x;
        }
      };
      auto load_page = [&](const int (&pos)[kRowsPer], int (&page)[kRowsPer]) {
#pragma unroll
        for (int e = 0; e < kRowsPer; ++e) page[e] = pos[e] >= 0 ? __ldg(tab + (unsigned)pos[e] / (unsigned)p.P) : -1;
      };
      int pos[kRowsPer], page[kRowsPer];
      load_pos(sg.t0, pos);
      load_page(pos, page);
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % R;
        long long row[kRowsPer];
#pragma unroll
        for (int e = 0; e < kRowsPer; ++e) {
          row[e] = -1;
          if (pos[e] >= 0) {
            if (page[e] >= 0 && page[e] < p.num_pages) row[e] = (long long)page[e] * p.P + (unsigned)pos[e] % (unsigned)p.P;
            else record_error(p.err, DSA_ERR_DEVICE_INDEX);
          }
        }
        load_pos(t + 1, pos);
        load_page(pos, page);
        if (i >= R && !mbar_wait(bar_pv + 8 * sl, ((i / R) - 1) & 1, s_abort, p.err, p.wait_limit)) { stop = true; break; }
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const uint32_t dst = L::chunk(sKV, sl, c);
#pragma unroll
          for (int e = 0; e < kRowsPer; ++e) {
            const int r = (gt >> 3) + (kGather / 8) * e;
            const bool ok = row[e] >= 0;
            cp_async16(dst + sw128_off(r, uc), p.cache + (ok ? (size_t)row[e] * DQK + c * 64 + uc * 8 : 0), ok ? 16u : 0u);
          }
        }
        cp_async_arrive(bar_kv + 8 * sl);
        if (uc == 0) {
#pragma unroll
          for (int e = 0; e < kRowsPer; ++e) s_valid[sl * kTile + (gt >> 3) + (kGather / 8) * e] = row[e] >= 0 ? 1 : 0;
          mbar_arrive(bar_kv + 8 * sl);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ======================= softmax + epilogue =======================
    const int tid = threadIdx.x - 32, wk = warp - 1, qd = warp & 3, ch = wk >> 2;
    const int par = (lane >> 1) & 1;
    const int r = qd * 16 + (lane >> 2) + 8 * (lane & 1);  // key row of the tile
    const int bar_id = 1 + ch;
    const int n0 = ch * NHH + par * NQ;  // this thread's rows n0 .. n0 + NQ - 1 of the group
    auto load_q = [&](const Seg& s) {
      constexpr int UNITS = NH * NCH * 8;
      const uint64_t pol = l2_evict_first_policy();
      for (int x = tid; x < UNITS; x += kWorkers) {
        const int hh = x / (NCH * 8), rem = x - hh * (NCH * 8), c = rem >> 3, uc = rem & 7;
        const bool ok = hh < s.rows;
        cp_async16_hint(sQ + c * L::Q_CHUNK + sw128_off(hh, uc),
                        p.q + (ok ? (size_t)(s.row0 + hh) * DQK + c * 64 + uc * 8 : 0), ok ? 16u : 0u, pol);
      }
      cp_async_arrive(bar_q);
    };
    // over the warp's 16 keys: the lanes of one parity hold the same rows
    auto reduce_keys = [&](float v, bool is_max) -> float {
#pragma unroll
      for (int o = 1; o <= 16; o <<= 1) {
        if (o == 2) continue;
        const float x = __shfl_xor_sync(0xffffffffu, v, o);
        v = is_max ? fmaxf(v, x) : v + x;
      }
      return v;
    };
    Walk walk(p, plan);
    Seg sg, nx;
    bool have = walk.next(sg);
    if (have) load_q(sg);
    bool aborted = false;
    int i = 0;
    while (have && !aborted) {
      const bool more = walk.next(nx);
      float l_part[NQ];
#pragma unroll
      for (int j = 0; j < NQ; ++j) l_part[j] = 0.f;
      if (qd == 0 && lane < NHH) s_stat[ch * NHH + lane] = -INFINITY;  // (read only after a barrier of the half)
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int sl = i % R, sb = i % NS;
        bool bad = !mbar_wait(bar_s + 8 * sb, (i / NS) & 1, s_abort, p.err, p.wait_limit);
        // (complete since before S^T was issued: orders the row flags before their reads below)
        bad = bad || !mbar_wait(bar_kv + 8 * sl, (i / R) & 1, s_abort, p.err, p.wait_limit);
        // P of tile i overwrites what P.V of an earlier tile read: of the tile before with the shared block, else
        // of the one before that
        constexpr int kBack = L::OVERLAY ? 1 : 2;
        if (!L::OVERLAY && i >= kBack)
          bad = bad || !mbar_wait(bar_pv + 8 * ((i - kBack) % R), ((i - kBack) / R) & 1, s_abort, p.err, p.wait_limit);
        tc_fence_after();
        uint32_t raw[NQ];
        tmem_ld16x64b<NQ>(tmem_addr(tmem + sb * NH + ch * NHH, qd * 32, 0), raw);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf + 8 * sb);
        if (t + 1 == sg.t1 && more && !bad) load_q(nx);  // S^T of the segment is done: Q is free
        // alternate columns of the half -> NQ consecutive rows: swap half of them with the key's other thread
        float z[NQ];
#pragma unroll
        for (int j = 0; j < NQ / 2; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, par ? raw[j] : raw[NQ / 2 + j], 2);
          z[2 * j] = __uint_as_float(par ? got : raw[j]);
          z[2 * j + 1] = __uint_as_float(par ? raw[NQ / 2 + j] : got);
        }
        const bool valid = s_valid[sl * kTile + r] != 0;
        const int pos = t * kTile + r;
        if (p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0) {  // some token may not see all of the tile
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const int seen = sg.seen0 + (sg.head0 + n0 + j) / p.H;
            z[j] = (valid && pos < seen) ? z[j] * p.sl2e : -INFINITY;
          }
        } else {
#pragma unroll
          for (int j = 0; j < NQ; ++j) z[j] = valid ? z[j] * p.sl2e : -INFINITY;
        }
        bool mine = t == sg.t0;
        if (!mine) {
#pragma unroll
          for (int j = 0; j < NQ; ++j) mine |= z[j] > s_stat[n0 + j] + kRaise;
        }
        bool raise = false;
        if (named_bar_or(bar_id, 128, mine || bad)) {
          if (named_bar_or(bar_id, 128, bad)) { aborted = true; break; }
          raise = true;
        }
        if (raise) {
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const float wmax = reduce_keys(z[j], true);
            if ((lane & ~2) == 0) s_red[qd * NH + n0 + j] = wmax;
          }
          named_bar(bar_id, 128);
          if (qd == 0 && lane < NHH) {
            const int n = ch * NHH + lane;
            const float bm = fmaxf(fmaxf(s_red[n], s_red[NH + n]), fmaxf(s_red[2 * NH + n], s_red[3 * NH + n]));
            const float mo = s_stat[n], mn = fmaxf(mo, bm);
            s_stat[n] = mn;
            s_fac[n] = mo == -INFINITY ? 0.f : exp2f(mo - mn);
          }
          named_bar(bar_id, 128);
#pragma unroll
          for (int j = 0; j < NQ; ++j) l_part[j] *= s_fac[n0 + j];
          if (t > sg.t0) {
            bool okw = mbar_wait(bar_pv + 8 * ((i - 1) % R), ((i - 1) / R) & 1, s_abort, p.err, p.wait_limit);
            if (named_bar_or(bar_id, 128, !okw)) { aborted = true; break; }
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < (NH == 64 ? 7 : 8); ++x) {
              const uint32_t ta = tmem_addr(tmem + L::o_col(x >> 1) + (x & 1) * NH + ch * NHH, qd * 32, 0);
              uint32_t ov[NHH];
              tmem_ld_n<NHH>(ta, ov);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < NHH; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * s_fac[ch * NHH + h]);
              tmem_st_n<NHH>(ta, ov);
            }
            tmem_st_wait();
          }
        }
        uint32_t hi[NQ / 2], lo[NQ / 2];
#pragma unroll
        for (int j = 0; j < NQ; j += 2) {
          const float ma = s_stat[n0 + j], mb2 = s_stat[n0 + j + 1];
          const float pa = exp2f(z[j] - (ma == -INFINITY ? 0.f : ma));
          const float pb = exp2f(z[j + 1] - (mb2 == -INFINITY ? 0.f : mb2));
          l_part[j] += pa;
          l_part[j + 1] += pb;
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(pa, pb);
          const float2 hf = __bfloat1622float2(h2);
          hi[j / 2] = *reinterpret_cast<const uint32_t*>(&h2);
          lo[j / 2] = pack_bf16x2(pa - hf.x, pb - hf.y);
        }
        if (L::OVERLAY && i >= 1) {
          const bool okp = mbar_wait(bar_pv + 8 * ((i - 1) % R), ((i - 1) / R) & 1, s_abort, p.err, p.wait_limit);
          if (!okp) bad = true;  // (the store below then goes unused: no product is formed after an abort)
        }
        const uint32_t sP = L::p(sKV, i);
        if constexpr (NH == 64) {
          const int u0 = n0 / 8;
          st_shared_v4(sP + sw128_off(r, u0), hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(sP + sw128_off(r, u0 + 1), hi[4], hi[5], hi[6], hi[7]);
          st_shared_v4(sP + 8192 + sw128_off(r, u0), lo[0], lo[1], lo[2], lo[3]);
          st_shared_v4(sP + 8192 + sw128_off(r, u0 + 1), lo[4], lo[5], lo[6], lo[7]);
        } else {
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const int n = n0 + j;
            const uint32_t at = sP + (uint32_t)(n * 128 + (((r >> 3) ^ (n & 7)) << 4) + (r & 7) * 2);
            st_shared_u16(at, (uint16_t)(hi[j / 2] >> (16 * (j & 1))));
            st_shared_u16(at + NH * 128, (uint16_t)(lo[j / 2] >> (16 * (j & 1))));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !bad) mbar_arrive(bar_p + 8 * (i & 1));
      }
      if (!aborted) {
        const bool got = mbar_wait(bar_pv + 8 * ((i - 1) % R), ((i - 1) / R) & 1, s_abort, p.err, p.wait_limit);
        aborted = named_bar_or(bar_id, 128, !got);
        tc_fence_after();
      }
      if (aborted) break;
      // ---- the segment's rows: out and lse, or the workspace's partial sums ----
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        const float l = reduce_keys(l_part[j], false);
        if ((lane & ~2) == 0) s_red[qd * NH + n0 + j] = l;
      }
      named_bar(bar_id, 128);
      const bool whole = sg.t0 == 0 && sg.t1 == sg.T;
      const int slot = 2 * blockIdx.x + (sg.t0 == 0 ? 1 : 0);
      if (qd == 0 && lane < NHH) {
        const int n = ch * NHH + lane;
        const float l = s_red[n] + s_red[NH + n] + s_red[2 * NH + n] + s_red[3 * NH + n];
        const float m = s_stat[n];
        float fac = 1.f;
        if (whole) {
          const float s2 = (p.sink && n < sg.rows) ? __ldg(p.sink + (sg.head0 + n) % p.H) * kLog2e : -INFINITY;
          const float mf = fmaxf(m, s2), base = mf == -INFINITY ? 0.f : mf;
          const float keep = m == -INFINITY ? 1.f : exp2f(m - base);  // (no finite score: l is 0, or NaN from a NaN)
          const float lt = l * keep + exp2f(s2 - base);
          fac = lt == 0.f ? 0.f : keep / lt;
          if (n < sg.rows) p.lse[sg.row0 + n] = lt == 0.f ? -INFINITY : base * kLn2 + logf(lt);
        } else {
          p.stats[(size_t)slot * 128 + n] = m;
          p.stats[(size_t)slot * 128 + 64 + n] = l;
        }
        s_fac[n] = fac;
      }
      named_bar(bar_id, 128);
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t oh[NHH];
        const uint32_t ta = tmem_addr(tmem + L::o_col(mt) + ch * NHH, qd * 32, 0);
        tmem_ld_n<NHH>(ta, oh);
        if (NH != 64 || mt < 3) {
          uint32_t ol[NHH];
          tmem_ld_n<NHH>(ta + NH, ol);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < NHH; ++h) oh[h] = __float_as_uint(__uint_as_float(oh[h]) + __uint_as_float(ol[h]));
        } else {
          tmem_ld_wait();
        }
        const int c = mt * 128 + qd * 32 + lane;
        if (whole) {
#pragma unroll
          for (int h = 0; h < NHH; ++h) {
            const int n = ch * NHH + h;
            const float f = s_fac[n];
            if (n < sg.rows) p.out[(size_t)(sg.row0 + n) * kDv + c] = __float2bfloat16_rn(f == 0.f ? 0.f : __uint_as_float(oh[h]) * f);
          }
        } else {
#pragma unroll
          for (int h = 0; h < NHH; ++h) {
            const int n = ch * NHH + h;
            if (n < sg.rows) p.partial[((size_t)slot * 64 + n) * kDv + c] = __uint_as_float(oh[h]);
          }
        }
      }
      tc_fence_before();
      named_bar(bar_id, 128);  // s_red, s_stat and s_fac have been read
      sg = nx;
      have = more;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TM_COLS);
  }
}

// Joins the pieces of the groups that went over several CTAs: one row per half CTA at a time, 128 threads with 4
// channels each.  Pieces are read in CTA order, so the result does not depend on which came first.
__global__ void __launch_bounds__(256) paged_mla_join_kernel(const int4* __restrict__ records, int ctas,
                                                            const float* __restrict__ stats,
                                                            const float* __restrict__ partial,
                                                            const float* __restrict__ sink, int H,
                                                            __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ int4 rec[kMaxCtas];
  __shared__ int first[kMaxCtas + 1];
  for (int c = threadIdx.x; c < ctas; c += 256) rec[c] = records[c];
  __syncthreads();
  if (threadIdx.x < 32) {  // rows before each record
    int base = 0;
    for (int c0 = 0; c0 < ctas; c0 += 32) {
      const int c = c0 + threadIdx.x;
      const int v = c < ctas ? rec[c].y : 0;
      int inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if ((int)threadIdx.x >= o) inc += x;
      }
      if (c < ctas) first[c] = base + inc - v;
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (threadIdx.x == 0) first[ctas] = base;
  }
  __syncthreads();
  const int total = first[ctas];
  const int half = threadIdx.x >> 7, x = threadIdx.x & 127;
  for (int it = blockIdx.x * 2 + half; it < total; it += gridDim.x * 2) {
    int lo = 0, hi = ctas;  // last c with first[c] <= it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= it) lo = mid; else hi = mid;
    }
    const int4 rc = rec[lo];
    const int n = it - first[lo];
    const float s2 = sink ? __ldg(sink + (rc.z + n) % H) * kLog2e : -INFINITY;
    float m = s2;
    for (int c = lo; c <= rc.w; ++c) m = fmaxf(m, __ldg(stats + (size_t)(2 * c + (c == lo)) * 128 + n));
    const float base = m == -INFINITY ? 0.f : m;
    float l = exp2f(s2 - base);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = lo; c <= rc.w; ++c) {
      const int slot = 2 * c + (c == lo);
      const float f = exp2f(__ldg(stats + (size_t)slot * 128 + n) - base);
      const float4 v = __ldg(reinterpret_cast<const float4*>(partial + ((size_t)slot * 64 + n) * kDv) + x);
      l += f * __ldg(stats + (size_t)slot * 128 + 64 + n);
      o.x += f * v.x;
      o.y += f * v.y;
      o.z += f * v.z;
      o.w += f * v.w;
    }
    const bool empty = l == 0.f;  // nothing is seen, and there is no sink
    const float inv = empty ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(out + (size_t)(rc.x + n) * kDv)[x] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (x == 0) lse[rc.x + n] = empty ? -INFINITY : base * kLn2 + logf(l);
  }
}

constexpr size_t kRecordBytes = kMaxCtas * sizeof(int4);
constexpr size_t kStatBytes = (size_t)2 * kMaxCtas * 128 * sizeof(float);
constexpr size_t kPartialBytes = (size_t)2 * kMaxCtas * 64 * kDv * sizeof(float);

// SMs of the current device, at most kMaxCtas.
int cta_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n < kMaxCtas ? n : kMaxCtas;
}

template <int DQK, int NH>
dsa_status_t launch(Params& p, int ctas, cudaStream_t s) {
  using L = Smem<DQK, NH>;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_mla_kernel<DQK, NH>), L::TOTAL,
                                          "configuring paged_mla_kernel");
  if (st != DSA_OK) return st;
  p.G = p.topk_idx ? 1 : (p.H <= NH ? NH / p.H : 1);
  p.HB = (p.H + NH - 1) / NH;
  paged_mla_kernel<DQK, NH><<<ctas, kThreads, L::TOTAL, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching paged_mla_kernel");
}

}  // namespace pmla
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_paged_mla_workspace_size(void) {
  return kErrorWordBytes + pmla::kRecordBytes + pmla::kStatBytes + pmla::kPartialBytes;
}

extern "C" dsa_status_t dsa_paged_mla(const dsa_bf16_t* q, const dsa_bf16_t* cache, const int32_t* block_table,
                                      const int32_t* seq_lens, const int32_t* cu_q, const int32_t* topk_idx,
                                      const int32_t* topk_len, int32_t N, int32_t B, int32_t H, int32_t Dqk, int32_t Dv,
                                      int32_t K, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                      float softmax_scale, const float* attn_sink, dsa_bf16_t* out, float* lse,
                                      void* workspace, size_t workspace_bytes, dsa_stream_t stream) {
  const char* who = "dsa_paged_mla";
  if (N < 0 || B < 0 || H < 1 || K < 0 || num_pages < 0 || page_size < 1 || max_pages < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT,
                "%s: need N, B, K, num_pages, max_pages >= 0, H >= 1, page_size >= 1 (got %d, %d, %d, %d, %d, %d, %d)", who,
                N, B, K, num_pages, max_pages, H, page_size);
  if (Dqk != 576 && Dqk != 512) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: Dqk must be 576 or 512 (got %d)", who, Dqk);
  if (Dv != 512) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: Dv must be 512 (got %d)", who, Dv);
  if ((int64_t)N * H > 0x7fffffffll) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: N * H must be below 2^31", who);
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: softmax_scale must be finite and > 0", who);
  if (!cu_q && N != B)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: without cu_q every request has one token (N = %d, B = %d)", who, N, B);
  if ((topk_idx != nullptr) != (K > 0)) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: topk_idx and K > 0 go together", who);
  if (topk_len && !topk_idx) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: topk_len needs topk_idx", who);
  if (N > 0 && (!q || !out || !lse)) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if (B > 0 && (!seq_lens || (max_pages > 0 && !block_table) || (num_pages > 0 && !cache)))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: q, cache and out must be 16-byte aligned", who);
  dsa_status_t st = check_workspace(workspace, workspace_bytes, dsa_paged_mla_workspace_size(), who);
  if (st != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (N == 0 || B == 0) return ok();
  const int ctas = pmla::cta_count();
  if (ctas < 1) return fail(DSA_ERR_CUDA, "%s: the device's SM count cannot be read", who);
  pmla::Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.cache = reinterpret_cast<const __nv_bfloat16*>(cache);
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.topk_idx = topk_idx;
  p.topk_len = topk_len;
  p.N = N;
  p.B = B;
  p.H = H;
  p.K = K;
  p.num_pages = num_pages;
  p.P = page_size;
  p.max_pages = max_pages;
  p.sl2e = softmax_scale * pmla::kLog2e;
  p.sink = attn_sink;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  char* ws = reinterpret_cast<char*>(workspace);
  p.err = reinterpret_cast<int*>(ws);
  p.records = reinterpret_cast<int4*>(ws + kErrorWordBytes);
  p.stats = reinterpret_cast<float*>(ws + kErrorWordBytes + pmla::kRecordBytes);
  p.partial = reinterpret_cast<float*>(ws + kErrorWordBytes + pmla::kRecordBytes + pmla::kStatBytes);
  p.wait_limit = wait_limit_cycles();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // 16 columns while all rows of a request (or of a list) fit: fewer products of zero columns, a longer ring
  const int64_t rows = (int64_t)H * (topk_idx ? 1 : (N + B - 1) / B);
  if (rows <= 16) st = Dqk == 576 ? pmla::launch<576, 16>(p, ctas, s) : pmla::launch<512, 16>(p, ctas, s);
  else st = Dqk == 576 ? pmla::launch<576, 64>(p, ctas, s) : pmla::launch<512, 64>(p, ctas, s);
  if (st != DSA_OK) return st;
  pmla::paged_mla_join_kernel<<<2 * ctas, 256, 0, s>>>(p.records, ctas, p.stats, p.partial, attn_sink, H, p.out, lse);
  st = cuda_check(cudaGetLastError(), "launching paged_mla_join_kernel");
  return st == DSA_OK ? ok() : st;
}
