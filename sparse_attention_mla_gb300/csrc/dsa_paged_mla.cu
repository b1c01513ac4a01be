// dsa_paged_mla.cu -- attention of new tokens over a paged latent cache (sm_103a).
//
// For new token j of request b (n_b of them, at the end of seq_lens[b] tokens) and
// head h:  z_p = scale <q, kv_p> over the positions p it sees (its own and all
// before, or the ones of its list),  lse = ln sum e^{z_p},
// out = sum e^{z_p - lse} kv_p[0:512].  One latent row serves all heads, so the
// floor is one read of every visible row; at 64 heads the tensor core needs about
// three quarters of the time that DRAM needs for a tile (2340 of 3135 cycles).
//
// Split: the (token, head) rows of a request that share its cache are packed into
// groups of NH = 16 or 64 MMA columns; a group's positions are cut into tiles of 64,
// and the tiles of all groups, laid end to end, are cut into equal ranges, one per
// CTA (one CTA per SM); a group's end, in which no tile is copied, counts as some tiles.
// Every CTA finds its range from the lengths on the device
// (a sum over the requests), so no plan is made on the host and a captured step
// follows the lengths.  A group inside one range is finished there; the pieces of
// a group over several CTAs go to the workspace as (max, sum, unnormalised O) in
// fp32 and a second kernel joins them in a fixed order.
//
// A tile: S^T[key, row] = KV Q^T (M = 64 keys), an online softmax with a lazily
// raised maximum, O^T[channel, row] += V^T P^T (M = 128 channels), P as bf16 hi + lo
// side by side on the N axis, so that O keeps about fp32 accuracy (P in bf16 alone
// would add as much error as the output's own rounding).  Rows that follow one another
// in whole pages come by TMA, 32 rows of 64 channels a copy; lists, other page sizes and
// a request's end by 16-byte cp.async, which takes any row and zero-fills what is masked
// (no stale page, NaN included, reaches a product).
//
// Warps: 0 issues S^T, 1-8 softmax and epilogue, 9-12 copy tiles into a ring, 13
// issues P.V, 14 announces the runs of tiles (segments) that the CTA's range consists
// of.  At width 576 and NH = 64 the ring's two tiles, Q and P need all the shared
// memory: P^T lies over the tile's last chunk (positions, read only by S^T) and an
// 8 KiB block that the two tiles share.
//
// Measured: 674,000 positions of 64 requests, 64 heads, 159 us (4.9 TB/s); 131072
// positions, two tokens of 128 heads, 116 us (four groups of rows, each reading the cache,
// three times of four from L2); 48 lists of 2048 rows 55 us; 1000 positions, 16 heads, 13 us.
// What bounds it: a tile passes its copy (1350 cycles, as fast as an SM takes one), S^T
// (1700), the softmax (1600) and P.V (1200) one after the other, and shared memory holds two,
// so that a tile takes 3600 cycles; the start (from the launch to the first softmax 6 us in the call of 1000
// positions, 9 to 13 in the others), the end of a group and the join (3 us after the last CTA in that call, 6 to 10 in the
// others) come on top.
#include <climits>
#include <cmath>

#include "dsa_f32x2.cuh"
#include "dsa_paged_groups.cuh"

namespace dsa {
namespace pmla {

using namespace pgroups;

constexpr int kTile = 64;
constexpr int kWorkers = 256;
constexpr int kGather = 128;
constexpr int kThreads = 32 + kWorkers + kGather + 64;
constexpr float kRaise = 8.0f;  // log2 units: the running maximum is raised only past this

template <int DQK, int NH>
struct Smem {
  static constexpr int NCH = DQK / 64;
  static constexpr int CHUNK = kTile * 128;
  static constexpr int Q_CHUNK = NH * 128;
  // P over the ring only where nothing else fits
  static constexpr bool OVERLAY = NH == 64 && DQK == 576;
  static constexpr int R = 2;  // tiles in the ring
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
  // of the matrix descriptors (16-byte units): from chunk to chunk, from slot to slot
  static constexpr int STEP = CHUNK >> 4, SLOT = (OVERLAY ? 11 : NCH) * STEP;
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

// misc (bytes).  A tile's chunks land in groups of three, each with its own barrier (S^T starts on the first), and are
// given back in pairs as P.V reads them.
constexpr int kLand = 3, kGroups = 3, kPairs = 4;
constexpr int M_KV = 0, M_PV = 48, M_S = 112, M_SF = 128, M_P = 144, M_Q = 160, M_FIN = 168;  // [2][3] [2][4] [2] [2] [2] 1 [2]
constexpr int M_SEGF = 184, M_SEGE = M_SEGF + 8 * kSegs;  // [kSegs] each: announced, read by all
constexpr int M_TMEM = 312, M_ABORT = 316, M_PLAN = 320;  // plan: 56 bytes
constexpr int M_VALID = 376;                  // uint8 [2][64]
constexpr int M_SEG = 512;                    // int4 [kSegs][2]
constexpr int M_RED = 768;                    // float [4][64]; the first row also holds the factors of a rescale
constexpr int M_STAT = M_RED + 1024;          // float [64]
static_assert(M_SEGE + 8 * kSegs <= M_TMEM && M_VALID + 128 <= M_SEG && M_SEG + 32 * kSegs <= M_RED && M_STAT + 256 <= 2048,
              "misc layout");

struct Params : GroupParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* cache;
  int box;  // rows of a TMA box (32 or a smaller page), 0: every row by cp.async
  float sl2e;
};

// A latent's 512 channels in shared memory (its 128 bytes of the first chunk at `at`): values that are not finite become 0.
// (A function of its own, for the same reason as read_announcement.)
__device__ __noinline__ void zero_not_finite(uint32_t at, uint32_t landed, uint32_t parity) {
  if (!mbar_test(landed, parity) || !mbar_test(landed + 8, parity)) return;  // (they have long landed: orders what is read here)
#pragma unroll 1
  for (int x = 0; x < kDv / 8; ++x, at += (x & 7) ? 16 : kTile * 128 - 112) {
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
    bool found = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool lo = (v[k] & 0x7f80u) == 0x7f80u, hi = (v[k] & 0x7f800000u) == 0x7f800000u;
      found |= lo || hi;
      v[k] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
    }
    if (found) st_shared_v4(at, v[0], v[1], v[2], v[3]);
  }
}

constexpr int kReaders = 2 + kWorkers / 32 + kGather / 32;  // warps that read an announcement

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
template <int DQK, int NH>
__global__ void __launch_bounds__(kThreads, 1) paged_mla_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map) {
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
  float* s_fac = reinterpret_cast<float*>(misc + M_RED);  // a column's factor replaces its first maximum or sum
  float* s_red = reinterpret_cast<float*>(misc + M_RED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // tile i: group g of its chunks has landed; P.V has read pair m of its channels (3: all of it)
  auto wait_kv = [&](int i, int g) {
    return wait_for(bar_kv + 8 * ((i % R) * kGroups + g), (i / R) & 1, s_abort, p.wait_limit);
  };
  auto wait_pv = [&](int i, int m) {
    return wait_for(bar_pv + 8 * ((i % R) * kPairs + m), (i / R) & 1, s_abort, p.wait_limit);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      for (int g = 0; g < kGroups; ++g) mbar_init(bar_kv + 8 * (s * kGroups + g), 2);  // the slot's two gather warps
      for (int m = 0; m < kPairs; ++m) mbar_init(bar_pv + 8 * (s * kPairs + m), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_s + 8 * b, 1);
      mbar_init(bar_sf + 8 * b, 8);
      mbar_init(bar_p + 8 * b, 8);
      mbar_init(bar_fin + 8 * b, 1);
    }
    mbar_init(bar_q, kWorkers);
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(mb + M_SEGF + 8 * k, 1);
      mbar_init(mb + M_SEGE + 8 * k, kReaders);
    }
    if (p.box > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    *s_abort = 0;
    fence_mbar_init();
  }
  make_plan<kTile, kThreads>(p, s_plan, reinterpret_cast<long long*>(s_red));
  const Plan plan = *s_plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the joining kernel waits for this one's end itself)
  if (plan.w1 <= plan.w0 || plan.w1 - plan.w0 <= plan.skip) return;  // (the whole CTA)
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), L::TM_COLS);
    tmem_relinquish();
  }
  uint32_t tmem = 0;
  if (warp <= 8 || warp == 13) {  // the others neither need it nor wait for it
    named_bar(3, 320);
    tmem = (uint32_t)warp_value((int)*s_tmem);
  }

  // announcement k, once per warp
  auto read_seg = [&](int k, Seg& s) -> bool {
    return read_announcement(mb + M_SEGF, mb + M_SEGE, reinterpret_cast<const int4*>(misc + M_SEG), k, s_abort, p.wait_limit, s);
  };
  if (warp == 0) {
    // ======================= S^T issuer =======================
    constexpr uint32_t kIdS = idesc_bf16(kTile, NH, false, false);
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      if (!warp_all(wait_for(bar_q, seg & 1, s_abort, p.wait_limit))) break;
      fence_proxy_async_smem();  // (the queries came by cp.async)
      // what the loop needs in registers of the warp (a call does not keep them)
      const int n = warp_value(sg.n);
      const uint32_t d0 = (uint32_t)warp_value((int)tmem), q0 = (uint32_t)warp_value((int)sQ), kv0 = (uint32_t)warp_value((int)sKV);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const int sl = i % R, sb = i % NS;
        if (i >= NS && !warp_all(wait_for(bar_sf + 8 * sb, ((i / NS) - 1) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        // the chunks' descriptors by constant steps from the tile's (chunk 8 lies elsewhere in the overlaid ring)
        const uint64_t a0 = sdesc_sw128(kv0, 16, 1024) + (uint64_t)(uint32_t)(sl * L::SLOT);
        const uint64_t a8 = sdesc_sw128(kv0, 16, 1024) + (uint64_t)(uint32_t)((L::OVERLAY ? (sl ? 10 : 8) * L::STEP : sl * L::SLOT + 8 * L::STEP));
        const uint64_t b0 = sdesc_sw128(q0, 16, 1024);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if (c % kLand == 0) {
            if (!warp_all(wait_kv(i, c / kLand))) { stop = true; break; }
            tc_fence_after();
          }
          mma4_w<2, 2>(d0 + sb * NH, c == 8 ? a8 : a0 + c * L::STEP, b0 + c * (L::Q_CHUNK >> 4), kIdS, c);
        }
        if (stop) break;
        mma_commit_w(bar_s + 8 * sb);
      }
      if (stop) break;
    }
    mma_commit_w(bar_fin);
    volatile int dummy = 0;
    mbar_wait(bar_fin, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 13) {
    // ======================= P.V issuer =======================
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      const int n = warp_value(sg.n);
      const uint32_t d0 = (uint32_t)warp_value((int)tmem), kv0 = (uint32_t)warp_value((int)sKV);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const int sl = i % R;
        const uint32_t add = k0 > 0;  // the segment's first tile overwrites O^T
        if (!warp_all(wait_for(bar_p + 8 * (i & 1), (i >> 1) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        tc_fence_after();
        const uint64_t va = sdesc_sw128(L::chunk(kv0, sl, 0), L::CHUNK, 1024);
        constexpr uint64_t kPair = (2 * L::CHUNK) >> 4;
        const uint32_t sP = L::p(kv0, i);
        if constexpr (NH == 64) {  // P^T rows are keys (MN-major), hi and lo blocks of 64 rows' columns 8 KiB apart
          constexpr uint32_t kId2 = idesc_bf16(128, 128, true, true), kId1 = idesc_bf16(128, 64, true, true);
          const uint64_t pb = sdesc_sw128(sP, 8192, 1024);
#pragma unroll 1
          for (int s = 0; s < 5; ++s) {  // channel tiles 0-2, tile 3 with hi, tile 3 with lo
            const int m = min(s, 3);
            const uint32_t id = s < 3 ? kId2 : kId1, on = add | (s == 4);
            const uint64_t a = va + m * kPair, b = pb + (s == 4 ? 512 : 0);
            mma4_w<128, 128>(d0 + L::o_col(m), a, b, id, on);
            if (s != 3) mma_commit_w(bar_pv + 8 * (sl * kPairs + m));
          }
        } else {  // P^T rows are [hi rows | lo rows], keys along K
          constexpr uint32_t kId = idesc_bf16(128, 2 * NH, true, false);
          const uint64_t pb = sdesc_sw128(sP, 16, 1024);
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            mma4_w<128, 2>(d0 + L::o_col(m), va + m * kPair, pb, kId, add);
            mma_commit_w(bar_pv + 8 * (sl * kPairs + m));
          }
        }
      }
      if (stop) break;
    }
    mma_commit_w(bar_fin + 8);
    volatile int dummy = 0;
    mbar_wait(bar_fin + 8, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 14) {
    announce<kTile>(p, plan, mb + M_SEGF, mb + M_SEGE, reinterpret_cast<int4*>(misc + M_SEG), s_abort);
  } else if (warp >= 9) {
    // ======================= gather: two warps per slot of the ring, 32 rows of a tile each =======================
    // A lane looks one row up, in steps whose loads have a tile of the slot to come back: the list's entry (three tiles
    // of the slot ahead), the page (two ahead), the row number (one ahead).  Whole rows of whole pages come by TMA (one
    // lane issues a box of 64 channels; it needs no thread while it lands and no fence before the tensor core reads
    // it); lists, odd page sizes and the end of a request by 16-byte cp.async, which zero-fills what is masked.
    const int sl = (warp - 9) >> 1, gw = (warp - 9) & 1, uc = lane & 7;
    Seg sg;
    int seg = 0, base = 0, end = 0, limit = 0;  // this CTA's tiles [base, end) are the segment's
    int n_tiles = INT_MAX;                      // this CTA's tiles, known once one past them has been looked for
    struct Look {
      int pos, b, limit;  // position (then its place in the page), or -1; request; what the position has to stay below
    };
    bool bad_index = false, stop = false;
    auto position = [&](int i) -> Look {
      Look k{-1, 0, 0};
      if (i < n_tiles && !stop) {
#pragma unroll 1
        while (i >= end) {
          if (seg > 0 && sg.last) { n_tiles = end; return k; }
          if (!read_seg(seg, sg)) { stop = true; return k; }
          ++seg;
          base = end;
          end += sg.n;
          limit = (int)min((long long)p.max_pages * p.P, (long long)(p.topk_idx ? sg.seen0 : sg.keys));
        }
        k.b = sg.b;
        k.limit = limit;
        const int j = (sg.t0 + i - base) * kTile + gw * 32 + lane;
        if (j < sg.keys) k.pos = p.topk_idx ? __ldg(p.topk_idx + (size_t)(sg.row0 / p.H) * p.K + j) : j;
      }
      return k;
    };
    auto page_of = [&](Look& k) -> int {
      if (k.pos < -1 || k.pos >= k.limit) {
        bad_index |= k.pos != -1;
        k.pos = -1;
      }
      if (k.pos < 0) return -1;
      const unsigned at = (unsigned)k.pos / (unsigned)p.P;
      k.pos -= (int)at * p.P;
      return __ldg(p.table + (size_t)k.b * p.max_pages + at);
    };
    auto row_of = [&](int pos, int page) -> long long {
      if (pos < 0) return -1;
      if (page >= 0 && page < p.num_pages) return (long long)page * p.P + pos;
      bad_index = true;
      return -1;
    };
    Look look[3];
    int page[2];
    long long row[2];  // rows of the slot's next two tiles
#pragma unroll
    for (int k = 0; k < 3; ++k) look[k] = position(sl + k * R);
    page[0] = page_of(look[0]);
    page[1] = page_of(look[1]);
    row[0] = row_of(look[0].pos, page[0]);
    row[1] = row_of(look[1].pos, page[1]);
    look[0] = look[2];
    page[0] = page_of(look[0]);
    look[1] = position(sl + 3 * R);
    // where this warp's rows of the slot go (chunk 8 apart), and the slot's barriers
    const uint32_t land = (uint32_t)warp_value((int)(L::chunk(sKV, sl, 0) + gw * 4096));
    const uint32_t land8 = (uint32_t)warp_value((int)(L::chunk(sKV, sl, NCH - 1) + gw * 4096));
    const uint32_t landed_bar = (uint32_t)warp_value((int)(bar_kv + 8 * sl * kGroups));
    int armed = -1, next = sl;  // the slot's last tile that this warp has answered for, and the one after it
#pragma unroll 1
    for (int i = sl; i < n_tiles && !stop; i += R) {
      const long long row_d = row[0];
      // the chunks of pair m (with the last, the ninth too) are free
      auto slot_free = [&](int m) { return i < R || warp_all(wait_pv(i - R, m)); };
      // all 32 rows are there, in whole boxes
      if (p.box > 0 && __all_sync(0xffffffffu, row_d >= 0)) {
        const int boxes = 32 / p.box;
#pragma unroll 1
        for (int m = 0; m < kPairs; ++m) {
          // (a tile once begun is issued to its end: what is on its way can then be waited for)
          if (!stop && !slot_free(m)) {
            stop = true;
            if (m == 0) break;
          }
          if (m == 0) {
            s_valid[sl * kTile + gw * 32 + lane] = 1;
            __syncwarp();
            if (lane < kGroups) mbar_expect_tx(bar_kv + 8 * (sl * kGroups + lane), min(kLand, NCH - kLand * lane) * 4096);
            __syncwarp();
          }
#pragma unroll 1
          for (int bx = 0; bx < boxes; ++bx) {
            const int at = warp_value((int)__shfl_sync(0xffffffffu, row_d, (bx * p.box) & 31));
            const uint32_t to = land + bx * p.box * 128;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              tma_load_2d_w(to + (2 * m + x) * L::CHUNK, &map, (2 * m + x) * 64, at, landed_bar + 8 * ((2 * m + x) / kLand));
            if (NCH == 9 && m == 3) tma_load_2d_w(land8 + bx * p.box * 128, &map, 512, at, landed_bar + 16);
          }
          armed = i;
          next = i + R;
        }
        if (stop) break;
        // the slot's next tile on its way to L2 (the ring's room bounds what can be on its way to the SM)
        if (__all_sync(0xffffffffu, row[1] >= 0)) {
#pragma unroll 1
          for (int bx = 0; bx < boxes; ++bx) {
            const int at = warp_value((int)__shfl_sync(0xffffffffu, row[1], (bx * p.box) & 31));
#pragma unroll
            for (int c = 0; c < NCH; ++c) tma_prefetch_2d_w(&map, c * 64, at);
          }
        }
      } else {
        const __nv_bfloat16* src[8];
        uint32_t ok = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const long long at = __shfl_sync(0xffffffffu, row_d, e * 4 + (lane >> 3));
          ok |= (at >= 0 ? 1u : 0u) << e;
          src[e] = p.cache + (at >= 0 ? (size_t)at * DQK + uc * 8 : 0);
        }
#pragma unroll 1
        for (int c = 0; c < NCH; ++c) {
          if ((c & 1) == 0 && c < 8 && !slot_free(c >> 1)) { stop = true; break; }
          if (c == 0) s_valid[sl * kTile + gw * 32 + lane] = row_d >= 0 ? 1 : 0;
          const uint32_t dst = L::chunk(sKV, sl, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool on = (ok >> e) & 1u;
            cp_async16(dst + sw128_off(gw * 32 + e * 4 + (lane >> 3), uc), src[e] + (on ? c * 64 : 0), on ? 16u : 0u);
          }
          if (c % kLand == kLand - 1 || c == NCH - 1) asm volatile("cp.async.commit_group;" ::: "memory");
        }
        if (stop) break;
        // landings in order
        auto landed = [&](int g) {
          fence_proxy_async_smem();  // the copies -> visible to the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_kv + 8 * (sl * kGroups + g));
        };
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        landed(0);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        landed(1);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        landed(2);
        armed = i;
        next = i + R;
      }
      row[0] = row[1];
      row[1] = row_of(look[0].pos, page[0]);
      look[0] = look[1];
      page[0] = page_of(look[0]);
      look[1] = position(i + 4 * R);
    }
    if (bad_index) record_error(p.err, DSA_ERR_DEVICE_INDEX);
    asm volatile("cp.async.wait_all;" ::: "memory");
    // Nothing lands after the CTA has left: the slot's last tile is waited for, and where the wait for room ran out, the
    // other warp of the slot, which may have begun the next one, gets this warp's part of it.
    volatile int dummy = 0;
    if (armed >= 0)
      for (int g = 0; g < kGroups; ++g) mbar_wait(bar_kv + 8 * (sl * kGroups + g), (armed / R) & 1, &dummy, p.err);
    __syncwarp();
    if (next < n_tiles && lane < kGroups) mbar_arrive(bar_kv + 8 * (sl * kGroups + lane));
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
#pragma unroll 2
      for (int x = tid; x < UNITS; x += kWorkers) {
        const int hh = x / (NCH * 8), rem = x - hh * (NCH * 8), c = rem >> 3, uc = rem & 7;
        const bool ok = hh < s.rows;
        cp_async16_hint(sQ + c * L::Q_CHUNK + sw128_off(hh, uc),
                        p.q + (ok ? (size_t)(s.row0 + hh) * DQK + c * 64 + uc * 8 : 0), ok ? 16u : 0u, pol);
      }
      cp_async_arrive(bar_q);
    };
    // Maxima or sums over the warp's 16 keys of all NQ rows of a thread: the result is that of row sum_row.
    auto over_keys = [&](float (&v)[NQ], bool is_max) -> float {
      constexpr int kBit[4] = {16, 8, 4, 1};  // the lanes of one parity
      int w = 8;
#pragma unroll
      for (int s = 0; s < 4; ++s, w >>= 1) {
        const bool upper = (lane & kBit[s]) != 0;
        if (w >= NQ) {
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const float x = __shfl_xor_sync(0xffffffffu, v[j], kBit[s]);
            v[j] = is_max ? fmaxf(v[j], x) : v[j] + x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < w; ++j) {
            const float send = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
            const float x = __shfl_xor_sync(0xffffffffu, send, kBit[s]);
            v[j] = is_max ? fmaxf(keep, x) : keep + x;
          }
        }
      }
      return v[0];
    };
    const int sum_row = n0 + (((lane >> 1) & 14) | (lane & 1)) % NQ;
    Seg sg, nx;
    // (one answer for the half: its warps meet at barriers from here on)
    bool aborted = named_bar_or(bar_id, 128, !read_seg(0, sg));
    if (!aborted) load_q(sg);
    nx = sg;
    int i = 0;
    for (int seg = 1; !aborted; ++seg) {
      const bool more = !sg.last;
      bool bad_seg = more && !read_seg(seg, nx);
      // this thread's first row: its token in the group, and how many rows of that token there are from it on
      const int tok0 = (sg.head0 + n0) / p.H, head_left = p.H - ((sg.head0 + n0) - tok0 * p.H);
      // sums and minus the running maxima (log2 units) of this thread's rows, in pairs; a row without a finite score yet
      // has a maximum of -3e38, which any finite score passes and which leaves e^-inf at 0
      float2 l_part[NQ / 2], m_neg[NQ / 2];
#pragma unroll
      for (int j = 0; j < NQ / 2; ++j) { l_part[j] = make_float2(0.f, 0.f); m_neg[j] = make_float2(3.0e38f, 3.0e38f); }
      if (qd == 0 && lane < NHH) s_stat[ch * NHH + lane] = -INFINITY;  // (read only after a barrier of the half)
      const int t_end = sg.t0 + sg.n;
#pragma unroll 1
      for (int t = sg.t0; t < t_end; ++t, ++i) {
        const int sl = i % R, sb = i % NS;
        bool bad = bad_seg || !wait_for(bar_s + 8 * sb, (i / NS) & 1, s_abort, p.wait_limit);
        // (complete since before S^T was issued: orders the row flags before their reads below)
        bad = bad || !wait_kv(i, kGroups - 1);
        // with its own buffers, P of tile i overwrites what P.V of tile i - 2 read
        if (!L::OVERLAY && i >= 2) bad = bad || !wait_pv(i - 2, 3);
        tc_fence_after();
        uint32_t raw[NQ];
        tmem_ld16x64b<NQ>(tmem_addr(tmem + sb * NH + ch * NHH, qd * 32, 0), raw);
        const bool valid = s_valid[sl * kTile + r] != 0;
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf + 8 * sb);
        if (t + 1 == t_end && more && !bad) load_q(nx);  // S^T of the segment is done: Q is free
        // alternate columns of the half -> NQ consecutive rows: swap half of them with the key's other thread
        float z[NQ];
#pragma unroll
        for (int j = 0; j < NQ / 2; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, par ? raw[j] : raw[NQ / 2 + j], 2);
          z[2 * j] = __uint_as_float(par ? got : raw[j]);
          z[2 * j + 1] = __uint_as_float(par ? raw[NQ / 2 + j] : got);
        }
        const int pos = t * kTile + r;
        if (!valid) {
#pragma unroll
          for (int j = 0; j < NQ; ++j) z[j] = -INFINITY;
        } else if (p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0) {  // some token may not see all of it
          // The rows share the latent, and a weight of 0 times an infinity is NaN: where a token does not see this position,
          // what is not finite in its channels becomes 0 before P.V.  (Any row's score tells: with such a latent all are
          // infinite or NaN.  A row that sees it has NaN for its weight then, unless its score is -inf.)
          if (pos >= sg.seen0 && !(fabsf(z[0]) < INFINITY))
            zero_not_finite(L::chunk(sKV, sl, 0) + (uint32_t)r * 128, bar_kv + 8 * (sl * kGroups), (i / R) & 1);
          int seen = sg.seen0 + tok0, left = head_left;
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            if (pos >= seen) z[j] = -INFINITY;
            if (--left == 0) { left = p.H; ++seen; }
          }
        }
        // the exponents; a score may pass its row's maximum by the threshold
        const float2 scale = make_float2(p.sl2e, p.sl2e);
        float2 e[NQ / 2];
        bool mine = t == sg.t0;
#pragma unroll
        for (int j = 0; j < NQ / 2; ++j) {
          e[j] = fma2(make_float2(z[2 * j], z[2 * j + 1]), scale, m_neg[j]);
          mine |= e[j].x > kRaise || e[j].y > kRaise;
        }
        bool raise = false;
        if (named_bar_or(bar_id, 128, mine || bad)) {
          if (named_bar_or(bar_id, 128, bad)) { aborted = true; break; }
          raise = true;
        }
        if (raise) {
          float top[NQ];
#pragma unroll
          for (int j = 0; j < NQ; ++j) top[j] = z[j];
          s_red[qd * NH + sum_row] = over_keys(top, true) * p.sl2e;
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
          for (int j = 0; j < NQ / 2; ++j) {
            l_part[j] = mul2(l_part[j], make_float2(s_fac[n0 + 2 * j], s_fac[n0 + 2 * j + 1]));
            m_neg[j] = make_float2(-fmaxf(s_stat[n0 + 2 * j], -3.0e38f), -fmaxf(s_stat[n0 + 2 * j + 1], -3.0e38f));
            e[j] = fma2(make_float2(z[2 * j], z[2 * j + 1]), scale, m_neg[j]);
          }
          if (t > sg.t0) {
            const bool okw = wait_pv(i - 1, 3);
            if (named_bar_or(bar_id, 128, !okw)) { aborted = true; break; }
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < (NH == 64 ? 7 : 8) * (NHH / 8); ++x) {  // 8 columns at a time
              const int part = x / (NHH / 8), h0 = ch * NHH + (x % (NHH / 8)) * 8;
              const uint32_t ta = tmem_addr(tmem + L::o_col(part >> 1) + (part & 1) * NH + h0, qd * 32, 0);
              uint32_t ov[8];
              tmem_ld8(ta, ov);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 8; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * s_fac[h0 + h]);
              tmem_st8(ta, ov);
            }
            tmem_st_wait();
          }
        }
        uint32_t hi[NQ / 2], lo[NQ / 2];
#pragma unroll
        for (int j = 0; j < NQ / 2; ++j) {
          const float2 w = make_float2(ex2(e[j].x), ex2(e[j].y));
          l_part[j] = add2(l_part[j], w);
          hi[j] = pack_bf16x2(w.x, w.y);
          const float2 rest = add2(w, make_float2(__uint_as_float((hi[j] << 16) ^ 0x80000000u),
                                                  __uint_as_float((hi[j] & 0xffff0000u) ^ 0x80000000u)));
          lo[j] = pack_bf16x2(rest.x, rest.y);
        }
        if (L::OVERLAY && i >= 1) {
          if (!wait_pv(i - 1, 3)) bad = true;  // (the store below then goes unused: no product is formed after an abort)
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
      if (aborted) break;
      // ---- the segment's rows: out and lse, or the workspace's partial sums ----
      float sums[NQ];
#pragma unroll
      for (int j = 0; j < NQ / 2; ++j) { sums[2 * j] = l_part[j].x; sums[2 * j + 1] = l_part[j].y; }
      named_bar(bar_id, 128);  // the factors of a rescale in the last tile have been read (the sums take their place)
      s_red[qd * NH + sum_row] = over_keys(sums, false);
      named_bar(bar_id, 128);
      const bool whole = sg.whole;
      const int slot = 2 * blockIdx.x + (sg.opens ? 1 : 0);
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
      const bool got = wait_pv(i - 1, 3);  // (the sums above while the last P.V is under way)
      aborted = named_bar_or(bar_id, 128, !got);
      if (aborted) break;
      tc_fence_after();
      // a few rows of 32 channels at a time, in a loop: unrolled, this code is longer than the time it takes to fetch it
      constexpr int kStep = NHH < 16 ? NHH : 16;
#pragma unroll 1
      for (int x = 0; x < 4 * NHH / kStep; ++x) {
        const int mt = x / (NHH / kStep), h0 = ch * NHH + (x % (NHH / kStep)) * kStep;
        uint32_t oh[kStep], ol[kStep];
        const uint32_t ta = tmem_addr(tmem + L::o_col(mt) + h0, qd * 32, 0);
        const bool split = NH != 64 || mt < 3;
        const uint32_t tl = split ? ta + NH : ta;  // (the last tile's hi and lo are one sum)
        if constexpr (kStep == 16) {
          tmem_ld16(ta, oh);
          tmem_ld16(tl, ol);
        } else {
          tmem_ld8(ta, oh);
          tmem_ld8(tl, ol);
        }
        tmem_ld_wait();
        const int c = mt * 128 + qd * 32 + lane, rows = sg.rows - h0;
        float o[kStep];
#pragma unroll
        for (int h = 0; h < kStep; ++h) o[h] = __uint_as_float(oh[h]) + (split ? __uint_as_float(ol[h]) : 0.f);
        // (one branch for all rows: with one for each, every store waits for the one before, 66 cycles in place of 5)
        if (whole) {
          __nv_bfloat16* dst = p.out + (size_t)(sg.row0 + h0) * kDv + c;
          float f[kStep];
#pragma unroll
          for (int h = 0; h < kStep; ++h) f[h] = s_fac[h0 + h];
#pragma unroll
          for (int h = 0; h < kStep; ++h)
            if (h < rows) dst[h * kDv] = __float2bfloat16_rn(f[h] == 0.f ? 0.f : o[h] * f[h]);
        } else {
          float* part = p.partial + ((size_t)slot * 64 + h0) * kDv + c;
#pragma unroll
          for (int h = 0; h < kStep; ++h)
            if (h < rows) part[h * kDv] = o[h];
        }
      }
      tc_fence_before();
      named_bar(bar_id, 128);  // s_red, s_stat and s_fac have been read
      if (!more) break;
      sg = nx;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TM_COLS);
    if (lane == 0 && *s_abort) record_error(p.err, DSA_ERR_TIMEOUT);
  }
}

template <int DQK, int NH>
dsa_status_t launch(Params& p, const CUtensorMap& map, int ctas, cudaStream_t s) {
  using L = Smem<DQK, NH>;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_mla_kernel<DQK, NH>), L::TOTAL,
                                          "configuring paged_mla_kernel");
  if (st != DSA_OK) return st;
  p.G = p.topk_idx ? 1 : (p.H <= NH ? NH / p.H : 1);
  // a group's end takes 15,000 cycles: 4 tiles of whole pages, 2 of listed rows (100 requests of 3000: 72 us, 80 when the
  // ends count for nothing; 48 lists of 2048: 55.4 and 57.5)
  p.extra = p.topk_idx ? 2 : 4;
  p.HB = (p.H + NH - 1) / NH;
  paged_mla_kernel<DQK, NH><<<ctas, kThreads, L::TOTAL, s>>>(p, map);
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
  // (lists of no tokens have no address)
  if (topk_idx ? K == 0 : K > 0 && N > 0)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: topk_idx and K > 0 go together", who);
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
  // rows that follow one another in the cache, 32 or a whole page of them at a time
  p.box = 0;
  CUtensorMap map{};
  if (!topk_idx && num_pages > 0 && (page_size % 32 == 0 || 32 % page_size == 0) && page_size >= 8 &&
      (int64_t)num_pages * page_size <= 0x7fffffffll) {
    p.box = page_size < 32 ? page_size : 32;
    if ((st = make_map_2d_bf16(&map, cache, (uint64_t)num_pages * page_size, Dqk, Dqk, 64, p.box)) != DSA_OK) return st;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // 16 columns where a request has no more rows on the average (or a list): fewer products of zero columns, a longer ring
  const int64_t rows = (int64_t)H * (topk_idx ? 1 : (N + B - 1) / B);
  if (rows <= 16) st = Dqk == 576 ? pmla::launch<576, 16>(p, map, ctas, s) : pmla::launch<512, 16>(p, map, ctas, s);
  else st = Dqk == 576 ? pmla::launch<576, 64>(p, map, ctas, s) : pmla::launch<512, 64>(p, map, ctas, s);
  if (st != DSA_OK) return st;
  st = pmla::launch_join(p, ctas, s);
  return st == DSA_OK ? ok() : st;
}
