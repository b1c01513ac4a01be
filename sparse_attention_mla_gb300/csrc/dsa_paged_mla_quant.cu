// dsa_paged_mla_quant.cu -- attention of new tokens over a paged cache of quantised latents (sm_103a).
//
// For new token j of request b and head h:  z_p = scale <q, kv_p> over the positions p it sees,
// lse = ln sum e^{z_p},  out = sum e^{z_p - lse} kv_p[0:512],  kv_p = v_p s_p with v_p = code (8 bits) or code * block
// (4 bits) for the first 512 channels and s_p the row's scale.
//
// What a code stands for without s is exact in fp16 (4 or 6 bits between 2^-10 and 2688), so the products run in fp16
// and s stays outside of them: z_p = s_p <q, v_p> + <q', kv'_p>, with the position channels' part in bf16, divided by
// s_p (a power of two); and the output sums the weights w_p = e^{z_p} s_p.  The running maximum is that of w, not of
// e^{z}: w in fp16 (11 bits, 2^15 down to 2^-24 around a maximum of 2^7) then loses nothing that counts, whatever the
// rows' scales are.  The denominator adds w_p / s_p in fp32.  A query row is divided by a power of two so that its
// largest channel lies in [2^14, 2^15): the channels that this takes out of fp16 are below 2^-38 of that one.
//
// Split of the work as in dsa_paged_groups.cuh, with tiles of 128 positions and groups of NH = 16 or 64 columns.
// A tile: 16 warps take the codes from global memory to registers (their loads run a tile ahead of them), form fp16
// and write it twice: to TMEM, position by lane, as the A operand of S^T[position, column] = V Q^T, and to shared memory
// as the A operand of O^T[channel, column] += V^T W^T, 128 channels at a time as P.V of the tile before is done
// with them.  Then the same warps do the softmax, a position a thread.  In this way shared memory, whose 128 bytes a
// cycle are what the whole thing runs into, sees a latent written once and read once: 131 KB each for a tile, and 74 KB
// of Q, 66 KB of W, 131 KB / 4 ... of codes not at all.
//
// Warps: 0-15 convert, softmax, epilogue; 16 issues S^T, 17 P.V, 18 announces the runs of tiles, 19 looks rows up.
#include <climits>
#include <cmath>

#include "dsa_f32x2.cuh"
#include "dsa_paged_groups.cuh"
#include "dsa_paged_quant.cuh"

namespace dsa {
namespace pmlaq {

using namespace pgroups;

constexpr int kTile = 128;
constexpr int kWarps = 16;  // that convert and do the softmax
constexpr int kThreads = 32 * (kWarps + 4);
constexpr int kReaders = kWarps + 3;  // warps that read an announcement
constexpr int kRing = 4;              // tiles whose rows are looked up ahead
constexpr float kRaise = 15.0f;       // log2 units: the running maximum is raised when a weight passes 2^15
constexpr float kTop = 7.0f;          // a new maximum is 2^7
constexpr float kLeast = 3.5527136788005009e-15f;  // 2^-48, the least s

template <int DQK, int NH>
struct Smem {
  static constexpr bool kRope = DQK == 576;
  static constexpr int CHUNK = kTile * 128;    // 64 channels of a tile
  static constexpr int Q_CHUNK = NH * 128;
  static constexpr int OFF_Q = 8 * CHUNK;
  static constexpr int OFF_P = OFF_Q + (kRope ? 9 : 8) * Q_CHUNK;
  static constexpr int OFF_MISC = OFF_P + kTile * NH * 2;
  static constexpr int MISC = 8192;
  static constexpr int TOTAL = OFF_MISC + MISC + 1024;  // + alignment slack
  static_assert(TOTAL <= 232448, "shared memory budget");
  // TMEM columns: O^T, S^T, the position channels and the slots of 128 channels of the A operand
  static constexpr int TM_S = 4 * NH, TM_R = TM_S + (NH < 32 ? 32 : NH), TM_A = TM_R + 32;
  static constexpr int SLOTS = NH == 64 ? 2 : 4;
  static_assert(TM_A + SLOTS * 64 <= 512, "TMEM budget");
};

// misc (bytes)
constexpr int M_LAND = 0;      // [5]: position channels, then 128 channels each: converted by all warps
constexpr int M_PV = 40;       // [4]: P.V is done with 128 channels
constexpr int M_A = 72;        // [2]: S^T is done with a slot
constexpr int M_S = 88, M_P = 96, M_Q = 104, M_FIN = 112;  // 1, 1, 1, [2]
constexpr int M_ROWF = 128, M_ROWE = 160;                   // [kRing] each
constexpr int M_SEGF = 192, M_SEGE = 256;                   // [kSegs] each
constexpr int M_TMEM = 320, M_ABORT = 324, M_PLAN = 328;    // plan: 56 bytes
constexpr int M_SEG = 384;                                  // int4 [kSegs][2]
constexpr int M_COL = 640;                                  // float [2][64]: a column's factor of the score, by run
constexpr int M_NEG = 1152;                                 // float [64]: minus the running maxima
constexpr int M_RED = 1408;                                 // float [4][64]; the first row also holds the factors of a rescale
constexpr int M_STAT = 2432;                                // float [64]
constexpr int M_SCALE = 2688;                               // float [2][128]: s of a tile's rows, -1: masked
constexpr int M_ROW = 3712;                                 // long long [kRing][128]: where the rows lie, -1: masked
static_assert(M_SEGE + 8 * kSegs <= M_TMEM && M_PLAN + 56 <= M_SEG && M_ROW + kRing * kTile * 8 <= 8192, "misc layout");

struct Params : GroupParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  float sl2e;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));  // A and B format: fp16
}

// 16 TMEM lanes x 256 bits, N times: thread t of the warp gives lane t / 4 (registers 4j, 4j + 1) and lane t / 4 + 8 (4j + 2,
// 4j + 3) the columns 8j + 2 (t % 4) and the next one.
__device__ __forceinline__ void tmem_st16x256b(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st16x256b(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(a, r);
  } else {
    static_assert(N == 4, "columns of a thread");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_st16(a, r);
  else asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Four MMAs on consecutive 16-element steps of K, A in TMEM (8 columns a step), issued by one elected lane (as mma4_w).
template <int SB>
__device__ __forceinline__ void mma4_ts_w(uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add_first) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, %5;\n\tadd.s64 b2, %2, %6;\n\tadd.s64 b3, %2, %7;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(idesc), "r"(add_first), "n"(SB), "n"(2 * SB), "n"(3 * SB)
      : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

// What a thread holds of a tile between its loads and its conversion: 16 channels of every 64 of half the chunks, of two rows.
template <int BITS, bool ROPE>
struct Raw {
  uint32_t code[4][2][BITS / 2];  // step (128 channels), row
  uint32_t block[2];              // the scales of two blocks of four (4 bits)
  uint32_t rope[2][ROPE ? 4 : 1];
  float s[2];                     // -1: masked
};

template <int DQK, int NH, int BITS>
__global__ void __launch_bounds__(kThreads, 1) paged_mla_quant_kernel(const __grid_constant__ Params p) {
  using L = Smem<DQK, NH>;
  constexpr bool ROPE = L::kRope;
  constexpr int NC = NH / 4;  // columns of a softmax thread
  constexpr QuantRow LAY = quant_row(DQK, kDv, BITS);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sV = smem_u32(smem), sQ = sV + L::OFF_Q, sP = sV + L::OFF_P;
  uint8_t* misc = smem + L::OFF_MISC;
  const uint32_t mb = smem_u32(misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + M_ABORT);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  Plan* s_plan = reinterpret_cast<Plan*>(misc + M_PLAN);
  long long* s_row = reinterpret_cast<long long*>(misc + M_ROW);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](int off, uint32_t parity) { return wait_for(mb + off, parity, s_abort, p.wait_limit); };

  if (threadIdx.x == 0) {
    for (int k = 0; k < 5; ++k) mbar_init(mb + M_LAND + 8 * k, kWarps);
    for (int k = 0; k < 4; ++k) mbar_init(mb + M_PV + 8 * k, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(mb + M_A + 8 * k, 1);
      mbar_init(mb + M_FIN + 8 * k, 1);
    }
    mbar_init(mb + M_S, 1);
    mbar_init(mb + M_P, kWarps);
    mbar_init(mb + M_Q, kWarps);
    for (int k = 0; k < kRing; ++k) {
      mbar_init(mb + M_ROWF + 8 * k, 1);
      mbar_init(mb + M_ROWE + 8 * k, kWarps);
    }
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(mb + M_SEGF + 8 * k, 1);
      mbar_init(mb + M_SEGE + 8 * k, kReaders);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  make_plan<kTile, kThreads>(p, s_plan, reinterpret_cast<long long*>(misc + M_RED));
  const Plan plan = *s_plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the joining kernel waits for this one's end itself)
  if (plan.w1 <= plan.w0 || plan.w1 - plan.w0 <= plan.skip) return;  // (the whole CTA)
  if (warp == 16) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  uint32_t tmem = 0;
  if (warp < 18) {  // the others neither need it nor wait for it
    named_bar(5, 32 * 18);
    tmem = (uint32_t)warp_value((int)*s_tmem);
  }
  auto read_seg = [&](int k, Seg& s) -> bool {
    return read_announcement(mb + M_SEGF, mb + M_SEGE, reinterpret_cast<const int4*>(misc + M_SEG), k, s_abort, p.wait_limit, s);
  };
  if (warp == 16) {
    // ======================= S^T issuer =======================
    constexpr uint32_t kIdR = idesc_bf16(kTile, NH, false, false), kId = idesc_f16(kTile, NH, false, false);
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      if (!warp_all(wait(M_Q, seg & 1))) break;
      const int n = warp_value(sg.n);
      const uint32_t t0 = (uint32_t)warp_value((int)tmem), q0 = (uint32_t)warp_value((int)sQ);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const uint64_t b0 = sdesc_sw128(q0, 16, 1024);
        if (ROPE) {
          if (!warp_all(wait(M_LAND, i & 1))) { stop = true; break; }
          tc_fence_after();
          mma4_ts_w<2>(t0 + L::TM_S, t0 + L::TM_R, b0 + (8 * L::Q_CHUNK >> 4), kIdR, 0);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (!warp_all(wait(M_LAND + 8 * (1 + m), i & 1))) { stop = true; break; }
          tc_fence_after();
          const uint32_t a = t0 + L::TM_A + (m % L::SLOTS) * 64;
          mma4_ts_w<2>(t0 + L::TM_S, a, b0 + (2 * m * L::Q_CHUNK >> 4), kId, ROPE || m > 0);
          mma4_ts_w<2>(t0 + L::TM_S, a + 32, b0 + ((2 * m + 1) * L::Q_CHUNK >> 4), kId, 1);
          if (L::SLOTS == 2 && m < 2) mma_commit_w(mb + M_A + 8 * m);
        }
        if (stop) break;
        mma_commit_w(mb + M_S);
      }
      if (stop) break;
    }
    mma_commit_w(mb + M_FIN);
    volatile int dummy = 0;
    mbar_wait(mb + M_FIN, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 17) {
    // ======================= P.V issuer =======================
    constexpr uint32_t kId = idesc_f16(128, NH, true, NH == 64);
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      const int n = warp_value(sg.n);
      const uint32_t t0 = (uint32_t)warp_value((int)tmem), v0 = (uint32_t)warp_value((int)sV), w0 = (uint32_t)warp_value((int)sP);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        if (!warp_all(wait(M_P, i & 1))) { stop = true; break; }
        tc_fence_after();
        const uint64_t va = sdesc_sw128(v0, L::CHUNK, 1024), wb = sdesc_sw128(w0, 16, 1024);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t a = va + m * (2 * L::CHUNK >> 4);
          if constexpr (NH == 64) {  // W^T rows are positions (MN-major)
            mma4_w<128, 128>(t0 + m * NH, a, wb, kId, k0 > 0);
            mma4_w<128, 128>(t0 + m * NH, a + 512, wb + 512, kId, 1);
          } else {  // W^T rows are columns, 64 positions along K, then the other 64
            mma4_w<128, 2>(t0 + m * NH, a, wb, kId, k0 > 0);
            mma4_w<128, 2>(t0 + m * NH, a + 512, wb + (NH * 128 >> 4), kId, 1);
          }
          mma_commit_w(mb + M_PV + 8 * m);
        }
      }
      if (stop) break;
    }
    mma_commit_w(mb + M_FIN + 8);
    volatile int dummy = 0;
    mbar_wait(mb + M_FIN + 8, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 18) {
    announce<kTile>(p, plan, mb + M_SEGF, mb + M_SEGE, reinterpret_cast<int4*>(misc + M_SEG), s_abort);
  } else if (warp == 19) {
    // ======================= rows of the tiles =======================
    bool bad_index = false;
    int i = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!read_seg(seg, sg)) break;
      last = sg.last;
      const int limit = (int)min((long long)p.max_pages * p.P, (long long)(p.topk_idx ? sg.seen0 : sg.keys));
      const int32_t* table = p.table + (size_t)sg.b * p.max_pages;
      const int32_t* list = p.topk_idx ? p.topk_idx + (size_t)(sg.row0 / p.H) * p.K : nullptr;
      bool stop = false;
#pragma unroll 1
      for (int t = sg.t0; t < sg.t0 + sg.n; ++t, ++i) {
        int pos[4], page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = t * kTile + 32 * k + lane;
          pos[k] = j >= sg.keys ? -1 : list ? __ldg(list + j) : j;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (pos[k] < -1 || pos[k] >= limit) {
            bad_index |= pos[k] != -1;
            pos[k] = -1;
          }
          page[k] = -1;
          if (pos[k] >= 0) {
            const unsigned at = (unsigned)pos[k] / (unsigned)p.P;
            pos[k] -= (int)at * p.P;
            page[k] = __ldg(table + at);
          }
        }
        const int slot = i % kRing;
        if (i >= kRing && !warp_all(wait(M_ROWE + 8 * slot, (i / kRing - 1) & 1))) { stop = true; break; }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          long long at = -1;
          if (pos[k] >= 0) {
            if (page[k] >= 0 && page[k] < p.num_pages) at = ((long long)page[k] * p.P + pos[k]) * LAY.bytes;
            else bad_index = true;
          }
          s_row[slot * kTile + 32 * k + lane] = at;
          if (at >= 0)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.cache + at), "n"(LAY.bytes) : "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + M_ROWF + 8 * slot);
      }
      if (stop) break;
    }
    if (bad_index) record_error(p.err, DSA_ERR_DEVICE_INDEX);
  } else {
    // ======================= conversion, softmax, epilogue =======================
    float* s_col = reinterpret_cast<float*>(misc + M_COL);
    float* s_neg = reinterpret_cast<float*>(misc + M_NEG);
    float* s_red = reinterpret_cast<float*>(misc + M_RED);
    float* s_fac = s_red;  // a column's factor replaces its first maximum or sum
    float* s_stat = reinterpret_cast<float*>(misc + M_STAT);
    volatile float* s_scale = reinterpret_cast<volatile float*>(misc + M_SCALE);
    // conversion: rows r0 and r0 + 8 of the tile, 16 channels of chunk 2m + half in step m
    const int qd = warp & 3, half = warp >> 3, quad = lane & 3;
    const int r0 = qd * 32 + ((warp >> 2) & 1) * 16 + (lane >> 2);
    const uint32_t to0 = sV + half * L::CHUNK + sw128_off(r0, 2 * quad), to1 = sV + half * L::CHUNK + sw128_off(r0, 2 * quad + 1);
    const uint32_t tm_a = tmem_addr(tmem, (r0 & ~15) & 127, 0);
    // softmax: position `row` of the tile, columns n0 .. n0 + NC - 1, together with the other warps of the column group
    const int cg = warp >> 2, n0 = cg * NC, row = qd * 32 + lane, bar_id = 1 + cg;
    Raw<BITS, ROPE> raw;
    auto load_tile = [&](int i) -> bool {
      const int slot = i % kRing;
      if (!warp_all(wait(M_ROWF + 8 * slot, (i / kRing) & 1))) return false;
      long long at[2] = {s_row[slot * kTile + r0], s_row[slot * kTile + r0 + 8]};
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_ROWE + 8 * slot);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool on = at[k] >= 0;
        const uint8_t* src = p.cache + (on ? at[k] : 0);
        raw.s[k] = -1.f;
        if (on) {  // (a row that was never written, of zero bytes, holds zeros)
          const float v = __ldg(reinterpret_cast<const float*>(src + LAY.scale));
          raw.s[k] = v < kLeast ? kLeast : v;
        }
        if constexpr (ROPE) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (on) v = __ldg(reinterpret_cast<const uint4*>(src + LAY.tail + half * 64 + quad * 16));
          raw.rope[k][0] = v.x; raw.rope[k][1] = v.y; raw.rope[k][2] = v.z; raw.rope[k][3] = v.w;
        }
        if constexpr (BITS == 4)  // of chunk 2 quad + half; the lanes exchange them
          raw.block[k] = on ? __ldg(reinterpret_cast<const uint32_t*>(src + LAY.blocks) + 2 * quad + half) : 0u;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if constexpr (BITS == 4) {
            uint2 v = make_uint2(0, 0);
            if (on) v = __ldg(reinterpret_cast<const uint2*>(src + (2 * m + half) * 32) + quad);
            raw.code[m][k][0] = v.x; raw.code[m][k][1] = v.y;
          } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (on) v = __ldg(reinterpret_cast<const uint4*>(src + (2 * m + half) * 64) + quad);
            raw.code[m][k][0] = v.x; raw.code[m][k][1] = v.y; raw.code[m][k][2] = v.z; raw.code[m][k][3] = v.w;
          }
        }
      }
      return true;
    };
    auto landed = [&](int step) {
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_LAND + 8 * step);
    };
    // Tile i from registers to TMEM and shared memory; false when a wait ran out.
    auto convert = [&](int i) -> bool {
      if (half == 0 && quad == 0) {
        s_scale[(i & 1) * kTile + r0] = raw.s[0];
        s_scale[(i & 1) * kTile + r0 + 8] = raw.s[1];
      }
      tc_fence_after();  // (the tile before has left S^T's operands: its scores have been waited for)
      if constexpr (ROPE) {
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float inv = raw.s[k] < 0.f ? 1.f : __frcp_rn(raw.s[k]);
          const uint32_t by = pack_bf16x2(inv, inv);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[(j >> 1) * 4 + 2 * k + (j & 1)] = mul_bf16x2(raw.rope[k][j], by);
        }
        tmem_st16x256b(tm_a + L::TM_R + half * 16, v);
        landed(0);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[8];
          if constexpr (BITS == 4) {
            const uint32_t b4 = __shfl_sync(0xffffffffu, raw.block[k], (lane & 28) | m);
            const uint32_t by = e4m3x2_f16x2((uint16_t)__byte_perm(b4, 0, quad * 0x11));
            uint32_t lo[4], hi[4];
            e2m1x8_f16x2(raw.code[m][k][0], lo);
            e2m1x8_f16x2(raw.code[m][k][1], hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              h[j] = mul_f16x2(lo[j], by);
              h[4 + j] = mul_f16x2(hi[j], by);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              h[2 * j] = e4m3x2_f16x2((uint16_t)raw.code[m][k][j]);
              h[2 * j + 1] = e4m3x2_f16x2((uint16_t)(raw.code[m][k][j] >> 16));
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) v[(j >> 1) * 4 + 2 * k + (j & 1)] = h[j];
        }
        if (i > 0 && !warp_all(wait(M_PV + 8 * m, (i - 1) & 1))) return false;
        if (L::SLOTS == 2 && m >= 2) {
          if (!warp_all(wait(M_A + 8 * (m - 2), i & 1))) return false;
          tc_fence_after();
        }
        __syncwarp();
        tmem_st16x256b(tm_a + L::TM_A + (m % L::SLOTS) * 64 + half * 32, v);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          st_shared_v4(to0 + m * 2 * L::CHUNK + k * 1024, v[2 * k], v[2 * k + 1], v[4 + 2 * k], v[5 + 2 * k]);
          st_shared_v4(to1 + m * 2 * L::CHUNK + k * 1024, v[8 + 2 * k], v[9 + 2 * k], v[12 + 2 * k], v[13 + 2 * k]);
        }
        landed(1 + m);
      }
      return true;
    };
    // The run's queries: a row a warp, divided by a power of two, its channels in the order in which they lie in TMEM.
    auto load_q = [&](const Seg& s, int run) {
#pragma unroll 1
      for (int hh = warp; hh < NH; hh += kWarps) {
        constexpr int UNITS = DQK / 8;
        uint4 v[3];
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const int u = lane + 32 * x;
          v[x] = make_uint4(0, 0, 0, 0);
          if (hh < s.rows && u < UNITS) v[x] = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)(s.row0 + hh) * DQK) + u);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[x].x & 0x7fff7fffu, v[x].y & 0x7fff7fffu),
                                       __vmaxu2(v[x].z & 0x7fff7fffu, v[x].w & 0x7fff7fffu)));
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int e = max((int)(most >> 7) - 127, -112);
        const float by = pow2(14 - e);
        if (lane == 0) s_col[(run & 1) * 64 + hh] = pow2(e - 14) * p.sl2e;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const int u = lane + 32 * x;
          if (u >= UNITS) continue;
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
          for (int g = 0; g < 2; ++g) {  // four channels, and their place among the 64
            uint32_t a, b;
            int at;
            if (u < 64) {
              a = pack_f16x2(__uint_as_float(w[2 * g] << 16) * by, __uint_as_float(w[2 * g] & 0xffff0000u) * by);
              b = pack_f16x2(__uint_as_float(w[2 * g + 1] << 16) * by, __uint_as_float(w[2 * g + 1] & 0xffff0000u) * by);
              const int c4 = 2 * (u & 7) + g;
              at = (c4 & 3) * 4 + (c4 >> 2);
            } else {
              const uint32_t by2 = pack_bf16x2(by, by);
              a = mul_bf16x2(w[2 * g], by2);
              b = mul_bf16x2(w[2 * g + 1], by2);
              at = ((u - 64) >> 2) * 8 + g * 4 + ((u - 64) & 3);
            }
            const uint32_t dst = sQ + (u >> 3) * L::Q_CHUNK + sw128_off(hh, at >> 1) + (at & 1) * 8;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(a), "r"(b) : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_Q);
    };
    // Maxima or sums over the warp's 32 positions of a thread's columns: the result is that of column n0 + lane / (32 / NC).
    auto over_lanes = [&](float (&v)[NC], bool is_max) -> float {
      int w = NC / 2;
#pragma unroll
      for (int bit = 16; bit >= 1; bit >>= 1, w >>= 1) {
        if (w >= 1) {
          const bool upper = (lane & bit) != 0;
#pragma unroll
          for (int j = 0; j < w; ++j) {
            const float send = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
            const float x = __shfl_xor_sync(0xffffffffu, send, bit);
            v[j] = is_max ? fmaxf(keep, x) : keep + x;
          }
        } else {
          const float x = __shfl_xor_sync(0xffffffffu, v[0], bit);
          v[0] = is_max ? fmaxf(v[0], x) : v[0] + x;
        }
      }
      return v[0];
    };
    const int own_col = n0 + lane / (32 / NC);
    Seg sg;
    bool aborted = named_bar_or(bar_id, 128, !read_seg(0, sg));
    bool bad = false;
    if (!aborted) {
      load_q(sg, 0);
      bad = !load_tile(0);
    }
    int i = 0;
    for (int seg = 0; !aborted; ++seg) {
      const bool more = !sg.last;
      // this thread's first row: its token in the group, and how many rows of that token there are from it on
      const int tok0 = (sg.head0 + n0) / p.H, head_left = p.H - ((sg.head0 + n0) - tok0 * p.H);
      float2 l_part[NC / 2];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) l_part[j] = make_float2(0.f, 0.f);
      // a column without a finite score yet has a maximum of -3e38, which any finite score passes and which leaves e^-inf at 0
      if (qd == 0 && lane < NC) {
        s_stat[n0 + lane] = -INFINITY;
        s_neg[n0 + lane] = 3.0e38f;
      }
      named_bar(bar_id, 128);
      const float* col = s_col + (seg & 1) * 64 + n0;
      const int t_end = sg.t0 + sg.n;
#pragma unroll 1
      for (int t = sg.t0; t < t_end; ++t, ++i) {
        const bool end = t + 1 == t_end;
        bad = bad || !convert(i);
        if ((!end || more) && !bad) bad = !load_tile(i + 1);
        bad = bad || !warp_all(wait(M_S, i & 1));
        // (complete since before S^T was issued: orders the columns' factors and the rows' scales before their reads below)
        bad = bad || !warp_all(wait(M_Q, seg & 1) && wait(M_LAND + 32, i & 1));
        tc_fence_after();
        __syncwarp();
        uint32_t zr[NC];
        tmem_ld<NC>(tmem_addr(tmem, qd * 32, L::TM_S + n0), zr);
        const float s = s_scale[(i & 1) * kTile + row];
        const bool plain = s > 0.f;  // neither masked nor NaN
        const int ls = plain ? (int)(__float_as_uint(s) >> 23) - 127 : 0;
        const float log_s = (float)ls, inv_s = pow2(-ls);
        tmem_ld_wait();
        // scores in log2 units; the exponents of the weights: with s, above the running maximum
        float2 z[NC / 2], e[NC / 2];
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          const float2 f = mul2(*reinterpret_cast<const float2*>(col + 2 * j), make_float2(s, s));
          z[j] = fma2(make_float2(__uint_as_float(zr[2 * j]), __uint_as_float(zr[2 * j + 1])), f, make_float2(log_s, log_s));
        }
        const int pos = t * kTile + row;
        if (s < 0.f) {
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) z[j] = make_float2(-INFINITY, -INFINITY);
        } else if (p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0) {  // some token may not see all of it
          int seen = sg.seen0 + tok0, left = head_left;
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            if (pos >= seen) (j & 1 ? z[j / 2].y : z[j / 2].x) = -INFINITY;
            if (--left == 0) { left = p.H; ++seen; }
          }
        }
        bool mine = t == sg.t0;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          e[j] = add2(z[j], *reinterpret_cast<const float2*>(s_neg + n0 + 2 * j));
          mine |= e[j].x > kRaise || e[j].y > kRaise;
        }
        bool raise = false;
        if (named_bar_or(bar_id, 128, mine || bad)) {
          if (named_bar_or(bar_id, 128, bad)) { aborted = true; break; }
          raise = true;
        }
        if (raise) {
          float top[NC];
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) { top[2 * j] = z[j].x; top[2 * j + 1] = z[j].y; }
          s_red[qd * 64 + own_col] = over_lanes(top, true);
          named_bar(bar_id, 128);
          if (qd == 0 && lane < NC) {
            const int n = n0 + lane;
            const float bm = fmaxf(fmaxf(s_red[n], s_red[64 + n]), fmaxf(s_red[128 + n], s_red[192 + n])) - kTop;
            const float mo = s_stat[n], mn = fmaxf(mo, bm);
            s_stat[n] = mn;
            s_neg[n] = -fmaxf(mn, -3.0e38f);
            s_fac[n] = mo == -INFINITY ? 0.f : exp2f(mo - mn);
          }
          named_bar(bar_id, 128);
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) {
            l_part[j] = mul2(l_part[j], *reinterpret_cast<const float2*>(s_fac + n0 + 2 * j));
            e[j] = add2(z[j], *reinterpret_cast<const float2*>(s_neg + n0 + 2 * j));
          }
          if (t > sg.t0) {  // (P.V of the tile before has been waited for)
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              const uint32_t ta = tmem_addr(tmem, qd * 32, m * NH + n0);
              uint32_t ov[NC];
              tmem_ld<NC>(ta, ov);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < NC; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * s_fac[n0 + j]);
              tmem_st<NC>(ta, ov);
            }
            tmem_st_wait();
          }
          named_bar(bar_id, 128);  // the factors have been read
        }
        uint32_t w[NC / 2];
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          const float2 x = make_float2(ex2(e[j].x), ex2(e[j].y));
          l_part[j] = fma2(x, make_float2(inv_s, inv_s), l_part[j]);
          w[j] = pack_f16x2(x.x, x.y);
        }
        if constexpr (NH == 64) {
          st_shared_v4(sP + sw128_off(row, 2 * cg), w[0], w[1], w[2], w[3]);
          st_shared_v4(sP + sw128_off(row, 2 * cg + 1), w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const int n = n0 + j;
            st_shared_u16(sP + (row >> 6) * (NH * 128) + n * 128 + ((((row >> 3) & 7) ^ (n & 7)) << 4) + (row & 7) * 2,
                          (uint16_t)(w[j / 2] >> (16 * (j & 1))));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + M_P);
      }
      if (aborted) break;
      Seg nx = sg;
      if (more) {
        if (!read_seg(seg + 1, nx)) bad = true;
        else load_q(nx, seg + 1);  // (S^T of the run is done: Q is free)
      }
      // ---- the run's rows: out and lse, or the workspace's partial sums ----
      float sums[NC];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) { sums[2 * j] = l_part[j].x; sums[2 * j + 1] = l_part[j].y; }
      s_red[qd * 64 + own_col] = over_lanes(sums, false);
      named_bar(bar_id, 128);
      const bool whole = sg.whole;
      const int slot = 2 * blockIdx.x + (sg.opens ? 1 : 0);
      if (qd == 0 && lane < NC) {
        const int n = n0 + lane;
        const float l = s_red[n] + s_red[64 + n] + s_red[128 + n] + s_red[192 + n];
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
      const bool got = wait(M_PV + 24, (i - 1) & 1);
      aborted = named_bar_or(bar_id, 128, !got || bad);
      if (aborted) break;
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        uint32_t ov[NC];
        tmem_ld<NC>(tmem_addr(tmem, qd * 32, m * NH + n0), ov);
        tmem_ld_wait();
        const int c = m * 128 + qd * 32 + lane, rows = sg.rows - n0;
        // (one branch for all rows: with one for each, every store waits for the one before)
        if (whole) {
          __nv_bfloat16* dst = p.out + (size_t)(sg.row0 + n0) * kDv + c;
          float f[NC];
#pragma unroll
          for (int h = 0; h < NC; ++h) f[h] = s_fac[n0 + h];
#pragma unroll
          for (int h = 0; h < NC; ++h)
            if (h < rows) dst[h * kDv] = __float2bfloat16_rn(f[h] == 0.f ? 0.f : __uint_as_float(ov[h]) * f[h]);
        } else {
          float* part = p.partial + ((size_t)slot * 64 + n0) * kDv + c;
#pragma unroll
          for (int h = 0; h < NC; ++h)
            if (h < rows) part[h * kDv] = __uint_as_float(ov[h]);
        }
      }
      tc_fence_before();
      named_bar(bar_id, 128);  // s_red, s_stat and s_fac have been read
      if (!more) break;
      sg = nx;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    if (lane == 0 && *s_abort) record_error(p.err, DSA_ERR_TIMEOUT);
  }
}

constexpr size_t kRecordOff = kErrorWordBytes, kStatOff = kRecordOff + kRecordBytes, kPartialOff = kStatOff + kStatBytes;

template <int DQK, int NH, int BITS>
dsa_status_t launch(Params& p, int ctas, cudaStream_t s) {
  using L = Smem<DQK, NH>;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_mla_quant_kernel<DQK, NH, BITS>), L::TOTAL,
                                          "configuring paged_mla_quant_kernel");
  if (st != DSA_OK) return st;
  p.G = p.topk_idx ? 1 : (p.H <= NH ? NH / p.H : 1);
  p.extra = 2;
  p.HB = (p.H + NH - 1) / NH;
  paged_mla_quant_kernel<DQK, NH, BITS><<<ctas, kThreads, L::TOTAL, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching paged_mla_quant_kernel");
}
template <int DQK, int NH>
dsa_status_t launch(Params& p, int bits, int ctas, cudaStream_t s) {
  return bits == 8 ? launch<DQK, NH, 8>(p, ctas, s) : launch<DQK, NH, 4>(p, ctas, s);
}

}  // namespace pmlaq
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_paged_mla_quant_workspace_size(void) {
  return pmlaq::kPartialOff + pgroups::kPartialBytes;
}

extern "C" dsa_status_t dsa_paged_mla_quant(const dsa_bf16_t* q, const uint8_t* cache, const int32_t* block_table,
                                            const int32_t* seq_lens, const int32_t* cu_q, const int32_t* topk_idx,
                                            const int32_t* topk_len, int32_t N, int32_t B, int32_t H, int32_t Dqk,
                                            int32_t Dv, int32_t bits, int32_t K, int32_t num_pages, int32_t page_size,
                                            int32_t max_pages, float softmax_scale, const float* attn_sink,
                                            dsa_bf16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                            dsa_stream_t stream) {
  const char* who = "dsa_paged_mla_quant";
  if (N < 0 || B < 0 || H < 1 || K < 0 || num_pages < 0 || page_size < 1 || max_pages < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT,
                "%s: need N, B, K, num_pages, max_pages >= 0, H >= 1, page_size >= 1 (got %d, %d, %d, %d, %d, %d, %d)", who,
                N, B, K, num_pages, max_pages, H, page_size);
  if (Dqk != 576 && Dqk != 512) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: Dqk must be 576 or 512 (got %d)", who, Dqk);
  if (Dv != 512) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: Dv must be 512 (got %d)", who, Dv);
  if (bits != 8 && bits != 4) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: bits must be 8 or 4 (got %d)", who, bits);
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
  dsa_status_t st = check_workspace(workspace, workspace_bytes, dsa_paged_mla_quant_workspace_size(), who);
  if (st != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (N == 0 || B == 0) return ok();
  const int ctas = pgroups::cta_count();
  if (ctas < 1) return fail(DSA_ERR_CUDA, "%s: the device's SM count cannot be read", who);
  pmlaq::Params p{};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.cache = cache;
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
  p.sl2e = softmax_scale * pgroups::kLog2e;
  p.sink = attn_sink;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  char* ws = reinterpret_cast<char*>(workspace);
  p.err = reinterpret_cast<int*>(ws);
  p.records = reinterpret_cast<int4*>(ws + pmlaq::kRecordOff);
  p.stats = reinterpret_cast<float*>(ws + pmlaq::kStatOff);
  p.partial = reinterpret_cast<float*>(ws + pmlaq::kPartialOff);
  p.wait_limit = wait_limit_cycles();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // 16 columns while all rows of a request (or of a list) fit
  const int64_t rows = (int64_t)H * (topk_idx ? 1 : (N + B - 1) / B);
  if (rows <= 16) st = Dqk == 576 ? pmlaq::launch<576, 16>(p, bits, ctas, s) : pmlaq::launch<512, 16>(p, bits, ctas, s);
  else st = Dqk == 576 ? pmlaq::launch<576, 64>(p, bits, ctas, s) : pmlaq::launch<512, 64>(p, bits, ctas, s);
  if (st != DSA_OK) return st;
  st = pgroups::launch_join(p, ctas, s);
  return st == DSA_OK ? ok() : st;
}
