// dsa_paged_mla_quant.cu -- attention of new tokens over a paged cache of quantised latents (sm_103a): the kernel for rows of
// 4 bits, and the entry point for both (8 bits: dsa_paged_mla_e4m3.cu).
//
// For new token j of request b and head h:  z_p = scale <q, kv_p> over the positions p it sees,
// lse = ln sum e^{z_p},  out = sum e^{z_p - lse} kv_p[0:512],  kv_p = v_p s_p with v_p = code * block (e2m1 times
// e4m3) for the first 512 channels and s_p the row's scale, a power of two.
//
// v is exact in fp16 (6 bits between 2^-10 and 2688), so the products run in fp16 and s stays outside of them:
// z_p = s_p <q, v_p> + <q', kv'_p>, with the position channels' part in bf16, divided by s_p (a power of two); and the
// output sums the weights w_p = e^{z_p} s_p.  The running maximum is that of w, not of e^{z}: w in fp16 (11 bits, 2^15 down
// to 2^-24 around a maximum of 2^7) then loses nothing that counts, whatever the rows' scales are.  The denominator adds
// e^{z_p} in fp32.  A query row is divided by a power of two so that the largest of its first 512 channels lies in [2^14, 2^15):
// channels down to 2^-31 of that one are exact in fp16, smaller ones off by half a step of 2^-24, 2^-39 of it.  Not by the
// largest of all: one large position channel would take the others out of fp16, which count where s is large.  Where a position
// channel is more than 2^kOver of the others' largest, it takes part for 2^-kOver of it, so that the scores do not overflow.
//
// Split of the work as in dsa_paged_groups.cuh, with tiles of 96 positions and groups of NH = 64 columns, or of 16 where a
// request has no more rows on the average, or a list.  A tile: two warps copy its rows as they are to shared memory; 12 warps
// take the codes from there to registers and form fp16, which is the A operand of S^T[position, column] = V Q^T and, as V^T, of
// O^T[channel, column] += V^T W^T.  Two quarters of the channels are written to TMEM, position by lane, before P.V of the tile
// before has left shared memory; one quarter to shared memory, from where both products read it, and the last to TMEM; then the
// three quarters in TMEM to shared memory too, while S^T is under way.  Then the same warps do the softmax, a position a
// thread.  96 positions, since an fp16 tile of 128, its queries and W leave no room for the next tile's rows as they come (with
// 16 columns, which take the same form, 57 KB are free).
//
// A thread's four blocks of 16 channels lie side by side in a row (one load for four scales), but 16 channels apart in every
// 128 of the products: O^T's row 128 m + 16 y + e is channel 64 y + 16 m + e, and the queries' channels follow.
//
// What bounds it: 64 requests of 4000 to 16384 positions, 64 heads: 159 us, where the same over bf16 rows of 2.7 times the
// bytes takes 161 and over 8 bits (dsa_paged_mla_e4m3.cu, which converts nothing) 133.  A tile takes about 5500 cycles, of which
// the warps convert for 3900 and do the softmax for 1400, never waiting for a product; shared memory moves 424 KB (rows in
// and out 84, V in and out 192, W 60, queries 88), 3400 cycles at 128 bytes each.  Measured beside it: with 64 registers
// a thread and twice the warps 209 us, the next tile's rows in registers during the softmax 171 (half of them: 163), loads by the
// converting warps themselves 190 and more, three quarters in TMEM before the one in shared memory 161.5.
//
// Warps: three of four convert and do softmax and epilogue (they reach the TMEM lanes 0-95); of the others one issues the
// products, one announces the runs of tiles, two copy.
#include <climits>
#include <cmath>

#include "dsa_f32x2.cuh"
#include "dsa_paged_groups.cuh"
#include "dsa_paged_mla_quant.h"
#include "dsa_paged_quant.cuh"

namespace dsa {
namespace pmlaq {

using namespace pgroups;

constexpr int kTile = 96;
constexpr int kThreads = 512;
constexpr int kWorkers = 12;              // warps that convert and do the softmax: number w with w % 4 < 3
constexpr int kReaders = kWorkers + 6;    // readings of an announcement: two copying warps' two each, the announcing warp's own
constexpr int kTeam = 96;                 // threads of a column group
constexpr float kRaise = 15.0f;           // log2 units: the running maximum is raised when a weight passes 2^15
constexpr float kTop = 7.0f;              // a new maximum is 2^7
constexpr float kLeast = 3.5527136788005009e-15f;  // 2^-48, the least s
constexpr int kOver = 24;  // position channels of 2^(15 + 24), times 64 keys' below 2^82 s, are sums below 2^127

template <int DQK, int NH>
struct Smem {
  static constexpr bool kRope = DQK == 576;
  static constexpr QuantRow LAY = quant_row(DQK, kDv, 4);
  static constexpr int CHUNK = kTile * 128;  // 64 channels of a tile
  static constexpr int Q_CHUNK = NH * 128;
  static constexpr int P_BYTES = NH == 64 || kRope ? kTile * 128 : 2 * NH * 128;  // (position channels lie there before W)
  static constexpr int OFF_Q = 8 * CHUNK;
  static constexpr int OFF_P = OFF_Q + (kRope ? 9 : 8) * Q_CHUNK;
  static constexpr int OFF_MISC = OFF_P + P_BYTES;
  static constexpr int MISC = 3584;
  static constexpr int OFF_RAW = OFF_MISC + MISC;
  static constexpr int TOTAL = OFF_RAW + kTile * LAY.bytes;
  static_assert(TOTAL <= 232448 && LAY.bytes % 32 == 16, "shared memory budget");
  // TMEM columns: O^T, S^T and three slots of 128 channels of the A operand
  static constexpr int TM_S = 4 * NH, TM_A = TM_S + (NH < 32 ? 32 : NH);
  static_assert(TM_A + 3 * 64 <= 512, "TMEM budget");
};

// misc (bytes)
constexpr int M_LAND = 0;      // [3]: S^T's operand is there: 256 channels in TMEM, the last 128 in shared memory, the others
constexpr int M_PV = 40;       // P.V is done
constexpr int M_S = 88, M_P = 96, M_Q = 104, M_FIN = 112;
constexpr int M_RAW = 120, M_READ = 128;                    // a tile's rows have come, have been read
constexpr int M_SEGF = 144, M_SEGE = 208;                   // [kSegs] each
constexpr int M_TMEM = 272, M_ABORT = 276, M_PLAN = 280;    // plan: 56 bytes
constexpr int M_FAC = 3192, M_EPI = 3200;                   // a run's factors are there; its lanes 96-127 are stored
constexpr int M_FLAG = 3208;                                // uint8 [2][4]: a tile's raise, by column group
constexpr int M_VALID = 3240;                               // uint8 [96]: rows that are not masked
constexpr int M_SEG = 336;                                  // int4 [kSegs][2]
constexpr int M_COL = 592;                                  // float [2][64]: a column's factor of the score, by run
constexpr int M_NEG = 1104;                                 // float [64]: minus the running maxima
constexpr int M_RED = 1360;                                 // float [3][64]
constexpr int M_STAT = 2128;                                // float [64]
constexpr int M_SCL = 2384;                                 // float [64]: factors of a rescale
constexpr int M_OUT = 2640;                                 // float [2][64]: factors of the output, by run
static_assert(M_SEGE + 8 * kSegs <= M_TMEM && M_PLAN + 56 <= M_SEG && M_OUT + 512 <= M_FAC && M_FLAG + 32 <= M_VALID &&
                  M_VALID + kTile <= 3584, "misc layout");

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
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]) : "memory");
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

// Two MMAs on consecutive steps, added to D (as mma4_w).
template <int SA, int SB>
__device__ __forceinline__ void mma2_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred q, e;\n\t.reg .b64 a1, b1;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "add.s64 a1, %1, %4;\n\tadd.s64 b1, %2, %5;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "n"(SA), "n"(SB)
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

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t at) {
  float v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// A quarter (32 lanes of TMEM) of the channels of NC columns from n0 on: out, or the workspace's partial sums.
template <int NH>
__device__ __noinline__ void store_quarter(const Params& p, const Seg& sg, uint32_t tmem, int qd, int n0, const float* fac) {
  constexpr int NC = NH / 4;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int m = 0; m < 4; ++m) {
    uint32_t ov[NC];
    tmem_ld<NC>(tmem_addr(tmem, qd * 32, m * NH + n0), ov);
    tmem_ld_wait();
    const int c = (qd * 32 + lane) / 16 * 64 + m * 16 + lane % 16, rows = sg.rows - n0;
    // (one branch for all rows: with one for each, every store waits for the one before)
    if (sg.whole) {
      __nv_bfloat16* dst = p.out + (size_t)(sg.row0 + n0) * kDv + c;
      float f[NC];
#pragma unroll
      for (int h = 0; h < NC; ++h) f[h] = fac[n0 + h];
#pragma unroll
      for (int h = 0; h < NC; ++h)
        if (h < rows) dst[h * kDv] = __float2bfloat16_rn(f[h] == 0.f ? 0.f : __uint_as_float(ov[h]) * f[h]);
    } else {
      float* part = p.partial + ((size_t)(2 * blockIdx.x + (sg.opens ? 1 : 0)) * 64 + n0) * kDv + c;
#pragma unroll
      for (int h = 0; h < NC; ++h)
        if (h < rows) part[h * kDv] = __uint_as_float(ov[h]);
    }
  }
}

template <int DQK, int NH>
__global__ void __launch_bounds__(kThreads, 1) paged_mla_quant_kernel(const __grid_constant__ Params p) {
  using L = Smem<DQK, NH>;
  constexpr bool ROPE = L::kRope;
  constexpr int NC = NH / 4;  // columns of a softmax thread
  constexpr QuantRow LAY = L::LAY;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sV = smem_u32(smem), sQ = sV + L::OFF_Q, sP = sV + L::OFF_P, sRaw = sV + L::OFF_RAW;
  uint8_t* misc = smem + L::OFF_MISC;
  const uint32_t mb = smem_u32(misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + M_ABORT);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  Plan* s_plan = reinterpret_cast<Plan*>(misc + M_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](int off, uint32_t parity) -> bool {
    return warp_all(wait_for(mb + off, parity, s_abort, p.wait_limit));
  };

  // rows that follow one another in pages of some size come by copies of whole runs, others one by one
  const bool runs = p.topk_idx == nullptr && p.P >= 16;
  if (threadIdx.x == 0) {
    for (int k = 0; k < 3; ++k) mbar_init(mb + M_LAND + 8 * k, kWorkers);
    mbar_init(mb + M_PV, 1);
    mbar_init(mb + M_FIN, 1);
    mbar_init(mb + M_S, 1);
    mbar_init(mb + M_P, kWorkers);
    mbar_init(mb + M_Q, kWorkers);
    mbar_init(mb + M_RAW, runs ? 2 : 2 * 33);  // two warps' copies, and their stores
    mbar_init(mb + M_READ, kWorkers);
    mbar_init(mb + M_FAC, 4);
    mbar_init(mb + M_EPI, 3);
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
  if (warp == 3) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  __syncthreads();
  const uint32_t tmem = (uint32_t)warp_value((int)*s_tmem);
  auto read_seg = [&](int k, Seg& s) -> bool {
    const int4* ring = reinterpret_cast<const int4*>(misc + M_SEG);
    return read_announcement_here(mb + M_SEGF, mb + M_SEGE, ring, k, s_abort, p.wait_limit, s);
  };
  // The lanes 96-127 of TMEM hold no positions, but channels of O^T: the four warps that reach them store them, a column
  // group each (the one that issues the products rescales them too).  Run k, whose last tile is number i - 1 of the CTA's.
  const float* s_out = reinterpret_cast<const float*>(misc + M_OUT);
  auto last_quarter = [&](int k, int& i) -> bool {
    Seg sg;
    if (!warp_all(read_seg(k, sg))) return false;
    i += sg.n;
    if (!(wait(M_FAC, k & 1) && wait(M_PV, (i - 1) & 1))) return false;
    tc_fence_after();
    store_quarter<NH>(p, sg, tmem, 3, (warp >> 2) * NC, s_out + (k & 1) * 64);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(mb + M_EPI);
    return true;
  };
  if (warp == 3) {
    // ======================= the products: S^T of a tile as its steps are converted, then P.V =======================
    constexpr uint32_t kIdR = idesc_bf16(128, NH, false, false), kIdS = idesc_f16(128, NH, false, false);
    constexpr uint32_t kIdV = idesc_f16(128, NH, true, NH == 64);
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      if (!wait(M_Q, seg & 1)) break;
      const int n = warp_value(sg.n);
      const uint32_t t0 = (uint32_t)warp_value((int)tmem), q0 = (uint32_t)warp_value((int)sQ), v0 = (uint32_t)warp_value((int)sV),
                     w0 = (uint32_t)warp_value((int)sP);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const uint64_t b0 = sdesc_sw128(q0, 16, 1024);
        auto from_tmem = [&](int m) {
          const uint32_t a = t0 + L::TM_A + m * 64;
          mma4_ts_w<2>(t0 + L::TM_S, a, b0 + (2 * m * L::Q_CHUNK >> 4), kIdS, m > 0);
          mma4_ts_w<2>(t0 + L::TM_S, a + 32, b0 + ((2 * m + 1) * L::Q_CHUNK >> 4), kIdS, 1);
        };
        if (!wait(M_LAND, i & 1)) { stop = true; break; }
        tc_fence_after();
        from_tmem(0);
        from_tmem(1);
        // a quarter from where P.V will read it (of its 128 rows those past 96 are anything: no one looks at them)
        if (!wait(M_LAND + 8, i & 1)) { stop = true; break; }
        tc_fence_after();
        const uint64_t a0 = sdesc_sw128(v0, 16, 1024);
        mma4_w<2, 2>(t0 + L::TM_S, a0 + (6 * L::CHUNK >> 4), b0 + (6 * L::Q_CHUNK >> 4), kIdS, 1);
        mma4_w<2, 2>(t0 + L::TM_S, a0 + (7 * L::CHUNK >> 4), b0 + (7 * L::Q_CHUNK >> 4), kIdS, 1);
        if (ROPE) mma4_w<2, 2>(t0 + L::TM_S, sdesc_sw128(w0, 16, 1024), b0 + (8 * L::Q_CHUNK >> 4), kIdR, 1);
        if (!wait(M_LAND + 16, i & 1)) { stop = true; break; }
        tc_fence_after();
        from_tmem(2);
        mma_commit_w(mb + M_S);
        if (!wait(M_P, i & 1)) { stop = true; break; }
        tc_fence_after();
        if (k0 == 0) {  // the run before has left O^T
          if (seg > 0 && !wait(M_EPI, (seg - 1) & 1)) { stop = true; break; }
          tc_fence_after();
        } else {
          const uint32_t flags = lds32(mb + M_FLAG + (i & 1) * 4);
          const float* scl = reinterpret_cast<const float*>(misc + M_SCL);
#pragma unroll 1
          for (int g = 0; flags != 0 && g < 4; ++g) {
            if (!((flags >> (8 * g)) & 1u)) continue;
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              const uint32_t ta = tmem_addr(tmem, 96, m * NH + g * NC);
              uint32_t ov[NC];
              tmem_ld<NC>(ta, ov);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < NC; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * scl[g * NC + j]);
              tmem_st<NC>(ta, ov);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            tc_fence_after();
          }
        }
        const uint64_t va = sdesc_sw128(v0, L::CHUNK, 1024), wb = sdesc_sw128(w0, 16, 1024);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t a = va + m * (2 * L::CHUNK >> 4);
          if constexpr (NH == 64) {  // W^T rows are positions (MN-major)
            mma4_w<128, 128>(t0 + m * NH, a, wb, kIdV, k0 > 0);
            mma2_w<128, 128>(t0 + m * NH, a + 512, wb + 512, kIdV);
          } else {  // W^T rows are columns, 64 positions along K, then the other 32
            mma4_w<128, 2>(t0 + m * NH, a, wb, kIdV, k0 > 0);
            mma2_w<128, 2>(t0 + m * NH, a + 512, wb + (NH * 128 >> 4), kIdV);
          }
        }
        mma_commit_w(mb + M_PV);
      }
      if (stop) break;
      // (as last_quarter, of the first column group)
      if (!(wait(M_FAC, seg & 1) && wait(M_PV, (i - 1) & 1))) break;
      tc_fence_after();
      store_quarter<NH>(p, sg, tmem, 3, 0, s_out + (seg & 1) * 64);
      tc_fence_before();
      __syncwarp();
    }
    mma_commit_w(mb + M_FIN);
    volatile int dummy = 0;
    mbar_wait(mb + M_FIN, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == 7) {
    int told = 0, stored = 0, i = 0;
    bool ok = true;
    auto store = [&](int upto) {
      while (ok && stored < upto) ok = last_quarter(stored++, i);
    };
    announce<kTile>(p, plan, mb + M_SEGF, mb + M_SEGE, reinterpret_cast<int4*>(misc + M_SEG), s_abort, [&](int k) {
      told = k + 1;
      store(told - 4);  // (runs are announced some ahead)
    });
    store(told);
  } else if ((warp & 3) == 3) {
    // ======================= copies: 48 rows of every tile each =======================
    // Rows that follow one another by bulk copies; lists and small pages by cp.async, a warp's instruction up to 512 bytes of
    // one row.  Not the converting warps' own loads: their fences before the tensor core's reads would wait for all that
    // they have under way, and loads to registers need lines of L1, of which there are few beside 227 KB of shared memory.
    // A lane looks up to two rows up, in steps whose loads have a tile's time to come back: the list's entry (three tiles
    // ahead), the page (two), the row number (one).
    constexpr int kHalf = kTile / 2;
    const int gw = warp == 15;
    Seg sg;
    int seg = 0, base = 0, end = 0, limit = 0, n_tiles = INT_MAX;
    bool bad_index = false, stop = false;
    struct Look {
      int pos[2], b, limit;  // positions (then their places in the page), or -1; request; what they have to stay below
    };
    auto position = [&](int i) -> Look {
      Look k{{-1, -1}, 0, 0};
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
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned j = (unsigned)(sg.t0 + i - base) * kTile + gw * kHalf + e * 32 + lane;  // (may pass 2^31)
          if (j < (unsigned)sg.keys && (e == 0 || lane < kHalf - 32))
            k.pos[e] = p.topk_idx ? __ldg(p.topk_idx + (size_t)(sg.row0 / p.H) * p.K + j) : (int)j;
        }
      }
      return k;
    };
    auto page_of = [&](Look& k, int (&page)[2]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        page[e] = -1;
        if (k.pos[e] < -1 || k.pos[e] >= k.limit) {
          bad_index |= k.pos[e] != -1;
          k.pos[e] = -1;
        }
        if (k.pos[e] < 0) continue;
        const unsigned at = (unsigned)k.pos[e] / (unsigned)p.P;
        k.pos[e] -= (int)at * p.P;
        page[e] = __ldg(p.table + (size_t)k.b * p.max_pages + at);
      }
    };
    auto row_of = [&](const Look& k, const int (&page)[2], int (&row)[2]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row[e] = -1;
        if (k.pos[e] >= 0) {
          if (page[e] >= 0 && page[e] < p.num_pages) row[e] = page[e] * p.P + k.pos[e];
          else bad_index = true;
        }
      }
    };
    constexpr int kUnits = LAY.bytes / 16;  // of a row: a lane copies one
    static_assert(kUnits <= 32, "a row by one instruction");
    const uint32_t stage = sRaw + gw * kHalf * LAY.bytes;
    volatile uint8_t* s_valid = misc + M_VALID + gw * kHalf;
    int armed = -1;                // the last tile that this warp's bulk copies belong to
    int stored = 0, store_at = 0;  // runs whose last quarter is stored, and the tiles before the next one
    bool ok = true;
    Look ahead = position(0), next = position(1);
    int page[2], row[2], row_next[2];
    int in_page[2], in_page_next[2];
    page_of(ahead, page);
    row_of(ahead, page, row_next);
    in_page_next[0] = ahead.pos[0];
    in_page_next[1] = ahead.pos[1];
    page_of(next, page);
    ahead = next;
    next = position(2);
#pragma unroll 1
    for (int i = 0; i < n_tiles && !stop; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row[e] = row_next[e];
        in_page[e] = in_page_next[e];
        in_page_next[e] = ahead.pos[e];
      }
      row_of(ahead, page, row_next);
      ahead = next;
      page_of(ahead, page);
      next = position(i + 3);
      if (i > 0 && !wait(M_READ, (i - 1) & 1)) { stop = true; break; }
      s_valid[lane] = row[0] >= 0;
      if (lane < kHalf - 32) s_valid[32 + lane] = row[1] >= 0;
      if (runs) {
        // a run's first lane copies it (up to where the warp's first 32 rows or its others end)
        unsigned on[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) on[e] = __ballot_sync(0xffffffffu, row[e] >= 0);
        armed = i;
        __syncwarp();  // (all lanes' flags come before the arrival that gives them to the other warps: votes order no memory)
        if (lane == 0) mbar_expect_tx(mb + M_RAW, (__popc(on[0]) + __popc(on[1])) * LAY.bytes);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (row[e] >= 0 && (lane == 0 || in_page[e] == 0 || !((on[e] >> ((lane + 31) & 31)) & 1u))) {
            const unsigned stop_at = ~(on[e] >> lane);  // (its lowest set bit: the first row after this one that is masked)
            const int n = min(min(p.P - in_page[e], 32 - lane), stop_at ? __ffs(stop_at) - 1 : 32);
            bulk_copy(stage + (e * 32 + lane) * LAY.bytes, p.cache + (size_t)row[e] * LAY.bytes, n * LAY.bytes, mb + M_RAW);
          }
        }
        __syncwarp();
      } else {
        // eight rows at a time: what a copy reads from registers is free only when it has been taken
#pragma unroll 1
        for (int x0 = 0; x0 < kHalf; x0 += 8) {
          const uint8_t* src[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int at = __shfl_sync(0xffffffffu, x0 < 32 ? row[0] : row[1], (x0 + y) & 31);
            src[y] = at >= 0 ? p.cache + (size_t)at * LAY.bytes + lane * 16 : nullptr;
          }
          const uint32_t dst = stage + x0 * LAY.bytes + lane * 16;
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (src[y] && lane < kUnits) cp_async16(dst + y * LAY.bytes, src[y], 16);
        }
        cp_async_arrive(mb + M_RAW);
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + M_RAW);
      }
      // a run that ended before this tile (its announcement stays until it is read for the second time)
      if (ok && store_at + reinterpret_cast<const volatile int*>(misc + M_SEG)[8 * (stored % kSegs) + 1] <= i)
        ok = last_quarter(stored++, store_at);
    }
    if (!stop)
      while (ok && stored < seg) ok = last_quarter(stored++, store_at);
    if (bad_index) record_error(p.err, DSA_ERR_DEVICE_INDEX);
    // Nothing lands after the CTA has left: bulk copies are waited for too, and where a wait ran out, the other warp, which may
    // have begun the next tile, gets this warp's part of it.
    asm volatile("cp.async.wait_all;" ::: "memory");
    volatile int dummy = 0;
    if (armed >= 0) mbar_wait(mb + M_RAW, armed & 1, &dummy, p.err);
    __syncwarp();
    if (runs && stop && lane == 0) mbar_arrive(mb + M_RAW);
  } else {
    // ======================= conversion, softmax, epilogue =======================
    float* s_col = reinterpret_cast<float*>(misc + M_COL);
    float* s_neg = reinterpret_cast<float*>(misc + M_NEG);
    float* s_red = reinterpret_cast<float*>(misc + M_RED);
    float* s_fac = reinterpret_cast<float*>(misc + M_SCL);
    float* s_fin = reinterpret_cast<float*>(misc + M_OUT);
    volatile uint8_t* s_flag = misc + M_FLAG;
    float* s_stat = reinterpret_cast<float*>(misc + M_STAT);
    // conversion: rows r0 and r0 + 8 of the tile, of every 128 channels 16 (16 quad and on) of 64 (half)
    const int qd = warp & 3, cg = warp >> 2, half = cg & 1, quad = lane & 3;
    const int r0 = qd * 32 + (cg >> 1) * 16 + (lane >> 2);
    const uint32_t to0 = sV + half * L::CHUNK + sw128_off(r0, 2 * quad), to1 = sV + half * L::CHUNK + sw128_off(r0, 2 * quad + 1);
    const uint32_t raw0 = sRaw + r0 * LAY.bytes;
    const uint32_t tm_a = tmem_addr(tmem, qd * 32 + (cg >> 1) * 16, 0);
    // softmax: position `row` of the tile, columns n0 .. n0 + NC - 1, together with the two other warps of the column group
    const int n0 = cg * NC, row = qd * 32 + lane, bar_id = 1 + cg;
    auto scale_of = [&](int r) {  // (a row that was never written, of zero bytes, holds zeros; -1: masked)
      const float s = lds4(sRaw + r * LAY.bytes + LAY.scale);
      return !lds1(mb + M_VALID + r) ? -1.f : s < kLeast ? kLeast : s;
    };
    // Tile i's rows to registers (the copies of the next tile take their place), and s of this thread's position; false when
    // a wait ran out.  Done while S^T of the tile before is under way.
    uint4 code[2][2], rope[2];
    uint32_t blk[2];
    float sc[2], s_row;
    auto read = [&](int i) -> bool {
      if (!wait(M_RAW, i & 1)) return false;
      s_row = scale_of(row);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t at = raw0 + k * 8 * LAY.bytes;
        code[k][0] = lds16(at + (half * 4 + quad) * 32);
        code[k][1] = lds16(at + (half * 4 + quad) * 32 + 16);
        blk[k] = lds32(at + LAY.blocks + (half * 4 + quad) * 4);
        if (ROPE) rope[k] = lds16(at + LAY.tail + half * 64 + quad * 16);
        sc[k] = scale_of(r0 + 8 * k);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (sc[k] < 0.f) {  // (what lies in a masked row's place may be anything; codes are numbers, and zeros times a zero)
          blk[k] = 0;
          rope[k] = make_uint4(0, 0, 0, 0);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_READ);
      return true;
    };
    // ... and to TMEM and shared memory.
    auto convert = [&](int i) -> bool {
      tc_fence_after();  // (TMEM: S^T of the tile before is done)
      // 128 channels' codes as fp16, the halves of a row's four channels side by side as TMEM takes them
      auto to_fp16 = [&](int m, uint32_t (&v)[16]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[8], lo[4], hi[4];
          const uint32_t by = e4m3x2_f16x2((uint16_t)(((blk[k] >> (8 * m)) & 255u) * 0x101u));
          const uint4 c = code[k][m >> 1];
          e2m1x8_f16x2(m & 1 ? c.z : c.x, lo);
          e2m1x8_f16x2(m & 1 ? c.w : c.y, hi);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[j] = mul_f16x2(lo[j], by);
            h[4 + j] = mul_f16x2(hi[j], by);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) v[(j >> 1) * 4 + 2 * k + (j & 1)] = h[j];
        }
      };
      auto to_tmem = [&](int m, const uint32_t (&v)[16]) { tmem_st16x256b(tm_a + L::TM_A + m * 64 + half * 32, v); };
      // (seen by the tensor core with the weights, which every thread stores after this)
      auto to_shared = [&](int m, const uint32_t (&v)[16]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t at = m * 2 * L::CHUNK + k * 1024;
          st_shared_v4(to0 + at, v[2 * k], v[2 * k + 1], v[4 + 2 * k], v[5 + 2 * k]);
          st_shared_v4(to1 + at, v[8 + 2 * k], v[9 + 2 * k], v[12 + 2 * k], v[13 + 2 * k]);
        }
      };
      // S^T's operand: two quarters while P.V of the tile before is under way, one to where P.V will read it, and the last
      uint32_t v[3][16];
      auto quarter = [&](int m) {
        to_fp16(m, v[m]);
        to_tmem(m, v[m]);
      };
      auto in_tmem = [&](int bar) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + bar);
      };
      quarter(0);
      quarter(1);
      in_tmem(M_LAND);
      if (i > 0 && !wait(M_PV, (i - 1) & 1)) return false;
      to_fp16(3, v[2]);
      to_shared(3, v[2]);
      if constexpr (ROPE) {  // P.V has read all of W: the position channels take its place
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float inv = sc[k] < 0.f ? 1.f : __frcp_rn(sc[k]);
          const uint32_t by = pack_bf16x2(inv, inv);
          st_shared_v4(sP + sw128_off(r0 + 8 * k, 4 * half + quad), mul_bf16x2(rope[k].x, by), mul_bf16x2(rope[k].y, by),
                       mul_bf16x2(rope[k].z, by), mul_bf16x2(rope[k].w, by));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_LAND + 8);
      quarter(2);
      in_tmem(M_LAND + 16);
      // the channels that only P.V reads from shared memory, while S^T is under way
#pragma unroll
      for (int m = 0; m < 3; ++m) to_shared(m, v[m]);
      return true;
    };
    // The run's queries: a row a warp, divided by a power of two, its channels in the order in which they lie in TMEM.  A warp
    // asks for all its rows at once and has them come to where they will lie; each is then read before it is written.
    auto load_q = [&](const Seg& s, int run) {
      constexpr int UNITS = DQK / 8;
      auto raw_at = [&](int hh, int u) { return sQ + (u >> 3) * L::Q_CHUNK + sw128_off(hh, u & 7); };
#pragma unroll 1
      for (int hh = cg * 3 + qd; hh < NH; hh += kWorkers) {
        const __nv_bfloat16* src = p.q + (size_t)(hh < s.rows ? s.row0 + hh : s.row0) * DQK + lane * 8;
        const uint32_t size = hh < s.rows ? 16 : 0;
        cp_async16(raw_at(hh, lane), src, size);
        cp_async16(raw_at(hh, lane + 32), src + 256, size);
        if (ROPE && lane < UNITS - 64) cp_async16(raw_at(hh, lane + 64), src + 512, size);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll 1
      for (int hh = cg * 3 + qd; hh < NH; hh += kWorkers) {
        if (hh >= s.rows) {  // (zeros, as they have come)
          if (lane == 0) s_col[(run & 1) * 64 + hh] = 0.f;
          continue;
        }
        uint4 v[3];
        uint32_t top[2] = {0, 0};  // of the first 512 channels, of the position channels
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const int u = lane + 32 * x;
          v[x] = u < UNITS ? lds16(raw_at(hh, u)) : make_uint4(0, 0, 0, 0);
          top[x / 2] = __vmaxu2(top[x / 2], __vmaxu2(__vmaxu2(v[x].x & 0x7fff7fffu, v[x].y & 0x7fff7fffu),
                                                     __vmaxu2(v[x].z & 0x7fff7fffu, v[x].w & 0x7fff7fffu)));
        }
        __syncwarp();
        auto exponent = [&](uint32_t t) {
          return (int)(__reduce_max_sync(0xffffffffu, max(t & 0xffffu, t >> 16)) >> 7) - 127;
        };
        int e = max(exponent(top[0]), -112);
        if (ROPE) e = max(e, exponent(top[1]) - kOver);
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
            int at, chunk = 8;
            if (u < 64) {
              a = pack_f16x2(__uint_as_float(w[2 * g] << 16) * by, __uint_as_float(w[2 * g] & 0xffff0000u) * by);
              b = pack_f16x2(__uint_as_float(w[2 * g + 1] << 16) * by, __uint_as_float(w[2 * g + 1] & 0xffff0000u) * by);
              const int c4 = (u >> 3 & 3) * 4 + 2 * (u & 1) + g;
              chunk = (u >> 1 & 3) * 2 + (u >> 5);
              at = chunk < 6 ? (c4 & 3) * 4 + (c4 >> 2) : c4;
            } else {
              const uint32_t by2 = pack_bf16x2(by, by);
              a = mul_bf16x2(w[2 * g], by2);
              b = mul_bf16x2(w[2 * g + 1], by2);
              at = 2 * (u - 64) + g;  // (these are read from shared memory, as they lie)
            }
            const uint32_t dst = sQ + chunk * L::Q_CHUNK + sw128_off(hh, at >> 1) + (at & 1) * 8;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(a), "r"(b) : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb + M_Q);
    };
    // Maxima or sums over the warp's 32 positions of a thread's columns: the result is that of column own_col.
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
    bool aborted = named_bar_or(bar_id, kTeam, !read_seg(0, sg));
    bool bad = false;
    if (!aborted) load_q(sg, 0);
    int i = 0;
    for (int seg = 0; !aborted; ++seg) {
      const bool more = !sg.last;
      float2 l_part[NC / 2], neg[NC / 2];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) {
        l_part[j] = make_float2(0.f, 0.f);
        neg[j] = make_float2(3.0e38f, 3.0e38f);
      }
      // a column without a finite score yet has a maximum of -3e38, which any finite score passes and which leaves e^-inf at 0
      if (qd == 0 && lane < NC) s_stat[n0 + lane] = -INFINITY;
      named_bar(bar_id, kTeam);
      const float* col = s_col + (seg & 1) * 64 + n0;
      const int t_end = sg.t0 + sg.n;
#pragma unroll 1
      for (int t = sg.t0; t < t_end; ++t, ++i) {
        bad = bad || !read(i);
        bad = bad || !convert(i);
        // the weights without s are 2^(S f - m), m the running maximum of those with it
        if (t == sg.t0) bad = bad || !wait(M_Q, seg & 1);  // (orders the columns' factors before their reads)
        const float s = bad ? -1.f : s_row;
        const float log_s = s > 0.f ? (float)((int)(__float_as_uint(s) >> 23) - 127) : 0.f;  // (masked, or NaN: 0)
        float2 f[NC / 2];
#pragma unroll
        for (int j = 0; j < NC / 4; ++j) {
          const float4 c = *reinterpret_cast<const float4*>(col + 4 * j);
          f[2 * j] = mul2(make_float2(c.x, c.y), make_float2(s, s));
          f[2 * j + 1] = mul2(make_float2(c.z, c.w), make_float2(s, s));
        }
        bad = bad || !wait(M_S, i & 1);
        tc_fence_after();
        __syncwarp();
        const int pos = (int)((unsigned)t * kTile + row);  // (past 2^31: masked by its s)
        const bool partly = p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0;  // some token may not see all of it
        float2 e[NC / 2];
        auto exponents = [&](auto&& add) {
          uint32_t zr[NC];
          tmem_ld<NC>(tmem_addr(tmem, qd * 32, L::TM_S + n0), zr);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < NC / 2; ++j)
            e[j] = fma2(make_float2(__uint_as_float(zr[2 * j]), __uint_as_float(zr[2 * j + 1])), f[j], add(j));
          if (s < 0.f) {
#pragma unroll
            for (int j = 0; j < NC / 2; ++j) e[j] = make_float2(-INFINITY, -INFINITY);
          } else if (partly) {
            const int tok0 = (sg.head0 + n0) / p.H;
            int seen = sg.seen0 + tok0, left = p.H - ((sg.head0 + n0) - tok0 * p.H);
#pragma unroll
            for (int j = 0; j < NC; ++j) {
              if (pos >= seen) (j & 1 ? e[j / 2].y : e[j / 2].x) = -INFINITY;
              if (--left == 0) { left = p.H; ++seen; }
            }
          }
        };
        exponents([&](int j) { return neg[j]; });
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) most = fmaxf(most, fmaxf(e[j].x, e[j].y));
        const bool mine = t == sg.t0 || most > kRaise - log_s;
        bool raise = false;
        if (named_bar_or(bar_id, kTeam, mine || bad)) {
          if (named_bar_or(bar_id, kTeam, bad)) { aborted = true; break; }
          raise = true;
        }
        if (raise) {
          exponents([&](int) { return make_float2(log_s, log_s); });
          float top[NC];
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) { top[2 * j] = e[j].x; top[2 * j + 1] = e[j].y; }
          s_red[qd * 64 + own_col] = over_lanes(top, true);
          named_bar(bar_id, kTeam);
          if (qd == 0 && lane < NC) {
            const int n = n0 + lane;
            const float bm = fmaxf(fmaxf(s_red[n], s_red[64 + n]), s_red[128 + n]) - kTop;
            const float mo = s_stat[n], mn = fmaxf(mo, bm);
            s_stat[n] = mn;
            s_neg[n] = -fmaxf(mn, -3.0e38f);
            s_fac[n] = mo == -INFINITY ? 0.f : exp2f(mo - mn);
          }
          named_bar(bar_id, kTeam);
#pragma unroll
          for (int j = 0; j < NC / 2; ++j) {
            l_part[j] = mul2(l_part[j], *reinterpret_cast<const float2*>(s_fac + n0 + 2 * j));
            neg[j] = *reinterpret_cast<const float2*>(s_neg + n0 + 2 * j);
            e[j] = add2(e[j], add2(neg[j], make_float2(-log_s, -log_s)));
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
          named_bar(bar_id, kTeam);  // the factors have been read
        }
        if (qd == 0 && lane == 0) s_flag[(i & 1) * 4 + cg] = raise;
        const float times = s > 0.f ? s : 1.f;  // (a NaN is in x where the row is seen, and only there)
        uint32_t w[NC / 2];
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          const float2 x = make_float2(ex2(e[j].x), ex2(e[j].y));
          l_part[j] = add2(l_part[j], x);
          const float2 ws = mul2(x, make_float2(times, times));
          w[j] = pack_f16x2(ws.x, ws.y);
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
      if (seg > 0 && !wait(M_EPI, (seg - 1) & 1)) bad = true;  // (its factors have been read)
      // ---- the run's rows: out and lse, or the workspace's partial sums ----
      float sums[NC];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) { sums[2 * j] = l_part[j].x; sums[2 * j + 1] = l_part[j].y; }
      s_red[qd * 64 + own_col] = over_lanes(sums, false);
      named_bar(bar_id, kTeam);
      const bool whole = sg.whole;
      const int slot = 2 * blockIdx.x + (sg.opens ? 1 : 0);
      if (qd == 0 && lane < NC) {
        const int n = n0 + lane;
        const float l = s_red[n] + s_red[64 + n] + s_red[128 + n];
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
        s_fin[(seg & 1) * 64 + n] = fac;
      }
      if (qd == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(mb + M_FAC);
      }
      named_bar(bar_id, kTeam);
      const bool got = wait(M_PV, (i - 1) & 1);
      aborted = named_bar_or(bar_id, kTeam, !got || bad);
      if (aborted) break;
      tc_fence_after();
      store_quarter<NH>(p, sg, tmem, qd, n0, s_out + (seg & 1) * 64);
      tc_fence_before();
      named_bar(bar_id, kTeam);  // s_red, s_stat and s_fac have been read
      if (!more) break;
      sg = nx;
    }
    tmem_st_wait();  // (a wait that ran out may have left one under way)
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    if (lane == 0 && *s_abort) record_error(p.err, DSA_ERR_TIMEOUT);
  }
}

constexpr size_t kRecordOff = kErrorWordBytes, kStatOff = kRecordOff + kRecordBytes, kPartialOff = kStatOff + kStatBytes;

template <int DQK, int NH>
dsa_status_t launch(Params& p, int ctas, cudaStream_t s) {
  using L = Smem<DQK, NH>;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_mla_quant_kernel<DQK, NH>), L::TOTAL,
                                          "configuring paged_mla_quant_kernel");
  if (st != DSA_OK) return st;
  p.G = p.topk_idx ? 1 : (p.H <= NH ? NH / p.H : 1);
  // (64 x 16384, 64 heads, in the state then: 161 us with 2 to 4, 164 with 1; 96 x 4097, 8 heads: 61.9 with 1, 62.7 with 2)
  p.extra = NH == 16 ? 1 : 2;
  p.HB = (p.H + NH - 1) / NH;
  paged_mla_quant_kernel<DQK, NH><<<ctas, kThreads, L::TOTAL, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching paged_mla_quant_kernel");
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
  if ((int64_t)num_pages * page_size > 0x7fffffffll)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: num_pages * page_size must be below 2^31", who);
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
  // 16 columns where a request has no more rows on the average (the host does not know cu_q), or a list: 96 requests to 4097,
  // 8 heads, 61 us and 72 with 64 columns at 4 bits, 52 and 65 at 8; 8 x 8191, 16 heads, 30 and 31, 24 and 28.  An uneven
  // batch under that average pays for it: one chunk of 128 tokens, 16384 positions, beside 127 single tokens of 4096 takes 280 us
  // at 4 bits and 212 at 8, one of 130, which takes the average past 16 rows, 185 and 152.
  const int64_t rows = (int64_t)H * (topk_idx ? 1 : (N + B - 1) / B);
  if (bits == 8) st = launch_paged_mla_e4m3(p, p.q, cache, Dqk, p.sl2e, rows <= 16, ctas, s);
  else if (rows <= 16) st = Dqk == 576 ? pmlaq::launch<576, 16>(p, ctas, s) : pmlaq::launch<512, 16>(p, ctas, s);
  else st = Dqk == 576 ? pmlaq::launch<576, 64>(p, ctas, s) : pmlaq::launch<512, 64>(p, ctas, s);
  if (st != DSA_OK) return st;
  st = pgroups::launch_join(p, ctas, s);
  return st == DSA_OK ? ok() : st;
}
