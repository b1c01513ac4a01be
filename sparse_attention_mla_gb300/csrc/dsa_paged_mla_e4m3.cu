// dsa_paged_mla_e4m3.cu -- attention of new tokens over a paged cache of latents in 8 bits (sm_103a).
//
// For new token j of request b and head h:  z_p = scale <q, kv_p> over the positions p it sees,
// lse = ln sum e^{z_p},  out = sum e^{z_p - lse} kv_p[0:512],  kv_p = code_p s_p (e4m3 times the row's power of two) for the
// first 512 channels, bf16 for the position channels.
//
// The codes go into the products as they lie in the cache: nothing is converted, and shared memory holds 640 bytes a
// position in place of 1152.  s_p stays outside: z_p = s_p <q, code_p> + <q', kv'_p>, the output sums the weights
// w_p = e^{z_p} s_p, and the running maximum is that of w.  The other operands become sums of 8-bit numbers:
//  - a query row, divided by a power of two so that its largest channel lies in [2^7, 2^8), is hi + lo, both e4m3: exact
//    down to 2^-2, and to 2^-10 (2^-17 of the largest channel) below;
//  - a weight is the sum of three e5m2 (2^15 down to 2^-16, 3 bits each): within 2^-11 of itself and, where they run out, to
//    2^-17; the largest weight of a row is between 2^11 and 2^15 (the maximum is raised lazily), so that this is 2^-28 of it.
//    With less a long tail far below one position is off as a whole: its weights are alike, and so are their errors.
// Position channels are multiplied in bf16 and added by the softmax, since s_p must not reach them.
//
// Split of the work as in dsa_paged_groups.cuh, with tiles of 64 positions and groups of 64 rows, or of 16 where a request has
// no more on the average, or a list.  A tile:
//  - 64 rows: S[row, key] = Q K^T with hi and lo of the queries as the 128 lanes (M = 128, N = 64 keys), so that a thread of
//    the softmax has keys of one row.  16 rows: S^T[key, row] = K Q^T (M = 64), hi and lo side by side, which keeps all warps
//    busy; with 64 rows it took the tensor core, whose M = 64 runs at half its rate, 2000 cycles a tile in place of 1300.
//  - an online softmax with a lazily raised maximum;
//  - O^T[channel, row] += V^T W^T (M = 128 channels, K = 32 keys, the weights' parts one after the other into the same
//    columns).  The codes of 128 channels of a key are a row of 128 bytes, which is K-major for the first product and M-major
//    for the second.
//
// What bounds it: 64 requests of 4000 to 16384 positions, 64 heads: 133 us (122 with weights of two parts, e5m2 and e4m3,
// which held 2^-15 of the largest), of which 10 pass before the first scores (cutting the line, the queries), 15 with the
// launches and the joining; the 430 MB of rows are read at 4.0 TB/s in between, where a copy reaches 6.8.  A tile takes 2700
// cycles, and its place in the ring (three tiles of 40 KB beside 72 KB of queries) is in use for 9200: 2000 for its copies,
// 1900 for S, 2300 for the softmax, 3000 for P.V, which is issued behind the next tiles' S; the products share shared memory's
// 128 bytes a cycle (260 KB a tile; with the copies and the softmax 82 % of its cycles are taken).  Measured beside it, with
// weights of two parts: the same rows converted to fp16 as the 4-bit kernel does, 220 us; queries in TMEM and four tiles in
// the ring, 136 (queries that a thread loads by its row cost 13 us a run); copies by TMA boxes, 206.
//
// Warps: 0 issues S, the next 16 (or 8) softmax and epilogue, four copy tiles into the ring, one issues P.V, one announces the
// runs of tiles that the CTA's range consists of.
#include <climits>
#include <cmath>

#include "dsa_f32x2.cuh"
#include "dsa_paged_groups.cuh"
#include "dsa_paged_mla_quant.h"
#include "dsa_paged_quant.cuh"

namespace dsa {
namespace pmla8 {

using namespace pgroups;

constexpr int kTile = 64;
constexpr int kGather = 4;       // warps that copy
constexpr float kRaise = 15.0f;    // log2 units: the running maximum is raised when a weight passes 2^15 (e5m2 ends at 1.75 2^15)
constexpr float kTop = 11.0f;      // a new maximum is 2^11 (2^9: fewer rescales, 2 % less time at 64 x 16384; four times the floor)
constexpr float kMost = 32768.0f;  // 2^kRaise
constexpr float kLeast = 3.5527136788005009e-15f;  // 2^-48, the least s

template <int DQK, int NH>
struct Smem {
  static constexpr bool ROPE = DQK == 576;
  static constexpr QuantRow LAY = quant_row(DQK, kDv, 8);
  static constexpr int NCH = ROPE ? 5 : 4;      // 128 codes each, then the position channels
  static constexpr int CHUNK = kTile * 128;
  static constexpr int Q_CHUNK = 2 * NH * 128;  // hi rows, lo rows
  static constexpr int R = NH == 64 ? 3 : 4;    // tiles in the ring
  // 64 rows: S[row, key], hi and lo rows as M = 128 (of each warp's 32 lanes the first 16 hi, the others lo);
  // 16 rows: S^T[key, row], M = 64 keys, hi and lo side by side.
  static constexpr bool ROWS = NH == 64;
  static constexpr int W = ROWS ? 16 : 8;       // softmax warps
  static constexpr int THREADS = 32 * (W + kGather + 3);
  static constexpr int READERS = W + kGather + 2;  // warps that read an announcement
  static constexpr int SW = ROWS ? (ROPE ? 2 : 1) * kTile : (ROPE ? 3 : 2) * NH;  // TMEM columns of S
  // W, two buffers.  64 rows: a row's 64 keys of the first part and of the second side by side, and the third parts of both
  // buffers so in a block of their own; 16 rows: the first part beside the third, then rows of the second.
  static constexpr int P_BLOCK = NH * 128 * (ROWS ? 1 : 2);
  static constexpr int P_BYTES = (ROWS ? 3 : 2) * P_BLOCK;
  static constexpr int QR_CHUNK = NH * 128;  // position channels
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_Q = R * NCH * CHUNK;
  static constexpr int OFF_P = OFF_Q + 4 * Q_CHUNK + (ROPE ? QR_CHUNK : 0);
  static constexpr int OFF_MISC = OFF_P + P_BYTES;
  static constexpr int MISC = 8192;
  static constexpr int TOTAL = OFF_MISC + MISC;
  static_assert(TOTAL <= 232448 && OFF_P % 1024 == 0 && P_BLOCK % 1024 == 0, "shared memory budget");
  static constexpr int TM_O = (2 * SW + 31) / 32 * 32;
  static constexpr int TM_COLS = NH == 64 ? 512 : 256;
  static_assert(TM_O + 4 * NH <= TM_COLS, "TMEM budget");
};

// misc (bytes)
constexpr int kSlots = 4;
constexpr int M_KV = 0, M_PV = 32, M_S = 64, M_SF = 80, M_P = 96, M_Q = 112, M_FIN = 120;  // [4] [4] [2] [2] [2] 1 [2]
constexpr int M_SEGF = 136, M_SEGE = M_SEGF + 8 * kSegs;  // [kSegs] each: announced, read by all
constexpr int M_TMEM = 264, M_ABORT = 268, M_PLAN = 272;  // plan: 56 bytes
constexpr int M_SEG = 336;                    // int4 [kSegs][2]
constexpr int M_RED = 592;                    // float [4][64]; the first row also holds the factors of a rescale
constexpr int M_STAT = M_RED + 1024;          // float [64]
constexpr int M_COL = M_STAT + 256;           // float [2][64]: a column's factor of the score, by run
constexpr int M_SCALE = M_COL + 512;          // float [kSlots][64]: s of the rows, -1: masked
constexpr int M_RAW = 4096;                   // float4 [kSlots][64]: s of the rows as it comes, -1: masked
constexpr int M_MASKED = M_SCALE + kSlots * 256;  // uint8 [kSlots]: some row of a tile is masked
static_assert(M_SEGE + 8 * kSegs <= M_TMEM && M_PLAN + 56 <= M_SEG && M_SEG % 16 == 0 && M_SCALE % 16 == 0 &&
                  M_MASKED + kSlots <= M_RAW, "misc layout");

struct Params : GroupParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  float sl2e;
};

// Instruction descriptor for kind::f8f6f4 with fp32 D: formats 0 e4m3, 1 e5m2.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_format, int b_format, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((uint32_t)a_format << 7) | ((uint32_t)b_format << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// As mma4_w, of two or four MMAs of 8-bit operands (32 elements of K each).
template <int N, int SA, int SB>
__device__ __forceinline__ void mma_f8_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add_first) {
  static_assert(N == 2 || N == 4, "MMAs");
  if constexpr (N == 4) {
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, %6;\n\tadd.s64 a3, %1, %7;\n\t"
        "add.s64 b1, %2, %8;\n\tadd.s64 b2, %2, %9;\n\tadd.s64 b3, %2, %10;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(add_first), "n"(SA), "n"(2 * SA), "n"(3 * SA), "n"(SB), "n"(2 * SB), "n"(3 * SB)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a1, b1;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "add.s64 a1, %1, %5;\n\tadd.s64 b1, %2, %6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(add_first), "n"(SA), "n"(SB)
        : "memory");
  }
}

// Two values to e4m3 or e5m2 (the first in the lower half), and e5m2 back.
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(float2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
  return r;
}
__device__ __forceinline__ float2 e5m2x2_floats(uint32_t v) {  // (the upper half of an fp16 number)
  return f16x2_floats(__byte_perm(v, 0, 0x1404));
}
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t v) { return f16x2_floats(e4m3x2_f16x2((uint16_t)v)); }
__device__ __forceinline__ float2 minus2(float2 a, float2 b) { return add2(a, make_float2(-b.x, -b.y)); }
// Two weights as sums of three e5m2 (what each leaves is exact in fp32).
__device__ __forceinline__ void parts(float2 w, uint32_t (&r)[3]) {
  r[0] = e5m2x2(w);
  w = minus2(w, e5m2x2_floats(r[0]));
  r[1] = e5m2x2(w);
  r[2] = e5m2x2(minus2(w, e5m2x2_floats(r[1])));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

// 16 TMEM lanes x 64 bits, four times: thread t of the warp gets lane base + (t >> 2) + 8 (t & 1) and the columns
// c + 2j + ((t >> 1) & 1), j = 0..3.
__device__ __forceinline__ void tmem_ld16x64b(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x64b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// 16 TMEM lanes, a thread 8 columns of one: threads 0-15 from column c, 16-31 from column c + 8.
__device__ __forceinline__ void tmem_ld16x32bx2(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(a));
}
__device__ __forceinline__ void st_shared_v2(uint32_t at, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float4 lds4f(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

template <int DQK, int NH>
__global__ void __launch_bounds__(Smem<DQK, NH>::THREADS, 1) paged_mla_e4m3_kernel(const __grid_constant__ Params p) {
  using L = Smem<DQK, NH>;
  constexpr bool ROPE = L::ROPE;
  constexpr int NCH = L::NCH, R = L::R;
  constexpr bool ROWS = L::ROWS;
  constexpr int W = L::W, NHH = NH / (W / 4), NQ = 4;  // columns of O^T of four softmax warps; rows of a thread (16 rows)
  constexpr int kKeys = 8;  // keys of a thread (64 rows)
  static_assert(R <= kSlots, "ring");
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sKV = smem_u32(smem) + L::OFF_KV, sQ = smem_u32(smem) + L::OFF_Q, sP = smem_u32(smem) + L::OFF_P;
  uint8_t* misc = smem + L::OFF_MISC;
  const uint32_t mb = smem_u32(misc);
  const uint32_t bar_kv = mb + M_KV, bar_pv = mb + M_PV, bar_s = mb + M_S, bar_sf = mb + M_SF, bar_p = mb + M_P,
                 bar_q = mb + M_Q, bar_fin = mb + M_FIN;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + M_ABORT);
  Plan* s_plan = reinterpret_cast<Plan*>(misc + M_PLAN);
  const uint32_t sScale = smem_u32(misc + M_SCALE), sRaw = smem_u32(misc + M_RAW);
  volatile float* s_raw = reinterpret_cast<volatile float*>(misc + M_RAW);
  volatile float* s_scale = reinterpret_cast<volatile float*>(misc + M_SCALE);
  auto scale_of = [&](int at) {  // (a row that was never written, of zero bytes, holds zeros; -1: masked)
    const float s = s_raw[4 * at];
    return s >= 0.f && s < kLeast ? kLeast : s;
  };
  volatile uint8_t* s_masked = misc + M_MASKED;
  float* s_stat = reinterpret_cast<float*>(misc + M_STAT);
  float* s_fac = reinterpret_cast<float*>(misc + M_RED);  // a column's factor replaces its first maximum or sum
  float* s_red = reinterpret_cast<float*>(misc + M_RED);
  float* s_col = reinterpret_cast<float*>(misc + M_COL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // tile i has landed; P.V has read it
  auto wait_kv = [&](int i) { return wait_for(bar_kv + 8 * (i % R), (i / R) & 1, s_abort, p.wait_limit); };
  auto wait_pv = [&](int i) { return wait_for(bar_pv + 8 * (i % R), (i / R) & 1, s_abort, p.wait_limit); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(bar_kv + 8 * s, 4 * 33);  // four warps: each lane's copies, and what the warp has stored
      mbar_init(bar_pv + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_s + 8 * b, ROWS ? 2 : 1);
      mbar_init(bar_sf + 8 * b, W);
      mbar_init(bar_p + 8 * b, W);
      mbar_init(bar_fin + 8 * b, 1);
    }
    mbar_init(bar_q, W);
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(mb + M_SEGF + 8 * k, 1);
      mbar_init(mb + M_SEGE + 8 * k, L::READERS);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  make_plan<kTile, L::THREADS>(p, s_plan, reinterpret_cast<long long*>(s_red));
  const Plan plan = *s_plan;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the joining kernel waits for this one's end itself)
  if (plan.w1 <= plan.w0 || plan.w1 - plan.w0 <= plan.skip) return;  // (the whole CTA)
  if (warp == 0) {
    tmem_alloc(smem_u32(s_tmem), L::TM_COLS);
    tmem_relinquish();
  }
  uint32_t tmem = 0;
  if (warp <= W || warp == W + 5) {  // the others neither need it nor wait for it
    named_bar(3, 32 * (W + 2));
    tmem = (uint32_t)warp_value((int)*s_tmem);
  }
  // announcement k, once per warp
  auto read_seg = [&](int k, Seg& s) -> bool {
    return read_announcement(mb + M_SEGF, mb + M_SEGE, reinterpret_cast<const int4*>(misc + M_SEG), k, s_abort, p.wait_limit, s);
  };
  if (warp == 0) {
    // ======================= S issuer =======================
    constexpr uint32_t kIdS = ROWS ? idesc_f8(128, kTile, 0, 0, false, false) : idesc_f8(kTile, 2 * NH, 0, 0, false, false);
    constexpr uint32_t kIdR = idesc_bf16(64, ROWS ? kTile : NH, false, false);
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      if (!warp_all(wait_for(bar_q, seg & 1, s_abort, p.wait_limit))) break;
      // what the loop needs in registers of the warp (a call does not keep them)
      const int n = warp_value(sg.n);
      const uint32_t d0 = (uint32_t)warp_value((int)tmem), q0 = (uint32_t)warp_value((int)sQ), kv0 = (uint32_t)warp_value((int)sKV);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const int sl = i % R, sb = i & 1;
        if (i >= 2 && !warp_all(wait_for(bar_sf + 8 * sb, ((i >> 1) - 1) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        const uint64_t a0 = sdesc_sw128(kv0, 16, 1024) + (uint64_t)(uint32_t)(sl * NCH * (L::CHUNK >> 4));
        const uint64_t b0 = sdesc_sw128(q0, 16, 1024);
        if (!warp_all(wait_kv(i))) { stop = true; break; }
        fence_proxy_async_smem();  // (the rows came by cp.async)
        tc_fence_after();
        if constexpr (ROWS) {
          // (position channels by M = 64, whose rows are the first 16 lanes of every 32, as the hi rows are of the others)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mma_f8_w<4, 2, 2>(d0 + sb * L::SW, b0 + c * (L::Q_CHUNK >> 4), a0 + c * (L::CHUNK >> 4), kIdS, c);
          if (ROPE) mma4_w<2, 2>(d0 + sb * L::SW + kTile, b0 + 4 * (L::Q_CHUNK >> 4), a0 + 4 * (L::CHUNK >> 4), kIdR, 0);
          // what the softmax needs of s, once for all rows: -1: masked; whether there are such
          bool masked = false;
#pragma unroll
          for (int x = 0; x < kTile; x += 32) {
            const float v = scale_of(sl * kTile + x + lane);
            s_scale[sl * kTile + x + lane] = v;
            masked |= v < 0.f;
          }
          masked = __any_sync(0xffffffffu, masked);
          if (lane == 0) s_masked[sl] = masked;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_s + 8 * sb);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mma_f8_w<4, 2, 2>(d0 + sb * L::SW, a0 + c * (L::CHUNK >> 4), b0 + c * (L::Q_CHUNK >> 4), kIdS, c);
          if (ROPE) mma4_w<2, 2>(d0 + sb * L::SW + 2 * NH, a0 + 4 * (L::CHUNK >> 4), b0 + 4 * (L::Q_CHUNK >> 4), kIdR, 0);
        }
        mma_commit_w(bar_s + 8 * sb);
      }
      if (stop) break;
    }
    mma_commit_w(bar_fin);
    volatile int dummy = 0;
    mbar_wait(bar_fin, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == W + 5) {
    // ======================= P.V issuer =======================
    int done = 0;
    for (int seg = 0, last = 0; !last; ++seg) {
      Seg sg;
      if (!warp_all(read_seg(seg, sg))) break;
      last = warp_value(sg.last ? 1 : 0);
      const int n = warp_value(sg.n);
      const uint32_t d0 = (uint32_t)warp_value((int)tmem), kv0 = (uint32_t)warp_value((int)sKV), p0 = (uint32_t)warp_value((int)sP);
      int i = warp_value(done);
      done += n;
      bool stop = false;
#pragma unroll 1
      for (int k0 = 0; k0 < n; ++k0, ++i) {
        const int sl = i % R;
        const uint32_t add = k0 > 0;  // the segment's first tile overwrites O^T
        if (!warp_all(wait_for(bar_p + 8 * (i & 1), (i >> 1) & 1, s_abort, p.wait_limit))) { stop = true; break; }
        fence_proxy_async_smem();
        tc_fence_after();
        constexpr uint32_t kId = idesc_f8(128, NH, 0, 1, true, false);
        const uint64_t va = sdesc_sw128(kv0, 16, 1024) + (uint64_t)(uint32_t)(sl * NCH * (L::CHUNK >> 4));
        // W: a row for each row of the group, keys along K
        const uint64_t pb = sdesc_sw128(p0, 16, 1024) + (uint64_t)(uint32_t)((i & 1) * (L::P_BLOCK >> 4));
        constexpr int kSecond = ROWS ? 64 >> 4 : NH * 128 >> 4, kStep = 2;
        const uint64_t pc = ROWS ? sdesc_sw128(p0 + 2 * L::P_BLOCK, 16, 1024) + (uint64_t)(uint32_t)((i & 1) * (64 >> 4))
                                 : pb + (64 >> 4);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t a = va + m * (L::CHUNK >> 4);
          mma_f8_w<2, (32 * 128 >> 4), kStep>(d0 + L::TM_O + m * NH, a, pb, kId, add);
          mma_f8_w<2, (32 * 128 >> 4), kStep>(d0 + L::TM_O + m * NH, a, pb + kSecond, kId, 1);
          mma_f8_w<2, (32 * 128 >> 4), kStep>(d0 + L::TM_O + m * NH, a, pc, kId, 1);
        }
        mma_commit_w(bar_pv + 8 * sl);
      }
      if (stop) break;
    }
    mma_commit_w(bar_fin + 8);
    volatile int dummy = 0;
    mbar_wait(bar_fin + 8, 0, &dummy, p.err);
    __syncwarp();
  } else if (warp == W + 6) {
    announce<kTile>(p, plan, mb + M_SEGF, mb + M_SEGE, reinterpret_cast<int4*>(misc + M_SEG), s_abort);
  } else if (warp > W) {
    // ======================= gather: 16 rows of every tile each =======================
    // By cp.async, which takes any row, a warp's instruction the 512 codes of one, and says itself when it has landed; what is
    // masked is filled with zeros.  A lane looks one row up, in steps whose loads have a tile's time to come back: the list's
    // entry (three tiles ahead), the page (two ahead), the row number (one ahead, and its lines are asked for in L2: without,
    // 132 us in place of 125; runs of rows by bulk prefetch, 126).  s comes as a copy too, of its 16 bytes (four would go through
    // L1: 122.5 us in place of 121): a load whose value moves from one register to another in the loop holds the warp up until it
    // is there.  L2 gives 995 bytes a row, since eight lanes' 128 bytes begin anywhere in a line; eight lanes a line of their own
    // took 124.
    constexpr int kRows = kTile / 4;
    const int gw = warp - W - 1;
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
        const int j = (sg.t0 + i - base) * kTile + gw * kRows + lane;
        if (lane < kRows && j < sg.keys) k.pos = p.topk_idx ? __ldg(p.topk_idx + (size_t)(sg.row0 / p.H) * p.K + j) : j;
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
    auto row_of = [&](int pos, int page) -> int {
      if (pos < 0) return -1;
      if (page >= 0 && page < p.num_pages) return page * p.P + pos;
      bad_index = true;
      return -1;
    };
    auto to_l2 = [&](int row) {
#pragma unroll
      for (int x = 0; x < kRows; x += 4) {  // four rows, eight lanes each
        const int at = __shfl_sync(0xffffffffu, row, x + (lane >> 3));
        if (at >= 0 && (lane & 7) * 128 < L::LAY.bytes)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cache + (size_t)at * L::LAY.bytes + (lane & 7) * 128));
      }
    };
    Look look[3];
    int page[2], row[2];  // rows of the next two tiles
#pragma unroll
    for (int k = 0; k < 3; ++k) look[k] = position(k);
    page[0] = page_of(look[0]);
    page[1] = page_of(look[1]);
    row[0] = row_of(look[0].pos, page[0]);
    row[1] = row_of(look[1].pos, page[1]);
    look[0] = look[2];
    page[0] = page_of(look[0]);
    look[1] = position(3);
    to_l2(row[1]);
#pragma unroll 1
    for (int i = 0; i < n_tiles && !stop; ++i) {
      const int sl = i % R;
      if (i >= R && !warp_all(wait_pv(i - R))) { stop = true; break; }
      if (lane < kRows) {
        const int r = sl * kTile + gw * kRows + lane;
        if (row[0] < 0) s_raw[4 * r] = -1.f;
        else cp_async16(sRaw + 16 * r, p.cache + (size_t)row[0] * L::LAY.bytes + L::LAY.scale, 16);
      }
      const uint32_t to = sKV + sl * NCH * L::CHUNK;
#pragma unroll
      for (int x0 = 0; x0 < kRows; x0 += 8) {  // eight rows at a time: a copy's registers are free only when it has been taken
        const uint8_t* src[8];
        uint32_t size[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int at = __shfl_sync(0xffffffffu, row[0], x0 + y);
          src[y] = p.cache + (size_t)max(at, 0) * L::LAY.bytes + lane * 16;
          size[y] = at >= 0 ? 16u : 0u;
        }
#pragma unroll
        for (int y = 0; y < 8; ++y)
          cp_async16(to + (lane >> 3) * L::CHUNK + sw128_off(gw * kRows + x0 + y, lane & 7), src[y], size[y]);
      }
      if constexpr (ROPE) {
#pragma unroll
        for (int x0 = 0; x0 < kRows; x0 += 4) {  // four rows' position channels
          const int at = __shfl_sync(0xffffffffu, row[0], x0 + (lane >> 3));
          cp_async16(to + 4 * L::CHUNK + sw128_off(gw * kRows + x0 + (lane >> 3), lane & 7),
                     p.cache + (size_t)max(at, 0) * L::LAY.bytes + L::LAY.tail + (lane & 7) * 16, at >= 0 ? 16u : 0u);
        }
      }
      cp_async_arrive(bar_kv + 8 * sl);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_kv + 8 * sl);
      row[0] = row[1];
      row[1] = row_of(look[0].pos, page[0]);
      look[0] = look[1];
      page[0] = page_of(look[0]);
      look[1] = position(i + 4);
      to_l2(row[1]);
    }
    if (bad_index) record_error(p.err, DSA_ERR_DEVICE_INDEX);
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing lands after the CTA has left
  } else {
    // ======================= softmax + epilogue =======================
    const int wk = warp - 1, qd = warp & 3, ch = wk >> 2;
    const int par = (lane >> 1) & 1;
    const int r = qd * 16 + (lane >> 2) + 8 * (lane & 1);  // key row of the tile
    const int n0 = ch * NHH + par * NQ;  // this thread's rows n0 .. n0 + NQ - 1 of the group
    // or (ROWS) its row of the group, and its keys of the tile
    const int my_row = qd * 16 + (lane & 15), k0 = ch * 16 + (lane >> 4) * kKeys;
    // warps that share rows, and meet at barriers
    const int bar_id = ROWS ? 1 : 1 + ch;
    constexpr int kTeam = ROWS ? 32 * W : 128;
    // row hh of the group in Q, its hi or its lo
    auto q_row = [&](int hh, int lo) { return ROWS ? (hh >> 4) * 32 + (hh & 15) + 16 * lo : hh + NH * lo; };
    // The run's queries: a row a warp, as hi and lo, and what the sums of a column are to be multiplied by.  A warp asks for
    // all its rows at once (one or two at a time, each with the time of a read from DRAM: 16000 cycles in place of 4000) and
    // has them come to where their hi and lo will lie, which are as large together; each is then read before it is written.
    auto load_q = [&](const Seg& s, int run) {
      auto raw_at = [&](int hh, int u) { return sQ + (u >> 4) * L::Q_CHUNK + sw128_off(q_row(hh, u >> 3 & 1), u & 7); };
#pragma unroll 1
      for (int hh = wk; hh < NH; hh += W) {
        const __nv_bfloat16* src = p.q + (size_t)(hh < s.rows ? s.row0 + hh : s.row0) * DQK + lane * 8;
        const uint32_t size = hh < s.rows ? 16 : 0;
        cp_async16(raw_at(hh, lane), src, size);
        cp_async16(raw_at(hh, lane + 32), src + 256, size);
        if (ROPE && lane < 8) cp_async16(sQ + 4 * L::Q_CHUNK + sw128_off(hh, lane), src + 512, size);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll 1
      for (int hh = wk; hh < NH; hh += W) {
        uint4 v[2];
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t at = raw_at(hh, lane + 32 * x);
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[x].x), "=r"(v[x].y), "=r"(v[x].z), "=r"(v[x].w) : "r"(at) : "memory");
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[x].x & 0x7fff7fffu, v[x].y & 0x7fff7fffu),
                                       __vmaxu2(v[x].z & 0x7fff7fffu, v[x].w & 0x7fff7fffu)));
        }
        __syncwarp();
        const uint32_t most = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const int e = max((int)(most >> 7) - 127, -119);
        const float by = pow2(7 - e);
        // (a row with a channel that is not finite gives NaN)
        const float factor = most >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e - 7) * (ROWS ? 1.f : p.sl2e);
        if (lane == 0) s_col[(run & 1) * 64 + hh] = factor;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int u = lane + 32 * x;
          const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float2 a = make_float2(__uint_as_float(w[g] << 16) * by, __uint_as_float(w[g] & 0xffff0000u) * by);
            hi[g] = e4m3x2(a);
            lo[g] = e4m3x2(minus2(a, e4m3x2_floats(hi[g])));
          }
          const uint32_t at = sQ + (u >> 4) * L::Q_CHUNK + (u & 1) * 8;
          st_shared_v2(at + sw128_off(q_row(hh, 0), (u & 15) >> 1), hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          st_shared_v2(at + sw128_off(q_row(hh, 1), (u & 15) >> 1), lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q);
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
    // the running maxima of the team's rows, from those of the tile in s_red, and the factors of what has been summed so far
    auto new_maxima = [&]() {
      if (qd == 0 && lane < NHH) {
        const int n = ch * NHH + lane;
        const float bm = fmaxf(fmaxf(s_red[n], s_red[NH + n]), fmaxf(s_red[2 * NH + n], s_red[3 * NH + n]));
        const float mo = s_stat[n], mn = fmaxf(mo, bm - kTop);
        s_stat[n] = mn;
        s_fac[n] = mo == -INFINITY ? 0.f : exp2f(mo - mn);
      }
    };
    auto rescale = [&]() {
#pragma unroll 1
      for (int x = 0; x < 4 * (NHH / 8); ++x) {  // 8 columns at a time
        const int h0 = ch * NHH + (x % (NHH / 8)) * 8;
        const uint32_t ta = tmem_addr(tmem + L::TM_O + x / (NHH / 8) * NH + h0, qd * 32, 0);
        uint32_t ov[8];
        tmem_ld8(ta, ov);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 8; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * s_fac[h0 + h]);
        tmem_st8(ta, ov);
      }
      tmem_st_wait();
    };
    Seg sg, nx;
    // (one answer for the team: its warps meet at barriers from here on)
    bool aborted = named_bar_or(bar_id, kTeam, !read_seg(0, sg));
    if (!aborted) load_q(sg, 0);
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
      if (qd == 0 && lane < NHH) s_stat[ch * NHH + lane] = -INFINITY;  // (read only after a barrier of the team)
      const float* col = s_col + ((seg - 1) & 1) * 64 + n0;
      float2 l_row = make_float2(0.f, 0.f);
      float neg = 3.0e38f, factor = 0.f;
      const int seen = sg.seen0 + (sg.head0 + my_row) / p.H;
      const int t_end = sg.t0 + sg.n;
#pragma unroll 1
      for (int t = sg.t0; t < t_end; ++t, ++i) {
        const int sl = i % R, sb = i & 1;
        bool bad = bad_seg || !warp_all(wait_for(bar_s + 8 * sb, (i >> 1) & 1, s_abort, p.wait_limit));
        // (complete since before S^T was issued: order the rows' scales and the columns' factors before their reads below)
        if (!ROWS) bad = bad || !warp_all(wait_kv(i));
        if (t == sg.t0) bad = bad || !warp_all(wait_for(bar_q, (seg - 1) & 1, s_abort, p.wait_limit));
        // W of tile i overwrites what P.V of tile i - 2 read
        if (i >= 2) bad = bad || !warp_all(wait_pv(i - 2));
        tc_fence_after();
        __syncwarp();
        if constexpr (ROWS) {
          if (t == sg.t0) factor = s_col[((seg - 1) & 1) * 64 + my_row];
          uint32_t v[kKeys], x[kKeys], w[kKeys];  // scores before softmax_scale; e^z; the weights
          const uint32_t ts = tmem_addr(tmem + sb * L::SW + ch * 16, qd * 32, 0);
          tmem_ld16x32bx2(ts, v);
          tmem_ld16x32bx2(ts + (16u << 16), x);
          if constexpr (ROPE) tmem_ld16x32bx2(ts + kTile, w);
          const uint32_t scales = sScale + (sl * kTile + k0) * 4;
          const float4 sx = lds4f(scales), sy = lds4f(scales + 16);
          const float2 s2[kKeys / 2] = {{sx.x, sx.y}, {sx.z, sx.w}, {sy.x, sy.y}, {sy.z, sy.w}};
          const bool some = s_masked[sl] || (p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sf + 8 * sb);
          auto at2 = [](const uint32_t (&a)[kKeys], int j) {
            return make_float2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
          };
          auto set2 = [](uint32_t (&a)[kKeys], int j, float2 y) {
            a[2 * j] = __float_as_uint(y.x);
            a[2 * j + 1] = __float_as_uint(y.y);
          };
#pragma unroll
          for (int j = 0; j < kKeys / 2; ++j) {
            const float2 sum = mul2(add2(at2(v, j), at2(x, j)), s2[j]), by = make_float2(factor, factor);
            set2(v, j, ROPE ? fma2(sum, by, at2(w, j)) : mul2(sum, by));
          }
          if (t + 1 == t_end && more && !bad) load_q(nx, seg);  // S of the segment is done: Q is free
          auto hidden = [&](int j) {
            return (j & 1 ? s2[j / 2].y : s2[j / 2].x) < 0.f || (p.topk_idx == nullptr && t * kTile + k0 + j >= seen);
          };
          auto weights = [&]() -> float {
#pragma unroll
            for (int j = 0; j < kKeys / 2; ++j) {
              const float2 e = fma2(at2(v, j), make_float2(p.sl2e, p.sl2e), make_float2(neg, neg));
              const float2 y = make_float2(ex2(e.x), ex2(e.y));
              set2(x, j, y);
              set2(w, j, mul2(y, s2[j]));
            }
            if (some) {
#pragma unroll
              for (int j = 0; j < kKeys; ++j)
                if (hidden(j)) x[j] = w[j] = 0;
            }
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) most = fmaxf(most, __uint_as_float(w[j]));
            return most;
          };
          const bool mine = weights() > kMost || t == sg.t0;
          if (named_bar_or(bar_id, kTeam, mine || bad)) {
            if (named_bar_or(bar_id, kTeam, bad)) { aborted = true; break; }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
              const float s = j & 1 ? s2[j / 2].y : s2[j / 2].x;
              const float z = __uint_as_float(v[j]) * p.sl2e + (float)((int)(__float_as_uint(s) >> 23) - 127);
              if (s > 0.f && !(some && hidden(j))) top = fmaxf(top, z);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (lane < 16) s_red[ch * NH + my_row] = top;
            named_bar(bar_id, kTeam);
            new_maxima();
            named_bar(bar_id, kTeam);
            l_row = mul2(l_row, make_float2(s_fac[my_row], s_fac[my_row]));
            neg = -fmaxf(s_stat[my_row], -3.0e38f);
            weights();
            if (t > sg.t0) {
              const bool okw = wait_pv(i - 1);
              if (named_bar_or(bar_id, kTeam, !okw)) { aborted = true; break; }
              tc_fence_after();
              rescale();
            }
          }
          uint32_t part[3][2];
#pragma unroll
          for (int j = 0; j < kKeys / 2; j += 2) {
            l_row = add2(l_row, add2(at2(x, j), at2(x, j + 1)));
            uint32_t w0[3], w1[3];
            parts(at2(w, j), w0);
            parts(at2(w, j + 1), w1);
#pragma unroll
            for (int k = 0; k < 3; ++k) part[k][j / 2] = w0[k] | w1[k] << 16;
          }
          const uint32_t to = sP + (i & 1) * L::P_BLOCK + (k0 & 8), third = sP + 2 * L::P_BLOCK + (k0 & 8);
          st_shared_v2(to + sw128_off(my_row, ch), part[0][0], part[0][1]);
          st_shared_v2(to + sw128_off(my_row, 4 + ch), part[1][0], part[1][1]);
          st_shared_v2(third + sw128_off(my_row, 4 * (i & 1) + ch), part[2][0], part[2][1]);
        } else {
          uint32_t raw[NQ];
          float2 z[NQ / 2];  // (alternate columns of the half first)
          const uint32_t ts = tmem_addr(tmem + sb * L::SW + ch * NHH, qd * 32, 0);
          {
            uint32_t lo[NQ], pos[NQ];
            tmem_ld16x64b(ts, raw);
            tmem_ld16x64b(ts + NH, lo);
            if constexpr (ROPE) tmem_ld16x64b(ts + 2 * NH, pos);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_sf + 8 * sb);
#pragma unroll
            for (int j = 0; j < NQ; ++j) raw[j] = __float_as_uint(__uint_as_float(raw[j]) + __uint_as_float(lo[j]));
            // -> NQ consecutive rows: swap half of them with the key's other thread
            auto rows_of = [&](uint32_t (&x)[NQ], int j) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, par ? x[j] : x[NQ / 2 + j], 2);
              return make_float2(__uint_as_float(par ? got : x[j]), __uint_as_float(par ? x[NQ / 2 + j] : got));
            };
            const float s = scale_of(sl * kTile + r);
            const float log_s0 = s > 0.f ? (float)((int)(__float_as_uint(s) >> 23) - 127) : 0.f;
#pragma unroll
            for (int j = 0; j < NQ / 2; ++j) {
              const float2 f = mul2(*reinterpret_cast<const float2*>(col + 2 * j), make_float2(s, s));
              float2 c = make_float2(log_s0, log_s0);
              if constexpr (ROPE) c = fma2(rows_of(pos, j), make_float2(p.sl2e, p.sl2e), c);
              z[j] = fma2(rows_of(raw, j), f, c);
            }
          }
          if (t + 1 == t_end && more && !bad) load_q(nx, seg);  // S^T of the segment is done: Q is free
          const float s = scale_of(sl * kTile + r);
          const float inv_s = s > 0.f ? pow2(127 - (int)(__float_as_uint(s) >> 23)) : 1.f;
          const int pos = t * kTile + r;
          if (s < 0.f) {
#pragma unroll
            for (int j = 0; j < NQ / 2; ++j) z[j] = make_float2(-INFINITY, -INFINITY);
          } else if (p.topk_idx == nullptr && (t + 1) * (long long)kTile > sg.seen0) {  // some token may not see all of it
            int seen = sg.seen0 + tok0, left = head_left;
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
              if (pos >= seen) (j & 1 ? z[j / 2].y : z[j / 2].x) = -INFINITY;
              if (--left == 0) { left = p.H; ++seen; }
            }
          }
          // the exponents of the weights; one may pass its row's maximum by the threshold
          float2 e[NQ / 2];
          bool mine = t == sg.t0;
#pragma unroll
          for (int j = 0; j < NQ / 2; ++j) {
            e[j] = add2(z[j], m_neg[j]);
            mine |= e[j].x > kRaise || e[j].y > kRaise;
          }
          bool raise = false;
          if (named_bar_or(bar_id, kTeam, mine || bad)) {
            if (named_bar_or(bar_id, kTeam, bad)) { aborted = true; break; }
            raise = true;
          }
          if (raise) {
            float top[NQ];
#pragma unroll
            for (int j = 0; j < NQ / 2; ++j) { top[2 * j] = z[j].x; top[2 * j + 1] = z[j].y; }
            s_red[qd * NH + sum_row] = over_keys(top, true);
            named_bar(bar_id, kTeam);
            new_maxima();
            named_bar(bar_id, kTeam);
#pragma unroll
            for (int j = 0; j < NQ / 2; ++j) {
              l_part[j] = mul2(l_part[j], make_float2(s_fac[n0 + 2 * j], s_fac[n0 + 2 * j + 1]));
              m_neg[j] = make_float2(-fmaxf(s_stat[n0 + 2 * j], -3.0e38f), -fmaxf(s_stat[n0 + 2 * j + 1], -3.0e38f));
              e[j] = add2(z[j], m_neg[j]);
            }
            if (t > sg.t0) {
              const bool okw = wait_pv(i - 1);
              if (named_bar_or(bar_id, kTeam, !okw)) { aborted = true; break; }
              tc_fence_after();
              rescale();
            }
          }
          uint32_t part[NQ / 2][3];
#pragma unroll
          for (int j = 0; j < NQ / 2; ++j) {
            const float2 w = make_float2(ex2(e[j].x), ex2(e[j].y));
            l_part[j] = fma2(w, make_float2(inv_s, inv_s), l_part[j]);
            parts(w, part[j]);
          }
          const uint32_t to = sP + (i & 1) * L::P_BLOCK;
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            const int n = n0 + j;
            const uint32_t at = to + (uint32_t)(n * 128 + (((r >> 4) ^ (n & 7)) << 4) + (r & 15));
            const uint32_t third = to + (uint32_t)(n * 128 + (((4 + (r >> 4)) ^ (n & 7)) << 4) + (r & 15));
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(part[j / 2][0] >> (8 * (j & 1))) : "memory");
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + NH * 128), "r"(part[j / 2][1] >> (8 * (j & 1))) : "memory");
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(third), "r"(part[j / 2][2] >> (8 * (j & 1))) : "memory");
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !bad) mbar_arrive(bar_p + 8 * (i & 1));
      }
      if (aborted) break;
      // ---- the segment's rows: out and lse, or the workspace's partial sums ----
      named_bar(bar_id, kTeam);  // the factors of a rescale in the last tile have been read (the sums take their place)
      if constexpr (ROWS) {
        float sum = l_row.x + l_row.y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (lane < 16) s_red[ch * NH + my_row] = sum;
      } else {
        float sums[NQ];
#pragma unroll
        for (int j = 0; j < NQ / 2; ++j) { sums[2 * j] = l_part[j].x; sums[2 * j + 1] = l_part[j].y; }
        s_red[qd * NH + sum_row] = over_keys(sums, false);
      }
      named_bar(bar_id, kTeam);
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
      named_bar(bar_id, kTeam);
      const bool got = wait_pv(i - 1);  // (the sums above while the last P.V is under way)
      aborted = named_bar_or(bar_id, kTeam, !got);
      if (aborted) break;
      tc_fence_after();
      // a few rows of 32 channels at a time, in a loop: unrolled, this code is longer than the time it takes to fetch it
      constexpr int kStep = NHH < 16 ? NHH : 16;
#pragma unroll 1
      for (int x = 0; x < 4 * NHH / kStep; ++x) {
        const int mt = x / (NHH / kStep), h0 = ch * NHH + (x % (NHH / kStep)) * kStep;
        uint32_t o[kStep];
        const uint32_t ta = tmem_addr(tmem + L::TM_O + mt * NH + h0, qd * 32, 0);
        if constexpr (kStep == 16) tmem_ld16(ta, o);
        else tmem_ld8(ta, o);
        tmem_ld_wait();
        const int c = mt * 128 + qd * 32 + lane, rows = sg.rows - h0;
        // (one branch for all rows: with one for each, every store waits for the one before, 66 cycles in place of 5)
        if (whole) {
          __nv_bfloat16* dst = p.out + (size_t)(sg.row0 + h0) * kDv + c;
          float f[kStep];
#pragma unroll
          for (int h = 0; h < kStep; ++h) f[h] = s_fac[h0 + h];
#pragma unroll
          for (int h = 0; h < kStep; ++h)
            if (h < rows) dst[h * kDv] = __float2bfloat16_rn(f[h] == 0.f ? 0.f : __uint_as_float(o[h]) * f[h]);
        } else {
          float* part = p.partial + ((size_t)slot * 64 + h0) * kDv + c;
#pragma unroll
          for (int h = 0; h < kStep; ++h)
            if (h < rows) part[h * kDv] = __uint_as_float(o[h]);
        }
      }
      tc_fence_before();
      named_bar(bar_id, kTeam);  // s_red, s_stat and s_fac have been read
      if (!more) break;
      sg = nx;
    }
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
dsa_status_t launch(Params& p, int ctas, cudaStream_t s) {
  using L = Smem<DQK, NH>;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(paged_mla_e4m3_kernel<DQK, NH>), L::TOTAL,
                                          "configuring paged_mla_e4m3_kernel");
  if (st != DSA_OK) return st;
  p.G = p.topk_idx ? 1 : (p.H <= NH ? NH / p.H : 1);
  // (queries, a pipeline that runs dry and the sums: as long as six tiles.  64 x 16384: 122.5 us, with 4 124.4, with 2 125.5; 48
  // lists of 2048: 42.9, with 4 43.4, with 2 47.1)
  p.extra = 6;
  p.HB = (p.H + NH - 1) / NH;
  paged_mla_e4m3_kernel<DQK, NH><<<ctas, L::THREADS, L::TOTAL, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching paged_mla_e4m3_kernel");
}

}  // namespace pmla8

dsa_status_t launch_paged_mla_e4m3(const pgroups::GroupParams& g, const __nv_bfloat16* q, const uint8_t* cache, int Dqk,
                                   float scale_log2e, bool few, int ctas, cudaStream_t s) {
  pmla8::Params p{};
  static_cast<pgroups::GroupParams&>(p) = g;
  p.q = q;
  p.cache = cache;
  p.sl2e = scale_log2e;
  if (few) return Dqk == 576 ? pmla8::launch<576, 16>(p, ctas, s) : pmla8::launch<512, 16>(p, ctas, s);
  return Dqk == 576 ? pmla8::launch<576, 64>(p, ctas, s) : pmla8::launch<512, 64>(p, ctas, s);
}

}  // namespace dsa
