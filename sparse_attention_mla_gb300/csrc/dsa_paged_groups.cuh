// dsa_paged_groups.cuh -- what the attention kernels over a paged cache of latents share: the (token, head) rows of a
// request packed into groups of MMA columns, the tiles of all groups laid end to end and cut into one range per CTA, the
// runs of tiles announced to a CTA's warps, and the joining of a group's pieces.
#pragma once
#include "dsa_host.h"
#include "dsa_paged.cuh"

namespace dsa {
namespace pgroups {

constexpr int kDv = 512;
constexpr int kSegs = 8;  // segments announced ahead
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct GroupParams {
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const int32_t* topk_idx;
  const int32_t* topk_len;
  int N, B, H, K, num_pages, P, max_pages;
  int G, HB;  // tokens per group, head blocks
  int extra;  // tiles that the end of a group counts as when the line is cut
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  int4* records;   // [kMaxCtas]: (first row, rows, first head, last CTA) of the group that a CTA opens; rows 0: none
  float* stats;    // [2 * kMaxCtas][2][64]
  float* partial;  // [2 * kMaxCtas][64][512]
  long long wait_limit;
};

// 2^x in one instruction (results below 2^-126 become 0)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Unit {
  int groups, tiles;  // groups of MMA columns, tiles of each
  int n0, n;          // first token, tokens
  int len, keys;      // length of the request; positions looked at, or entries of the list
};

// A unit is a request (all its tokens see the same cache) or, with lists, one token.
template <int TILE>
__device__ __forceinline__ Unit unit_of(const GroupParams& p, int u) {
  Unit r;
  if (p.topk_idx != nullptr) {
    const int end = p.cu_q ? min(max(__ldg(p.cu_q + p.B), 0), p.N) : p.N;
    const int begin = p.cu_q ? __ldg(p.cu_q) : 0;
    r.n0 = u;
    r.n = u >= begin && u < end ? 1 : 0;
    r.len = 0;
    r.keys = p.topk_len ? min(max(__ldg(p.topk_len + u), 0), p.K) : p.K;
  } else {
    const int lo = p.cu_q ? min(max(__ldg(p.cu_q + u), 0), p.N) : u;
    const int hi = p.cu_q ? min(max(__ldg(p.cu_q + u + 1), lo), p.N) : u + 1;
    r.n0 = lo;
    r.n = hi - lo;
    r.len = max(__ldg(p.seq_lens + u), 0);
    r.keys = (int)min((long long)r.len, (long long)p.max_pages * p.P);
  }
  r.tiles = max(1, (int)(((long long)r.keys + TILE - 1) / TILE));
  r.groups = (r.n + p.G - 1) / p.G * p.HB;
  return r;
}

// The CTA's range of tiles and the unit it starts in (in shared memory, written by make_plan).
struct Plan {
  long long w0, w1;  // this CTA's tiles of the whole line
  Unit un;
  int u, g, t;       // unit, group and tile of the first tile
  int skip;          // what lies before it: the end of a group
};

// A run of tiles [t0, t0 + n) of one group, as announced (two int4).
struct Seg {
  int t0, n;
  int row0;           // first row (token, head) of q, out and lse
  int rows, head0;    // rows; head of the first row
  bool whole, opens;  // all tiles of the group; its first one among them
  bool last;          // the CTA's last run
  int b;              // request
  int seen0;          // positions that the group's first token sees (may be <= 0)
  int keys;           // positions looked at by any token, or entries of the list
};
__device__ __forceinline__ Seg unpack(const int4 a, const int4 c) {
  Seg s;
  s.t0 = a.x;
  s.n = a.y;
  s.row0 = a.z;
  s.rows = a.w & 255;
  s.whole = a.w & 256;
  s.opens = a.w & 512;
  s.last = a.w & 1024;
  s.head0 = c.w;
  s.b = c.x;
  s.seen0 = c.y;
  s.keys = c.z;
  return s;
}

// Announcement k, read by a whole warp; false when the wait ran out.
__device__ __forceinline__ bool read_announcement_here(uint32_t full, uint32_t empty, const int4* ring, int k,
                                                       volatile int* abort, long long limit, Seg& s) {
  const int at = k % kSegs;
  if (!__all_sync(0xffffffffu, wait_for(full + 8 * at, (k / kSegs) & 1, abort, limit))) return false;
  s = unpack(ring[2 * at], ring[2 * at + 1]);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * at);
  return true;
}
// (As a function of its own: called once per segment, and kept out of the roles' loops.)
__device__ __noinline__ static bool read_announcement(uint32_t full, uint32_t empty, const int4* ring, int k,
                                                      volatile int* abort, long long limit, Seg& s) {
  return read_announcement_here(full, empty, ring, k, abort, limit, s);
}

// The announcing warp: the segments of the CTA's range, one after the other, into a ring that the other warps read.
// One copy of this code and of its loads, instead of one per role.
// after(k) is called when number k has been announced.
struct Nothing {
  __device__ __forceinline__ void operator()(int) const {}
};
template <int TILE, class F = Nothing>
__device__ __forceinline__ void announce(const GroupParams& p, const Plan& pl, uint32_t full, uint32_t empty, int4* ring,
                                         volatile int* abort, const F& after = F()) {
  const int lane = threadIdx.x & 31;
  long long left = pl.w1 - pl.w0 - pl.skip;
  int u = pl.u, g = pl.g, t = pl.t;
  Unit un = pl.un;
  bool cut = false;
#pragma unroll 1
  for (int k = 0; left > 0; ++k) {
#pragma unroll 1
    while (g >= un.groups) {  // (units are skipped only while tiles are left, so u stays in range)
      un = unit_of<TILE>(p, ++u);
      g = t = 0;
    }
    const int tb = g / p.HB, hb = g - tb * p.HB;
    const int n0 = un.n0 + tb * p.G;
    int4 a, c;
    a.x = t;
    a.y = (int)min((long long)(un.tiles - t), left);
    a.z = n0 * p.H + hb * 64;
    a.w = (p.HB > 1 ? min(64, p.H - hb * 64) : min(p.G, un.n - tb * p.G) * p.H) | (t == 0 ? 512 : 0) |
          (t == 0 && a.y == un.tiles ? 256 : 0);
    t += a.y;
    left -= a.y + (t >= un.tiles ? p.extra : 0);
    a.w |= left <= 0 ? 1024 : 0;
    c.x = u;
    c.y = un.len - un.n + tb * p.G + 1;
    c.z = un.keys;
    c.w = hb * 64;
    if (p.topk_idx != nullptr) {
      int lo = n0, hi = n0 + 1;
      c.x = n0;
      if (p.cu_q) {
        c.x = warp_last_le(p.cu_q, p.B, n0);
        lo = __ldg(p.cu_q + c.x);
        hi = __ldg(p.cu_q + c.x + 1);
      }
      c.y = max(__ldg(p.seq_lens + c.x), 0) - (hi - lo) + (n0 - lo) + 1;
    } else {
      cut |= un.keys < un.len;
    }
    const int at = k % kSegs;
    if (k >= kSegs && !warp_all(wait_for(empty + 8 * at, (k / kSegs - 1) & 1, abort, p.wait_limit))) break;
    if (lane == 0) {
      ring[2 * at] = a;
      ring[2 * at + 1] = c;
      mbar_arrive(full + 8 * at);
    }
    if (t >= un.tiles) { ++g; t = 0; }
    after(k);
  }
  if (cut && lane == 0) record_error(p.err, DSA_ERR_DEVICE_INDEX);  // the table does not hold a request
}

// Whole CTA: this CTA's share of the tiles, the unit it starts in, and the record of the group that it opens and
// does not finish.
template <int TILE, int NT>
__device__ __forceinline__ void make_plan(const GroupParams& p, Plan* plan, long long* scratch) {
  if (threadIdx.x == 0) p.records[blockIdx.x] = make_int4(0, 0, 0, 0);
  auto tiles_of = [&](int u) -> long long {
    const Unit x = unit_of<TILE>(p, u);
    return (long long)x.groups * (x.tiles + p.extra);
  };
  auto visit = [&](const TileRange& r, int u, long long lo, long long n) {
    const bool starts = lo <= r.w0 && r.w0 < lo + n, ends = lo <= r.w1 - 1 && r.w1 - 1 < lo + n;
    if (!starts && !ends) return;
    const Unit x = unit_of<TILE>(p, u);
    const int span = x.tiles + p.extra;
    if (starts) {
      const long long first = r.w0 - lo;
      int g = (int)(first / span), t = (int)(first - (long long)g * span);
      plan->skip = 0;
      if (t >= x.tiles) {
        plan->skip = span - t;
        ++g;
        t = 0;
      }
      plan->u = u;
      plan->un = x;
      plan->g = g;
      plan->t = t;
    }
    if (ends) {  // the range's last tile
      const long long off = r.w1 - 1 - lo;
      const int g = (int)(off / span), tl = (int)(off - (long long)g * span);
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
  const TileRange r = split_line<NT>(p.topk_idx ? p.N : p.B, tiles_of, scratch, visit);
  if (threadIdx.x == 0) {
    plan->w0 = r.w0;
    plan->w1 = r.w1;
  }
  __syncthreads();
}

// Joins the pieces of the groups that went over several CTAs.  A row of few pieces is a team's of 128 threads, 4 channels
// each; a row of many (one long request over the whole card) is a CTA's, whose teams take every fourth piece.  Pieces are
// added in a fixed order, whichever came first.  Two CTAs of 512 threads an SM, all at once: as one of 1024 (with its 64
// registers a thread) the second half of them waited for the first, and took 7 us longer.  The records are made lists of
// by ballots, since code that runs once costs the time to fetch it (a scan in a loop: 4 us more).
constexpr int kJoin = 512, kTeams = kJoin / 128, kMany = 16;
constexpr int kGroupsOf = 64 / kTeams;  // of a record's rows, a row for each team
static __global__ void __launch_bounds__(kJoin, 2) paged_mla_join_kernel(const int4* __restrict__ records, int ctas,
                                                                 const float* __restrict__ stats,
                                                                 const float* __restrict__ partial,
                                                                 const float* __restrict__ sink, int H,
                                                                 __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  __shared__ int4 rec[kMaxCtas];
  __shared__ int list[2][kMaxCtas];  // records of few pieces, of many
  __shared__ int count[2][kMaxCtas / 32];
  __shared__ float fac[kMaxCtas];
  __shared__ float4 acc[kTeams][128];
  __shared__ float s_l, s_base;
  const int tid = threadIdx.x, lane = tid & 31, team = tid >> 7, x = tid & 127;
  // launched while the pieces are still being made; what the first kernel writes is read from L2, not as constant data
  asm volatile("griddepcontrol.wait;" ::: "memory");
  unsigned mine[2] = {0, 0};
  if (tid < kMaxCtas) {
    const int4 rc = tid < ctas ? __ldcg(records + tid) : make_int4(0, 0, 0, 0);
    rec[tid] = rc;
    const bool many = rc.w - tid + 1 >= kMany;
    mine[0] = __ballot_sync(0xffffffffu, rc.y > 0 && !many);
    mine[1] = __ballot_sync(0xffffffffu, rc.y > 0 && many);
    if (lane < 2) count[lane][tid >> 5] = __popc(lane ? mine[1] : mine[0]);
  }
  __syncthreads();
  int total[2] = {0, 0};
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < kMaxCtas / 32; ++w) {
      before += w < (tid >> 5) ? count[m][w] : 0;
      total[m] += count[m][w];
    }
    if ((mine[m] >> lane) & 1u) list[m][before + __popc(mine[m] & ((1u << lane) - 1u))] = tid;
  }
  __syncthreads();
  auto piece = [&](int lo, int k, int n) -> size_t { return (size_t)(2 * (lo + k) + (k == 0 ? 1 : 0)) * 64 + n; };
  auto part = [&](int lo, int k, int n) { return __ldcg(reinterpret_cast<const float4*>(partial + piece(lo, k, n) * kDv) + x); };
  auto add = [](float4& o, float f, float4 v) {
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  };
  auto store = [&](int row, float4 o, float l, float base) {
    const bool empty = l == 0.f;  // nothing is seen, and there is no sink
    const float inv = empty ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(out + (size_t)row * kDv)[x] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (x == 0) lse[row] = empty ? -INFINITY : base * kLn2 + logf(l);
  };
  for (int it = blockIdx.x; it < total[0] * kGroupsOf; it += gridDim.x) {
    const int lo = list[0][it / kGroupsOf];
    const int4 rc = rec[lo];
    const int n = it % kGroupsOf * kTeams + team, pieces = rc.w - lo + 1;
    if (n >= rc.y) continue;
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < pieces ? part(lo, k, n) : make_float4(0.f, 0.f, 0.f, 0.f);
    // lane k holds piece k's maximum and sum
    const size_t at = lane < pieces ? piece(lo, lane, n) : 0;
    const float mc = lane < pieces ? __ldcg(stats + at / 64 * 128 + n) : -INFINITY;
    const float lc = lane < pieces ? __ldcg(stats + at / 64 * 128 + 64 + n) : 0.f;
    const float s2 = sink ? __ldg(sink + (rc.z + n) % H) * kLog2e : -INFINITY;
    float m = fmaxf(mc, s2);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = __shfl_sync(0xffffffffu, m, 0);
    const float base = m == -INFINITY ? 0.f : m;
    const float f = exp2f(mc - base);
    float l = lane < pieces ? f * lc : 0.f;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    l = __shfl_sync(0xffffffffu, l, 0) + exp2f(s2 - base);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < pieces; k0 += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k0 + k < pieces) {
          add(o, __shfl_sync(0xffffffffu, f, k0 + k), v[k]);
          if (k0 + 4 + k < pieces) v[k] = part(lo, k0 + 4 + k, n);
        }
      }
    }
    store(rc.x + n, o, l, base);
  }
  for (int it = blockIdx.x; it < total[1] * 64; it += gridDim.x) {
    const int lo = list[1][it / 64];
    const int4 rc = rec[lo];
    const int n = it % 64, pieces = rc.w - lo + 1;
    if (n >= rc.y) continue;
    // the first pieces' channels are on their way while the maxima are compared
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = part(lo, team + j * kTeams, n);  // (kMany >= 4 kTeams)
    if (tid < 32) {
      const float s2 = sink ? __ldg(sink + (rc.z + n) % H) * kLog2e : -INFINITY;
      float mc[kMaxCtas / 32], lc[kMaxCtas / 32], m = s2;
#pragma unroll
      for (int j = 0; j < kMaxCtas / 32; ++j) {
        const int k = j * 32 + lane;
        const size_t at = k < pieces ? piece(lo, k, n) / 64 * 128 + n : 0;
        mc[j] = k < pieces ? __ldcg(stats + at) : -INFINITY;
        lc[j] = k < pieces ? __ldcg(stats + at + 64) : 0.f;
        m = fmaxf(m, mc[j]);
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m;
      float l = lane == 0 ? exp2f(s2 - base) : 0.f;
#pragma unroll
      for (int j = 0; j < kMaxCtas / 32; ++j) {
        const int k = j * 32 + lane;
        const float f = exp2f(mc[j] - base);
        if (k < pieces) {
          fac[k] = f;
          l += f * lc[j];
        }
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) { s_l = l; s_base = base; }
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = team; k0 < pieces; k0 += 4 * kTeams) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * kTeams;
        if (k < pieces) {
          add(o, fac[k], v[j]);
          if (k + 4 * kTeams < pieces) v[j] = part(lo, k + 4 * kTeams, n);
        }
      }
    }
    acc[team][x] = o;
    __syncthreads();
    if (team == 0) {
#pragma unroll
      for (int k = 1; k < kTeams; ++k) add(o, 1.f, acc[k][x]);
      store(rc.x + n, o, s_l, s_base);
    }
    __syncthreads();
  }
}
static_assert(kMany >= 4 * kTeams && kMany <= 16 && 64 % kTeams == 0, "join: pieces and rows");

constexpr size_t kRecordBytes = kMaxCtas * sizeof(int4);
constexpr size_t kStatBytes = (size_t)2 * kMaxCtas * 128 * sizeof(float);
constexpr size_t kPartialBytes = (size_t)2 * kMaxCtas * 64 * kDv * sizeof(float);

// SMs of the current device, at most kMaxCtas.
inline int cta_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n < kMaxCtas ? n : kMaxCtas;
}

// The joining kernel, launched while the pieces are still being made.
inline dsa_status_t launch_join(const GroupParams& p, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * ctas);
  cfg.blockDim = dim3(kJoin);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, paged_mla_join_kernel, (const int4*)p.records, ctas, (const float*)p.stats,
                                       (const float*)p.partial, p.sink, p.H, p.out, p.lse),
                    "launching paged_mla_join_kernel");
}

}  // namespace pgroups
}  // namespace dsa
