// dsa_norm_rope.cu -- the norm of a row and the rotation of its positions in one
// pass, with the gradient, and the frequencies of a scaled rotation.
//
// Per row (t, h) of width D: the first n channels are normalised,
//   rms:    u = x r w,             r = (mean x^2 + eps)^(-1/2)
//   layer:  u = (x - mean x) r w + b,  r = (mean (x - mean x)^2 + eps)^(-1/2)
// then the R channels from r0 are turned in pairs (a, b) by the angle
// pos[t] inv_freq[i]:  (a, b) -> s (c a - sn b, sn a + c b).  A pair is (2i, 2i+1)
// (interleaved) or (i, i + R/2).  With g the rotated-back gradient
// (s (c ga + sn gb), s (c gb - sn ga)) and xh the normalised row:
//   dw = sum g xh, db = sum g,  gw = g w,
//   dx = r (gw - [mean gw] - xh mean(gw xh))     ([..] in the layer norm only).
//
// What bounds it: DRAM, 4 bytes a channel forward and 6 backward; at 8 channels a
// lane the instructions come close behind.  So the rows stay in registers between
// the one read and the one write, LPR lanes to a row (8 for 64 channels, 16 for
// 128, else a warp), 16 bytes a lane and two fp32 operations an instruction; a
// group of lanes takes U consecutive rows (up to 4) at once, the next U on their
// way meanwhile, and the CTAs stay, so that the table of frequencies is made once;
// a row's place is the last one's plus a step (as two products of 64 bits 6 % more).
// The cosines and sines depend on the token alone: they are formed once per token
// of a group's run of rows, spread over its lanes, in shared memory.  Measured: the
// position channels of 16384 x 64 heads (128 of every 1152 bytes) 54 us at 5.0 TB/s,
// 131104 rows of 128 with the norm 18 us at 3.7 TB/s, the gradient of 32768 rows of
// 128 with the layer norm 16 us at 1.5 TB/s (four batches of rows a group: latency).
//
// Angles: positions reach millions, and position times frequency in fp32 is then
// off by 0.1 rad.  The frequency is held as a 64-bit binary fraction of a turn, so
// that position times fraction modulo 2^64 drops whole turns exactly; its upper
// 32 bits are the angle.  Sums and statistics are fp32; rows are rounded to bf16
// once, when written.
#include <cmath>
#include <type_traits>

#include "dsa_device.cuh"
#include "dsa_f32x2.cuh"
#include "dsa_host.h"

namespace dsa {
namespace nrope {

constexpr int kThreads = 256;
constexpr int kMaxD = 1024;
constexpr int64_t kMaxRows = 0x7fffffffll - 64;  // (a run counts up to 32 rows past the last one)
constexpr int kMaxPartials = 608;  // CTAs of a backward launch with parameters: each leaves one row of dw and db
enum { kAny = -1, kNone = 0, kRms = 1, kLayer = 2 };  // (kAny: a kernel that reads the norm from its arguments)

// CTAs of an SM, by the registers that a lane's channels take.
__host__ __device__ constexpr int ctas_per_sm(int VEC, int NIT) { return NIT <= 2 && VEC == 8 ? 2 : 1; }

// Steps in elements from a token and from a head to the next, and from a token's last head to the next token's first.
struct Step {
  int64_t t, h, wrap;
};
inline Step step_of(int64_t t, int64_t h, int H) { return Step{t, h, t - (int64_t)(H - 1) * h}; }

struct Rows {
  const __nv_bfloat16* x;
  Step xs;
  int T, H, D;
  int kind, n;
  const float* w;
  const float* b;
  float eps;
  int r0, R, inter;
  const int32_t* pos;
  const float* inv_freq;
  float rscale;
  int rows, run;  // T * H; consecutive rows of a group of lanes (a multiple of U)
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A row in registers: per lane NIT accesses of VEC channels, channel c = (it * LPR + l) * VEC + e; in fp32 as pairs of
// neighbours (on the scalar path a pair is one channel and a zero).
template <int VEC, int LPR, int NIT>
struct Row {
  static constexpr int PP = VEC == 8 ? 4 : 1, P = PP * NIT;  // pairs per access, per lane
  uint4 v[VEC == 8 ? NIT : 1];
  uint16_t s[VEC == 8 ? 1 : NIT];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int D, int l, bool on) {
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int c = (it * LPR + l) * VEC;
      if constexpr (VEC == 8) {
        v[it] = make_uint4(0, 0, 0, 0);
        if (on && c < D) v[it] = *reinterpret_cast<const uint4*>(row + c);
      } else {
        s[it] = 0;
        if (on && c < D) s[it] = *reinterpret_cast<const uint16_t*>(row + c);
      }
    }
  }
  __device__ __forceinline__ void values(float2 (&f)[P]) const {
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      if constexpr (VEC == 8) {
        const uint32_t u[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) f[it * 4 + k] = make_float2(bf_lo(u[k]), bf_hi(u[k]));
      } else {
        f[it] = make_float2(__uint_as_float((uint32_t)s[it] << 16), 0.f);
      }
    }
  }
};

template <int VEC, int LPR, int NIT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int D, int l, const float2 (&f)[Row<VEC, LPR, NIT>::P]) {
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int c = (it * LPR + l) * VEC;
    if (c >= D) continue;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack_bf16x2(f[it * 4].x, f[it * 4].y), pack_bf16x2(f[it * 4 + 1].x, f[it * 4 + 1].y),
                     pack_bf16x2(f[it * 4 + 2].x, f[it * 4 + 2].y), pack_bf16x2(f[it * 4 + 3].x, f[it * 4 + 3].y));
    } else {
      row[c] = __float2bfloat16_rn(f[it].x);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Shared memory: the fractions of a turn per position [R/2], then per group of lanes the (scaled) cosines and sines of
// the last U tokens [U][R/2] (token t in slot t % U) and R channels for the exchange between the two of a pair.
struct Shared {
  uint64_t* turn;
  float2* cs;
  float* stage;
};
template <int U>
__device__ __forceinline__ Shared carve(uint8_t* raw, int R, int group) {
  const int half = R >> 1;
  Shared s;
  s.turn = reinterpret_cast<uint64_t*>(raw);
  uint8_t* mine = raw + (size_t)half * 8 + (size_t)group * half * 8 * (U + 1);
  s.cs = reinterpret_cast<float2*>(mine);
  s.stage = reinterpret_cast<float*>(mine + (size_t)half * 8 * U);
  return s;
}
inline int shared_bytes(int R, int groups, int U) { return (R >> 1) * 8 * (1 + groups * (U + 1)); }

__device__ __forceinline__ void fill_turns(uint64_t* turn, const Rows& p) {
  for (int i = threadIdx.x; i < (p.R >> 1); i += kThreads) {
    double f = (double)__ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    turn[i] = (uint64_t)(f * 18446744073709551616.0);  // f < 1: below 2^64
  }
}

template <int LPR>
__device__ __forceinline__ void fill_cos_sin(float2* cs, const uint64_t* turn, const Rows& p, int64_t pos, int l) {
  for (int i = l; i < (p.R >> 1); i += LPR) {
    const int32_t frac = (int32_t)(((uint64_t)pos * turn[i]) >> 32);  // signed: [-1/2, 1/2) of a turn
    float sn, c;
    sincospif((float)frac * 4.656612873077393e-10f, &sn, &c);  // 2^-31: half turns
    cs[i] = make_float2(c * p.rscale, sn * p.rscale);
  }
}

// How a rotation reaches the other half of a pair.  kPairs: interleaved pairs inside a lane's whole accesses.  kLanes:
// half layout, the other half is the same channel of the lane R / 16 away, and all rotated channels are in access `it`
// of the row.  kShared: any layout, through shared memory.
enum { kShared = 0, kPairs = 1, kLanes = 2 };

// A token's cosines and sines as this lane needs them, and the turn of a row by them; back = -1 turns the other way
// (the transpose).
template <int VEC, int LPR, int NIT, int ROT>
struct Turn {
  static constexpr int PP = Row<VEC, LPR, NIT>::PP, P = Row<VEC, LPR, NIT>::P;
  float2 a[ROT == kPairs ? P : 4], b[4];
  int it, other;
  bool in;
  const float2* cs;
  // `table`: any of the group's tables (a group without rows turns zeros by whatever is there)
  __device__ __forceinline__ void init(const float2* table, const Rows& p, int l) {
    cs = table;
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < (ROT == kPairs ? P : 4); ++i) a[i] = make_float2(1.f, 0.f);
    it = ROT == kLanes ? p.r0 / (LPR * VEC) : 0;
    const int u0 = (it * LPR + l) * VEC - p.r0;
    in = u0 >= 0 && u0 < p.R;
    const int half = p.R >> 1;
    other = (l + (u0 >= half ? -(half / 8) : half / 8)) & (LPR - 1);
  }
  __device__ __forceinline__ void load(const float2* table, const Rows& p, int l, float back) {
    cs = table;
    if constexpr (ROT == kPairs) {
#pragma unroll
      for (int k = 0; k < NIT; ++k) {
        const int u0 = (k * LPR + l) * VEC - p.r0;
        if (u0 < 0 || u0 >= p.R) continue;
        const float4* q = reinterpret_cast<const float4*>(table + (u0 >> 1));
        const float4 x = q[0], y = q[1];
        a[k * PP] = make_float2(x.x, x.y * back);
        a[k * PP + 1 % PP] = make_float2(x.z, x.w * back);
        a[k * PP + 2 % PP] = make_float2(y.x, y.y * back);
        a[k * PP + 3 % PP] = make_float2(y.z, y.w * back);
      }
    } else if constexpr (ROT == kLanes) {
      const int u0 = (it * LPR + l) * VEC - p.r0, half = p.R >> 1;
      const bool second = u0 >= half;
      const float4* q = reinterpret_cast<const float4*>(table + (in ? (second ? u0 - half : u0) : 0));
      const float sign = second ? back : -back;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 c = q[e];
        a[e] = make_float2(c.x, c.z);
        b[e] = make_float2(c.y * sign, c.w * sign);
      }
    }
  }
  __device__ __forceinline__ void apply(float2 (&f)[P], float* stage, const Rows& p, int l, float back) const {
    // (channels that are not turned are left out, not turned by 0: 0 times a neighbour's infinity is no 0)
    if constexpr (ROT == kPairs) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int u0 = ((i / PP) * LPR + l) * VEC - p.r0;
        const float2 x = f[i];
        if (u0 >= 0 && u0 < p.R) f[i] = make_float2(x.x * a[i].x - x.y * a[i].y, x.y * a[i].x + x.x * a[i].y);
      }
    } else if constexpr (ROT == kLanes) {
#pragma unroll
      for (int k = 0; k < NIT; ++k) {
        if (NIT > 1 && k != it) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (k * PP + e) % P;  // (the remainder only keeps the unused scalar shape in range)
          const float2 y = make_float2(__shfl_sync(0xffffffffu, f[i].x, other, LPR), __shfl_sync(0xffffffffu, f[i].y, other, LPR));
          if (in) f[i] = fma2(f[i], a[e], mul2(y, b[e]));
        }
      }
    } else {
      if (p.R == 0) return;
      const int half = p.R >> 1;
      constexpr int W = VEC == 8 ? 2 : 1;  // channels of a pair of values
      __syncwarp();  // the row before has been read
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int u = ((i / PP) * LPR + l) * VEC + (i % PP) * 2 + e - p.r0;
          if (u >= 0 && u < p.R) stage[u] = e ? f[i].y : f[i].x;
        }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int u = ((i / PP) * LPR + l) * VEC + (i % PP) * 2 + e - p.r0;
          if (u < 0 || u >= p.R) continue;
          const bool second = p.inter ? (u & 1) : (u >= half);
          const int k = p.inter ? (u >> 1) : (second ? u - half : u);
          const int partner = p.inter ? (u ^ 1) : (second ? u - half : u + half);
          const float2 c = cs[k];
          const float sn = second ? c.y * back : -c.y * back;
          float& x = e ? f[i].y : f[i].x;
          x = x * c.x + stage[partner] * sn;
        }
    }
  }
};

// weight or bias of this lane's channels below n (`none` where there is no array; 16-byte loads on the vector path,
// where n is a multiple of 8)
template <int VEC, int LPR, int NIT>
__device__ __forceinline__ void load_param(float2 (&v)[Row<VEC, LPR, NIT>::P], const float* a, float none, int n, int l) {
  constexpr int PP = Row<VEC, LPR, NIT>::PP;
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int c0 = (it * LPR + l) * VEC;
    const bool on = a != nullptr && c0 < n;
    if constexpr (VEC == 8) {
      float4 x = make_float4(none, none, none, none), y = x;
      if (on) {
        x = __ldg(reinterpret_cast<const float4*>(a + c0));
        y = __ldg(reinterpret_cast<const float4*>(a + c0) + 1);
      }
      v[it * PP] = make_float2(x.x, x.y);
      v[it * PP + 1] = make_float2(x.z, x.w);
      v[it * PP + 2] = make_float2(y.x, y.y);
      v[it * PP + 3] = make_float2(y.z, y.w);
    } else {
      v[it] = make_float2(on ? __ldg(a + c0) : none, 0.f);
    }
  }
}

// A group's run of rows, U at a time: their tokens and heads, where they lie in NA arrays (by steps: a row's place costs
// no products), and the tokens' cosines and sines as they come up.
template <int LPR, int U, int NA>
struct Run {
  int row, end, t, h;  // next row, end of the run; token and head of the next row
  int filled;          // last token whose cosines and sines are there
  int64_t at[NA];      // the next row in each array
  __device__ __forceinline__ void begin(const Rows& p, int64_t first, const Step (&st)[NA]) {
    row = first < p.rows ? (int)first : p.rows;
    end = (int)min((int64_t)p.rows, first + p.run);
    t = row / p.H;
    h = row - t * p.H;
    filled = t - 1;
#pragma unroll
    for (int a = 0; a < NA; ++a) at[a] = t * st[a].t + h * st[a].h;
  }
  // the next U rows (t = -1: none), their places and their positions
  __device__ __forceinline__ void batch(const Rows& p, const Step (&st)[NA], int (&tt)[U], int (&hh)[U], int (&pos)[U],
                                        int64_t (&place)[NA][U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = row < end;
      tt[u] = on ? t : -1;
      hh[u] = h;
      pos[u] = p.R > 0 && on ? __ldg(p.pos + t) : 0;
      const bool last = h + 1 == p.H;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        place[a][u] = on ? at[a] : 0;
        at[a] += last ? st[a].wrap : st[a].h;
      }
      ++row;
      t += last ? 1 : 0;
      h = last ? 0 : h + 1;
    }
  }
  // the cosines and sines of a batch's tokens
  __device__ __forceinline__ void cos_sin(const Rows& p, const Shared& s, const int (&tt)[U], const int (&pos)[U], int l) {
    if (p.R == 0) return;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tt[u] > filled) {
        fill_cos_sin<LPR>(s.cs + (size_t)(tt[u] % U) * (p.R >> 1), s.turn, p, pos[u], l);
        filled = tt[u];
      }
    }
    __syncwarp();
  }
};

// ROWS: out_rows may say where a token's rows go; else they follow one another.
template <int VEC, int LPR, int NIT, int ROT, int U, int KIND, bool ROWS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(VEC, NIT))
    norm_rope_fwd_kernel(const Rows p, __nv_bfloat16* out, const Step os, const int32_t* __restrict__ out_rows,
                         int64_t num_rows, int* __restrict__ err) {
  using R = Row<VEC, LPR, NIT>;
  const int kind = KIND == kAny ? p.kind : KIND;
  const bool by_rows = ROWS && out_rows != nullptr;
  constexpr int GPB = kThreads / LPR, P = R::P, PP = R::PP;
  extern __shared__ __align__(16) uint8_t raw_sh[];
  const int lane = threadIdx.x & 31, l = lane & (LPR - 1), group = threadIdx.x / LPR;
  const Shared s = carve<U>(raw_sh, p.R, group);
  // rows on their way while the ones before are worked on
  Run<LPR, U, 1> run;
  const Step steps[1] = {p.xs};
  int nt[U], nh[U], np[U], no[U];
  R nraw[U];
  auto fetch = [&]() {
    int64_t place[1][U];
    run.batch(p, steps, nt, nh, np, place);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nraw[u].load(p.x + place[0][u], p.D, l, nt[u] >= 0);
      no[u] = by_rows && nt[u] >= 0 ? __ldg(out_rows + nt[u]) : nt[u];
    }
  };
  int64_t first = ((int64_t)blockIdx.x * GPB + group) * p.run;
  run.begin(p, first, steps);
  fetch();
  fill_turns(s.turn, p);
  const float inv_n = p.n > 0 ? 1.f / (float)p.n : 0.f;
  float2 w[NIT == 1 ? P : 1];  // the weights stay in registers where a lane has 8 channels
  if constexpr (NIT == 1) load_param<VEC, LPR, NIT>(w, p.w, 1.f, p.n, l);
  Turn<VEC, LPR, NIT, ROT> turn;
  turn.init(s.cs, p, l);
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * GPB * p.run;
  // the groups of a warp run the same trip counts
  for (int64_t warp_first = first - (int64_t)(lane / LPR) * p.run; warp_first < p.rows; warp_first += step) {
    int turned = -1;  // the token whose cosines and sines `turn` holds
    int64_t to = nt[0] * os.t + nh[0] * os.h;  // where the next row goes
#pragma unroll 1
    for (int k = 0; k < p.run; k += U) {
      int tt[U], hh[U], pos[U], o[U];
      R raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        tt[u] = nt[u];
        hh[u] = nh[u];
        pos[u] = np[u];
        o[u] = no[u];
        raw[u] = nraw[u];
        if (by_rows && tt[u] >= 0 && (o[u] < -1 || o[u] >= num_rows)) {
          if (l == 0) record_error(err, DSA_ERR_DEVICE_INDEX);
          o[u] = -1;
        }
      }
      run.cos_sin(p, s, tt, pos, l);
      if (k + U >= p.run) {
        first += step;
        run.begin(p, first, steps);
      }
      fetch();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 f[P];
        raw[u].values(f);
        if (kind != kNone) {
          float2 mean = make_float2(0.f, 0.f), ss = mean;
          if (kind == kLayer) {
#pragma unroll
            for (int i = 0; i < P; ++i)
              if (((i / PP) * LPR + l) * VEC < p.n) mean = add2(mean, f[i]);
            const float m = -group_sum<LPR>(mean.x + mean.y) * inv_n;
            mean = make_float2(m, VEC == 8 ? m : 0.f);
          }
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (((i / PP) * LPR + l) * VEC < p.n) {
              if (kind == kLayer) f[i] = add2(f[i], mean);
              ss = fma2(f[i], f[i], ss);
            }
          const float r = rsqrtf(group_sum<LPR>(ss.x + ss.y) * inv_n + p.eps);
          const float2 r2 = make_float2(r, r);
          float2 v[P];
          if constexpr (NIT > 1) load_param<VEC, LPR, NIT>(v, p.w, 1.f, p.n, l);
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (((i / PP) * LPR + l) * VEC < p.n) f[i] = mul2(mul2(f[i], r2), NIT == 1 ? w[i % (NIT == 1 ? P : 1)] : v[i]);
          if (kind == kLayer && p.b != nullptr) {
            load_param<VEC, LPR, NIT>(v, p.b, 0.f, p.n, l);
#pragma unroll
            for (int i = 0; i < P; ++i)
              if (((i / PP) * LPR + l) * VEC < p.n) f[i] = add2(f[i], v[i]);
          }
        }
        if (p.R > 0) {
          if (tt[u] >= 0 && tt[u] != turned) {
            turn.load(s.cs + (size_t)(tt[u] % U) * (p.R >> 1), p, l, 1.f);
            turned = tt[u];
          }
          turn.apply(f, s.stage, p, l, 1.f);
        }
        if (o[u] >= 0) store_row<VEC, LPR, NIT>(out + (by_rows ? o[u] * os.t + hh[u] * os.h : to), p.D, l, f);
        to += hh[u] + 1 == p.H ? os.wrap : os.h;
      }
    }
  }
}

template <int VEC, int LPR, int NIT, int ROT, int U>
__global__ void __launch_bounds__(kThreads, NIT == 1 ? 2 : ctas_per_sm(VEC, NIT))
    norm_rope_bwd_kernel(const Rows p, const __nv_bfloat16* dout, const Step gs, __nv_bfloat16* dx, const Step ds,
                         float* __restrict__ partials) {
  using R = Row<VEC, LPR, NIT>;
  const int kind = p.kind;
  constexpr int GPB = kThreads / LPR, P = R::P, PP = R::PP;
  extern __shared__ __align__(16) uint8_t raw_sh[];
  const int lane = threadIdx.x & 31, l = lane & (LPR - 1), group = threadIdx.x / LPR;
  const Shared s = carve<U>(raw_sh, p.R, group);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the sum over the CTAs waits for this kernel's end)
  // rows on their way while the ones before are worked on
  Run<LPR, U, 2> run;
  const Step steps[2] = {gs, p.xs};
  int nt[U], nh[U], np[U];
  R ng[U], nx[U];
  auto fetch = [&]() {
    int64_t place[2][U];
    run.batch(p, steps, nt, nh, np, place);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = nt[u] >= 0;
      ng[u].load(dout + place[0][u], p.D, l, on);
      if (kind != kNone) nx[u].load(p.x + place[1][u], p.n, l, on);
    }
  };
  int64_t first = ((int64_t)blockIdx.x * GPB + group) * p.run;
  run.begin(p, first, steps);
  fetch();
  fill_turns(s.turn, p);
  const float inv_n = p.n > 0 ? 1.f / (float)p.n : 0.f;
  float2 w1[NIT == 1 ? P : 1];
  if constexpr (NIT == 1) load_param<VEC, LPR, NIT>(w1, p.w, 1.f, p.n, l);
  Turn<VEC, LPR, NIT, ROT> turn;
  turn.init(s.cs, p, l);
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * GPB * p.run;
  float2 dw[P], db[P];
#pragma unroll
  for (int i = 0; i < P; ++i) dw[i] = db[i] = make_float2(0.f, 0.f);
  for (int64_t warp_first = first - (int64_t)(lane / LPR) * p.run; warp_first < p.rows; warp_first += step) {
    int turned = -1;
    int64_t to = nt[0] * ds.t + nh[0] * ds.h;  // where the next row goes
#pragma unroll 1
    for (int k = 0; k < p.run; k += U) {
      int tt[U], hh[U], pos[U];
      R graw[U], xraw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        tt[u] = nt[u];
        hh[u] = nh[u];
        pos[u] = np[u];
        graw[u] = ng[u];
        xraw[u] = nx[u];
      }
      run.cos_sin(p, s, tt, pos, l);
      if (k + U >= p.run) {
        first += step;
        run.begin(p, first, steps);
      }
      fetch();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = tt[u] >= 0;
        float2 g[P];
        graw[u].values(g);
        if (p.R > 0) {
          if (on && tt[u] != turned) {
            turn.load(s.cs + (size_t)(tt[u] % U) * (p.R >> 1), p, l, -1.f);
            turned = tt[u];
          }
          turn.apply(g, s.stage, p, l, -1.f);
        }
        if (kind != kNone) {
          float2 x[P], v[NIT == 1 ? 1 : P];
          xraw[u].values(x);
          if constexpr (NIT > 1) load_param<VEC, LPR, NIT>(v, p.w, 1.f, p.n, l);
          auto weight = [&](int i) -> float2 {
            if constexpr (NIT == 1) return w1[i];
            else return v[i];
          };
          float2 sx = make_float2(0.f, 0.f), sg = sx;
          if (kind == kLayer) {
#pragma unroll
            for (int i = 0; i < P; ++i)
              if (((i / PP) * LPR + l) * VEC < p.n) {
                sx = add2(sx, x[i]);
                sg = fma2(g[i], weight(i), sg);
              }
            const float a = -group_sum<LPR>(sx.x + sx.y) * inv_n, c = -group_sum<LPR>(sg.x + sg.y) * inv_n;
            sx = make_float2(a, VEC == 8 ? a : 0.f);
            sg = make_float2(c, VEC == 8 ? c : 0.f);
          }
          float2 ss = make_float2(0.f, 0.f), sgx = ss;
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (((i / PP) * LPR + l) * VEC < p.n) {
              x[i] = add2(x[i], sx);
              ss = fma2(x[i], x[i], ss);
              sgx = fma2(mul2(g[i], weight(i)), x[i], sgx);
            }
          const float sum = group_sum<LPR>(ss.x + ss.y), dot = group_sum<LPR>(sgx.x + sgx.y);
          const float r = rsqrtf(sum * inv_n + p.eps);
          const float2 r2 = make_float2(r, r), m2 = make_float2(-dot * r * inv_n, -dot * r * inv_n);  // -mean(gw xh)
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (on && ((i / PP) * LPR + l) * VEC < p.n) {
              const float2 xh = mul2(x[i], r2);
              dw[i] = fma2(g[i], xh, dw[i]);
              db[i] = add2(db[i], g[i]);
              g[i] = mul2(r2, fma2(xh, m2, fma2(g[i], weight(i), sg)));
            }
        }
        if (on) store_row<VEC, LPR, NIT>(dx + to, p.D, l, g);
        to += hh[u] + 1 == p.H ? ds.wrap : ds.h;
      }
    }
  }
  if (partials == nullptr) return;
  // the CTA's sums: the groups of a warp by shuffles, then the warps one after the other in shared memory
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
      dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
      db[i].x += __shfl_xor_sync(0xffffffffu, db[i].x, o);
      db[i].y += __shfl_xor_sync(0xffffffffu, db[i].y, o);
    }
  }
  __shared__ float acc[2][VEC * LPR * NIT];
  for (int q = 0; q < kThreads / 32; ++q) {
    if ((threadIdx.x >> 5) == q && lane < LPR) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < (VEC == 8 ? 2 : 1); ++e) {
          const int c = ((i / PP) * LPR + l) * VEC + (i % PP) * 2 + e;
          const float a = e ? dw[i].y : dw[i].x, d = e ? db[i].y : db[i].x;
          acc[0][c] = q ? acc[0][c] + a : a;
          acc[1][c] = q ? acc[1][c] + d : d;
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < p.n; c += kThreads) {
    partials[(size_t)blockIdx.x * 2 * p.n + c] = acc[0][c];
    partials[(size_t)blockIdx.x * 2 * p.n + p.n + c] = acc[1][c];
  }
}

// Sums the CTAs' partial rows in a fixed order: 32 channels per CTA, 32 warps along the rows.
__global__ void __launch_bounds__(1024)
    norm_rope_sum_kernel(const float* partials, int count, int n, float* __restrict__ dweight,
                         float* __restrict__ dbias, int accumulate) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the rows are still being worked on
  if (c < 2 * n) {
#pragma unroll 8
    for (int r = w; r < count; r += 32) v += __ldcg(partials + (size_t)r * 2 * n + c);
  }
  sh[w][lane] = v;
  __syncthreads();
  v = sh[lane][w];  // channel w of this CTA, warp `lane`'s sum
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int ch = blockIdx.x * 32 + w;
  if (lane == 0 && ch < 2 * n) {
    float* out = ch < n ? dweight : dbias;
    const int at = ch < n ? ch : ch - n;
    if (out != nullptr) out[at] = accumulate ? out[at] + v : v;
  }
}

template <int V, int L, int N, int T, int K = kAny>
struct Shape {
  static constexpr int VEC = V, LPR = L, NIT = N, ROT = T, KIND = K;
};

// A forward kernel for each norm where a row's instructions count: the 16-byte path with a rotation in registers.
// (131104 rows of 128, rms and rotation: 18 us, 25 us with the norm as an argument; in the backward 1 %, not worth its
// kernels.)
template <int LPR, int NIT, int ROT, class F>
dsa_status_t dispatch_norm(const Rows& p, F&& f) {
  if (p.kind == kRms) return f(Shape<8, LPR, NIT, ROT, kRms>{});
  if (p.kind == kLayer) return f(Shape<8, LPR, NIT, ROT, kLayer>{});
  return f(Shape<8, LPR, NIT, ROT, kNone>{});
}

// The 16-byte path with LPR lanes to a row: whole accesses are rotated where r0 and R are multiples of 8 (the tables of
// cosines then start on 16 bytes too).
template <int LPR, int NIT, class F>
dsa_status_t dispatch_rotation(const Rows& p, F&& f) {
  if (p.r0 % 8 == 0 && p.R % 8 == 0) {
    if (p.inter || p.R == 0) return dispatch_norm<LPR, NIT, kPairs>(p, f);
    if (p.R % 16 == 0 && p.r0 / 8 / LPR == ((p.r0 + p.R) / 8 - 1) / LPR) return dispatch_norm<LPR, NIT, kLanes>(p, f);
  }
  return f(Shape<8, LPR, NIT, kShared>{});
}

// Calls f with the lanes of a row: 16-byte accesses where every row and the parameters start on a 16-byte boundary and
// the norm covers whole accesses; else one channel at a time.
template <class F>
dsa_status_t dispatch(bool vec, const Rows& p, F&& f) {
  if (vec) {
    if (p.D <= 64) return dispatch_rotation<8, 1>(p, f);
    if (p.D <= 128) return dispatch_rotation<16, 1>(p, f);
    if (p.D <= 256) return dispatch_rotation<32, 1>(p, f);
    if (p.D <= 512) return dispatch_rotation<32, 2>(p, f);
    if (p.D <= 768) return dispatch_rotation<32, 3>(p, f);
    return dispatch_rotation<32, 4>(p, f);
  }
  return p.D <= 128 ? f(Shape<1, 32, 4, kShared>{}) : f(Shape<1, 32, 32, kShared>{});
}

// Shared memory beyond the 48 KiB that every kernel has (wide rotations; `fixed`: what the kernel declares itself).
inline dsa_status_t allow_shared(const void* kernel, int bytes, int fixed) {
  if (bytes + fixed <= 48 * 1024) return DSA_OK;
  return cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 104 * 1024),
                    "shared memory of the norm and rotation");
}

// Rows of a group's run: the rows over the groups that the card holds at once, so that one wave of CTAs takes them all,
// while that is at most 32; 16 beyond it (many waves, whose last one matters less).  A token's heads in one run share
// its cosines and sines.
inline int run_of(int64_t rows, int LPR, int U, int per_sm) {
  const int64_t groups = (int64_t)152 * per_sm * (kThreads / LPR);
  const int64_t run = ((rows + groups - 1) / groups + U - 1) / U * U;
  return run <= 32 ? (int)(run < U ? U : run) : 16;
}

dsa_status_t check_rows(const char* who, Rows& p, int norm, int norm_dim, const float* weight, const float* bias,
                        float eps, int rope_start, int rope_dim, int interleaved, const int32_t* positions,
                        const float* inv_freq, float rope_scale) {
  if (p.T < 0 || p.H < 1 || p.D < 1 || p.D > kMaxD)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: need T >= 0, H >= 1, 1 <= D <= %d (got %d, %d, %d)", who, kMaxD, p.T,
                p.H, p.D);
  if (norm < kNone || norm > kLayer)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: norm must be 0 (none), 1 (rms) or 2 (layer), got %d", who, norm);
  if (norm == kNone ? norm_dim != 0 : (norm_dim < 1 || norm_dim > p.D))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: norm_dim must be 0 without a norm, else in [1, D] (got %d)", who, norm_dim);
  if (norm == kNone && (weight || bias))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: weight and bias belong to a norm", who);
  if (norm != kNone && !(std::isfinite(eps) && eps >= 0.f))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: eps must be finite and >= 0", who);
  if (rope_dim < 0 || (rope_dim & 1) || rope_start < 0 || rope_start > p.D - rope_dim)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: the rotated channels [%d, %d + %d) must be an even number inside [0, D)",
                who, rope_start, rope_start, rope_dim);
  if (interleaved != 0 && interleaved != 1)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: interleaved must be 0 or 1", who);
  if (rope_dim > 0 && !std::isfinite(rope_scale))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: rope_scale must be finite", who);
  if (rope_dim > 0 && (!inv_freq || (p.T > 0 && !positions)))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: a rotation needs positions and inv_freq", who);
  p.kind = norm;
  p.n = norm_dim;
  p.w = weight;
  p.b = bias;
  p.eps = eps;
  p.r0 = rope_start;
  p.R = rope_dim;
  p.inter = interleaved;
  p.pos = positions;
  p.inv_freq = inv_freq;
  p.rscale = rope_scale;
  if ((int64_t)p.T * p.H > kMaxRows)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: T * H must be at most %lld", who, (long long)kMaxRows);
  p.rows = p.T * p.H;
  return DSA_OK;
}

// Rows that are written must not share channels: one stride steps over D, the other over all that the first spans.
inline bool strides_apart(int64_t rows, int H, int D, int64_t st, int64_t sh) {
  if (rows <= 1) return H <= 1 || sh >= D;
  if (H <= 1) return st >= D;
  return (sh >= D && st / sh >= H - 1 && st - (H - 1) * sh >= D) ||
         (st >= D && sh / st >= rows - 1 && sh - (rows - 1) * st >= D);
}
inline bool vec_rows(const void* p, int64_t st, int64_t sh) { return aligned16(p) && st % 8 == 0 && sh % 8 == 0; }

}  // namespace nrope
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_norm_rope_fwd(const dsa_bf16_t* x, int64_t x_stride_t, int64_t x_stride_h, int32_t T,
                                          int32_t H, int32_t D, int32_t norm, int32_t norm_dim, const float* weight,
                                          const float* bias, float eps, int32_t rope_start, int32_t rope_dim,
                                          int32_t interleaved, const int32_t* positions, const float* inv_freq,
                                          float rope_scale, dsa_bf16_t* out, int64_t out_stride_t,
                                          int64_t out_stride_h, const int32_t* out_rows, int64_t num_out_rows,
                                          void* workspace, size_t workspace_bytes, dsa_stream_t stream) {
  const char* who = "dsa_norm_rope_fwd";
  nrope::Rows p{};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.xs = nrope::step_of(x_stride_t, x_stride_h, H);
  p.T = T;
  p.H = H;
  p.D = D;
  dsa_status_t st = nrope::check_rows(who, p, norm, norm_dim, weight, bias, eps, rope_start, rope_dim, interleaved,
                                      positions, inv_freq, rope_scale);
  if (st != DSA_OK) return st;
  if (norm == nrope::kRms && bias) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: the rms norm has no bias", who);
  if (T > 0 && (!x || !out)) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 1)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: x and out must be 2-byte aligned", who);
  if (x_stride_t < 0 || x_stride_h < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: strides must be >= 0", who);
  if (out_rows && (num_out_rows < 0 || num_out_rows > 0x7fffffffll))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: num_out_rows must be in [0, 2^31)", who);
  if (!nrope::strides_apart(out_rows ? num_out_rows : T, H, D, out_stride_t, out_stride_h))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: the rows of out overlap (strides %lld, %lld)", who,
                (long long)out_stride_t, (long long)out_stride_h);
  if ((st = check_workspace(workspace, workspace_bytes, kErrorWordBytes, who)) != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (T == 0) return ok();
  const bool vec = D % 8 == 0 && nrope::vec_rows(x, x_stride_t, x_stride_h) &&
                   nrope::vec_rows(out, out_stride_t, out_stride_h) && norm_dim % 8 == 0 && aligned16(weight) &&
                   aligned16(bias);
  st = nrope::dispatch(vec, p, [&](auto shape) -> dsa_status_t {
    using S = decltype(shape);
    constexpr int U = S::VEC == 1 || S::NIT > 2 ? 1 : S::NIT > 1 ? 2 : 4, GPB = nrope::kThreads / S::LPR;
    p.run = nrope::run_of(p.rows, S::LPR, U, nrope::ctas_per_sm(S::VEC, S::NIT));
    const int64_t want = ((int64_t)p.rows + (int64_t)GPB * p.run - 1) / ((int64_t)GPB * p.run);
    const int64_t most = 152 * nrope::ctas_per_sm(S::VEC, S::NIT);  // (a CTA that stays forms its table once)
    const int blocks = (int)(want < most ? want : most);
    const int smem = nrope::shared_bytes(p.R, GPB, U);
    auto kernel = out_rows ? nrope::norm_rope_fwd_kernel<S::VEC, S::LPR, S::NIT, S::ROT, U, S::KIND, true>
                           : nrope::norm_rope_fwd_kernel<S::VEC, S::LPR, S::NIT, S::ROT, U, S::KIND, S::KIND == nrope::kAny>;
    dsa_status_t ok_smem = nrope::allow_shared(reinterpret_cast<const void*>(kernel), smem, 0);
    if (ok_smem != DSA_OK) return ok_smem;
    kernel<<<blocks, nrope::kThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(
        p, reinterpret_cast<__nv_bfloat16*>(out), nrope::step_of(out_stride_t, out_stride_h, H), out_rows, num_out_rows,
        reinterpret_cast<int*>(workspace));
    return cuda_check(cudaGetLastError(), "launching norm_rope_fwd_kernel");
  });
  return st == DSA_OK ? ok() : st;
}

extern "C" size_t dsa_norm_rope_bwd_workspace_size(int32_t norm_dim) {
  return kErrorWordBytes + (size_t)nrope::kMaxPartials * 2 * sizeof(float) * (norm_dim > 0 ? norm_dim : 0);
}

extern "C" dsa_status_t dsa_norm_rope_bwd(const dsa_bf16_t* dout, int64_t dout_stride_t, int64_t dout_stride_h,
                                          const dsa_bf16_t* x, int64_t x_stride_t, int64_t x_stride_h, int32_t T,
                                          int32_t H, int32_t D, int32_t norm, int32_t norm_dim, const float* weight,
                                          float eps, int32_t rope_start, int32_t rope_dim, int32_t interleaved,
                                          const int32_t* positions, const float* inv_freq, float rope_scale,
                                          dsa_bf16_t* dx, int64_t dx_stride_t, int64_t dx_stride_h, float* dweight,
                                          float* dbias, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                          dsa_stream_t stream) {
  const char* who = "dsa_norm_rope_bwd";
  nrope::Rows p{};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.xs = nrope::step_of(x_stride_t, x_stride_h, H);
  p.T = T;
  p.H = H;
  p.D = D;
  dsa_status_t st = nrope::check_rows(who, p, norm, norm_dim, weight, nullptr, eps, rope_start, rope_dim, interleaved,
                                      positions, inv_freq, rope_scale);
  if (st != DSA_OK) return st;
  if (T > 0 && (!dout || !dx || (norm && !x))) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if ((norm == nrope::kNone && (dweight || dbias)) || (norm == nrope::kRms && dbias))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: dweight belongs to a norm and dbias to the layer norm", who);
  if (accumulate != 0 && accumulate != 1) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: accumulate must be 0 or 1", who);
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dx)) & 1)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: x, dout and dx must be 2-byte aligned", who);
  if (x_stride_t < 0 || x_stride_h < 0 || dout_stride_t < 0 || dout_stride_h < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: strides must be >= 0", who);
  if (!nrope::strides_apart(T, H, D, dx_stride_t, dx_stride_h))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: the rows of dx overlap (strides %lld, %lld)", who,
                (long long)dx_stride_t, (long long)dx_stride_h);
  if ((st = check_workspace(workspace, workspace_bytes, dsa_norm_rope_bwd_workspace_size(norm_dim), who)) != DSA_OK)
    return st;
  if ((st = check_device()) != DSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* partials = (dweight || dbias) ? reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kErrorWordBytes)
                                       : nullptr;
  int blocks = 0;
  if (T > 0) {
    const bool vec = D % 8 == 0 && nrope::vec_rows(dout, dout_stride_t, dout_stride_h) &&
                     nrope::vec_rows(dx, dx_stride_t, dx_stride_h) &&
                     (!norm || (norm_dim % 8 == 0 && nrope::vec_rows(x, x_stride_t, x_stride_h))) && aligned16(weight);
    st = nrope::dispatch(vec, p, [&](auto shape) -> dsa_status_t {
      using S = decltype(shape);
      constexpr int U = S::VEC == 1 || S::NIT > 1 ? 1 : 2, GPB = nrope::kThreads / S::LPR;
      p.run = nrope::run_of(p.rows, S::LPR, U, S::NIT == 1 ? 2 : nrope::ctas_per_sm(S::VEC, S::NIT));
      const int64_t want = ((int64_t)p.rows + (int64_t)GPB * p.run - 1) / ((int64_t)GPB * p.run);
      const int most = partials ? nrope::kMaxPartials : 152 * 4;
      blocks = (int)(want < most ? want : most);
      const int smem = nrope::shared_bytes(p.R, GPB, U);
      auto kernel = nrope::norm_rope_bwd_kernel<S::VEC, S::LPR, S::NIT, S::ROT, U>;
      dsa_status_t ok_smem = nrope::allow_shared(reinterpret_cast<const void*>(kernel), smem, 8192);
      if (ok_smem != DSA_OK) return ok_smem;
      kernel<<<blocks, nrope::kThreads, smem, s>>>(p, reinterpret_cast<const __nv_bfloat16*>(dout),
                                                   nrope::step_of(dout_stride_t, dout_stride_h, H),
                                                   reinterpret_cast<__nv_bfloat16*>(dx),
                                                   nrope::step_of(dx_stride_t, dx_stride_h, H), partials);
      return cuda_check(cudaGetLastError(), "launching norm_rope_bwd_kernel");
    });
    if (st != DSA_OK) return st;
  }
  if (partials) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((2 * norm_dim + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = blocks > 0 ? 1 : 0;
    st = cuda_check(cudaLaunchKernelEx(&cfg, nrope::norm_rope_sum_kernel, (const float*)partials, blocks, norm_dim, dweight,
                                       dbias, accumulate),
                    "launching norm_rope_sum_kernel");
    if (st != DSA_OK) return st;
  }
  return ok();
}

extern "C" dsa_status_t dsa_rope_frequencies(int32_t rope_dim, double base, double factor, int32_t original_context,
                                             double beta_fast, double beta_slow, float* inv_freq_host,
                                             float* rope_scale_host) {
  const char* who = "dsa_rope_frequencies";
  if (rope_dim < 2 || (rope_dim & 1)) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: rope_dim must be even and >= 2", who);
  if (!(std::isfinite(base) && base > 1.0) || !(std::isfinite(factor) && factor >= 1.0))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: need base > 1 and factor >= 1", who);
  if (factor > 1.0 && (original_context < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0) || !std::isfinite(beta_fast)))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: scaling needs original_context >= 1 and beta_fast > beta_slow > 0", who);
  if (!inv_freq_host || !rope_scale_host) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null pointer", who);
  const double two_pi = 6.283185307179586476925;
  // the pair whose wave turns `r` times over the original context
  auto pair_of = [&](double r) { return rope_dim * std::log(original_context / (r * two_pi)) / (2.0 * std::log(base)); };
  double low = 0.0, high = 0.0;
  if (factor > 1.0) {
    low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(beta_slow)), (double)(rope_dim - 1));
    if (!(high > low)) high = low + 0.001;
  }
  for (int i = 0; i < rope_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rope_dim);
    double ramp = 0.0;
    if (factor > 1.0) ramp = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
    inv_freq_host[i] = (float)(f * (1.0 - ramp) + f / factor * ramp);
  }
  *rope_scale_host = factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return ok();
}
