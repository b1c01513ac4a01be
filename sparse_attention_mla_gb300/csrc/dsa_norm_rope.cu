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
// What bounds it: DRAM, 4 bytes a channel forward and 6 backward.  So the rows
// stay in registers between the one read and the one write, LPR lanes to a row
// (8 for 64 channels, 16 for 128, else a warp), 16 bytes a lane, the next row's
// loads in flight while this one is worked on.  The cosines and sines depend on
// the token alone: a group of lanes keeps one token and walks its heads, so they
// are formed once for up to 16 heads, spread over the lanes, and kept in shared
// memory.
//
// Angles: positions reach millions, and position times frequency in fp32 is then
// off by 0.1 rad.  The frequency is held as a 64-bit binary fraction of a turn, so
// that position times fraction modulo 2^64 drops whole turns exactly; its upper
// 32 bits are the angle.  Sums and statistics are fp32; rows are rounded to bf16
// once, when written.
#include <cmath>

#include "dsa_device.cuh"
#include "dsa_host.h"

namespace dsa {
namespace nrope {

constexpr int kThreads = 128;
constexpr int kMaxD = 1024;
constexpr int kMaxPartials = 608;  // CTAs of a backward launch: each leaves one row of dw and db
enum { kNone = 0, kRms = 1, kLayer = 2 };

struct Rows {
  const __nv_bfloat16* x;
  int64_t xs_t, xs_h;
  int T, H, D;
  int kind, n;
  const float* w;
  const float* b;
  float eps;
  int r0, R, inter;
  const int32_t* pos;
  const float* inv_freq;
  float rscale;
  int hpt;        // heads that a group of lanes takes of one token
  int64_t tasks;  // T * ceil(H / hpt)
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A row in registers: E = VEC * NIT channels per lane, channel c = (it * LPR + l) * VEC + e.
template <int VEC, int LPR, int NIT>
struct Raw {
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
  __device__ __forceinline__ void values(float (&f)[VEC * NIT]) const {
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      if constexpr (VEC == 8) {
        const uint32_t u[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[it * 8 + 2 * k] = bf_lo(u[k]);
          f[it * 8 + 2 * k + 1] = bf_hi(u[k]);
        }
      } else {
        f[it] = __uint_as_float((uint32_t)s[it] << 16);
      }
    }
  }
};

template <int VEC, int LPR, int NIT>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int D, int l, const float (&f)[VEC * NIT]) {
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int c = (it * LPR + l) * VEC;
    if (c >= D) continue;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack_bf16x2(f[it * 8], f[it * 8 + 1]), pack_bf16x2(f[it * 8 + 2], f[it * 8 + 3]),
                     pack_bf16x2(f[it * 8 + 4], f[it * 8 + 5]), pack_bf16x2(f[it * 8 + 6], f[it * 8 + 7]));
    } else {
      row[c] = __float2bfloat16_rn(f[it]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Shared memory: the fractions of a turn per position [R/2], then per group of lanes the token's
// (scaled) cosines and sines [R/2] and R channels for the exchange between the two of a pair.
struct Shared {
  uint64_t* turn;
  float2* cs;
  float* stage;
};
__device__ __forceinline__ Shared carve(uint8_t* raw, int R, int group) {
  const int half = R >> 1;
  Shared s;
  s.turn = reinterpret_cast<uint64_t*>(raw);
  uint8_t* mine = raw + (size_t)half * 8 + (size_t)group * half * 16;
  s.cs = reinterpret_cast<float2*>(mine);
  s.stage = reinterpret_cast<float*>(mine + (size_t)half * 8);
  return s;
}
inline int shared_bytes(int R, int groups) { return (R >> 1) * 8 + groups * (R >> 1) * 16; }

__device__ __forceinline__ void fill_turns(uint64_t* turn, const Rows& p) {
  for (int i = threadIdx.x; i < (p.R >> 1); i += kThreads) {
    double f = (double)__ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    turn[i] = (uint64_t)(f * 18446744073709551616.0);  // f < 1: below 2^64
  }
}

template <int LPR>
__device__ __forceinline__ void fill_cos_sin(const Shared& s, const Rows& p, int t, int l) {
  const int64_t pos = __ldg(p.pos + t);
  for (int i = l; i < (p.R >> 1); i += LPR) {
    const int32_t frac = (int32_t)(((uint64_t)pos * s.turn[i]) >> 32);  // signed: [-1/2, 1/2) of a turn
    float sn, c;
    sincospif((float)frac * 4.656612873077393e-10f, &sn, &c);  // 2^-31: half turns
    s.cs[i] = make_float2(c * p.rscale, sn * p.rscale);
  }
}

// Turns the row's rotated channels in place; back = -1 turns the other way (the transpose).
template <int VEC, int LPR, int NIT>
__device__ __forceinline__ void rotate(float (&f)[VEC * NIT], const Shared& s, const Rows& p, int l, float back) {
  if (p.R == 0) return;
  const int half = p.R >> 1;
  if (VEC == 8 && p.inter) {  // both of a pair are in this lane (r0 is even on this path)
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int u0 = (it * LPR + l) * VEC - p.r0;
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const int u = u0 + e;
        if (u < 0 || u >= p.R) continue;
        const float2 c = s.cs[u >> 1];
        const float sn = c.y * back, a = f[it * VEC + e], b = f[it * VEC + (e | (VEC > 1))];
        f[it * VEC + e] = a * c.x - b * sn;
        f[it * VEC + (e | (VEC > 1))] = b * c.x + a * sn;
      }
    }
    return;
  }
  __syncwarp();  // the row before has been read
#pragma unroll
  for (int it = 0; it < NIT; ++it)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int u = (it * LPR + l) * VEC + e - p.r0;
      if (u >= 0 && u < p.R) s.stage[u] = f[it * VEC + e];
    }
  __syncwarp();
#pragma unroll
  for (int it = 0; it < NIT; ++it)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int u = (it * LPR + l) * VEC + e - p.r0;
      if (u < 0 || u >= p.R) continue;
      const bool second = p.inter ? (u & 1) : (u >= half);
      const int i = p.inter ? (u >> 1) : (second ? u - half : u);
      const int other = p.inter ? (u ^ 1) : (second ? u - half : u + half);
      const float2 c = s.cs[i];
      const float sn = second ? c.y * back : -c.y * back;
      f[it * VEC + e] = f[it * VEC + e] * c.x + s.stage[other] * sn;
    }
}

// weight or bias of this lane's channels below n (`none` where there is no array)
template <int VEC, int LPR, int NIT>
__device__ __forceinline__ float param(const float* a, float none, int n, int l, int k) {
  const int c = ((k / VEC) * LPR + l) * VEC + (k % VEC);
  return (a != nullptr && c < n) ? __ldg(a + c) : none;
}

template <int VEC, int LPR, int NIT>
__global__ void __launch_bounds__(kThreads)
    norm_rope_fwd_kernel(const Rows p, __nv_bfloat16* out, int64_t os_t, int64_t os_h,
                         const int32_t* __restrict__ out_rows, int64_t num_rows, int* __restrict__ err) {
  constexpr int E = VEC * NIT, GPW = 32 / LPR, GPB = kThreads / LPR;
  extern __shared__ __align__(16) uint8_t raw_sh[];
  const int lane = threadIdx.x & 31, l = lane & (LPR - 1), group = threadIdx.x / LPR;
  const Shared s = carve(raw_sh, p.R, group);
  fill_turns(s.turn, p);
  __syncthreads();
  const int nhb = (p.H + p.hpt - 1) / p.hpt;
  const float inv_n = p.n > 0 ? 1.f / (float)p.n : 0.f;
  // the groups of a warp run the same trip counts; `on` marks the ones that have a row
  const int64_t first = (int64_t)blockIdx.x * GPB + group, step = (int64_t)gridDim.x * GPB;
  const int64_t warp_first = first - (lane / LPR);
  Raw<VEC, LPR, NIT> cur;
  auto row_of = [&](int64_t task, int hh, bool& on, int& t, int& h) {
    t = (int)(task / nhb);
    h = (int)(task - (int64_t)t * nhb) * p.hpt + hh;
    on = task < p.tasks && h < p.H;
  };
  auto fetch = [&](int64_t task, int hh) {
    bool on;
    int t, h;
    row_of(task, hh, on, t, h);
    cur.load(p.x + (on ? t * p.xs_t + h * p.xs_h : 0), p.D, l, on);
  };
  fetch(first, 0);
  for (int64_t k = 0; warp_first + k * step < p.tasks; ++k) {
    const int64_t task = first + k * step;
    if (p.R > 0) {
      __syncwarp();
      if (task < p.tasks) fill_cos_sin<LPR>(s, p, (int)(task / nhb), l);
      __syncwarp();
    }
    for (int hh = 0; hh < p.hpt; ++hh) {
      bool on;
      int t, h;
      row_of(task, hh, on, t, h);
      float f[E];
      cur.values(f);
      if (hh + 1 < p.hpt) fetch(task, hh + 1);
      else fetch(task + step, 0);
      if (p.kind != kNone) {
        float mean = 0.f, ss = 0.f;
        if (p.kind == kLayer) {
#pragma unroll
          for (int i = 0; i < E; ++i) mean += (((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n) ? f[i] : 0.f;
          mean = group_sum<LPR>(mean) * inv_n;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const bool in = ((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n;
          if (in) f[i] -= mean;
          ss += in ? f[i] * f[i] : 0.f;
        }
        const float r = rsqrtf(group_sum<LPR>(ss) * inv_n + p.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n)
            f[i] = f[i] * r * param<VEC, LPR, NIT>(p.w, 1.f, p.n, l, i) + param<VEC, LPR, NIT>(p.b, 0.f, p.n, l, i);
        }
      }
      rotate<VEC, LPR, NIT>(f, s, p, l, 1.f);
      if (on) {
        int64_t o = t;
        if (out_rows != nullptr) {
          o = __ldg(out_rows + t);
          if (o < -1 || o >= num_rows) {
            if (l == 0) record_error(err, DSA_ERR_DEVICE_INDEX);
            o = -1;
          }
        }
        if (o >= 0) store_row<VEC, LPR, NIT>(out + o * os_t + h * os_h, p.D, l, f);
      }
    }
  }
}

template <int VEC, int LPR, int NIT>
__global__ void __launch_bounds__(kThreads)
    norm_rope_bwd_kernel(const Rows p, const __nv_bfloat16* dout, int64_t gs_t, int64_t gs_h, __nv_bfloat16* dx,
                         int64_t ds_t, int64_t ds_h, float* __restrict__ partials) {
  constexpr int E = VEC * NIT, GPB = kThreads / LPR;
  extern __shared__ __align__(16) uint8_t raw_sh[];
  const int lane = threadIdx.x & 31, l = lane & (LPR - 1), group = threadIdx.x / LPR;
  const Shared s = carve(raw_sh, p.R, group);
  fill_turns(s.turn, p);
  __syncthreads();
  const int nhb = (p.H + p.hpt - 1) / p.hpt;
  const float inv_n = p.n > 0 ? 1.f / (float)p.n : 0.f;
  const int64_t first = (int64_t)blockIdx.x * GPB + group, step = (int64_t)gridDim.x * GPB;
  const int64_t warp_first = first - (lane / LPR);
  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
  Raw<VEC, LPR, NIT> gcur, xcur;
  auto row_of = [&](int64_t task, int hh, bool& on, int& t, int& h) {
    t = (int)(task / nhb);
    h = (int)(task - (int64_t)t * nhb) * p.hpt + hh;
    on = task < p.tasks && h < p.H;
  };
  auto fetch = [&](int64_t task, int hh) {
    bool on;
    int t, h;
    row_of(task, hh, on, t, h);
    gcur.load(dout + (on ? t * gs_t + h * gs_h : 0), p.D, l, on);
    if (p.kind != kNone) xcur.load(p.x + (on ? t * p.xs_t + h * p.xs_h : 0), p.n, l, on);
  };
  fetch(first, 0);
  for (int64_t k = 0; warp_first + k * step < p.tasks; ++k) {
    const int64_t task = first + k * step;
    if (p.R > 0) {
      __syncwarp();
      if (task < p.tasks) fill_cos_sin<LPR>(s, p, (int)(task / nhb), l);
      __syncwarp();
    }
    for (int hh = 0; hh < p.hpt; ++hh) {
      bool on;
      int t, h;
      row_of(task, hh, on, t, h);
      float g[E], x[E];
      gcur.values(g);
      if (p.kind != kNone) xcur.values(x);
      if (hh + 1 < p.hpt) fetch(task, hh + 1);
      else fetch(task + step, 0);
      rotate<VEC, LPR, NIT>(g, s, p, l, -1.f);
      if (p.kind != kNone) {
        float sx = 0.f, sg = 0.f;
        if (p.kind == kLayer) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const bool in = ((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n;
            sx += in ? x[i] : 0.f;
            sg += in ? g[i] * param<VEC, LPR, NIT>(p.w, 1.f, p.n, l, i) : 0.f;
          }
          sx = group_sum<LPR>(sx) * inv_n;
          sg = group_sum<LPR>(sg) * inv_n;
        }
        float ss = 0.f, sgx = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const bool in = ((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n;
          x[i] = in ? x[i] - sx : 0.f;
          ss += x[i] * x[i];
          sgx += in ? g[i] * param<VEC, LPR, NIT>(p.w, 1.f, p.n, l, i) * x[i] : 0.f;
        }
        ss = group_sum<LPR>(ss);
        sgx = group_sum<LPR>(sgx);
        const float r = rsqrtf(ss * inv_n + p.eps);
        const float m = sgx * r * inv_n;  // mean(gw xh)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const bool in = ((i / VEC) * LPR + l) * VEC + (i % VEC) < p.n;
          if (!in || !on) continue;
          const float xh = x[i] * r;
          dw[i] += g[i] * xh;
          db[i] += g[i];
          g[i] = r * (g[i] * param<VEC, LPR, NIT>(p.w, 1.f, p.n, l, i) - sg - xh * m);
        }
      }
      if (on) store_row<VEC, LPR, NIT>(dx + t * ds_t + h * ds_h, p.D, l, g);
    }
  }
  if (partials == nullptr) return;
  // the CTA's sums: the groups of a warp by shuffles, then the warps one after the other in shared memory
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
    }
  }
  __shared__ float acc[2][kMaxD];
  for (int w = 0; w < kThreads / 32; ++w) {
    if ((threadIdx.x >> 5) == w && lane < LPR) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = ((i / VEC) * LPR + l) * VEC + (i % VEC);
        if (c < p.n) {
          acc[0][c] = w ? acc[0][c] + dw[i] : dw[i];
          acc[1][c] = w ? acc[1][c] + db[i] : db[i];
        }
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
    norm_rope_sum_kernel(const float* __restrict__ partials, int count, int n, float* __restrict__ dweight,
                         float* __restrict__ dbias, int accumulate) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < 2 * n)
    for (int r = w; r < count; r += 32) v += __ldg(partials + (size_t)r * 2 * n + c);
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

// Calls f<VEC, LPR, NIT>: 16-byte accesses where every row starts on a 16-byte boundary and the pairs of an
// interleaved rotation stay inside one; else one channel at a time.
template <class F>
dsa_status_t dispatch(bool vec, int D, F&& f) {
  if (vec) {
    if (D <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    if (D <= 128) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (D <= 256) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    if (D <= 512) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
    if (D <= 768) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 3>{});
    return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  }
  if (D <= 128) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
}

// Heads a group of lanes takes of one token: up to 16 share a token's cosines and sines, fewer while the
// launch has too few groups to fill the card (152 SMs x 64 groups).
inline int heads_per_task(int64_t T, int H, int R) {
  if (R == 0) return 1;
  int hpt = 1;
  while (hpt < 16 && hpt < H && T * ((H + 2 * hpt - 1) / (2 * hpt)) >= 152 * 64) hpt *= 2;
  return hpt;
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
  p.hpt = heads_per_task(p.T, p.H, rope_dim);
  p.tasks = (int64_t)p.T * ((p.H + p.hpt - 1) / p.hpt);
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
  p.xs_t = x_stride_t;
  p.xs_h = x_stride_h;
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
                   nrope::vec_rows(out, out_stride_t, out_stride_h) && !(interleaved && (rope_start & 1));
  st = nrope::dispatch(vec, D, [&](auto v, auto lpr, auto nit) -> dsa_status_t {
    constexpr int VEC = decltype(v)::value, LPR = decltype(lpr)::value, NIT = decltype(nit)::value;
    constexpr int GPB = nrope::kThreads / LPR;
    const int64_t want = (p.tasks + GPB - 1) / GPB;
    const int blocks = (int)(want < 152 * 16 ? want : 152 * 16);
    nrope::norm_rope_fwd_kernel<VEC, LPR, NIT>
        <<<blocks, nrope::kThreads, nrope::shared_bytes(p.R, GPB), reinterpret_cast<cudaStream_t>(stream)>>>(
            p, reinterpret_cast<__nv_bfloat16*>(out), out_stride_t, out_stride_h, out_rows, num_out_rows,
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
  p.xs_t = x_stride_t;
  p.xs_h = x_stride_h;
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
                     nrope::vec_rows(dx, dx_stride_t, dx_stride_h) && !(interleaved && (rope_start & 1)) &&
                     (!norm || (norm_dim % 8 == 0 && nrope::vec_rows(x, x_stride_t, x_stride_h)));
    st = nrope::dispatch(vec, D, [&](auto v, auto lpr, auto nit) -> dsa_status_t {
      constexpr int VEC = decltype(v)::value, LPR = decltype(lpr)::value, NIT = decltype(nit)::value;
      constexpr int GPB = nrope::kThreads / LPR;
      const int64_t want = (p.tasks + GPB - 1) / GPB;
      const int most = partials ? nrope::kMaxPartials : 152 * 16;
      blocks = (int)(want < most ? want : most);
      nrope::norm_rope_bwd_kernel<VEC, LPR, NIT><<<blocks, nrope::kThreads, nrope::shared_bytes(p.R, GPB), s>>>(
          p, reinterpret_cast<const __nv_bfloat16*>(dout), dout_stride_t, dout_stride_h,
          reinterpret_cast<__nv_bfloat16*>(dx), dx_stride_t, dx_stride_h, partials);
      return cuda_check(cudaGetLastError(), "launching norm_rope_bwd_kernel");
    });
    if (st != DSA_OK) return st;
  }
  if (partials) {
    nrope::norm_rope_sum_kernel<<<(2 * norm_dim + 31) / 32, 1024, 0, s>>>(partials, blocks, norm_dim, dweight, dbias,
                                                                         accumulate);
    if ((st = cuda_check(cudaGetLastError(), "launching norm_rope_sum_kernel")) != DSA_OK) return st;
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
