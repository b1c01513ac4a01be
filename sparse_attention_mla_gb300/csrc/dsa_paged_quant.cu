// dsa_paged_quant.cu -- rows quantised as they are written to a paged cache, and read back (sm_103a).
//
// A row's scale s is a power of two (codes that have an exponent of their own lose nothing by that), a block's scale
// e4m3, a code the nearest of e4m3 or e2m1: x / s and every value read back are exact, and a code does not depend on
// how a quotient was rounded (see nearest_side).  Both directions are bound by memory: a row is read once and written
// once, 1152 + 420 bytes for a latent in 4 bits.  Reading 12 requests of 7500 to 30000 latents of 4 bits back: 66 us, 5.7
// TB/s, where a copy reaches 6.8 (8 channels a thread in place of 16, and stores of 16 bytes in place of 32: 73.7); writing
// 8191 latents of 4 bits and reading them: 11.0 us, two kernels of little more than their launch.  Writing 131072 rows of 128
// channels of 8 bits: 13.8 us where their bytes take 7.6, 131072 latents 49 (8 bits; bytes 35) and 58 (4 bits; bytes 30): a row's
// loads wait for another one, its place, and a thread has one row and is gone.
#include <climits>

#include "dsa_host.h"
#include "dsa_paged.cuh"
#include "dsa_paged_quant.cuh"

namespace dsa {
namespace pquant {

constexpr int kThreads = 256;
constexpr int kSms = 152;

struct Rows {
  const __nv_bfloat16* x;
  long long stride;
  int T, D, Q;
  uint8_t* cache;
  long long num_rows;
  const int32_t* out_rows;
  int* err;
  bool vec;  // 16-byte aligned rows of x
};

__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(h + 2 * i) | ((uint32_t)__ldg(h + 2 * i + 1) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A quotient q = v * (1 / block) with relative error below 2^-22, to 12 bits: q then lies on the side of every border
// between two codes that the exact quotient lies on, or on the border when that does.  v has 8 bits and block 4, so that
// v / block = X / m 2^i with integers X < 256, 8 <= m < 16, and a border is b = T 2^j with T in {1, 3, 5, 7}: where the two
// differ, they do by a part in X at least when i <= j, or in m T < 106 otherwise, more than 2^-8; 12 bits change it by 2^-12.
__device__ __forceinline__ float nearest_side(float q) {
  return __uint_as_float((__float_as_uint(q) + 0x800u) & 0xfffff000u);
}

// Two values to e4m3, e2m1 (the first in the lower half); magnitudes past the largest code become that code.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, z;\n\tmov.b16 {z, b}, 0;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tmov.b32 %0, {b, z, z, z};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// LPR lanes a row (a power of two), 16 channels each: one block of 4 bits, 16 bytes of 8.  NIT: rounds of them.
template <int BITS, int LPR, int NIT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Rows p) {
  const int lane = threadIdx.x & 31, sub = lane & (LPR - 1);
  const long long row_t = ((long long)blockIdx.x * kThreads + threadIdx.x) / LPR;
  const int t = row_t < p.T ? (int)row_t : -1;
  const QuantRow lay = quant_row(p.D, p.Q, BITS);
  long long to = -1;
  if (t >= 0) {
    to = p.out_rows ? __ldg(p.out_rows + t) : t;
    if (to < -1 || to >= p.num_rows) {
      if (sub == 0) record_error(p.err, DSA_ERR_DEVICE_INDEX);
      to = -1;
    }
  }
  const __nv_bfloat16* x = p.x + (t < 0 ? 0 : t) * p.stride;
  uint4 a[NIT][2];
  uint32_t top[NIT];  // the largest magnitude of the lane's block, as its bits
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < NIT; ++k) {
    const int c = (k * LPR + sub) * 16;
    a[k][0] = a[k][1] = make_uint4(0, 0, 0, 0);
    if (to >= 0 && c < p.Q) {
      a[k][0] = load8(x + c, p.vec);
      a[k][1] = load8(x + c + 8, p.vec);
    }
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m = __vmaxu2(m, a[k][h].x & 0x7fff7fffu);
      m = __vmaxu2(m, a[k][h].y & 0x7fff7fffu);
      m = __vmaxu2(m, a[k][h].z & 0x7fff7fffu);
      m = __vmaxu2(m, a[k][h].w & 0x7fff7fffu);
    }
    top[k] = max(m & 0xffffu, m >> 16);
    most = max(most, top[k]);
  }
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (to < 0) return;
  // s = 2^e: 448 = 1.75 2^8, 2688 = 1.3125 2^11; infinities and NaN have the largest exponent
  const uint32_t bits = most << 16;
  int e = (int)(bits >> 23) - 127 - (BITS == 8 ? 8 : 11) + ((bits & 0x7fffffu) > (BITS == 8 ? 0x600000u : 0x280000u) ? 1 : 0);
  const bool bad = e > 48;
  e = max(e, -48);
  const float inv_s = __uint_as_float((uint32_t)(127 - e) << 23);
  uint8_t* row = p.cache + (size_t)to * lay.bytes;
#pragma unroll
  for (int k = 0; k < NIT; ++k) {
    const int unit = k * LPR + sub;
    if (unit * 16 >= p.Q) continue;
    float factor = inv_s;
    if constexpr (BITS == 4) {
      const float a6 = __fdiv_rn(__uint_as_float(top[k] << 16) * inv_s, 6.f);
      const uint32_t code = bad ? 0 : to_e4m3x2(a6, 0.f) & 0xff;
      const float block = f16x2_floats(e4m3x2_f16x2((uint16_t)code)).x;
      factor = block > 0.f ? inv_s / block : 0.f;
      row[lay.blocks + unit] = (uint8_t)code;
    }
    uint32_t w[8] = {a[k][0].x, a[k][0].y, a[k][0].z, a[k][0].w, a[k][1].x, a[k][1].y, a[k][1].z, a[k][1].w};
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float lo = __uint_as_float(w[i] << 16) * factor, hi = __uint_as_float(w[i] & 0xffff0000u) * factor;
      if constexpr (BITS == 8) code[i] = to_e4m3x2(lo, hi);
      else code[i] = to_e2m1x2(nearest_side(lo), nearest_side(hi));
    }
    if constexpr (BITS == 8) {
      uint4 v = make_uint4(code[0] | code[1] << 16, code[2] | code[3] << 16, code[4] | code[5] << 16, code[6] | code[7] << 16);
      if (bad) v = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(row + unit * 16) = v;
    } else {
      uint2 v = make_uint2(code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                           code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24);
      if (bad) v = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(row + unit * 8) = v;
    }
  }
  if (sub < (lay.tail - lay.scale) / 4)
    reinterpret_cast<uint32_t*>(row + lay.scale)[sub] = sub == 0 ? (bad ? 0x7fc00000u : (uint32_t)(127 + e) << 23) : 0u;
  for (int c = sub * 8; c < p.D - p.Q; c += LPR * 8)
    *reinterpret_cast<uint4*>(row + lay.tail + 2 * c) = load8(x + p.Q + c, p.vec);
}

struct Back {
  const uint8_t* cache;
  const int32_t *table, *first, *cu;
  int N, B, D, Q, num_pages, P, max_pages;
  int rows;                  // of a CTA: 32 a warp that looks them up
  // ceil(2^21 / units) of both parts, of 16 and 8 channels: a unit's row is (i inv) >> 21 for i < 64 * 128
  unsigned inv_q, inv_tail;
  __nv_bfloat16* out;
  long long stride;
  int* err;
  int align;  // of the rows of out: 32, 16 or 2 bytes
};
constexpr int kBackRows = 64;  // at most

// A CTA reads rows that follow one another in the output: a warp finds where 32 of them lie (together: a search of its own
// for each row is a chain of loads, and a CTA has little else to do), then all threads take units of 16 channels (a
// block), so that a warp writes 1024 bytes that follow one another; two units at a time, loads before stores.
template <int BITS>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Back p) {
  __shared__ long long s_row[kBackRows];  // row of the cache; -1: zeros, -2: not to be written
  const long long t0 = (long long)blockIdx.x * p.rows;
  if (threadIdx.x < p.rows) {
    const long long first = t0 + (threadIdx.x & ~31);  // of this warp's
    const int begin = min(max(__ldg(p.cu), 0), p.N), end = min(max(__ldg(p.cu + p.B), 0), p.N);
    const int from = (int)max(first, (long long)begin), to = (int)min(first + 32, (long long)end) - 1;
    long long row = -2;
    if (from <= to) {  // (of the whole warp)
      // the last requests that begin at the first row or before, and at the last one or before
      int lo = warp_last_le(p.cu, p.B, from), hi = lo + 1;
      if (__ldg(p.cu + hi) <= to) hi = warp_last_le(p.cu, p.B, to) + 1;
      const long long t = t0 + threadIdx.x;
      if (t >= from && t <= to) {
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.cu + mid) <= t) lo = mid;
          else hi = mid;
        }
        const long long pos = t - __ldg(p.cu + lo) + (p.first ? __ldg(p.first + lo) : 0);
        row = -1;
        if (pos >= 0 && pos < (long long)p.max_pages * p.P) {
          const unsigned at = (unsigned long long)pos <= UINT_MAX ? (unsigned)pos / (unsigned)p.P : (unsigned)(pos / p.P);
          const int page = __ldg(p.table + (size_t)lo * p.max_pages + at);
          if (page >= 0 && page < p.num_pages) row = (long long)page * p.P + (pos - (long long)at * p.P);
        }
        if (row < 0) record_error(p.err, DSA_ERR_DEVICE_INDEX);
      }
    }
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  const QuantRow lay = quant_row(p.D, p.Q, BITS);
  const int rows = (int)min((long long)p.rows, p.N - t0), q16 = p.Q / 16, tail8 = (p.D - p.Q) / 8;
  auto store8 = [&](__nv_bfloat16* dst, uint4 v) {
    if (p.align >= 16) {
      *reinterpret_cast<uint4*>(dst) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) reinterpret_cast<uint16_t*>(dst)[k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
  };
  constexpr int kAtOnce = 2;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < rows * q16; i0 += kThreads * kAtOnce) {
    int r[kAtOnce];
    bool zero[kAtOnce];
    uint4 code[kAtOnce];
    uint32_t block[kAtOnce];
    float scale[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads;
      r[k] = (int)(((unsigned)i * p.inv_q) >> 21);
      const long long at = i < rows * q16 ? s_row[r[k]] : -2;
      const int u = i - r[k] * q16;
      const uint8_t* row = p.cache + (size_t)(at < 0 ? 0 : at) * lay.bytes;
      zero[k] = at == -1;
      if (at == -2) r[k] = -1;
      code[k] = make_uint4(0, 0, 0, 0);
      block[k] = 0;
      scale[k] = 0.f;
      if (at >= 0) {
        scale[k] = __ldg(reinterpret_cast<const float*>(row + lay.scale));
        if constexpr (BITS == 8) {
          code[k] = __ldg(reinterpret_cast<const uint4*>(row) + u);
        } else {
          block[k] = __ldg(row + lay.blocks + u);
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(row) + u);
          code[k].x = c.x;
          code[k].y = c.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (r[k] < 0) continue;
      uint32_t h[8], o[8];
      if constexpr (BITS == 8) {
        const uint32_t c[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          h[2 * x] = e4m3x2_f16x2((uint16_t)c[x]);
          h[2 * x + 1] = e4m3x2_f16x2((uint16_t)(c[x] >> 16));
        }
      } else {
        const uint32_t by = e4m3x2_f16x2((uint16_t)(block[k] | block[k] << 8));
        uint32_t lo[4], hi[4];
        e2m1x8_f16x2(code[k].x, lo);
        e2m1x8_f16x2(code[k].y, hi);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          h[x] = mul_f16x2(lo[x], by);
          h[4 + x] = mul_f16x2(hi[x], by);
        }
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float2 f = f16x2_floats(h[x]);
        o[x] = zero[k] ? 0u : pack_bf16x2(f.x * scale[k], f.y * scale[k]);
      }
      __nv_bfloat16* dst = p.out + (t0 + r[k]) * p.stride + (i0 + k * kThreads - r[k] * q16) * 16;
      if (p.align == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]),
                     "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
      } else {
        store8(dst, make_uint4(o[0], o[1], o[2], o[3]));
        store8(dst + 8, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < rows * tail8; i += kThreads) {
    const int r = (int)(((unsigned)i * p.inv_tail) >> 21), u = i - r * tail8;
    const long long at = s_row[r];
    if (at == -2) continue;
    const uint4* src = reinterpret_cast<const uint4*>(p.cache + (size_t)(at < 0 ? 0 : at) * lay.bytes + lay.tail) + u;
    store8(p.out + (t0 + r) * p.stride + p.Q + u * 8, at < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src));
  }
}

inline bool share(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

template <int BITS>
dsa_status_t quantize(const Rows& p, cudaStream_t s) {
  auto go = [&](auto kernel, int lpr) -> dsa_status_t {
    const int64_t blocks = ((int64_t)p.T * lpr + kThreads - 1) / kThreads;
    kernel<<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cuda_check(cudaGetLastError(), "launching quantize_kernel");
  };
  if (p.Q <= 64) return go(quantize_kernel<BITS, 4, 1>, 4);
  if (p.Q <= 128) return go(quantize_kernel<BITS, 8, 1>, 8);
  if (p.Q <= 256) return go(quantize_kernel<BITS, 16, 1>, 16);
  if (p.Q <= 512) return go(quantize_kernel<BITS, 32, 1>, 32);
  return go(quantize_kernel<BITS, 32, 2>, 32);
}

}  // namespace pquant
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_paged_quant_row_bytes(int32_t D, int32_t quant_dim, int32_t bits) {
  return quant_row_ok(D, quant_dim, bits) ? (size_t)quant_row(D, quant_dim, bits).bytes : 0;
}

static dsa_status_t check_format(const char* who, int32_t D, int32_t quant_dim, int32_t bits) {
  if (quant_row_ok(D, quant_dim, bits)) return DSA_OK;
  return fail(DSA_ERR_INVALID_ARGUMENT,
              "%s: need bits 8 or 4, quant_dim a multiple of 64, D <= 1024 and D - quant_dim >= 0 a multiple of 8 (got %d, %d, %d)",
              who, bits, quant_dim, D);
}

extern "C" dsa_status_t dsa_paged_quantize(const dsa_bf16_t* x, int64_t x_stride_t, int32_t T, int32_t D,
                                           int32_t quant_dim, int32_t bits, uint8_t* cache, int64_t num_rows,
                                           const int32_t* out_rows, void* workspace, size_t workspace_bytes,
                                           dsa_stream_t stream) {
  const char* who = "dsa_paged_quantize";
  dsa_status_t st = check_format(who, D, quant_dim, bits);
  if (st != DSA_OK) return st;
  if (T < 0 || x_stride_t < 0) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: T and the stride must be >= 0", who);
  if (num_rows < 0 || num_rows > 0x7fffffffll || (!out_rows && num_rows < T))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: num_rows must be in [0, 2^31), and at least T without out_rows", who);
  if (T > 0 && (!x || (num_rows > 0 && !cache))) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if ((reinterpret_cast<uintptr_t>(x) & 1) || !aligned16(cache))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: x must be 2-byte and cache 16-byte aligned", who);
  const uint64_t row = quant_row(D, quant_dim, bits).bytes;
  if (T > 0 && pquant::share(x, 2 * ((uint64_t)(T - 1) * x_stride_t + D), cache, row * num_rows))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: x and cache share memory", who);
  if ((st = check_workspace(workspace, workspace_bytes, kErrorWordBytes, who)) != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (T == 0) return ok();
  pquant::Rows p{};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.stride = x_stride_t;
  p.T = T;
  p.D = D;
  p.Q = quant_dim;
  p.cache = cache;
  p.num_rows = num_rows;
  p.out_rows = out_rows;
  p.err = reinterpret_cast<int*>(workspace);
  p.vec = aligned16(x) && (x_stride_t % 8 == 0 || T == 1);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = bits == 8 ? pquant::quantize<8>(p, s) : pquant::quantize<4>(p, s);
  return st == DSA_OK ? ok() : st;
}

extern "C" dsa_status_t dsa_paged_dequantize(const uint8_t* cache, const int32_t* block_table, const int32_t* first,
                                             const int32_t* cu_rows, int32_t N, int32_t B, int32_t D, int32_t quant_dim,
                                             int32_t bits, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                             dsa_bf16_t* out, int64_t out_stride_t, void* workspace,
                                             size_t workspace_bytes, dsa_stream_t stream) {
  const char* who = "dsa_paged_dequantize";
  dsa_status_t st = check_format(who, D, quant_dim, bits);
  if (st != DSA_OK) return st;
  if (N < 0 || B < 0 || num_pages < 0 || page_size < 1 || max_pages < 0)
    return fail(DSA_ERR_INVALID_ARGUMENT,
                "%s: need N, B, num_pages, max_pages >= 0, page_size >= 1 (got %d, %d, %d, %d, %d)", who, N, B, num_pages,
                max_pages, page_size);
  if (out_stride_t < D) return fail(DSA_ERR_INVALID_ARGUMENT, "%s: the rows of out overlap", who);
  if ((N > 0 && !out) || !cu_rows || (B > 0 && max_pages > 0 && !block_table) || (num_pages > 0 && !cache))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: null tensor pointer", who);
  if ((reinterpret_cast<uintptr_t>(out) & 1) || !aligned16(cache))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: out must be 2-byte and cache 16-byte aligned", who);
  const uint64_t row = quant_row(D, quant_dim, bits).bytes;
  if (N > 0 && pquant::share(out, 2 * ((uint64_t)(N - 1) * out_stride_t + D), cache, row * num_pages * page_size))
    return fail(DSA_ERR_INVALID_ARGUMENT, "%s: out and cache share memory", who);
  if ((st = check_workspace(workspace, workspace_bytes, kErrorWordBytes, who)) != DSA_OK) return st;
  if ((st = check_device()) != DSA_OK) return st;
  if (N == 0 || B == 0) return ok();
  pquant::Back p{};
  p.cache = cache;
  p.table = block_table;
  p.first = first;
  p.cu = cu_rows;
  p.N = N;
  p.B = B;
  p.D = D;
  p.Q = quant_dim;
  p.num_pages = num_pages;
  p.P = page_size;
  p.max_pages = max_pages;
  const unsigned q16 = quant_dim / 16, tail8 = (D - quant_dim) / 8;
  p.inv_q = ((1u << 21) + q16 - 1) / q16;
  p.inv_tail = tail8 ? ((1u << 21) + tail8 - 1) / tail8 : 0;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.stride = out_stride_t;
  p.err = reinterpret_cast<int*>(workspace);
  const uintptr_t lie = reinterpret_cast<uintptr_t>(out) | (N == 1 ? 0 : (uintptr_t)out_stride_t * 2);
  p.align = lie % 32 == 0 ? 32 : lie % 16 == 0 ? 16 : 2;
  // 64 rows a CTA while that leaves four an SM (131104 rows of 128, written and read, 24.0 us, 26.8 with 32; 12 x 30000 of 576 read
  // 65.8 and 65.0; 8191 of 576, written and read, 12.3 and 11.0)
  p.rows = N / 64 >= 4 * pquant::kSms ? 64 : 32;
  const unsigned blocks = (unsigned)(((int64_t)N + p.rows - 1) / p.rows);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (bits == 8) pquant::dequantize_kernel<8><<<blocks, pquant::kThreads, 0, s>>>(p);
  else pquant::dequantize_kernel<4><<<blocks, pquant::kThreads, 0, s>>>(p);
  st = cuda_check(cudaGetLastError(), "launching dequantize_kernel");
  return st == DSA_OK ? ok() : st;
}
