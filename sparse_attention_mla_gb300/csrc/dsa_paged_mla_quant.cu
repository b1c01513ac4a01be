// dsa_paged_mla_quant.cu -- attention of new tokens over a paged cache of quantised latents (sm_103a).
//
// For new token j of request b and head h:  z_p = scale <q, kv_p> over the positions p it sees,
// lse = ln sum e^{z_p},  out = sum e^{z_p - lse} kv_p[0:512],  kv_p = code * block * s for the first 512 channels.
//
// One CTA per token and 8 heads walks the positions in tiles of 32: the tile's rows as fp32 in shared memory, scores in
// fp32, a running maximum and sum, the output in registers.
#include <cmath>

#include "dsa_host.h"
#include "dsa_paged_quant.cuh"

namespace dsa {
namespace pmlaq {

constexpr int kDv = 512, kThreads = 256, kHeads = 8, kTile = 32;

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t *table, *seq_lens, *cu_q, *topk_idx, *topk_len;
  int N, B, H, K, num_pages, P, max_pages;
  float scale;
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

template <int DQK, int BITS>
__global__ void __launch_bounds__(kThreads) mla_quant_kernel(const Params p) {
  extern __shared__ float smem[];
  float* s_kv = smem;                     // [kTile][DQK + 1]
  float* s_q = s_kv + kTile * (DQK + 1);  // [kHeads][DQK]
  __shared__ float s_z[kHeads][kTile];
  __shared__ long long s_row[kTile];
  constexpr QuantRow lay = quant_row(DQK, kDv, BITS);
  const int n = blockIdx.x, h0 = blockIdx.y * kHeads, tid = threadIdx.x;
  int b = n, lo = n, hi = n + 1;
  if (p.cu_q) {
    const int begin = max(__ldg(p.cu_q), 0), end = min(__ldg(p.cu_q + p.B), p.N);
    if (n < begin || n >= end) return;
    int l = 0, r = p.B;
    while (r - l > 1) {
      const int m = (l + r) >> 1;
      if (__ldg(p.cu_q + m) <= n) l = m;
      else r = m;
    }
    b = l;
    lo = __ldg(p.cu_q + b);
    hi = __ldg(p.cu_q + b + 1);
  }
  const int seen = max(__ldg(p.seq_lens + b), 0) - (hi - lo) + (n - lo) + 1;
  const long long held = (long long)p.max_pages * p.P;
  const int keys = p.topk_idx ? (p.topk_len ? min(max(__ldg(p.topk_len + n), 0), p.K) : p.K)
                              : (int)min((long long)max(seen, 0), held);
  const int limit = (int)min((long long)seen, held);
  if (!p.topk_idx && keys < seen && tid == 0) record_error(p.err, DSA_ERR_DEVICE_INDEX);
  for (int x = tid; x < kHeads * DQK; x += kThreads) {
    const int h = h0 + x / DQK;
    s_q[x] = h < p.H ? __bfloat162float(p.q[((size_t)n * p.H + h) * DQK + x % DQK]) : 0.f;
  }
  float acc[kHeads][2], m[kHeads], l[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    acc[h][0] = acc[h][1] = l[h] = 0.f;
    m[h] = -INFINITY;
  }
  for (int t0 = 0; t0 < keys; t0 += kTile) {
    __syncthreads();
    if (tid < kTile) {
      const int j = t0 + tid;
      int pos = j >= keys ? -1 : p.topk_idx ? __ldg(p.topk_idx + (size_t)n * p.K + j) : j;
      long long row = -1;
      if (pos < -1 || pos >= limit) {
        record_error(p.err, DSA_ERR_DEVICE_INDEX);
        pos = -1;
      }
      if (pos >= 0) {
        const int page = __ldg(p.table + (size_t)b * p.max_pages + pos / p.P);
        if (page >= 0 && page < p.num_pages) row = (long long)page * p.P + pos % p.P;
        else record_error(p.err, DSA_ERR_DEVICE_INDEX);
      }
      s_row[tid] = row;
    }
    __syncthreads();
    for (int x = tid; x < kTile * DQK; x += kThreads) {
      const int k = x / DQK, c = x % DQK;
      float v = 0.f;
      if (s_row[k] >= 0) {
        const uint8_t* row = p.cache + (size_t)s_row[k] * lay.bytes;
        if (c >= kDv) {
          v = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row + lay.tail)[c - kDv]);
        } else if (BITS == 8) {
          v = f16x2_floats(e4m3x2_f16x2(row[c])).x;
        } else {
          uint32_t r[4];
          e2m1x8_f16x2((uint32_t)row[c / 2] >> (4 * (c & 1)), r);
          v = f16x2_floats(r[0]).x * f16x2_floats(e4m3x2_f16x2(row[lay.blocks + c / 16])).x;
        }
        if (c < kDv) v *= *reinterpret_cast<const float*>(row + lay.scale);
      }
      s_kv[k * (DQK + 1) + c] = v;
    }
    __syncthreads();
    {
      const int h = tid / kTile, k = tid % kTile;
      float z = 0.f;
      for (int c = 0; c < DQK; ++c) z += s_q[h * DQK + c] * s_kv[k * (DQK + 1) + c];
      s_z[h][k] = s_row[k] >= 0 ? z * p.scale : -INFINITY;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float top = m[h];
      for (int k = 0; k < kTile; ++k) top = fmaxf(top, s_z[h][k]);
      const float base = top == -INFINITY ? 0.f : top, f = expf(m[h] - base);
      m[h] = top;
      l[h] *= f;
      acc[h][0] *= f;
      acc[h][1] *= f;
      for (int k = 0; k < kTile; ++k) {
        if (s_row[k] < 0) continue;
        const float w = expf(s_z[h][k] - base);
        l[h] += w;
        acc[h][0] += w * s_kv[k * (DQK + 1) + tid];
        acc[h][1] += w * s_kv[k * (DQK + 1) + tid + 256];
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h0 + h >= p.H) continue;
    const float s = p.sink ? __ldg(p.sink + h0 + h) : -INFINITY, top = fmaxf(m[h], s);
    const float base = top == -INFINITY ? 0.f : top, f = expf(m[h] - base), total = l[h] * f + expf(s - base);
    const size_t at = (size_t)n * p.H + h0 + h;
    const float inv = total == 0.f ? 0.f : f / total;
    p.out[at * kDv + tid] = __float2bfloat16_rn(acc[h][0] * inv);
    p.out[at * kDv + tid + 256] = __float2bfloat16_rn(acc[h][1] * inv);
    if (tid == 0) p.lse[at] = total == 0.f ? -INFINITY : base + logf(total);
  }
}

template <int DQK, int BITS>
dsa_status_t launch(const Params& p, cudaStream_t s) {
  constexpr int bytes = (kTile * (DQK + 1) + kHeads * DQK) * 4;
  dsa_status_t st = configure_kernel_smem(reinterpret_cast<const void*>(mla_quant_kernel<DQK, BITS>), bytes,
                                          "configuring mla_quant_kernel");
  if (st != DSA_OK) return st;
  mla_quant_kernel<DQK, BITS><<<dim3(p.N, (p.H + kHeads - 1) / kHeads), kThreads, bytes, s>>>(p);
  return cuda_check(cudaGetLastError(), "launching mla_quant_kernel");
}

}  // namespace pmlaq
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_paged_mla_quant_workspace_size(void) { return kErrorWordBytes; }

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
  p.scale = softmax_scale;
  p.sink = attn_sink;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = reinterpret_cast<int*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (Dqk == 576) st = bits == 8 ? pmlaq::launch<576, 8>(p, s) : pmlaq::launch<576, 4>(p, s);
  else st = bits == 8 ? pmlaq::launch<512, 8>(p, s) : pmlaq::launch<512, 4>(p, s);
  return st == DSA_OK ? ok() : st;
}
