// dsa_paged_mla_quant.h -- the kernels behind dsa_paged_mla_quant.
#pragma once
#include "dsa_paged_groups.cuh"

namespace dsa {

// The attention's pieces over a cache of 8 bits, without the joining; few: groups of 16 rows, in place of 64.
dsa_status_t launch_paged_mla_e4m3(const pgroups::GroupParams& g, const __nv_bfloat16* q, const uint8_t* cache, int Dqk,
                                   float scale_log2e, bool few, int ctas, cudaStream_t s);

}  // namespace dsa
