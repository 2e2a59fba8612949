/*
 * block.h -- internal launch interface of the operators around the layer:
 * residual addition with root-mean-square norm (norm.hip), the quantised
 * matrix product with its epilogue (linear.hip), the paged int8 cache's append
 * and read-back (kv_cache.hip) and the attention over it (kv_attention.hip).
 * block_api.hip validates; the launchers assume validated arguments.
 */
#ifndef COLI_BLOCK_H
#define COLI_BLOCK_H

#include "../../include/colibri_block.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace coli {

hipError_t launch_add_rms_norm(const coli_norm& n, hipStream_t s);

struct LinearArgs {
    const void* w;
    const float* w_scale;
    const int8_t* xq;
    const float* xd;
    const float* bias;
    const void* residual;
    void* out;
    void* ws;
    int32_t S, N, K, qtype, group, act, out_type;
};

/* What one call of S tokens needs; the most that one of 1 .. S tokens does. */
size_t linear_workspace_need(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type);
size_t linear_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type);
hipError_t launch_linear_q(const LinearArgs& a, hipStream_t s);

hipError_t launch_kv_append(const coli_kv_cache& c, const coli_kv_batch& b, const void* k, const void* v,
                            int32_t type, int64_t k_stride, int64_t v_stride, hipStream_t s);
hipError_t launch_kv_read(const coli_kv_cache& c, const coli_kv_batch& b, void* k, void* v, int32_t type,
                          hipStream_t s);

/* What one call of these sizes needs; the most that one of these or smaller sizes does. */
size_t kv_attention_workspace_need(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a);
size_t kv_attention_workspace_bytes(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a);
hipError_t launch_kv_attention(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a, void* ws,
                               hipStream_t s);

} // namespace coli

#endif
