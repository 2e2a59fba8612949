/*
 * step.h -- internal launch interface of the operators of a serving step: the
 * embedding lookup (embed.hip), the paged cache's sequences (kv_pages.hip), the
 * linear product with one activation scale per token (linear_i8.hip) and what is done
 * to logits (logits.hip).
 * step_api.hip validates; the launchers assume validated arguments.
 */
#ifndef COLI_STEP_H
#define COLI_STEP_H

#include "../../include/colibri_step.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace coli {

hipError_t launch_embed_q(const coli_qbank& W, const void* ids, int32_t id_type, int32_t n, float scale, void* out,
                          int32_t out_type, hipStream_t s);

size_t kv_pages_workspace_bytes(int32_t n_pages, int32_t n_seq);
hipError_t launch_kv_extend(const coli_kv_pages& p, const int32_t* add, int32_t* granted, int32_t* src, int32_t* dst,
                            void* ws, hipStream_t s);
hipError_t launch_kv_trim(const coli_kv_pages& p, const int32_t* new_len, hipStream_t s);
hipError_t launch_kv_fork(const coli_kv_pages& p, const int32_t* parent, const int32_t* child, int32_t n,
                          hipStream_t s);
hipError_t launch_kv_compact(const coli_kv_pages& p, int32_t* src, int32_t* dst, int32_t* n_live, void* ws,
                             hipStream_t s);
hipError_t launch_kv_copy(const coli_kv_cache& from, const coli_kv_cache& to, const int32_t* src, const int32_t* dst,
                          int32_t n, hipStream_t s);

hipError_t launch_quantize_i8(const void* x, int32_t type, int64_t stride, int32_t rows, int32_t K, int8_t* q, float* d,
                              hipStream_t s);

struct LinearI8Args {
    const void* w;
    const float* w_scale;
    const int8_t* xq;
    const float* xd;
    const float* bias;
    const void* residual;
    void* out;
    void* ws;
    int32_t S, N, K, qtype, act, out_type;
};

/* What one call of S tokens needs; the most that one of 1 .. S tokens does. */
size_t linear_i8_workspace_need(int32_t S, int32_t N, int32_t K, int32_t bits);
size_t linear_i8_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t bits);
hipError_t launch_linear_i8(const LinearI8Args& a, hipStream_t s);

size_t logits_workspace_bytes(int32_t rows, int32_t vocab);
hipError_t launch_adjust_logits(const coli_logits& a, void* ws, hipStream_t s);

} // namespace coli

#endif
