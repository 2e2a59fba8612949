/*
 * embed.hip -- embedding lookup in a quantised table:
 *
 *   out[i][c] = (code[id][c] * scale[id][c / group]) * scale
 *
 * A thread takes eight consecutive dims, which lie under one scale: 2, 4 or 8
 * bytes of codes in, 16 or 32 bytes out.  Bound by the output's bytes: 8191 x 6144 bf16
 * from int8 with groups of 128 24.5 us (6.2 TB/s, the reads partly from the last-level cache);
 * one row of 6144 2 us.
 */
#include "block_device.h"
#include "step.h"

namespace coli {

namespace {

constexpr int kThreads = 256;
constexpr int kDims = 8;

template <int BITS>
__device__ __forceinline__ void codes8(const uint8_t* p, float* v)
{
    if constexpr (BITS == 8) {
        const uint2 w = *(const uint2*)p;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    } else if constexpr (BITS == 4) {
        const uint32_t w = *(const uint32_t*)p; /* the first of a byte's two in its upper half */
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)((int32_t)(w << (24 - 8 * (j / 2) + 4 * (j & 1))) >> 28);
    } else {
        const uint32_t w = *(const uint16_t*)p; /* the first of a byte's four in bits 7..6 */
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)((int32_t)(w << (24 - 8 * (j / 4) + 2 * (j & 3))) >> 30);
    }
}

template <int BITS, typename ID, typename TO>
__global__ __launch_bounds__(kThreads) void embed_kernel(coli_qbank W, const ID* ids, int parts, float scale, TO* out)
{
    const int i = blockIdx.x / parts, c = (blockIdx.x % parts * kThreads + threadIdx.x) * kDims;
    if (c >= W.K)
        return;
    const int64_t id = ids[i];
    float v[kDims] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (id >= 0 && id < W.rows) {
        codes8<BITS>((const uint8_t*)W.data + (id * W.K + c) * BITS / 8, v);
        const float s = W.group ? W.row_scale[id * (W.K / W.group) + c / W.group] : W.row_scale[id];
#pragma unroll
        for (int j = 0; j < kDims; ++j)
            v[j] = v[j] * s * scale;
    }
    TO* o = out + (int64_t)i * W.K + c;
    store4(o, make_float4(v[0], v[1], v[2], v[3]));
    store4(o + 4, make_float4(v[4], v[5], v[6], v[7]));
}

template <int BITS, typename ID>
void launch(const coli_qbank& W, const ID* ids, int32_t n, float scale, void* out, int32_t out_type, hipStream_t s)
{
    const int parts = (W.K + kThreads * kDims - 1) / (kThreads * kDims);
    const dim3 grid((uint32_t)(n * parts)); /* at most 2^16 rows of 2^4 parts */
    if (out_type == COLI_F32)
        hipLaunchKernelGGL((embed_kernel<BITS, ID, float>), grid, dim3(kThreads), 0, s, W, ids, parts, scale, (float*)out);
    else
        hipLaunchKernelGGL((embed_kernel<BITS, ID, bf16>), grid, dim3(kThreads), 0, s, W, ids, parts, scale, (bf16*)out);
}

template <int BITS>
void launch_ids(const coli_qbank& W, const void* ids, int32_t id_type, int32_t n, float scale, void* out,
                int32_t out_type, hipStream_t s)
{
    if (id_type == COLI_I32)
        launch<BITS>(W, (const int32_t*)ids, n, scale, out, out_type, s);
    else
        launch<BITS>(W, (const int64_t*)ids, n, scale, out, out_type, s);
}

} // namespace

hipError_t launch_embed_q(const coli_qbank& W, const void* ids, int32_t id_type, int32_t n, float scale, void* out,
                          int32_t out_type, hipStream_t s)
{
    switch (W.qtype) {
    case COLI_Q8: launch_ids<8>(W, ids, id_type, n, scale, out, out_type, s); break;
    case COLI_Q4: launch_ids<4>(W, ids, id_type, n, scale, out, out_type, s); break;
    default: launch_ids<2>(W, ids, id_type, n, scale, out, out_type, s); break;
    }
    return hipGetLastError();
}

} // namespace coli
