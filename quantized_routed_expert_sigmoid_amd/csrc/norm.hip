/*
 * norm.hip -- residual addition, root-mean-square norm and Q8_0 of the result.
 *
 *   t = x + r,  y = t * (1 / sqrt(mean(t^2) + eps)) * w,  Q8_0(y)
 *
 * One workgroup per row; the row stays in registers between the sum of
 * squares and the outputs, so x and r are read once.  Bound by those bytes:
 * 8191 x 6144 bf16, every output written, 85 us = 5.4 TB/s (a plain copy: 5.15);
 * one row of 6144 fp32 5.0 us.  Eight lanes share a 32-element block, whose
 * largest value needs three exchanges.
 */
#include "block_device.h"

#include <algorithm>

namespace coli {

namespace {

constexpr int kThreads = 256;

/* NV: groups of four values per thread, K <= NV * 1024. */
template <typename TX, typename TR, typename TY, int NV>
__global__ __launch_bounds__(kThreads) void add_rms_norm_kernel(coli_norm n, int64_t row0)
{
    __shared__ float part[kThreads / kWave];
    const int K = n.K, n4 = K / 4;
    const int64_t row = row0 + blockIdx.x;
    const TX* x = (const TX*)n.x + row * n.x_stride;
    const TR* r = n.residual ? (const TR*)n.residual + row * n.residual_stride : nullptr;
    /* loads are unconditional, past the row's end of its last group: one under a
     * branch would be waited for by itself */
    float4 t[NV], v[NV], w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        t[j] = load4(x + 4 * min((int)threadIdx.x + kThreads * j, n4 - 1));
    if (r) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            v[j] = load4(r + 4 * min((int)threadIdx.x + kThreads * j, n4 - 1));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        w[j] = load4(n.weight + 4 * min((int)threadIdx.x + kThreads * j, n4 - 1));
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (r) {
            t[j].x += v[j].x;
            t[j].y += v[j].y;
            t[j].z += v[j].z;
            t[j].w += v[j].w;
        }
        const float q = t[j].x * t[j].x + t[j].y * t[j].y + t[j].z * t[j].z + t[j].w * t[j].w;
        ss += threadIdx.x + kThreads * j < n4 ? q : 0.0f;
    }
    ss = wave_sum(ss);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < kThreads / kWave; ++w)
        ss += part[w];
    const float rs = 1.0f / __builtin_sqrtf(ss / (float)K + n.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + kThreads * j;
        if (i >= n4) /* whole groups of 8 lanes: K is a multiple of 32 */
            break;
        if (n.sum)
            store4((TR*)n.sum + row * K + 4 * i, t[j]);
        const float4 y =
            make_float4(t[j].x * rs * w[j].x, t[j].y * rs * w[j].y, t[j].z * rs * w[j].z, t[j].w * rs * w[j].w);
        if (n.y)
            store4((TY*)n.y + row * K + 4 * i, y);
        if (n.q) {
            float a = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
            a = fmaxf(a, shfl_xor(a, 1));
            a = fmaxf(a, shfl_xor(a, 2));
            a = fmaxf(a, shfl_xor(a, 4));
            const float d = a / 127.0f;
            const float inv = a == 0.0f ? 0.0f : 1.0f / d;
            ((uint32_t*)(n.q + row * K))[i] =
                (uint32_t)(q8_code(y.x, inv) & 0xFF) | ((uint32_t)(q8_code(y.y, inv) & 0xFF) << 8) |
                ((uint32_t)(q8_code(y.z, inv) & 0xFF) << 16) | ((uint32_t)(q8_code(y.w, inv) & 0xFF) << 24);
            if ((i & 7) == 0)
                n.d[row * (K / 32) + i / 8] = d;
        }
    }
}

template <typename TX, typename TR, typename TY>
hipError_t launch(const coli_norm& n, hipStream_t s)
{
    /* a launch's threads are counted in 32 bits */
    constexpr int kRows = 1 << 22;
    for (int64_t row0 = 0; row0 < n.rows; row0 += kRows) {
        const dim3 grid((uint32_t)std::min<int64_t>(n.rows - row0, kRows)), block(kThreads);
        if (n.K <= 1024)
            hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 1>), grid, block, 0, s, n, row0);
        else if (n.K <= 2048)
            hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 2>), grid, block, 0, s, n, row0);
        else if (n.K <= 4096)
            hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 4>), grid, block, 0, s, n, row0);
        else if (n.K <= 6144)
            hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 6>), grid, block, 0, s, n, row0);
        else
            hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 8>), grid, block, 0, s, n, row0);
    }
    return hipGetLastError();
}

template <typename TX, typename TR>
hipError_t launch_y(const coli_norm& n, hipStream_t s)
{
    return n.y_type == COLI_F32 ? launch<TX, TR, float>(n, s) : launch<TX, TR, bf16>(n, s);
}

} // namespace

hipError_t launch_add_rms_norm(const coli_norm& n, hipStream_t s)
{
    if (n.x_type == COLI_F32)
        return n.residual_type == COLI_F32 ? launch_y<float, float>(n, s) : launch_y<float, bf16>(n, s);
    return n.residual_type == COLI_F32 ? launch_y<bf16, float>(n, s) : launch_y<bf16, bf16>(n, s);
}

} // namespace coli
