/*
 * norm.hip -- residual addition, root-mean-square norm and Q8_0 of the result.
 *
 *   t = x + r,  y = t * (1 / sqrt(mean(t^2) + eps)) * w,  Q8_0(y)
 *
 * One workgroup per row; the row stays in registers between the sum of
 * squares and the outputs, so x and r are read once.  Bound by those bytes.
 */
#include "block_device.h"

namespace coli {

namespace {

constexpr int kThreads = 256;

/* NV: groups of four values per thread, K <= NV * 1024. */
template <typename TX, typename TR, typename TY, int NV>
__global__ __launch_bounds__(kThreads) void add_rms_norm_kernel(coli_norm n)
{
    __shared__ float part[kThreads / kWave];
    const int K = n.K, n4 = K / 4;
    for (int64_t row = blockIdx.x; row < n.rows; row += gridDim.x) {
        const TX* x = (const TX*)n.x + row * n.x_stride;
        const TR* r = n.residual ? (const TR*)n.residual + row * n.residual_stride : nullptr;
        float4 t[NV];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + kThreads * j;
            t[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n4) {
                t[j] = load4(x + 4 * i);
                if (r) {
                    const float4 v = load4(r + 4 * i);
                    t[j].x += v.x;
                    t[j].y += v.y;
                    t[j].z += v.z;
                    t[j].w += v.w;
                }
            }
            ss += t[j].x * t[j].x + t[j].y * t[j].y + t[j].z * t[j].z + t[j].w * t[j].w;
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
            const float4 w = load4(n.weight + 4 * i);
            const float4 y = make_float4(t[j].x * rs * w.x, t[j].y * rs * w.y, t[j].z * rs * w.z, t[j].w * rs * w.w);
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
        __syncthreads(); /* `part` is free for the next row */
    }
}

template <typename TX, typename TR, typename TY>
hipError_t launch(const coli_norm& n, hipStream_t s)
{
    const dim3 grid((uint32_t)min(n.rows, 1 << 20)), block(kThreads);
    if (n.K <= 2048)
        hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 2>), grid, block, 0, s, n);
    else
        hipLaunchKernelGGL((add_rms_norm_kernel<TX, TR, TY, 8>), grid, block, 0, s, n);
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
