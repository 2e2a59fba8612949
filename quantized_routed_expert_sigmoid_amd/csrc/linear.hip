/*
 * linear.hip -- quantised matrix product of Q8_0 activations with bias,
 * activation and residual in its epilogue.
 *
 * One wave per weight row and up to four tokens: each lane takes whole
 * 32-element blocks, their exact integer dot products times the two scales
 * are summed in fp32, first in the lane and then over the wave.
 */
#include "block_device.h"

namespace coli {

namespace {

__device__ __forceinline__ float activate(float v, int act)
{
    if (act == COLI_ACT_RELU)
        return fmaxf(v, 0.0f);
    if (act == COLI_ACT_SILU)
        return canon_silu(v);
    if (act == COLI_ACT_GELU)
        return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v;
}

template <int BITS, typename TO>
__global__ __launch_bounds__(256) void linear_rows_kernel(LinearArgs a)
{
    constexpr int T = 4;
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x * 4 + (threadIdx.x >> 6), t0 = blockIdx.y * T;
    if (n >= a.N)
        return;
    const int nb = a.K / 32, gb = a.group ? a.group / 32 : nb;
    const uint32_t* w = (const uint32_t*)a.w + (int64_t)n * nb * BITS;
    const float* ws = a.w_scale + (int64_t)n * (nb / gb);
    float acc[T] = {0.f, 0.f, 0.f, 0.f};
    for (int b = lane; b < nb; b += 64) {
        uint32_t wb[BITS];
        for (int i = 0; i < BITS; ++i)
            wb[i] = w[(int64_t)b * BITS + i];
        const float sc = ws[b / gb];
        for (int t = 0; t < T; ++t) {
            const int64_t row = min(t0 + t, a.S - 1);
            uint32_t x[8], xa[8];
            for (int i = 0; i < 8; ++i)
                x[i] = ((const uint32_t*)(a.xq + row * a.K))[b * 8 + i];
            prep_dot<BITS>(x, xa);
            const float d = a.xd[row * nb + b];
            acc[t] = __builtin_fmaf(sc * d, (float)block_dot<BITS>(wb, xa), acc[t]);
        }
    }
    for (int t = 0; t < T; ++t) {
        const float v = wave_sum(acc[t]);
        if (lane == t && t0 + t < a.S) {
            const int64_t o = (int64_t)(t0 + t) * a.N + n;
            float y = activate(v + (a.bias ? a.bias[n] : 0.0f), a.act);
            if (a.residual)
                y += to_f32(((const TO*)a.residual)[o]);
            store1((TO*)a.out + o, y);
        }
    }
}

template <int BITS>
hipError_t launch(const LinearArgs& a, hipStream_t s)
{
    const dim3 grid((a.N + 3) / 4, (a.S + 3) / 4), block(256);
    if (a.out_type == COLI_F32)
        hipLaunchKernelGGL((linear_rows_kernel<BITS, float>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((linear_rows_kernel<BITS, bf16>), grid, block, 0, s, a);
    return hipGetLastError();
}

} // namespace

size_t linear_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t qtype, int32_t group, int32_t out_type)
{
    return 256;
}

hipError_t launch_linear_q(const LinearArgs& a, hipStream_t s)
{
    return a.qtype == COLI_Q8 ? launch<8>(a, s) : a.qtype == COLI_Q4 ? launch<4>(a, s) : launch<2>(a, s);
}

} // namespace coli
