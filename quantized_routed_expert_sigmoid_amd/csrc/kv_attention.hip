/*
 * kv_attention.hip -- softmax attention over the paged int8 cache.
 *
 * One wave per (query row, head): lane j scores token j of the current page,
 * the running maximum and sum carry the softmax across pages, and each lane
 * accumulates its dims of the output.
 */
#include "block_device.h"

namespace coli {

namespace {

template <typename T>
__global__ __launch_bounds__(kWave) void kv_attention_simple(coli_kv_cache c, coli_kv_batch b, coli_kv_attn a)
{
    __shared__ float qs[256], ps[COLI_KV_BLOCK];
    const int lane = threadIdx.x, h = blockIdx.y, s = blockIdx.z, D = c.head_dim;
    const int hk = h / (a.n_heads / c.n_heads);
    const SeqBounds q = seq_bounds(b, s);
    for (int i = blockIdx.x; i < q.q_len; i += gridDim.x) {
        const int64_t row = q.row0 + i;
        const T* qr = (const T*)a.q + row * a.q_stride + (int64_t)h * D;
        __syncthreads();
        for (int d = lane; d < D; d += kWave)
            qs[d] = to_f32(qr[d]);
        __syncthreads();
        const int end = a.causal ? q.first + i + 1 : q.kv_len;
        const int begin = a.window > 0 ? max(end - a.window, 0) : 0;
        float m = -__builtin_inff(), l = 0.0f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int blk = begin / COLI_KV_BLOCK; blk * COLI_KV_BLOCK < end; ++blk) {
            const int page = page_of(b, c.n_pages, s, blk);
            if (page < 0)
                continue;
            const int64_t at = (int64_t)page * c.n_heads + hk;
            const int8_t* pk = c.k + at * COLI_KV_BLOCK * D;
            const int8_t* pv = c.v + at * COLI_KV_BLOCK * D;
            float x = 0.0f;
            for (int d = 0; d < D; ++d)
                x += qs[d] * (float)pk[key_byte(lane, d, D)];
            const int j = blk * COLI_KV_BLOCK + lane;
            const bool seen = j >= begin && j < end;
            x = seen ? x * (c.k_scale[at] * a.scale) : -__builtin_inff();
            float mx = x;
            bool nan = x != x;
            for (int w = 32; w >= 1; w >>= 1)
                mx = fmaxf(mx, shfl_xor(mx, w));
            const float mn = fmaxf(m, mx);
            const float base = mn == -__builtin_inff() ? 0.0f : mn;
            const float f = expf(m - base), p = (seen || nan) ? expf(x - base) : 0.0f;
            l = l * f + wave_sum(p);
            __syncthreads();
            ps[lane] = p * c.v_scale[at];
            __syncthreads();
            for (int d = lane, e = 0; d < D; d += kWave, ++e) {
                float o = 0.0f;
                for (int t = 0; t < COLI_KV_BLOCK; ++t)
                    if (blk * COLI_KV_BLOCK + t >= begin && blk * COLI_KV_BLOCK + t < end)
                        o += ps[t] * (float)pv[value_byte(t, d, D)];
                acc[e] = acc[e] * f + o;
            }
            m = mn;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        for (int d = lane, e = 0; d < D; d += kWave, ++e)
            store1((T*)a.out + row * a.out_stride + (int64_t)h * D + d, acc[e] * inv);
        if (a.lse && lane == 0)
            a.lse[row * a.n_heads + h] = l == 0.0f ? -__builtin_inff() : m + logf(l);
    }
}

} // namespace

size_t kv_attention_workspace_bytes(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a)
{
    return 256;
}

hipError_t launch_kv_attention(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a, void* ws,
                               hipStream_t s)
{
    const dim3 grid((uint32_t)max(1, min(b.max_q, 65536)), (uint32_t)a.n_heads, (uint32_t)b.n_seq);
    if (a.type == COLI_F32)
        hipLaunchKernelGGL(kv_attention_simple<float>, grid, dim3(kWave), 0, s, c, b, a);
    else
        hipLaunchKernelGGL(kv_attention_simple<bf16>, grid, dim3(kWave), 0, s, c, b, a);
    return hipGetLastError();
}

} // namespace coli
