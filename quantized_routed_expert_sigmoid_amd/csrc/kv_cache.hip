/*
 * kv_cache.hip -- append to and read-back from the paged int8 cache.
 *
 * Append: one workgroup per (sequence, touched block, head) takes the block's
 * new scale from the old one and the new values' largest magnitude, then
 * requantises what the block held (only where the scale grew) and writes the
 * new codes.  It reads each new value once from memory (the second pass over
 * them hits the caches) and touches 64 tokens of one head at most.
 */
#include "block_device.h"

namespace coli {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ void append_one(const T* x, int64_t stride, int D, int H, int h, int64_t row0, int t0, int t1,
                           bool held, int8_t* page, float* scale, bool key, float* part)
{
    /* new tokens t0 .. t1 - 1 of the block from packed row row0 on */
    const int n4 = D / 4, n = (t1 - t0) * n4;
    float a = 0.0f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const float4 v = load4(x + (row0 + i / n4) * stride + (int64_t)h * D + 4 * (i % n4));
        a = fmaxf(a, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    }
    for (int m = 32; m >= 1; m >>= 1)
        a = fmaxf(a, shfl_xor(a, m));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = a;
    __syncthreads();
    a = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float old = held ? *scale : 0.0f;
    const float now = fmaxf(old, a / 127.0f);
    const float inv = now == 0.0f ? 0.0f : 1.0f / now;
    if (held && now != old) {
        const float f = old * inv;
        for (int i = threadIdx.x; i < t0 * D; i += kThreads) {
            const int t = i / D, c = i % D;
            int8_t* p = page + (key ? key_byte(t, c, D) : value_byte(t, c, D));
            *p = (int8_t)q8_code((float)*p, f);
        }
    }
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int t = t0 + i / n4, c = 4 * (i % n4);
        const float4 v = load4(x + (row0 + i / n4) * stride + (int64_t)h * D + c);
        const float e[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 4; ++j)
            page[key ? key_byte(t, c + j, D) : value_byte(t, c + j, D)] = (int8_t)q8_code(e[j], inv);
    }
    __syncthreads(); /* every thread has read the old scale */
    if (threadIdx.x == 0)
        *scale = now;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(coli_kv_cache c, coli_kv_batch b, const T* k,
                                                             const T* v, int64_t k_stride, int64_t v_stride)
{
    __shared__ float part[kThreads / kWave];
    const int h = blockIdx.y, s = blockIdx.z, D = c.head_dim;
    const SeqBounds q = seq_bounds(b, s);
    const int from = max(q.first, 0);
    if (q.kv_len <= from)
        return;
    const int blk0 = from / COLI_KV_BLOCK, blk1 = (q.kv_len - 1) / COLI_KV_BLOCK;
    for (int blk = blk0 + blockIdx.x; blk <= blk1; blk += gridDim.x) {
        const int page = page_of(b, c.n_pages, s, blk);
        if (page < 0)
            continue;
        const int base = blk * COLI_KV_BLOCK;
        const int t0 = max(from - base, 0), t1 = min(q.kv_len - base, COLI_KV_BLOCK);
        const int64_t row0 = (int64_t)q.row0 + (base + t0 - q.first);
        const int64_t at = (int64_t)page * c.n_heads + h, bytes = (int64_t)COLI_KV_BLOCK * D;
        append_one(k, k_stride, D, c.n_heads, h, row0, t0, t1, t0 > 0, c.k + at * bytes, c.k_scale + at, true,
                   part);
        append_one(v, v_stride, D, c.n_heads, h, row0, t0, t1, t0 > 0, c.v + at * bytes, c.v_scale + at, false,
                   part);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(coli_kv_cache c, coli_kv_batch b, T* k, T* v)
{
    const int s = blockIdx.z, D = c.head_dim, H = c.n_heads, n4 = H * D / 4;
    const SeqBounds q = seq_bounds(b, s);
    for (int i = blockIdx.x; i < q.q_len; i += gridDim.x) {
        const int tok = q.first + i;
        const int page = tok < 0 ? -1 : page_of(b, c.n_pages, s, tok / COLI_KV_BLOCK);
        const int t = tok & (COLI_KV_BLOCK - 1);
        const int64_t o = (int64_t)(q.row0 + i) * H * D;
        for (int e = threadIdx.x; e < n4; e += kThreads) {
            const int h = 4 * e / D, d = 4 * e % D;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (page >= 0) {
                const int64_t at = (int64_t)page * H + h;
                const float sk = c.k_scale[at], sv = c.v_scale[at];
                const int8_t* pk = c.k + at * COLI_KV_BLOCK * D;
                const int8_t* pv = c.v + at * COLI_KV_BLOCK * D;
                kk = make_float4(sk * pk[key_byte(t, d, D)], sk * pk[key_byte(t, d + 1, D)],
                                 sk * pk[key_byte(t, d + 2, D)], sk * pk[key_byte(t, d + 3, D)]);
                vv = make_float4(sv * pv[value_byte(t, d, D)], sv * pv[value_byte(t, d + 1, D)],
                                 sv * pv[value_byte(t, d + 2, D)], sv * pv[value_byte(t, d + 3, D)]);
            }
            if (k)
                store4(k + o + 4 * e, kk);
            if (v)
                store4(v + o + 4 * e, vv);
        }
    }
}

} // namespace

hipError_t launch_kv_append(const coli_kv_cache& c, const coli_kv_batch& b, const void* k, const void* v,
                            int32_t type, int64_t k_stride, int64_t v_stride, hipStream_t s)
{
    const dim3 grid((uint32_t)min(b.max_q / COLI_KV_BLOCK + 2, 1024), (uint32_t)c.n_heads, (uint32_t)b.n_seq);
    if (type == COLI_F32)
        hipLaunchKernelGGL(kv_append_kernel<float>, grid, dim3(kThreads), 0, s, c, b, (const float*)k,
                           (const float*)v, k_stride, v_stride);
    else
        hipLaunchKernelGGL(kv_append_kernel<bf16>, grid, dim3(kThreads), 0, s, c, b, (const bf16*)k,
                           (const bf16*)v, k_stride, v_stride);
    return hipGetLastError();
}

hipError_t launch_kv_read(const coli_kv_cache& c, const coli_kv_batch& b, void* k, void* v, int32_t type,
                          hipStream_t s)
{
    const dim3 grid((uint32_t)max(1, min(b.max_q, 4096)), 1, (uint32_t)b.n_seq);
    if (type == COLI_F32)
        hipLaunchKernelGGL(kv_read_kernel<float>, grid, dim3(kThreads), 0, s, c, b, (float*)k, (float*)v);
    else
        hipLaunchKernelGGL(kv_read_kernel<bf16>, grid, dim3(kThreads), 0, s, c, b, (bf16*)k, (bf16*)v);
    return hipGetLastError();
}

} // namespace coli
