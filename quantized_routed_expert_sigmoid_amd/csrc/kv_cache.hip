/*
 * kv_cache.hip -- append to and read-back from the paged int8 cache.
 *
 * A workgroup takes the keys or the values of one (block, head).  Its units are
 * the 16-byte pieces in which the codes lie in the page: for keys 16 dims of
 * one token, for values 16 tokens of one dim (value_byte); neighbouring lanes
 * have neighbouring pieces, so a page is read and written in whole lines.  Rows
 * are read and written by eight dims of a token, whole lines too; LDS lies
 * between the two orders (read-back 17.5 -> 8.8 us, 8 k tokens of 8 heads of 128
 * dims as bf16, against single values written where their piece has them).
 *
 * Append: a = the new values' largest magnitude, s' = max(s, a / 127); held
 * codes become rnd(c s / s') where the scale grew, new ones rnd(v / s').  The
 * values stay in registers between the two, so each is read once; pieces that
 * neither hold a new token nor change are not touched.  Bound by the bytes of
 * the rows and codes, for a decode step by latency.
 */
#include "block_device.h"

#include <algorithm>
#include <type_traits>

namespace coli {

namespace {

constexpr int kThreads = 256;

/* Token (of the block) and dim of byte b of piece u. */
template <int D, bool KEY>
struct Piece {
    int token0, dim0;
    __device__ __forceinline__ explicit Piece(int u)
    {
        if (KEY) { /* half-block, 16 dims, token */
            token0 = u / (2 * D) * 32 + u % 32;
            dim0 = u / 32 % (D / 16) * 16;
        } else { /* half-block, dim, bit 2 of the token */
            token0 = u / (2 * D) * 32 + (u & 1) * 4;
            dim0 = u / 2 % D;
        }
    }
    __device__ __forceinline__ int token(int b) const { return KEY ? token0 : token0 + b / 4 * 8 + b % 4; }
};

/* The code of v as q8_code gives it, plus 128. */
__device__ __forceinline__ float code_up(float v, float inv)
{
    const float r = v * inv, t = __builtin_truncf(r);
    const float e = __builtin_fabsf(r - t) >= 0.5f ? t + __builtin_copysignf(1.0f, r) : t;
    return __builtin_amdgcn_fmed3f(e, -127.0f, 127.0f) + 128.0f;
}

/* Four codes, each converted into its byte. */
__device__ __forceinline__ uint32_t encode4(const float* v, float inv)
{
    uint32_t u = 0;
    u = __builtin_amdgcn_cvt_pk_u8_f32(code_up(v[0], inv), 0, u);
    u = __builtin_amdgcn_cvt_pk_u8_f32(code_up(v[1], inv), 1, u);
    u = __builtin_amdgcn_cvt_pk_u8_f32(code_up(v[2], inv), 2, u);
    u = __builtin_amdgcn_cvt_pk_u8_f32(code_up(v[3], inv), 3, u);
    return u ^ 0x80808080u;
}

/* Values' codes in LDS: the dims of a page four bytes further apart, so that
 * the bytes of neighbouring dims lie in different banks. */
constexpr int kDimBytes = 36;

__device__ __forceinline__ int value_at(int t, int c, int D)
{
    return (t / 32 * D + c) * kDimBytes + (t >> 2 & 1) * 16 + t % 32 / 8 * 4 + t % 4;
}

/* x is the row that token 0 of the block has or would have; only tokens t0 ..
 * t1 - 1 have rows.  A thread takes eight dims of a token at a time (loads are
 * unconditional, from the nearest row: one under a branch would be waited for by
 * itself); the codes go through LDS to the threads that own their pieces. */
template <typename T, int D, bool KEY>
__device__ void append_block(const T* x, int64_t stride, int t0, int t1, int8_t* page, float* scale)
{
    constexpr int N = D / 32, KT = D + 16; /* groups of eight values of a thread; bytes of a key row in LDS */
    __shared__ float part[kThreads / kWave];
    __shared__ __align__(16) uint8_t codes[KEY ? COLI_KV_BLOCK * KT : 2 * D * kDimBytes];
    float v[N][8], a = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + kThreads * n, t = min(max(i / (D / 8), t0), t1 - 1), c = i % (D / 8) * 8;
        const float4 lo = load4(x + t * stride + c), hi = load4(x + t * stride + c + 4);
        v[n][0] = lo.x;
        v[n][1] = lo.y;
        v[n][2] = lo.z;
        v[n][3] = lo.w;
        v[n][4] = hi.x;
        v[n][5] = hi.y;
        v[n][6] = hi.z;
        v[n][7] = hi.w;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            a = fmaxf(a, fabsf(v[n][j]));
    }
    const float old = t0 > 0 ? *scale : 0.0f;
    for (int m = 32; m >= 1; m >>= 1)
        a = fmaxf(a, shfl_xor(a, m));
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = a;
    __syncthreads(); /* and the block before has left `codes` */
    a = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float now = fmaxf(old, a / 127.0f);
    const float inv = now == 0.0f ? 0.0f : 1.0f / now, f = old * inv;
    const bool grew = t0 > 0 && now != old;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + kThreads * n, t = i / (D / 8), c = i % (D / 8) * 8;
        if (t < t0 || t >= t1)
            continue;
        const uint32_t w[2] = {encode4(v[n], inv), encode4(v[n] + 4, inv)};
        if (KEY) {
            *(uint2*)(codes + t * KT + c) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                codes[value_at(t, c + j, D)] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < D / 64; ++n) {
        const int u = threadIdx.x + kThreads * n;
        const Piece<D, KEY> p(u);
        bool any = false, whole = true, held = false;
#pragma unroll
        for (int b = 0; b < (KEY ? 1 : 16); ++b) {
            const int t = p.token(b);
            const bool fresh = t >= t0 && t < t1;
            any |= fresh;
            whole &= fresh;
            held |= t < t0;
        }
        if (!any && !(grew && held))
            continue;
        uint32_t w[4];
        const uint32_t* from = (const uint32_t*)(KEY ? codes + p.token0 * KT + p.dim0
                                                     : codes + u / 2 * kDimBytes + (u & 1) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = from[j];
        uint4* at = (uint4*)page + u;
        if (!whole) {
            /* some held, or behind the last token: these keep their bytes */
            const uint4 o = *at;
            const uint32_t was[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int b = 0; b < 16; ++b) {
                const int t = p.token(b), sh = 8 * (b & 3);
                if (t >= t0 && t < t1)
                    continue;
                int32_t c = (int8_t)(was[b / 4] >> sh);
                if (t < t0 && grew)
                    c = q8_code((float)c, f);
                w[b / 4] = (w[b / 4] & ~(0xFFu << sh)) | ((uint32_t)(c & 0xFF) << sh);
            }
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (threadIdx.x == 0)
        *scale = now; /* every wave has read the old one */
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(coli_kv_cache c, coli_kv_batch b, const T* k,
                                                             const T* v, int64_t k_stride, int64_t v_stride)
{
    const int h = blockIdx.y >> 1, s = blockIdx.z;
    const bool key = !(blockIdx.y & 1);
    const SeqBounds q = seq_bounds(b, s);
    const int from = max(q.first, 0);
    if (q.kv_len <= from)
        return;
    const int blk1 = (q.kv_len - 1) / COLI_KV_BLOCK;
    for (int blk = from / COLI_KV_BLOCK + blockIdx.x; blk <= blk1; blk += gridDim.x) {
        const int page = page_of(b, c.n_pages, s, blk);
        if (page < 0)
            continue;
        const int base = blk * COLI_KV_BLOCK;
        const int t0 = max(from - base, 0), t1 = min(q.kv_len - base, COLI_KV_BLOCK);
        const int64_t row0 = (int64_t)q.row0 + (base - q.first); /* the row that token 0 would have */
        const int64_t at = (int64_t)page * c.n_heads + h;
        if (key)
            append_block<T, D, true>(k + row0 * k_stride + (int64_t)h * D, k_stride, t0, t1,
                                     c.k + at * (COLI_KV_BLOCK * D), c.k_scale + at);
        else
            append_block<T, D, false>(v + row0 * v_stride + (int64_t)h * D, v_stride, t0, t1,
                                      c.v + at * (COLI_KV_BLOCK * D), c.v_scale + at);
    }
}

/* The rows' values of one block and head; a missing page (null) gives zeros.
 * The page goes through LDS, where the codes of a token's eight dims are picked
 * up by the lane that writes them: a row is written in whole lines. */
template <typename T, int D, bool KEY>
__device__ __forceinline__ void read_block(const int8_t* page, float scale, int t0, int t1, T* x, int64_t stride)
{
    constexpr int KT = D + 16;
    __shared__ __align__(16) uint8_t codes[KEY ? COLI_KV_BLOCK * KT : 2 * D * kDimBytes];
    __syncthreads(); /* the block before is written */
    if (page) {
#pragma unroll
        for (int n = 0; n < D / 64; ++n) {
            const int u = threadIdx.x + kThreads * n;
            const Piece<D, KEY> p(u);
            const uint4 o = ((const uint4*)page)[u];
            if (KEY) {
                *(uint4*)(codes + p.token0 * KT + p.dim0) = o;
            } else {
                uint32_t* w = (uint32_t*)(codes + u / 2 * kDimBytes + (u & 1) * 16);
                w[0] = o.x;
                w[1] = o.y;
                w[2] = o.z;
                w[3] = o.w;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (t1 - t0) * (D / 8); i += kThreads) {
        const int t = t0 + i / (D / 8), c = i % (D / 8) * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)(int8_t)codes[KEY ? t * KT + c + j : value_at(t, c + j, D)] * scale;
        if (!page) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = 0.0f;
        }
        T* o = x + t * stride + c;
        store4(o, make_float4(v[0], v[1], v[2], v[3]));
        store4(o + 4, make_float4(v[4], v[5], v[6], v[7]));
    }
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(coli_kv_cache c, coli_kv_batch b, T* k, T* v)
{
    const int h = blockIdx.y >> 1, s = blockIdx.z;
    const bool key = !(blockIdx.y & 1);
    if (!(key ? k : v))
        return;
    const SeqBounds q = seq_bounds(b, s);
    const int64_t stride = (int64_t)c.n_heads * D;
    /* rows before the first token (the rows outnumber the tokens) are in blocks
     * below 0, which have no page */
    const int blk0 = q.first >> 6, blk1 = (q.kv_len - 1) >> 6;
    for (int64_t blk = (int64_t)blk0 + blockIdx.x; q.q_len && blk <= blk1; blk += gridDim.x) {
        const int64_t base = blk * COLI_KV_BLOCK;
        const int page = blk < 0 ? -1 : page_of(b, c.n_pages, s, (int)blk);
        const int t0 = (int)max((int64_t)q.first - base, (int64_t)0);
        const int t1 = (int)min((int64_t)q.kv_len - base, (int64_t)COLI_KV_BLOCK);
        const int64_t row0 = (int64_t)q.row0 + (base - q.first), at = (int64_t)max(page, 0) * c.n_heads + h;
        if (key)
            read_block<T, D, true>(page < 0 ? nullptr : c.k + at * (COLI_KV_BLOCK * D), page < 0 ? 0.0f : c.k_scale[at],
                                   t0, t1, k + row0 * stride + (int64_t)h * D, stride);
        else
            read_block<T, D, false>(page < 0 ? nullptr : c.v + at * (COLI_KV_BLOCK * D), page < 0 ? 0.0f : c.v_scale[at],
                                    t0, t1, v + row0 * stride + (int64_t)h * D, stride);
    }
}

/* Workgroups of a sequence: a block each of the longest expected run of rows,
 * and one where the run straddles; longer runs take several turns.  An odd number:
 * workgroups are dealt to the CUs in turn, and a power of two would give the first
 * blocks of all short sequences to a few of them (append, 200 sequences of 40 rows
 * with 8 heads: 249 us with 16, 34 with 17). */
dim3 grid_of(const coli_kv_cache& c, const coli_kv_batch& b)
{
    const int rows = std::max(1, std::min(b.max_q, b.n_tokens));
    const int blocks = rows == 1 ? 1 : (rows - 2) / COLI_KV_BLOCK + 2;
    return dim3((uint32_t)std::min(blocks | 1, 1025), (uint32_t)c.n_heads * 2, (uint32_t)b.n_seq);
}

template <typename F>
void by_dim(int32_t head_dim, F f)
{
    switch (head_dim) {
    case 64: f(std::integral_constant<int, 64>()); break;
    case 128: f(std::integral_constant<int, 128>()); break;
    case 192: f(std::integral_constant<int, 192>()); break;
    default: f(std::integral_constant<int, 256>()); break;
    }
}

} // namespace

hipError_t launch_kv_append(const coli_kv_cache& c, const coli_kv_batch& b, const void* k, const void* v,
                            int32_t type, int64_t k_stride, int64_t v_stride, hipStream_t s)
{
    by_dim(c.head_dim, [&](auto d) {
        if (type == COLI_F32)
            hipLaunchKernelGGL((kv_append_kernel<float, d.value>), grid_of(c, b), dim3(kThreads), 0, s, c, b,
                               (const float*)k, (const float*)v, k_stride, v_stride);
        else
            hipLaunchKernelGGL((kv_append_kernel<bf16, d.value>), grid_of(c, b), dim3(kThreads), 0, s, c, b,
                               (const bf16*)k, (const bf16*)v, k_stride, v_stride);
    });
    return hipGetLastError();
}

hipError_t launch_kv_read(const coli_kv_cache& c, const coli_kv_batch& b, void* k, void* v, int32_t type,
                          hipStream_t s)
{
    by_dim(c.head_dim, [&](auto d) {
        if (type == COLI_F32)
            hipLaunchKernelGGL((kv_read_kernel<float, d.value>), grid_of(c, b), dim3(kThreads), 0, s, c, b, (float*)k,
                               (float*)v);
        else
            hipLaunchKernelGGL((kv_read_kernel<bf16, d.value>), grid_of(c, b), dim3(kThreads), 0, s, c, b, (bf16*)k,
                               (bf16*)v);
    });
    return hipGetLastError();
}

} // namespace coli
