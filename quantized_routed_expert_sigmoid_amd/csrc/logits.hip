/*
 * logits.hip -- penalties for repeated tokens, biases and grammar masks on logits,
 * the best token and the log of the sum (include/colibri_step.h gives the order of
 * the steps).
 *
 * A workgroup takes a chunk of one row's vocabulary.  It counts the row's tokens that
 * fall into the chunk in LDS (whole numbers: no order matters), adds up their
 * biases there, and then takes the chunk's logits through all steps in one pass,
 * which also yields the chunk's largest value and its sum of exponentials; a second
 * launch joins the chunks of a row.  Every chunk of a row reads all of the row's
 * tokens, from the last-level cache.
 */
#include "block_device.h"
#include "step.h"

#include <algorithm>

namespace coli {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 4096;                      /* tokens of a workgroup */
constexpr int kGroups = kChunk / (4 * kThreads); /* groups of four of a thread */
constexpr uint32_t kSeen = 0x80000000u;          /* among the tokens; below it the count of generated ones */

/* What a chunk has to say about its row: the key is the largest value in the order
 * of unsigned numbers, then the lowest token (key_of). */
struct Part {
    unsigned long long key;
    float sum; /* of exp(v - largest) */
    uint32_t pad;
};

/* Larger values have larger keys, NaN the largest, equal values larger ones for
 * lower tokens. */
__device__ __forceinline__ unsigned long long key_of(float v, int token)
{
    const uint32_t u = __float_as_uint(v + 0.0f); /* both zeros are one */
    const uint32_t k = v != v ? 0xFFFFFFFFu : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return (unsigned long long)k << 32 | (0xFFFFFFFFu - (uint32_t)token);
}

__device__ __forceinline__ float value_of(unsigned long long key)
{
    const uint32_t k = (uint32_t)(key >> 32);
    return k == 0xFFFFFFFFu ? __builtin_nanf("") : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

/* exp(v - top); 1 for the largest itself, whatever it is. */
__device__ __forceinline__ float exp_below(float v, float top)
{
    return v == top ? 1.0f : __builtin_amdgcn_exp2f((v - top) * 1.44269504088896340736f);
}

__device__ __forceinline__ unsigned long long wave_max(unsigned long long v)
{
    for (int m = 32; m >= 1; m >>= 1) {
        const unsigned long long x = __shfl_xor(v, m, 64);
        v = x > v ? x : v;
    }
    return v;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void adjust_kernel(coli_logits a, Part* part)
{
    extern __shared__ __align__(16) uint32_t counts[]; /* [kChunk], then sums and turns of the biases, each where there are any */
    float* const sums = (float*)(counts + (a.penalties ? kChunk : 0));
    int* const turn = (int*)(sums + kChunk);
    __shared__ unsigned long long keys[kWaves];
    __shared__ float exps[kWaves];
    const int r = blockIdx.y, c0 = blockIdx.x * kChunk, V = a.vocab;
    const T* x = (const T*)a.logits + (int64_t)r * a.logits_stride;

    /* the logits travel while the tokens are counted */
    float v[kGroups][4];
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const int t = c0 + 4 * (threadIdx.x + kThreads * j);
        if (t + 4 <= V) {
            const float4 f = load4_any(x + t);
            v[j][0] = f.x;
            v[j][1] = f.y;
            v[j][2] = f.z;
            v[j][3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[j][i] = t + i < V ? to_f32(x[t + i]) : -__builtin_inff();
        }
    }

    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    int h0 = 0, h1 = 0, made = 0;
    if (a.penalties) {
        rep = a.penalties[3 * r];
        freq = a.penalties[3 * r + 1];
        pres = a.penalties[3 * r + 2];
        h0 = max(a.spans[3 * r], 0);
        made = a.spans[3 * r + 1];
        h1 = min(a.spans[3 * r + 2], a.n_tokens);
    }
    /* neutral penalties change nothing, whatever the counts */
    const bool counted = h1 > h0 && !(rep == 1.0f && freq == 0.0f && pres == 0.0f);
    int b0 = 0, b1 = 0;
    if (a.cu_bias) {
        b0 = max(a.cu_bias[r], 0);
        b1 = min(a.cu_bias[r + 1], a.n_bias);
    }
    const bool biased = b1 > b0;
    if (counted)
        for (int i = threadIdx.x; i < kChunk; i += kThreads)
            counts[i] = 0;
    if (biased)
        for (int i = threadIdx.x; i < kChunk; i += kThreads) {
            sums[i] = 0.0f;
            turn[i] = 0x7FFFFFFF;
        }
    if (counted || biased)
        __syncthreads();
    if (counted) {
        auto count = [&](int token, int i) {
            const uint32_t at = (uint32_t)(token - c0);
            if (at < (uint32_t)kChunk) {
                if (i >= made)
                    atomicAdd(counts + at, 1u);
                else
                    atomicOr(counts + at, kSeen);
            }
        };
        for (int64_t i = h0 + 4 * (int64_t)threadIdx.x; i < h1; i += 4 * kThreads) {
            if (i + 4 <= h1) {
                int4 q;
                __builtin_memcpy(&q, a.tokens + i, 16);
                count(q.x, (int)i);
                count(q.y, (int)i + 1);
                count(q.z, (int)i + 2);
                count(q.w, (int)i + 3);
            } else {
                for (int64_t j = i; j < h1; ++j)
                    count(a.tokens[j], (int)j);
            }
        }
    }
    if (biased) {
        /* a token's entries are added in the list's order: of those that wait, the
         * first takes its turn */
        for (int base = b0; base < b1; base += kThreads) {
            const int i = base + threadIdx.x;
            const uint32_t at = i < b1 ? (uint32_t)(a.bias_ids[i] - c0) : 0xFFFFFFFFu;
            bool waits = at < (uint32_t)min(kChunk, V - c0);
            const float b = waits ? a.bias[i] : 0.0f;
            while (__syncthreads_or(waits)) {
                if (waits)
                    atomicMin(turn + at, i);
                __syncthreads();
                if (waits && turn[at] == i) {
                    sums[at] += b;
                    turn[at] = 0x7FFFFFFF;
                    waits = false;
                }
            }
        }
    }
    if (counted || biased)
        __syncthreads();

    const int m = a.mask ? a.mask_of[r] : -1;
    const uint32_t* mask = m >= 0 && m < a.n_masks ? a.mask + m * a.mask_stride : nullptr;
    unsigned long long key = 0;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const int at = 4 * (threadIdx.x + kThreads * j), t = c0 + at;
        if (t >= V)
            break;
        if (counted) {
            const uint4 q = *(const uint4*)(counts + at);
            const uint32_t c[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c[i])
                    v[j][i] = v[j][i] > 0.0f ? v[j][i] / rep : v[j][i] * rep;
                if (c[i] & ~kSeen)
                    v[j][i] -= freq * (float)(c[i] & ~kSeen) + pres;
            }
        }
        if (biased) {
            const float4 q = *(const float4*)(sums + at);
            v[j][0] += q.x;
            v[j][1] += q.y;
            v[j][2] += q.z;
            v[j][3] += q.w;
        }
        if (mask) {
            const uint32_t bits = mask[t / 32] >> (t % 32);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[j][i] = bits >> i & 1 ? v[j][i] : -__builtin_inff();
        }
        if (a.out) {
            T* o = (T*)a.out + (int64_t)r * a.out_stride + t;
            if (t + 4 <= V) {
                store4_any(o, make_float4(v[j][0], v[j][1], v[j][2], v[j][3]));
            } else {
                for (int i = 0; t + i < V; ++i)
                    store1(o + i, v[j][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned long long k = t + i < V ? key_of(v[j][i], t + i) : 0;
            key = k > key ? k : key;
        }
    }
    if (!part)
        return;
    key = wave_max(key);
    if ((threadIdx.x & 63) == 0)
        keys[threadIdx.x >> 6] = key;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        key = keys[i] > key ? keys[i] : key;
    const float top = value_of(key);
    float sum = 0.0f;
    if (top != -__builtin_inff()) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 4 * ((int)threadIdx.x + kThreads * j) + i < V)
                    sum += exp_below(v[j][i], top);
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0)
        exps[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0f;
        for (int i = 0; i < kWaves; ++i)
            sum += exps[i];
        part[(int64_t)r * gridDim.x + blockIdx.x] = Part{key, sum, 0};
    }
}

/* A wave joins the chunks of a row, at most 256. */
__global__ __launch_bounds__(64) void join_kernel(coli_logits a, const Part* part, int chunks)
{
    const int r = blockIdx.x;
    constexpr int N = COLI_MAX_VOCAB / kChunk / 64;
    Part p[N];
    unsigned long long key = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = threadIdx.x + 64 * i;
        p[i] = part[(int64_t)r * chunks + min(c, chunks - 1)];
        if (c >= chunks)
            p[i].key = 0;
        key = p[i].key > key ? p[i].key : key;
    }
    key = wave_max(key);
    const float top = value_of(key);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (p[i].key && p[i].sum != 0.0f) /* a chunk of -inf has no sum */
            sum += p[i].sum * exp_below(value_of(p[i].key), top);
    sum = wave_sum(sum);
    if (threadIdx.x == 0) {
        const bool none = top == -__builtin_inff();
        if (a.token)
            a.token[r] = none ? -1 : (int)(0xFFFFFFFFu - (uint32_t)key);
        if (a.lse)
            a.lse[r] = none ? top : top + logf(sum);
    }
}

int chunks_of(int32_t vocab)
{
    return (vocab + kChunk - 1) / kChunk;
}

template <typename T>
hipError_t launch(const coli_logits& a, Part* part, hipStream_t s)
{
    const int chunks = chunks_of(a.vocab);
    const int lds = (a.penalties ? kChunk : 0) * 4 + (a.cu_bias ? kChunk : 0) * 8;
    hipLaunchKernelGGL((adjust_kernel<T>), dim3(chunks, a.rows), dim3(kThreads), lds, s, a, part);
    if (part)
        hipLaunchKernelGGL(join_kernel, dim3(a.rows), dim3(64), 0, s, a, part, chunks);
    return hipGetLastError();
}

} // namespace

size_t logits_workspace_bytes(int32_t rows, int32_t vocab)
{
    return std::max<size_t>(256, ((size_t)rows * chunks_of(vocab) * sizeof(Part) + 255) / 256 * 256);
}

hipError_t launch_adjust_logits(const coli_logits& a, void* ws, hipStream_t s)
{
    Part* part = a.token || a.lse ? (Part*)ws : nullptr;
    return a.type == COLI_F32 ? launch<float>(a, part, s) : launch<bf16>(a, part, s);
}

} // namespace coli
