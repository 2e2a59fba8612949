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
constexpr int kTurn = 4 * kThreads;    /* tokens of a turn over the chunk; chunks are whole turns */
constexpr uint32_t kSeen = 0x80000000u; /* among the tokens; then whether there is a bias, */
constexpr uint32_t kBias = 0x40000000u;
constexpr uint32_t kCount = kBias - 1;  /* and the count of generated ones */

/* What a chunk has to say about its row: the key is the largest value in the order
 * of unsigned numbers, then the lowest token (key_of). */
struct Part {
    unsigned long long key;
    float sum; /* of exp(v - largest) */
    uint32_t pad;
};

/* Larger values have larger keys, NaN the largest, equal values larger ones for
 * lower tokens; 0 where there is nothing above -inf. */
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

/* exp(d) of a difference to the largest value; a sum that took inf - inf is not
 * looked at. */
__device__ __forceinline__ float exp_of(float d)
{
    return __builtin_amdgcn_exp2f(d * 1.44269504088896340736f);
}

__device__ __forceinline__ unsigned long long wave_max(unsigned long long v)
{
    for (int m = 32; m >= 1; m >>= 1) {
        const unsigned long long x = __shfl_xor(v, m, 64);
        v = x > v ? x : v;
    }
    return v;
}

/* Four logits from token t on, -inf past the vocabulary's end. */
template <typename T>
__device__ __forceinline__ float4 logits4(const T* x, int t, int V)
{
    if (t + 4 <= V)
        return load4_any(x + t);
    const float none = -__builtin_inff();
    return make_float4(t < V ? to_f32(x[t]) : none, t + 1 < V ? to_f32(x[t + 1]) : none,
                       t + 2 < V ? to_f32(x[t + 2]) : none, none);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void adjust_kernel(coli_logits a, int chunk, Part* part)
{
    /* [chunk] each: counts, then the biases' sums where there are any */
    extern __shared__ __align__(16) uint32_t counts[];
    float* const sums = (float*)(counts + chunk);
    __shared__ unsigned long long keys[kWaves];
    __shared__ float exps[kWaves];
    __shared__ int ids[kThreads], found[kWaves]; /* the chunk's among kThreads entries of the list */
    __shared__ float bias[kThreads];
    const int r = blockIdx.y, c0 = blockIdx.x * chunk, V = a.vocab, end = min(c0 + chunk, V);
    const T* x = (const T*)a.logits + (int64_t)r * a.logits_stride;

    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    int h0 = 0, h1 = 0, made = 0, b0 = 0, b1 = 0, m = -1;
    if (a.penalties) {
        rep = a.penalties[3 * r];
        freq = a.penalties[3 * r + 1];
        pres = a.penalties[3 * r + 2];
        h0 = max(a.spans[3 * r], 0);
        made = a.spans[3 * r + 1];
        h1 = min(a.spans[3 * r + 2], a.n_tokens);
    }
    if (a.cu_bias) {
        b0 = max(a.cu_bias[r], 0);
        b1 = min(a.cu_bias[r + 1], a.n_bias);
    }
    if (a.mask)
        m = a.mask_of[r];
    /* neutral penalties change nothing, whatever the counts */
    const bool counted = h1 > h0 && !(rep == 1.0f && freq == 0.0f && pres == 0.0f);
    const bool biased = b1 > b0;
    /* the first logits and entries travel while the counts are cleared and the tokens counted */
    float4 next = logits4(x, c0 + 4 * (int)threadIdx.x, V);
    if (counted || biased) {
        const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
        int id = -1, at = 0, n = 0;
        float b = 0.0f;
        uint64_t here = 0;
        auto look = [&](int i) {
            id = i < b1 ? a.bias_ids[i] : -1;
            b = i < b1 ? a.bias[i] : 0.0f;
            here = __ballot(id >= c0 && id < end);
            if (lane == 0)
                found[wv] = __popcll(here);
        };
        /* the entries that lie in the chunk, in the list's order */
        auto gather = [&]() {
            n = 0;
            at = __popcll(here & ((1ull << lane) - 1));
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                at += w < wv ? found[w] : 0;
                n += found[w];
            }
            if (here >> lane & 1) {
                ids[at] = id;
                bias[at] = b;
            }
        };
        /* the first entry of each token adds up all of them */
        auto add = [&]() {
            if ((int)threadIdx.x >= n)
                return;
            const int t = ids[threadIdx.x];
            bool first = true;
            for (int j = 0; j < (int)threadIdx.x; ++j)
                first &= ids[j] != t;
            if (!first)
                return;
            float s = counts[t - c0] & kBias ? sums[t - c0] : 0.0f;
            for (int j = threadIdx.x; j < n; ++j)
                s = ids[j] == t ? s + bias[j] : s;
            sums[t - c0] = s;
            counts[t - c0] |= kBias;
        };
        if (biased)
            look(b0 + threadIdx.x);
        for (int i = threadIdx.x; i < chunk / 4; i += kThreads)
            ((uint4*)counts)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (biased)
            gather();
        if (counted) {
            auto scan = [&](int from, int to, bool generated) {
                auto count = [&](int token) {
                    const uint32_t at = (uint32_t)(token - c0);
                    if (at < (uint32_t)chunk) {
                        if (generated)
                            atomicAdd(counts + at, 1u);
                        else
                            atomicOr(counts + at, kSeen);
                    }
                };
                /* four loads of four tokens at once: the tokens come from the caches, and their latency counts */
                constexpr int N = 4;
                int64_t i = from + 4 * (int64_t)threadIdx.x;
                for (; i + (N - 1) * kTurn + 4 <= to; i += N * kTurn) {
                    int4 q[N];
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        __builtin_memcpy(&q[j], a.tokens + i + j * kTurn, 16);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        count(q[j].x);
                        count(q[j].y);
                        count(q[j].z);
                        count(q[j].w);
                    }
                }
                /* up to three whole turns and a part */
                int4 q[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int64_t k = i + j * kTurn;
                    q[j] = make_int4(-1, -1, -1, -1);
                    if (k + 4 <= to) {
                        __builtin_memcpy(&q[j], a.tokens + k, 16);
                    } else if (k < to) {
                        q[j].x = a.tokens[k];
                        q[j].y = k + 1 < to ? a.tokens[k + 1] : -1;
                        q[j].z = k + 2 < to ? a.tokens[k + 2] : -1;
                    }
                }
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    count(q[j].x);
                    count(q[j].y);
                    count(q[j].z);
                    count(q[j].w);
                }
            };
            const int mid = min(max(made, h0), h1);
            scan(h0, mid, false);
            scan(mid, h1, true);
        }
        if (biased) {
            __syncthreads();
            add();
            for (int base = b0 + kThreads; base < b1; base += kThreads) {
                look(base + threadIdx.x);
                __syncthreads();
                gather();
                __syncthreads();
                add();
            }
        }
        __syncthreads();
    }

    const uint32_t* mask = m >= 0 && m < a.n_masks ? a.mask + m * a.mask_stride : nullptr;
    /* this thread's largest value and its token, its first NaN's, and the sum of exp(v - top) */
    float top = -__builtin_inff(), sum = 0.0f;
    int best = -1, nan = -1;
    for (int t = c0 + 4 * (int)threadIdx.x; t < end; t += kTurn) {
        float v[4] = {next.x, next.y, next.z, next.w};
        if (t + kTurn < end)
            next = logits4(x, t + kTurn, V);
        if (counted || biased) {
            const uint4 q = *(const uint4*)(counts + t - c0);
            const uint32_t c[4] = {q.x, q.y, q.z, q.w};
            if (q.x | q.y | q.z | q.w) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (c[i] & (kSeen | kCount))
                        v[i] = v[i] > 0.0f ? v[i] / rep : v[i] * rep;
                    if (c[i] & kCount)
                        v[i] -= freq * (float)(c[i] & kCount) + pres;
                    if (c[i] & kBias)
                        v[i] += sums[t - c0 + i];
                }
            }
        }
        if (mask) {
            const uint32_t bits = mask[t / 32] >> (t % 32);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = bits >> i & 1 ? v[i] : -__builtin_inff();
        }
        if (a.out) {
            T* o = (T*)a.out + (int64_t)r * a.out_stride + t;
            if (t + 4 <= V) {
                store4_any(o, make_float4(v[0], v[1], v[2], v[3]));
            } else {
                for (int i = 0; t + i < V; ++i)
                    store1(o + i, v[i]);
            }
        }
        if (part) { /* what lies past the vocabulary's end is -inf here */
            const float most = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
            if (most > top) {
                sum *= exp_of(top - most);
                top = most;
                best = t + (v[0] == most ? 0 : v[1] == most ? 1 : v[2] == most ? 2 : 3);
            }
            if (nan < 0 && (__builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3])))
                nan = t + (v[0] != v[0] ? 0 : v[1] != v[1] ? 1 : v[2] != v[2] ? 2 : 3);
            if (best >= 0)
                sum += exp_of(v[0] - top) + exp_of(v[1] - top) + (exp_of(v[2] - top) + exp_of(v[3] - top));
        }
    }
    if (!part)
        return;
    unsigned long long all = nan >= 0 ? key_of(__builtin_nanf(""), nan) : best >= 0 ? key_of(top, best) : 0;
    all = wave_max(all);
    if ((threadIdx.x & 63) == 0)
        keys[threadIdx.x >> 6] = all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        all = keys[i] > all ? keys[i] : all;
    if (best >= 0)
        sum *= exp_of(top - value_of(all));
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0)
        exps[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0f;
        for (int i = 0; i < kWaves; ++i)
            sum += exps[i];
        part[(int64_t)r * gridDim.x + blockIdx.x] = Part{all, sum, 0};
    }
}

/* A wave joins the chunks of a row. */
__global__ __launch_bounds__(64) void join_kernel(coli_logits a, const Part* part, int chunks)
{
    const int r = blockIdx.x;
    const Part* p = part + (int64_t)r * chunks;
    unsigned long long key = 0;
    for (int c = threadIdx.x; c < chunks; c += 64)
        key = p[c].key > key ? p[c].key : key;
    key = wave_max(key);
    const float top = value_of(key);
    float sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += 64)
        if (p[c].key)
            sum += p[c].sum * exp_of(value_of(p[c].key) - top);
    sum = wave_sum(sum);
    if (threadIdx.x == 0) {
        if (a.token)
            a.token[r] = key ? (int)(0xFFFFFFFFu - (uint32_t)key) : -1;
        if (a.lse)
            a.lse[r] = !key ? -__builtin_inff() : top == __builtin_inff() ? top : top + logf(sum);
    }
}

/* Tokens of a chunk.  A row's tokens are read by each of its chunks, so long histories want
 * large ones; what is in flight on a CU is bounded by its LDS, and a row alone by its
 * workgroups. */
int chunk_of(const coli_logits& a)
{
    const int turns = (a.vocab + kTurn - 1) / kTurn;
    const bool far = a.penalties && a.n_tokens / a.rows > 8192;
    const int most = a.cu_bias ? 2 : far ? 8 : 2;
    return kTurn * std::max(1, std::min(most, (int)((int64_t)a.rows * turns / 512)));
}

template <typename T>
hipError_t launch(const coli_logits& a, Part* part, hipStream_t s)
{
    const int chunk = chunk_of(a), chunks = (a.vocab + chunk - 1) / chunk;
    const int lds = chunk * (a.cu_bias ? 8 : a.penalties ? 4 : 0);
    hipLaunchKernelGGL((adjust_kernel<T>), dim3(chunks, a.rows), dim3(kThreads), lds, s, a, chunk, part);
    if (part)
        hipLaunchKernelGGL(join_kernel, dim3(a.rows), dim3(64), 0, s, a, part, chunks);
    return hipGetLastError();
}

} // namespace

size_t logits_workspace_bytes(int32_t rows, int32_t vocab)
{
    const size_t chunks = (vocab + kTurn - 1) / kTurn;
    return std::max<size_t>(256, ((size_t)rows * chunks * sizeof(Part) + 255) / 256 * 256);
}

hipError_t launch_adjust_logits(const coli_logits& a, void* ws, hipStream_t s)
{
    Part* part = a.token || a.lse ? (Part*)ws : nullptr;
    return a.type == COLI_F32 ? launch<float>(a, part, s) : launch<bf16>(a, part, s);
}

} // namespace coli
