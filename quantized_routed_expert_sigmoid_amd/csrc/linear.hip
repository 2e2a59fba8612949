/*
 * linear.hip -- quantised matrix product of Q8_0 activations with bias,
 * activation and residual in its epilogue.
 *
 * Few tokens (linear_rows_kernel): one wave per weight row and up to four
 * tokens; each lane takes whole 32-element blocks, whose exact integer dot
 * products times the two scales are summed in fp32, first in the lane and then
 * over the wave.
 *
 * Many tokens: linear_expand writes the activations once as fp16 and
 * linear_tiles runs the product on the fp16 matrix cores.  A weight code is
 * exact in fp16, so the matrix cores sum code * x in fp32 over a whole row (or
 * a group of one scale) with nothing to fold per 32-element block: the
 * per-block form on the int8 cores needs a conversion and an fma per block and
 * output, 32 VALU cycles beside 19 of the matrix core.  x = code * d is scaled
 * per token by a power of two so that its largest value lies in [2^14, 2^15)
 * and rounded to fp16 (2^-12 of each value) for bf16 outputs, an eighth of the
 * output's own rounding; for fp32 outputs a second fp16 term takes the
 * remainder (2^-22).
 */
#include "block_device.h"

namespace coli {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

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

/* ---- many tokens ---------------------------------------------------------- */

constexpr int kKB = 64;       /* k of one step */
constexpr int kTileTok = 32;  /* tokens of a matrix-core tile */
constexpr int kTileN = 128;   /* weight rows of a workgroup */
constexpr int kChunk = 16;    /* bytes that a lane loads at once */

/* Order of eight consecutive k in an operand: the one in which the packed
 * fields of a weight word come out of the unpacking below. */
template <int BITS>
__device__ __forceinline__ int k_order(int i)
{
    if constexpr (BITS == 8)
        return i;
    else if constexpr (BITS == 4)
        return (0x62734051 >> (4 * i)) & 7; /* 1 5 0 4 3 7 2 6 */
    else
        return (0x40516273 >> (4 * i)) & 7; /* 3 7 2 6 1 5 0 4 */
}

/*
 * Activations as fp16 operands: [step][tile of 32 tokens][term][chunk of 8 k][token] of 16 bytes, so that
 * a wave's operand load is one run of 1 KB.  The last step covers k = K - 64 .. K - 1; what an earlier step
 * has covered already is zero in it, as are tokens from S on.  A workgroup takes one token: its largest
 * value first, then its chunks.
 */
template <int BITS, int NT>
__global__ __launch_bounds__(256) void linear_expand(LinearArgs a, uint8_t* xh, float* xs, int tiles)
{
    __shared__ float part[4];
    const int t = blockIdx.x, nb = a.K / 32, steps = (a.K + kKB - 1) / kKB;
    const bool live = t < a.S;
    const float* d = a.xd + (int64_t)min(t, a.S - 1) * nb;
    const int8_t* q = a.xq + (int64_t)min(t, a.S - 1) * a.K;
    float top = 0.0f;
    for (int b = threadIdx.x; b < nb; b += 256)
        top = fmaxf(top, fabsf(d[b]));
    for (int m = 32; m >= 1; m >>= 1)
        top = fmaxf(top, shfl_xor(top, m));
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    /* 2^e > 127 top, so |x| 2^(15 - e) < 2^15 */
    int e = 0;
    if (top > 0.0f)
        (void)frexpf(top, &e);
    e = max(e + 7, -111); /* 2^(15 - e) stays finite */
    const float up = top > 0.0f ? ldexpf(1.0f, 15 - e) : 0.0f;
    if (threadIdx.x == 0 && live)
        xs[t] = ldexpf(1.0f, e - 15);
    for (int c = threadIdx.x; c < steps * 8; c += 256) {
        const int step = c >> 3, k0 = step * kKB, at = min(k0, a.K - kKB) + (c & 7) * 8;
        v8h hi = {0, 0, 0, 0, 0, 0, 0, 0}, lo = hi;
        if (live && at >= k0) {
            const uint2 w = *(const uint2*)(q + at);
            const float s = d[at >> 5] * up;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = k_order<BITS>(i);
                float x = (float)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3))) * s;
                /* pinned: the compiler may otherwise take hi from the unrounded
                 * product in one of its two uses, and a tie both ways */
                asm("" : "+v"(x));
                hi[i] = (_Float16)x;
                lo[i] = (_Float16)(x - (float)hi[i]);
            }
        }
        uint8_t* o = xh + ((((int64_t)step * tiles + t / kTileTok) * NT * 8 + (c & 7)) * kTileTok + t % kTileTok) * kChunk;
        *(v8h*)o = hi;
        if constexpr (NT == 2)
            *(v8h*)(o + 8 * kTileTok * kChunk) = lo;
    }
}

/* Sixteen bytes per lane from memory into LDS at dst + 16 lane (dst uniform). */
__device__ __forceinline__ void to_lds(const void* src, void* dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

__device__ __forceinline__ v2h as_h2(uint32_t u)
{
    v2h r;
    __builtin_memcpy(&r, &u, 4);
    return r;
}

/* Eight codes as fp16 in k_order: each field becomes the low mantissa bits of
 * 1024 + f 2^s, the offsets then subtracted (exact). */
template <int BITS>
__device__ __forceinline__ v8h codes_f16(uint32_t w0, uint32_t w1)
{
    v2h r[4];
    if constexpr (BITS == 8) {
        const uint32_t a = w0 ^ 0x80808080u, b = w1 ^ 0x80808080u;
        const v2h off = {(_Float16)-1152, (_Float16)-1152};
        r[0] = as_h2(__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) + off;
        r[1] = as_h2(__builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) + off;
        r[2] = as_h2(__builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) + off;
        r[3] = as_h2(__builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) + off;
    } else if constexpr (BITS == 4) {
        const uint32_t a = w0 ^ 0x88888888u, b = a >> 8;
        const v2h o0 = {(_Float16)-1032, (_Float16)-1032}, o1 = {(_Float16)-72, (_Float16)-72};
        const v2h s1 = {(_Float16)0.0625, (_Float16)0.0625};
        r[0] = as_h2((a & 0x000F000Fu) | 0x64006400u) + o0;
        r[1] = __builtin_elementwise_fma(as_h2((a & 0x00F000F0u) | 0x64006400u), s1, o1);
        r[2] = as_h2((b & 0x000F000Fu) | 0x64006400u) + o0;
        r[3] = __builtin_elementwise_fma(as_h2((b & 0x00F000F0u) | 0x64006400u), s1, o1);
    } else {
        /* w0: the eight fields' two bytes in bits 0..7 and 16..23 */
        const uint32_t a = w0 ^ 0x00AA00AAu;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sc = 1.0f / (float)(1 << (2 * i)), of = -(1024.0f * sc + 2.0f);
            const v2h s = {(_Float16)sc, (_Float16)sc}, o = {(_Float16)of, (_Float16)of};
            r[i] = __builtin_elementwise_fma(as_h2((a & (0x00030003u << (2 * i))) | 0x64006400u), s, o);
        }
    }
    v8h v;
    __builtin_memcpy(&v, r, 16);
    return v;
}

/*
 * A workgroup of 2 x 2 waves takes 128 weight rows x 64 TT tokens, a wave 64
 * rows x 32 TT tokens of them (2 x TT tiles of v_mfma_f32_32x32x16_f16), with
 * steps of 64 k: the next step's operands travel from memory to LDS under this
 * step's products.  Weights stay packed in LDS and are unpacked by the waves
 * that multiply them.  Lane (l % 32, h = l / 32) of instruction i of a step
 * takes k = 16 i + 8 h .. + 7 of a step, so that one instruction stays inside
 * one scale group.
 */
template <int BITS, int NT, int TT, bool GROUPED, typename TO>
__global__ __launch_bounds__(256, 2) void linear_tiles(LinearArgs a, const uint8_t* xh, const float* xs, int tiles,
                                                       int n_tiles, int t_tiles, int vec)
{
    constexpr int XB = 2 * TT * NT * 8 * kTileTok * kChunk; /* bytes of a step's activations */
    constexpr int WC = BITS / 2;                            /* 16-byte chunks of a row's step (int2: 1) */
    constexpr int WB = kTileN * WC * kChunk;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, h = lane >> 5, col = lane & 31;
    const int wn = wv & 1, wt = wv >> 1;

    /* Workgroups go to the eight XCDs in turn; each XCD takes a contiguous run
     * of tiles, eight token tiles to a column of weight tiles, so that the
     * tiles it works on at a time share operands in its L2. */
    const int total = n_tiles * t_tiles, per = (total + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if (id >= total || (int)(blockIdx.x >> 3) >= per)
        return;
    constexpr int GT = 8;
    const int band = id / (GT * n_tiles), in = id % (GT * n_tiles), wide = min(GT, t_tiles - band * GT);
    const int tn = in / wide, tt0 = band * GT + in % wide;

    const int steps = (a.K + kKB - 1) / kKB, n0 = tn * kTileN;
    const int64_t row_bytes = (int64_t)a.K * BITS / 8;
    const uint8_t* w = (const uint8_t*)a.w;

    /* this wave's share of a step's loads: runs of 64 chunks */
    auto fetch = [&](int step, uint8_t* buf) {
        const uint8_t* x = xh + ((int64_t)step * tiles + tt0 * 2 * TT) * (NT * 8 * kTileTok * kChunk);
#pragma unroll
        for (int i = 0; i < XB / 4096; ++i) {
            const int o = (i * 4 + wv) * 1024;
            to_lds(x + o + lane * 16, buf + o);
        }
        const int64_t kb = (int64_t)min(step * kKB, a.K - kKB) * BITS / 8;
        /* chunk c of row n at (c * 128 + n) * 16 */
#pragma unroll
        for (int i = 0; i < (WB / 1024 + 3) / 4; ++i) {
            const int run = i * 4 + wv;
            if (WB / 1024 % 4 && run >= WB / 1024)
                break;
            const int c = run * 64 / kTileN, n = min(n0 + run * 64 % kTileN + lane, a.N - 1);
            to_lds(w + n * row_bytes + kb + c * 16, buf + XB + run * 1024);
        }
    };

    v16f acc[2][TT];
    v16f part[GROUPED ? 2 : 1][GROUPED ? TT : 1];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[r][t][i] = 0.0f;
                if constexpr (GROUPED)
                    part[r][t][i] = 0.0f;
            }

    const int gpr = GROUPED ? a.K / a.group : 1;
    /* part *= scales of group g, added to acc */
    auto fold = [&](int g) {
        if constexpr (GROUPED) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int n = min(n0 + wn * 64 + r * 32 + 8 * (i / 4) + 4 * h + i % 4, a.N - 1);
                    const float s = a.w_scale[(int64_t)n * gpr + g];
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        acc[r][t][i] = __builtin_fmaf(part[r][t][i], s, acc[r][t][i]);
                        part[r][t][i] = 0.0f;
                    }
                }
        }
    };

    fetch(0, lds);
    __syncthreads();
    int g = 0;
    for (int step = 0; step < steps; ++step) {
        uint8_t* buf = lds + (step & 1) * (XB + WB);
        if (step + 1 < steps)
            fetch(step + 1, lds + (~step & 1) * (XB + WB));
        const int kb = min(step * kKB, a.K - kKB);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (GROUPED) {
                /* a step may start in an earlier group than the last one ended in:
                 * its activations there are zero */
                if (!(i & 1)) {
                    const int now = (kb + 16 * i) / a.group;
                    if (now > g) {
                        fold(g);
                        g = now;
                    }
                }
            }
            v8h wf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int n = wn * 64 + r * 32 + col;
                const uint8_t* p = buf + XB;
                if constexpr (BITS == 8) {
                    const uint2 v = *(const uint2*)(p + (i * kTileN + n) * 16 + h * 8);
                    wf[r] = codes_f16<8>(v.x, v.y);
                } else if constexpr (BITS == 4) {
                    wf[r] = codes_f16<4>(*(const uint32_t*)(p + ((i >> 1) * kTileN + n) * 16 + (i & 1) * 8 + h * 4), 0);
                } else {
                    const uint32_t v = *(const uint32_t*)(p + n * 16 + i * 4);
                    wf[r] = codes_f16<2>(__builtin_amdgcn_perm(0, v, h ? 0x0C030C02u : 0x0C010C00u), 0);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    const v8h x = *(const v8h*)(buf + (((wt * TT + t) * NT + e) * 8 + 2 * i) * (kTileTok * kChunk) +
                                                lane * 16);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        v16f& o = GROUPED ? part[GROUPED ? r : 0][GROUPED ? t : 0] : acc[r][t];
                        o = __builtin_amdgcn_mfma_f32_32x32x16_f16(wf[r], x, o, 0, 0, 0);
                    }
                }
        }
        __syncthreads();
    }
    fold(g);

    /* epilogue: lane (token col, rows 8 (i / 4) + 4 h + i % 4), one uniform
     * branch on the activation for all of them */
    const int tok0 = (tt0 * 2 * TT + wt * TT) * kTileTok + col;
    float scale[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        scale[t] = xs[min(tok0 + t * kTileTok, a.S - 1)];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = min(n0 + wn * 64 + r * 32 + 8 * (i / 4) + 4 * h + i % 4, a.N - 1);
            const float ws = GROUPED ? 1.0f : a.w_scale[n], bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
            for (int t = 0; t < TT; ++t)
                acc[r][t][i] = __builtin_fmaf(acc[r][t][i], scale[t] * ws, bias);
        }
    auto each = [&](auto f) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[r][t][i] = f(acc[r][t][i]);
    };
    if (a.act == COLI_ACT_RELU)
        each([](float v) { return activate(v, COLI_ACT_RELU); });
    else if (a.act == COLI_ACT_SILU)
        each([](float v) { return activate(v, COLI_ACT_SILU); });
    else if (a.act == COLI_ACT_GELU)
        each([](float v) { return activate(v, COLI_ACT_GELU); });
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int tok = tok0 + t * kTileTok;
        if (tok >= a.S)
            continue;
        TO* out = (TO*)a.out + (int64_t)tok * a.N;
        const TO* res = a.residual ? (const TO*)a.residual + (int64_t)tok * a.N : nullptr;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int n = n0 + wn * 64 + r * 32 + 2 * i + 4 * h;
                float4 y = make_float4(acc[r][t][i], acc[r][t][i + 1], acc[r][t][i + 2], acc[r][t][i + 3]);
                if (vec) {
                    if (n >= a.N)
                        continue;
                    if (res) {
                        const float4 v = load4(res + n);
                        y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                    }
                    store4(out + n, y);
                } else {
                    const float e[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < a.N)
                            store1(out + n + j, e[j] + (res ? to_f32(res[n + j]) : 0.0f));
                }
            }
    }
}

struct TilePlan {
    int tt, tiles, n_tiles, t_tiles, steps, terms;
    size_t x_bytes, total;
};

TilePlan tile_plan(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type)
{
    TilePlan p;
    p.terms = out_type == COLI_F32 ? 2 : 1;
    p.n_tiles = (N + kTileN - 1) / kTileN;
    const int most = p.terms == 1 && !group ? 4 : 2;
    /* the widest token tile that still gives every CU a workgroup or two */
    p.tt = most;
    while (p.tt > 1 && (int64_t)p.n_tiles * ((S + 64 * p.tt - 1) / (64 * p.tt)) < 256)
        p.tt /= 2;
    p.t_tiles = (S + 64 * p.tt - 1) / (64 * p.tt);
    p.tiles = p.t_tiles * 2 * p.tt;
    p.steps = (K + kKB - 1) / kKB;
    p.x_bytes = (size_t)p.steps * p.tiles * p.terms * 8 * kTileTok * kChunk;
    p.total = (p.x_bytes + (size_t)S * 4 + 255) / 256 * 256;
    return p;
}

bool use_tiles(int32_t S, int32_t K)
{
    return S > 16 && K >= kKB;
}

template <int BITS, int NT, int TT, bool GROUPED, typename TO>
hipError_t launch_tiles_t(const LinearArgs& a, const TilePlan& p, hipStream_t s)
{
    uint8_t* xh = (uint8_t*)a.ws;
    float* xs = (float*)(xh + p.x_bytes);
    hipLaunchKernelGGL((linear_expand<BITS, NT>), dim3(p.tiles * kTileTok), dim3(256), 0, s, a, xh, xs, p.tiles);
    constexpr int bytes = 2 * (2 * TT * NT * 8 * kTileTok * kChunk + kTileN * (BITS / 2) * kChunk);
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)linear_tiles<BITS, NT, TT, GROUPED, TO>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess)
            return e;
    }
    const int total = p.n_tiles * p.t_tiles;
    /* rows of whole, aligned groups of four outputs */
    const int vec = a.N % 4 == 0 && ((uintptr_t)a.out | (uintptr_t)a.residual) % (4 * sizeof(TO)) == 0;
    hipLaunchKernelGGL((linear_tiles<BITS, NT, TT, GROUPED, TO>), dim3((total + 7) / 8 * 8), dim3(256), bytes, s, a,
                       xh, xs, p.tiles, p.n_tiles, p.t_tiles, vec);
    return hipGetLastError();
}

template <int BITS, typename TO>
hipError_t launch_tiles(const LinearArgs& a, hipStream_t s)
{
    constexpr int NT = sizeof(TO) == 4 ? 2 : 1;
    const TilePlan p = tile_plan(a.S, a.N, a.K, a.group, a.out_type);
    if (a.group)
        return p.tt == 2 ? launch_tiles_t<BITS, NT, 2, true, TO>(a, p, s) : launch_tiles_t<BITS, NT, 1, true, TO>(a, p, s);
    if constexpr (NT == 1)
        if (p.tt == 4)
            return launch_tiles_t<BITS, NT, 4, false, TO>(a, p, s);
    return p.tt == 2 ? launch_tiles_t<BITS, NT, 2, false, TO>(a, p, s) : launch_tiles_t<BITS, NT, 1, false, TO>(a, p, s);
}

template <int BITS, typename TO>
hipError_t launch(const LinearArgs& a, hipStream_t s)
{
    if (use_tiles(a.S, a.K))
        return launch_tiles<BITS, TO>(a, s);
    hipLaunchKernelGGL((linear_rows_kernel<BITS, TO>), dim3((a.N + 3) / 4, (a.S + 3) / 4), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int BITS>
hipError_t launch_type(const LinearArgs& a, hipStream_t s)
{
    return a.out_type == COLI_F32 ? launch<BITS, float>(a, s) : launch<BITS, bf16>(a, s);
}

} // namespace

size_t linear_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t qtype, int32_t group, int32_t out_type)
{
    return use_tiles(S, K) ? tile_plan(S, N, K, group, out_type).total : 256;
}

hipError_t launch_linear_q(const LinearArgs& a, hipStream_t s)
{
    return a.qtype == COLI_Q8   ? launch_type<8>(a, s)
           : a.qtype == COLI_Q4 ? launch_type<4>(a, s)
                                : launch_type<2>(a, s);
}

} // namespace coli
