/*
 * linear_i8.hip -- matrix product in 8-bit integers with one scale per token and
 * one per channel, and the activations' quantisation that goes before it:
 *
 *   d[t] = max_k |x[t][k]| / 127,  q[t][k] = rnd(x[t][k] * (1 / d[t]))
 *   out[t][n] = act(s[n] d[t] sum_k w[n][k] q[t][k] + bias[n]) + residual[t][n]
 *
 * The sum over a whole row is exact in int32 (at most 2^15 products below 2^14), so
 * nothing is folded on the way and neither splits of a row nor their order change a
 * bit of the result.  Two forms:
 *
 * - i8_rows, few tokens: the weights are read once, from memory straight to the
 *   matrix cores' registers, and the activations again and again from the caches;
 * - i8_tiles, more: tiles of both in LDS.
 *
 * Codes of fewer bits are unpacked to the top of their bytes, 2^(8 - bits) times
 * their value, which the row's scale takes out again.
 */
#include "linear_device.h"
#include "step.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace coli {

namespace {

/* f(0) .. f(N - 1) with the number as a constant: large bodies that index registers
 * are not left to the unroller. */
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}

template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    each_of(f, std::make_integer_sequence<int, N>());
}

/* ---- activations ---------------------------------------------------------- */

/* A workgroup per row, which stays in its registers between the largest value and
 * the codes; NV groups of four values per thread.  Loads are unconditional, past the
 * row's end of its last group: one under a branch would be waited for by itself. */
template <typename T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void quantize_kernel(const T* x, int64_t stride, int K, int8_t* q, float* d)
{
    __shared__ float part[THREADS / 64];
    const int n4 = K / 4;
    const int64_t row = blockIdx.x;
    float4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        v[j] = load4(x + row * stride + 4 * min((int)threadIdx.x + THREADS * j, n4 - 1));
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        a = fmaxf(fmaxf(fmaxf(a, fabsf(v[j].x)), fmaxf(fabsf(v[j].y), fabsf(v[j].z))), fabsf(v[j].w));
    for (int m = 32; m >= 1; m >>= 1)
        a = fmaxf(a, shfl_xor(a, m));
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i)
        a = fmaxf(a, part[i]);
    const float s = a / 127.0f, inv = a == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + THREADS * j;
        if (i >= n4)
            break;
        ((uint32_t*)(q + row * K))[i] =
            (uint32_t)(q8_code(v[j].x, inv) & 0xFF) | ((uint32_t)(q8_code(v[j].y, inv) & 0xFF) << 8) |
            ((uint32_t)(q8_code(v[j].z, inv) & 0xFF) << 16) | ((uint32_t)(q8_code(v[j].w, inv) & 0xFF) << 24);
    }
    if (threadIdx.x == 0)
        d[row] = s;
}

/* ---- the last step -------------------------------------------------------- */

/* Sums of N x 4 rows n0 + 4 .. of token tok, finished and stored: s d sum + bias with
 * the scales' product and the sum rounded to fp32 once each. */
__device__ __forceinline__ void finish4(const LinearI8Args& a, float unit, float d, int n, const int* sum, float* v)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int m = min(n + j, a.N - 1);
        v[j] = __builtin_fmaf((float)sum[j], unit * a.w_scale[m] * d, a.bias ? a.bias[m] : 0.0f);
    }
}

/* ---- few tokens ----------------------------------------------------------- */

/* A lane's 32 codes of a step, as two operands of sixteen. */
template <int BITS>
struct Codes32 {
    uint32_t w[BITS];
};

template <int BITS>
__device__ __forceinline__ Codes32<BITS> load_codes(const uint8_t* p)
{
    Codes32<BITS> r;
    if constexpr (BITS == 2) {
        const uint2 v = *(const uint2*)p;
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < BITS; i += 4) {
            const uint4 v = *(const uint4*)(p + 4 * i);
            r.w[i] = v.x;
            r.w[i + 1] = v.y;
            r.w[i + 2] = v.z;
            r.w[i + 3] = v.w;
        }
    }
    return r;
}

template <int BITS>
__device__ __forceinline__ v4i operand(const Codes32<BITS>& c, int half)
{
    RawCodes<BITS> r;
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i)
        r.w[i] = c.w[half * (BITS / 2) + i];
    return codes_i8<BITS>(r);
}

/*
 * A workgroup takes 16 R rows x 16 T tokens, its W waves the row's steps of 128 k in
 * turn.  Lane (c = l % 16, g = l / 16) of a step reads the 32 codes from 32 g on of
 * row and of token c: a row's step is one or two whole lines.  Both operands of
 * v_mfma_i32_16x16x64_i8 take their k in this order, so any order is right.  The next
 * U steps travel under the products of these.
 */
template <int BITS, int R, int T, int W, int U, typename TO>
__global__ __launch_bounds__(W * 64) void i8_rows(LinearI8Args a)
{
    __shared__ int part[W][R * T][256];
    const int lane = threadIdx.x & 63, wv = wave_of(), c = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * (16 * R), t0 = blockIdx.y * (16 * T);
    const int steps = (a.K + 127) / 128;
    const int64_t row_bytes = (int64_t)a.K * BITS / 8;
    const uint8_t* w[R];
    const int8_t* x[T];
#pragma unroll
    for (int r = 0; r < R; ++r)
        w[r] = (const uint8_t*)a.w + min(n0 + 16 * r + c, a.N - 1) * row_bytes;
#pragma unroll
    for (int t = 0; t < T; ++t)
        x[t] = a.xq + (int64_t)min(t0 + 16 * t + c, a.S - 1) * a.K;

    Codes32<BITS> wc[2][U][R];
    Codes32<8> xc[2][U][T];
    auto load = [&](int first, int p) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (first + u * W) * 128 + g * 32, at = min(k, a.K - 32);
#pragma unroll
            for (int r = 0; r < R; ++r)
                wc[p][u][r] = load_codes<BITS>(w[r] + at * BITS / 8);
#pragma unroll
            for (int t = 0; t < T; ++t)
                xc[p][u][t] = load_codes<8>((const uint8_t*)x[t] + at);
        }
    };
    v4i acc[R][T];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t)
            acc[r][t] = v4i{0, 0, 0, 0};
    auto multiply = [&](int first, int p) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = (first + u * W) * 128 + g * 32 < a.K; /* past the row's end: zeros */
            v4i xo[T][2];
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    xo[t][i] = operand<8>(xc[p][u][t], i);
                    xo[t][i] = in ? xo[t][i] : v4i{0, 0, 0, 0};
                }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const v4i wo = operand<BITS>(wc[p][u][r], i);
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wo, xo[t][i], acc[r][t], 0, 0, 0);
                }
        }
    };
    load(wv, 0);
    for (int s = wv; s < steps; s += 2 * U * W) {
        load(s + U * W, 1);
        multiply(s, 0);
        load(s + 2 * U * W, 0);
        multiply(s + U * W, 1);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t)
            *(v4i*)(part[wv][r * T + t] + lane * 4) = acc[r][t];
    __syncthreads();
    for (int i = wv; i < R * T; i += W) {
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < W; ++j)
            sum += *(const v4i*)(part[j][i] + lane * 4);
        const int tok = t0 + 16 * (i % T) + c, n = n0 + 16 * (i / T) + 4 * g;
        const int e[4] = {sum[0], sum[1], sum[2], sum[3]};
        float v[4];
        finish4(a, 1.0f / (float)(1 << (8 - BITS)), a.xd[min(tok, a.S - 1)], n, e, v);
        activate_all<4>(v, a.act);
        store_rows<TO>(a, tok, n, v);
    }
}

/* ---- many tokens ---------------------------------------------------------- */

constexpr int kStageK = 64; /* k of a stage: two instructions deep */
constexpr int kStages = 4;

/* A workgroup of WR x WT waves, a wave of 32 RR rows x 32 TT tokens. */
template <int BITS, int RR, int TT, int WR, int WT>
struct TileShape {
    static constexpr int kWaves = WR * WT, kRows = 32 * RR * WR, kTok = 32 * TT * WT;
    static constexpr int kXC = kStageK / kChunk, kWC = kStageK * BITS / 8 / kChunk; /* chunks of a token, of a row: 4; 4, 2, 1 */
    static constexpr int kX = kTok * kStageK, kW = kRows * kStageK * BITS / 8, kStage = kX + kW;
    static constexpr int kXRuns = kX / 1024 / kWaves, kWRuns = (kW / 1024 + kWaves - 1) / kWaves;
    static constexpr int kLoads = kXRuns + kWRuns; /* of a wave and stage; where there are fewer runs than waves, waves load the same one */
};

struct I8TileArgs {
    int4* part; /* [split][tile][wave][r][t][i / 4][lane] */
    int n_tiles, t_tiles, stages, splits;
};

/*
 * Stages of 64 k travel from memory to LDS three ahead.  A wave reads the operands of
 * one instruction depth (32 k) while the products of the one before run; the wait
 * for the next stage and the workgroup's barrier lie in the middle of a stage, under
 * its first half's products.  Lane (col = l % 32, h = l / 32) of an operand takes k =
 * 16 h .. + 15 of row or token col.
 */
template <int BITS, int RR, int TT, int WR, int WT, int PER_CU, typename TO>
__global__ __launch_bounds__(WR* WT * 64, PER_CU* WR* WT / 4) void i8_tiles(LinearI8Args a, I8TileArgs ta)
{
    using L = TileShape<BITS, RR, TT, WR, WT>;
    constexpr int WC = L::kWC, XB = L::kX, NW = L::kWaves;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, wv = wave_of(), h = lane >> 5, col = lane & 31;
    const int unit = (int)xcd_unit(), total = ta.n_tiles * ta.t_tiles;
    if (unit >= total * ta.splits)
        return;
    const int id = unit / ta.splits, split = unit % ta.splits;
    const TileAt wg = tile_at<L::kRows, L::kTok>(id, ta.n_tiles, ta.t_tiles);
    const int wr = wv % WR * 32 * RR, wt = wv / WR * 32 * TT; /* the wave's rows and tokens in the tile */
    const int share = (ta.stages + ta.splits - 1) / ta.splits;
    const int s0 = split * share, s1 = min(s0 + share, ta.stages);
    const int row_bytes = (int)((int64_t)a.K * BITS / 8);

    /* Slot c of a token or row holds chunk c ^ f, so that 16 of them read at one
     * chunk fall into different banks. */
    auto xswz = [](int t) { return t / 4 % 4; };
    auto wswz = [](int n) { return n / (16 / WC) % WC; };
    const uint32_t lds0 = lds_address(lds);
    const uint8_t* w0 = (const uint8_t*)a.w + (int64_t)wg.n0 * row_bytes;
    const int8_t* x0 = a.xq + (int64_t)wg.tok0 * a.K;
    int xrow[L::kXRuns], xchunk[L::kXRuns], wrow[L::kWRuns], wchunk[L::kWRuns];
#pragma unroll
    for (int i = 0; i < L::kXRuns; ++i) {
        const int slot = (i * NW + wv) * 64 + lane, t = slot / L::kXC;
        xrow[i] = min(t, a.S - 1 - wg.tok0) * a.K;
        xchunk[i] = (slot % L::kXC ^ xswz(t)) * kChunk;
    }
#pragma unroll
    for (int i = 0; i < L::kWRuns; ++i) {
        const int slot = (i * NW + wv) % (L::kW / 1024) * 64 + lane, n = slot / WC;
        wrow[i] = min(n, a.N - 1 - wg.n0) * row_bytes;
        wchunk[i] = (slot % WC ^ wswz(n)) * kChunk;
    }
    /* Load i of a stage; past the row's end its last bytes, past the last stage that
     * one (loaded and not used). */
    auto fetch1 = [&](int stage, int i) {
        const uint32_t buf = lds0 + stage % kStages * L::kStage;
        stage = min(stage, ta.stages - 1);
        if (i < L::kXRuns) {
            const int k = stage * kStageK, b = min(k, a.K - kChunk);
            to_lds(x0 + b, xrow[i] + min(k + xchunk[i], a.K - kChunk) - b, buf + (i * NW + wv) * 1024);
        } else {
            const int j = i - L::kXRuns;
            const int k = stage * (WC * kChunk), last = row_bytes - kChunk, b = min(k, last);
            to_lds(w0 + b, wrow[j] + min(k + wchunk[j], last) - b,
                   buf + XB + (j * NW + wv) % (L::kW / 1024) * 1024);
        }
    };
    v16i acc[RR][TT];
#pragma unroll
    for (int r = 0; r < RR; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[r][t][i] = 0;

    const bool odd = a.K % kStageK != 0; /* the last stage has one depth only */
    RawCodes<BITS> wf[2][RR];
    v4i xf[2][TT];
    auto read1 = [&](int stage, auto kb, auto i) {
        const uint8_t* buf = lds + stage % kStages * L::kStage;
        if constexpr (i < RR) {
            const int n = wr + i * 32 + col;
            const int cc = BITS == 8 ? 2 * kb + h : BITS == 4 ? +kb : 0;
            /* an int2 row's odd last depth was loaded with the one before it */
            const int half = BITS == 2 && odd && stage == ta.stages - 1 ? 1 : +kb;
            wf[kb][i] = read_codes<BITS>(buf + XB + (n * WC + (cc ^ wswz(n))) * kChunk, half, h);
        } else {
            const int t = wt + (i - RR) * 32 + col;
            xf[kb][i - RR] = *(const v4i*)(buf + (t * L::kXC + ((2 * kb + h) ^ xswz(t))) * kChunk);
        }
    };
    constexpr int kReads = RR + TT, kMul = RR * TT;
    const std::integral_constant<int, 0> first{};
    const std::integral_constant<int, 1> second{};
    for (int s = 0; s < kStages - 1; ++s)
        each<L::kLoads>([&](auto i) { fetch1(s0 + s, i); });
    arrive_all<L::kLoads*(kStages - 2)>();
    each<kReads>([&](auto i) { read1(s0, first, i); });
    for (int stage = s0; stage < s1; ++stage) {
        /* the products of one depth, and after product m its share of what else is to be issued */
        auto multiply = [&](auto kb, auto other) {
            v4i wo[RR];
            each<RR>([&](auto r) { wo[r] = codes_i8<BITS>(wf[kb][r]); });
            each<kMul>([&](auto m) {
                acc[m / TT][m % TT] =
                    __builtin_amdgcn_mfma_i32_32x32x32_i8(wo[m / TT], xf[kb][m % TT], acc[m / TT][m % TT], 0, 0, 0);
                other(m);
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        multiply(first, [&](auto m) {
            each<kReads>([&](auto i) {
                if constexpr (i * kMul / kReads == m)
                    read1(stage, second, i);
            });
        });
        /* stage + 1 is there, and every wave has left stage - 1 */
        arrive_all<L::kLoads*(kStages - 3)>();
        /* the second depth of an odd row's last stage takes no part */
        const int part = odd && stage == ta.stages - 1 ? 0 : -1;
        each<TT>([&](auto t) { xf[1][t] &= part; });
        multiply(second, [&](auto m) {
            each<kReads>([&](auto i) {
                if constexpr (i * kMul / kReads == m)
                    read1(stage + 1, first, i);
            });
            each<L::kLoads>([&](auto i) {
                if constexpr (i * kMul / L::kLoads == m)
                    fetch1(stage + kStages - 1, i);
            });
        });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); /* no load outlives the workgroup's LDS */
    if (ta.splits > 1) {
        int4* o = ta.part + (((int64_t)split * total + id) * NW + wv) * (RR * TT * 4 * 64) + lane;
        each<kMul * 4>([&](auto q) {
            constexpr int m = q / 4, i = q % 4 * 4;
            const v16i& z = acc[m / TT][m % TT];
            o[q * 64] = make_int4(z[i], z[i + 1], z[i + 2], z[i + 3]);
        });
        return;
    }
    /* One 32 x 32 part at a time: the next one's scales are not loaded ahead, for which
     * there are no registers. */
    each<kMul>([&](auto m) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        constexpr int r = m / TT, t = m % TT;
        const int tok = wg.tok0 + wt + t * 32 + col, n = wg.n0 + wr + r * 32 + 4 * h;
        const float d = a.xd[min(tok, a.S - 1)];
        each<4>([&](auto i) {
            const v16i& z = acc[r][t];
            const int e[4] = {z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]};
            float v[4];
            finish4(a, 1.0f / (float)(1 << (8 - BITS)), d, n + 8 * i, e, v);
            activate_all<4>(v, a.act);
            store_rows<TO>(a, tok, n + 8 * i, v);
        });
    });
}

/* Adds the splits' sums and finishes them: a workgroup takes one of a tile's groups
 * of four rows, in the tiles' layout. */
template <int RR, int TT, int WR, int WT, typename TO>
__global__ __launch_bounds__(WR* WT * 64) void i8_join(LinearI8Args a, I8TileArgs ta, float unit)
{
    constexpr int NW = WR * WT;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, total = ta.n_tiles * ta.t_tiles;
    const int id = blockIdx.x, q = blockIdx.y, i = q & 3, t = (q >> 2) % TT, r = (q >> 2) / TT;
    const int4* o = ta.part + (((int64_t)id * NW + wv) * (RR * TT * 4) + q) * 64 + lane;
    const int64_t step = (int64_t)total * NW * (RR * TT * 4) * 64;
    int e[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < ta.splits; ++s) {
        const int4 x = o[s * step];
        e[0] += x.x;
        e[1] += x.y;
        e[2] += x.z;
        e[3] += x.w;
    }
    const TileAt wg = tile_at<32 * RR * WR, 32 * TT * WT>(id, ta.n_tiles, ta.t_tiles);
    const int tok = wg.tok0 + wv / WR * 32 * TT + t * 32 + (lane & 31);
    const int n = wg.n0 + wv % WR * 32 * RR + r * 32 + 8 * i + 4 * (lane >> 5);
    float v[4];
    finish4(a, unit, a.xd[min(tok, a.S - 1)], n, e, v);
    activate_all<4>(v, a.act);
    store_rows<TO>(a, tok, n, v);
}

/* ---- which form, and its shape ------------------------------------------- */

int64_t tiles_of(int32_t S, int32_t N, int rows, int toks)
{
    return (int64_t)((N + rows - 1) / rows) * ((S + toks - 1) / toks);
}

constexpr int kRowsTokens = 64;

bool use_rows(int32_t S, int32_t K)
{
    return S <= kRowsTokens || K < 128;
}

struct I8Plan {
    int shape, rows, toks, n_tiles, t_tiles, stages, splits;
    size_t total;
};

I8Plan plan_of(int32_t S, int32_t N, int32_t K)
{
    I8Plan p;
    p.stages = (K + kStageK - 1) / kStageK;
    p.shape = tiles_of(S, N, 256, 256) >= 256 ? 0 : tiles_of(S, N, 128, 128) >= 256 ? 1 : 2;
    p.rows = p.toks = p.shape == 0 ? 256 : p.shape == 1 ? 128 : 64;
    p.n_tiles = (N + p.rows - 1) / p.rows;
    p.t_tiles = (S + p.toks - 1) / p.toks;
    const int total = p.n_tiles * p.t_tiles;
    p.splits = p.shape == 2 ? std::max(1, std::min(512 / total, p.stages / 4)) : 1;
    p.total = p.splits > 1 ? (size_t)p.splits * total * p.rows * p.toks * 4 : 256;
    return p;
}

template <int BITS, int R, int T, int U, typename TO>
void launch_rows_w(const LinearI8Args& a, hipStream_t s)
{
    const int wgs = (a.N + 16 * R - 1) / (16 * R);
    const dim3 grid(wgs, (a.S + 16 * T - 1) / (16 * T));
    if (wgs >= 512)
        hipLaunchKernelGGL((i8_rows<BITS, R, T, 4, U, TO>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((i8_rows<BITS, R, T, 8, U, TO>), grid, dim3(512), 0, s, a);
}

template <int BITS, typename TO>
hipError_t launch_rows(const LinearI8Args& a, hipStream_t s)
{
    if (a.S <= 16) {
        if (a.N >= 16384)
            launch_rows_w<BITS, 2, 1, 2, TO>(a, s);
        else
            launch_rows_w<BITS, 1, 1, 4, TO>(a, s);
    } else if (a.S <= 32) {
        launch_rows_w<BITS, 2, 2, 2, TO>(a, s);
    } else {
        launch_rows_w<BITS, 2, 4, 1, TO>(a, s);
    }
    return hipGetLastError();
}

template <int BITS, int RR, int TT, int WR, int WT, int PER_CU, typename TO>
hipError_t launch_tiles(const LinearI8Args& a, const I8Plan& p, hipStream_t s)
{
    const I8TileArgs ta = {(int4*)a.ws, p.n_tiles, p.t_tiles, p.stages, p.splits};
    constexpr int bytes = TileShape<BITS, RR, TT, WR, WT>::kStage * kStages;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)i8_tiles<BITS, RR, TT, WR, WT, PER_CU, TO>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess)
            return e;
    }
    const int total = p.n_tiles * p.t_tiles;
    hipLaunchKernelGGL((i8_tiles<BITS, RR, TT, WR, WT, PER_CU, TO>), dim3((total * p.splits + 7) / 8 * 8),
                       dim3(WR * WT * 64), bytes, s, a, ta);
    if (p.splits > 1)
        hipLaunchKernelGGL((i8_join<RR, TT, WR, WT, TO>), dim3(total, RR * TT * 4), dim3(WR * WT * 64), 0, s, a, ta,
                           1.0f / (float)(1 << (8 - BITS)));
    return hipGetLastError();
}

template <int BITS, typename TO>
hipError_t launch(const LinearI8Args& a, hipStream_t s)
{
    if (use_rows(a.S, a.K))
        return launch_rows<BITS, TO>(a, s);
    const I8Plan p = plan_of(a.S, a.N, a.K);
    switch (p.shape) {
    case 0: return launch_tiles<BITS, 2, 4, 4, 2, 1, TO>(a, p, s);
    case 1: return launch_tiles<BITS, 2, 2, 2, 2, 2, TO>(a, p, s);
    default: return launch_tiles<BITS, 1, 1, 2, 2, 2, TO>(a, p, s);
    }
}

template <typename T>
hipError_t launch_quantize(const T* x, int64_t stride, int32_t rows, int32_t K, int8_t* q, float* d, hipStream_t s)
{
    const dim3 grid(rows);
    if (K <= 1024)
        hipLaunchKernelGGL((quantize_kernel<T, 256, 1>), grid, dim3(256), 0, s, x, stride, K, q, d);
    else if (K <= 2048)
        hipLaunchKernelGGL((quantize_kernel<T, 256, 2>), grid, dim3(256), 0, s, x, stride, K, q, d);
    else if (K <= 4096)
        hipLaunchKernelGGL((quantize_kernel<T, 256, 4>), grid, dim3(256), 0, s, x, stride, K, q, d);
    else if (K <= 8192)
        hipLaunchKernelGGL((quantize_kernel<T, 256, 8>), grid, dim3(256), 0, s, x, stride, K, q, d);
    else
        hipLaunchKernelGGL((quantize_kernel<T, 1024, 8>), grid, dim3(1024), 0, s, x, stride, K, q, d);
    return hipGetLastError();
}

} // namespace

hipError_t launch_quantize_i8(const void* x, int32_t type, int64_t stride, int32_t rows, int32_t K, int8_t* q, float* d,
                              hipStream_t s)
{
    return type == COLI_F32 ? launch_quantize((const float*)x, stride, rows, K, q, d, s)
                            : launch_quantize((const bf16*)x, stride, rows, K, q, d, s);
}

size_t linear_i8_workspace_need(int32_t S, int32_t N, int32_t K)
{
    return use_rows(S, K) ? 256 : plan_of(S, N, K).total;
}

/* The largest need of 1 .. S tokens: fewer tokens can be more splits of smaller
 * tiles.  The plan changes with every 64 tokens, and nothing is split from 256 tiles
 * of 128 x 128 on. */
size_t linear_i8_workspace_bytes(int32_t S, int32_t N, int32_t K)
{
    size_t most = linear_i8_workspace_need(S, N, K);
    if (use_rows(S, K))
        return most;
    const int ends = std::min((S + 63) / 64, 512 / (int)std::min<int64_t>(512, tiles_of(1, N, 128, 1)) + 1);
    for (int t = 1; t <= ends; ++t)
        most = std::max(most, linear_i8_workspace_need(std::min(S, 64 * t), N, K));
    return most;
}

hipError_t launch_linear_i8(const LinearI8Args& a, hipStream_t s)
{
    const bool f32 = a.out_type == COLI_F32;
    switch (a.qtype) {
    case COLI_Q8: return f32 ? launch<8, float>(a, s) : launch<8, bf16>(a, s);
    case COLI_Q4: return f32 ? launch<4, float>(a, s) : launch<4, bf16>(a, s);
    default: return f32 ? launch<2, float>(a, s) : launch<2, bf16>(a, s);
    }
}

} // namespace coli
