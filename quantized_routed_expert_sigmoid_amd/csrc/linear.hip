/*
 * linear.hip -- quantised matrix product of Q8_0 activations with bias,
 * activation and residual in its epilogue:
 *
 *   out[t][n] = act(sum_b s(n, b) d(t, b) sum_(k in b) w[n][k] q[t][k] + bias[n]) + residual[t][n]
 *
 * over 32-element blocks b, w and q small integers.  Three forms:
 *
 * - linear_rows_kernel, up to four tokens: the weights are read once and
 *   nothing else matters, so integer dot products on the VALU keep up.
 * - linear_fold, more tokens: the int8 matrix cores form the block products
 *   exactly, the VALU adds them in fp32 (a conversion and an fma per block and
 *   output, which bounds it: 32 VALU instructions, 128 cycles, beside 32 of the
 *   matrix core per 32 x 32 x 32 block).
 * - linear_tiles, bf16 outputs of very many tokens with one scale per row: the
 *   activations are written once as fp16 (linear_expand) and the fp16 matrix
 *   cores sum a whole row in fp32 with nothing to fold.  x = q d is scaled per
 *   token by a power of two and rounded to fp16, by up to 2^-11 of a value, an
 *   eighth of what the output's own rounding to bf16 takes; below fp16's normal
 *   range by up to 2^-25 of the scaled value, which is 2^-31 of the token's largest
 *   scale (127 of it lie above 2^13.98).  A weight code is exact.
 */
#include "block_device.h"

#include <algorithm>

namespace coli {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float activate(float v, int act)
{
    if (act == COLI_ACT_RELU) /* a NaN stays one */
        return v <= 0.0f ? 0.0f : v;
    if (act == COLI_ACT_SILU) /* the rounded exponent weighs 2^-23.4 |v|, power, sum, reciprocal and product 2^-21 */
        return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896340736f));
    if (act == COLI_ACT_GELU)
        return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v;
}

/* ---- few tokens ----------------------------------------------------------- */

/* Sum over the wave in lane 63, by lane moves within the VALU (device_common.h's
 * wave_reduce_u32 explains them). */
__device__ __forceinline__ float wave_sum63(float v)
{
#define COLI_ADD_DPP(ctrl, rows) \
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xF, false))
    COLI_ADD_DPP(0x111, 0xF);
    COLI_ADD_DPP(0x112, 0xF);
    COLI_ADD_DPP(0x114, 0xF);
    COLI_ADD_DPP(0x118, 0xF);
    COLI_ADD_DPP(0x142, 0xA);
    COLI_ADD_DPP(0x143, 0xC);
#undef COLI_ADD_DPP
    return v;
}

constexpr int kMaxRowsWg = 256; /* weight rows of a workgroup, most */

/*
 * A wave keeps the activations of up to T tokens in registers, NU units of a
 * weight row per lane (a unit: 16 bytes of an int8 or int4 row, 8 of an int2
 * row; unit 64 j + lane), and streams its rows past them, one row's loads
 * ahead of the products.  A unit lies inside one 32-element block, so its
 * exact integer dot product takes one pair of scales.  Rows longer than 64 NU
 * units go in several rounds, their sums kept in LDS.  Bound by the weights'
 * bytes: 1 x 10240 x 6144 int4 9.4 us with the weights in HBM (3.3 TB/s; 6.6 from the
 * last-level cache), 4 x 6144 x 8192 int8 with groups of 128 13.4 us (3.9 TB/s; 11.4).
 */
template <int BITS, int T, int NU, bool GROUPED, typename TO>
__global__ __launch_bounds__(256) void linear_rows_kernel(LinearArgs a, int rows_wg)
{
    constexpr int W = BITS == 2 ? 2 : 4;      /* words of a unit */
    constexpr int UK = W * 32 / BITS;         /* its codes: 16, 32, 32 */
    constexpr int X = BITS == 8 ? 4 : 8;      /* its activation words */
    __shared__ float sums[kMaxRowsWg][T];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int n0 = blockIdx.x * rows_wg, n1 = min(n0 + rows_wg, a.N), t0 = blockIdx.y * T;
    const int nb = a.K / 32, units = a.K / UK, gpr = GROUPED ? a.K / a.group : 1;
    const uint32_t* w = (const uint32_t*)a.w;

    for (int u0 = 0; u0 < units; u0 += 64 * NU) {
        uint32_t xa[T][NU][X];
        float xd[T][NU];
        int at[NU], grp[NU];
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int u = u0 + 64 * j + lane;
            at[j] = min(u, units - 1);
            if constexpr (GROUPED)
                grp[j] = at[j] * UK / a.group;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int64_t tok = min(t0 + t, a.S - 1);
                const uint32_t* x = (const uint32_t*)(a.xq + tok * a.K + (int64_t)at[j] * UK);
                xd[t][j] = u < units ? a.xd[tok * nb + at[j] * UK / 32] : 0.0f;
                if constexpr (BITS == 8) {
                    const uint4 v = *(const uint4*)x;
                    xa[t][j][0] = v.x;
                    xa[t][j][1] = v.y;
                    xa[t][j][2] = v.z;
                    xa[t][j][3] = v.w;
                } else {
                    const uint4 lo = *(const uint4*)x, hi = *(const uint4*)(x + 4);
                    const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    prep_dot<BITS>(v, xa[t][j]);
                }
            }
        }
        uint32_t wb[2][NU][W];
        float ws[2][GROUPED ? NU : 1];
        auto load = [&](int n, int p) {
            const int64_t row = min(n, n1 - 1);
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const uint32_t* q = w + (row * units + at[j]) * W;
                if constexpr (W == 4) {
                    const uint4 v = *(const uint4*)q;
                    wb[p][j][0] = v.x;
                    wb[p][j][1] = v.y;
                    wb[p][j][2] = v.z;
                    wb[p][j][3] = v.w;
                } else {
                    const uint2 v = *(const uint2*)q;
                    wb[p][j][0] = v.x;
                    wb[p][j][1] = v.y;
                }
                if constexpr (GROUPED)
                    ws[p][j] = a.w_scale[row * gpr + grp[j]];
            }
        };
        auto row = [&](int n, int p) {
            float acc[T];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                acc[t] = 0.0f;
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    int32_t s = 0;
                    if constexpr (BITS == 8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s = COLI_SDOT4(wb[p][j][i], xa[t][j][i], s);
                    } else {
                        s = block_dot<BITS>(wb[p][j], xa[t][j]);
                    }
                    const float d = GROUPED ? xd[t][j] * ws[p][GROUPED ? j : 0] : xd[t][j];
                    acc[t] = __builtin_fmaf(d, (float)s, acc[t]);
                }
                acc[t] = wave_sum63(acc[t]);
            }
            if (lane == 63 && n < n1) {
#pragma unroll
                for (int t = 0; t < T; ++t)
                    sums[n - n0][t] = u0 ? sums[n - n0][t] + acc[t] : acc[t];
            }
        };
        load(n0 + wv, 0);
        for (int n = n0 + wv; n < n1; n += 8) {
            load(n + 4, 1);
            row(n, 0);
            load(n + 8, 0);
            row(n + 4, 1);
        }
    }
    __syncthreads();
    /* rows of one token together, as they are stored */
    for (int i = threadIdx.x; i < rows_wg * T; i += 256) {
        const int t = t0 + i / rows_wg, n = n0 + i % rows_wg;
        if (n >= n1 || t >= a.S)
            continue;
        const int64_t o = (int64_t)t * a.N + n;
        const float v = sums[n - n0][i / rows_wg];
        float y = activate(__builtin_fmaf(v, GROUPED ? 1.0f : a.w_scale[n], a.bias ? a.bias[n] : 0.0f), a.act);
        if (a.residual)
            y += to_f32(((const TO*)a.residual)[o]);
        store1((TO*)a.out + o, y);
    }
}

/* Rows of a workgroup: one workgroup per CU, or more in equal shares.  Each
 * wave reads the activations once, so few long runs of rows are better (S = 4,
 * N = 6144, K = 8192, int8: 11.5 us with 24 rows, 16.4 with 12). */
inline int rows_per_wg(int N)
{
    int shares = 256;
    while (N / shares >= 32 && shares < (1 << 20))
        shares *= 2;
    return std::max(4, std::min(kMaxRowsWg, (N + shares - 1) / shares));
}

template <int BITS, int T, int NU, typename TO>
void launch_rows_nu(const LinearArgs& a, hipStream_t s)
{
    const int r = rows_per_wg(a.N);
    const dim3 grid((a.N + r - 1) / r, (a.S + T - 1) / T);
    if (a.group)
        hipLaunchKernelGGL((linear_rows_kernel<BITS, T, NU, true, TO>), grid, dim3(256), 0, s, a, r);
    else
        hipLaunchKernelGGL((linear_rows_kernel<BITS, T, NU, false, TO>), grid, dim3(256), 0, s, a, r);
}

template <int BITS, int T, typename TO>
void launch_rows_t(const LinearArgs& a, hipStream_t s)
{
    /* units per lane of a round: up to K = 2048, 4096 or 8192 */
    constexpr int per = BITS == 8 ? 2 : 1;
    const int need = (a.K / 32 + 63) / 64;
    if (need <= 1)
        launch_rows_nu<BITS, T, 1 * per, TO>(a, s);
    else if (need <= 2)
        launch_rows_nu<BITS, T, 2 * per, TO>(a, s);
    else if (need == 3)
        launch_rows_nu<BITS, T, 3 * per, TO>(a, s);
    else
        launch_rows_nu<BITS, T, 4 * per, TO>(a, s);
}

template <int BITS, typename TO>
hipError_t launch_rows(const LinearArgs& a, hipStream_t s)
{
    if (a.S == 1)
        launch_rows_t<BITS, 1, TO>(a, s);
    else if (a.S == 2)
        launch_rows_t<BITS, 2, TO>(a, s);
    else
        launch_rows_t<BITS, 4, TO>(a, s);
    return hipGetLastError();
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
 * Activations as fp16 operands: [step][tile of 32 tokens][chunk of 8 k][token] of 16 bytes, so that
 * a wave's operand load is one run of 1 KB.  Steps past the row's end cover k = K - 64 .. K - 1; what an
 * earlier step has covered already is zero in them, as are tokens from S on.  A workgroup takes a tile of 32 tokens and
 * per steps: eight threads find a token's largest scale, then 32 threads write the tokens of one
 * chunk as a run of 512 bytes.
 */
template <int BITS>
__global__ __launch_bounds__(256) void linear_expand(LinearArgs a, uint8_t* xh, float* xs, int tiles, int steps, int per)
{
    __shared__ float up_of[kTileTok];
    const int tile = blockIdx.x, step0 = blockIdx.y * per, nb = a.K / 32;
    {
        const int t = tile * kTileTok + (threadIdx.x >> 3);
        const float* d = a.xd + (int64_t)min(t, a.S - 1) * nb;
        float top = 0.0f;
        for (int b = threadIdx.x & 7; b < nb; b += 8)
            top = fmaxf(top, fabsf(d[b]));
        top = fmaxf(top, shfl_xor(top, 1));
        top = fmaxf(top, shfl_xor(top, 2));
        top = fmaxf(top, shfl_xor(top, 4));
        /* 2^e > 127 top, so |x| 2^(15 - e) < 2^15 */
        int e = 0;
        if (top > 0.0f)
            (void)frexpf(top, &e);
        e = max(e + 7, -111); /* 2^(15 - e) stays finite */
        if ((threadIdx.x & 7) == 0) {
            up_of[threadIdx.x >> 3] = top > 0.0f ? ldexpf(1.0f, 15 - e) : 0.0f;
            if (step0 == 0 && t < a.S)
                xs[t] = ldexpf(1.0f, e - 15);
        }
    }
    __syncthreads();
    const int t = tile * kTileTok + (threadIdx.x & 31);
    const bool live = t < a.S;
    const float* d = a.xd + (int64_t)min(t, a.S - 1) * nb;
    const int8_t* q = a.xq + (int64_t)min(t, a.S - 1) * a.K;
    const float up = live ? up_of[threadIdx.x & 31] : 0.0f;
    const int c = threadIdx.x >> 5;
    for (int step = step0; step < min(step0 + per, steps); ++step) {
        const int at = min(step * kKB, a.K - kKB) + c * 8;
        const uint2 w = *(const uint2*)(q + at);
        const float s = at >= step * kKB ? d[at >> 5] * up : 0.0f;
        v8h x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k_order<BITS>(i);
            x[i] = (_Float16)((float)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3))) * s);
        }
        *(v8h*)(xh + ((((int64_t)step * tiles + tile) * 8 + c) * kTileTok + (threadIdx.x & 31)) * kChunk) = x;
    }
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

/* Where a wave's part of a tile lies: rows n0 + 32 r, tokens tok0 + 32 t; lane
 * (col = l % 32, h = l / 32) of a 32 x 32 part holds token col and the rows 8 (i
 * / 4) + 4 h + i % 4 of accumulator register i. */
struct TileAt {
    int n0, tok0;
};

/* Tile id of a grid of n_tiles x t_tiles tiles of ROWS rows x TOKS tokens: bands
 * of eight token tiles, column by column of weight tiles, so that neighbours
 * share operands. */
template <int ROWS, int TOKS>
__device__ __forceinline__ TileAt tile_at(int id, int n_tiles, int t_tiles)
{
    constexpr int GT = 8;
    const int band = id / (GT * n_tiles), in = id % (GT * n_tiles), wide = min(GT, t_tiles - band * GT);
    return TileAt{in / wide * ROWS, (band * GT + in % wide) * TOKS};
}

/* One uniform branch on the activation for N values. */
template <int N>
__device__ __forceinline__ void activate_all(float* v, int act)
{
    if (act == COLI_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = activate(v[i], COLI_ACT_RELU);
    } else if (act == COLI_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = activate(v[i], COLI_ACT_SILU);
    } else if (act == COLI_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = activate(v[i], COLI_ACT_GELU);
    }
}

/* Residual and store of four consecutive rows n .. n + 3 of a token. */
template <typename TO>
__device__ __forceinline__ void store_rows(const LinearArgs& a, int tok, int n, const float* v)
{
    if (tok >= a.S || n >= a.N)
        return;
    TO* out = (TO*)a.out + (int64_t)tok * a.N + n;
    const TO* res = a.residual ? (const TO*)a.residual + (int64_t)tok * a.N + n : nullptr;
    if (n + 4 <= a.N) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        if (res)
            r = load4_any(res);
        store4_any(out, make_float4(v[0] + r.x, v[1] + r.y, v[2] + r.z, v[3] + r.w));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < a.N)
                store1(out + j, v[j] + (res ? to_f32(res[j]) : 0.0f));
    }
}

/* What the tile kernels take of a launch. */
struct TileArgs {
    const uint8_t* xh; /* linear_tiles: the expanded activations and their scales */
    const float* xs;
    float* part; /* linear_fold: [split][tile][wave][r][t][i / 4][lane] of four sums */
    int tiles, n_tiles, t_tiles, stages, splits;
};

/*
 * A workgroup of 2 x 2 waves takes 128 weight rows x 256 tokens, a wave 64 rows
 * x 128 tokens of them (2 x 4 tiles of v_mfma_f32_32x32x16_f16), in steps of 64
 * k: the next step's operands travel from memory to LDS under this step's
 * products, 36 KB of an int4 step, so that two workgroups share a CU.  Weights
 * stay packed in LDS and are unpacked by the waves that multiply them.  Lane
 * (l % 32, h = l / 32) of instruction i of a step takes k = 16 i + 8 h .. + 7.
 * Measured: 4096 x 10240 x 6144 int4 460 us and 23 us of linear_expand, 1.07
 * PFLOP/s (a bf16 library product of 8192^3: 1.45); without the unpacking 65 us
 * less; the matrix cores are busy half of the time, at 1.9 GHz.
 */
constexpr int kTileTT = 4;

template <int BITS>
struct TileLds {
    static constexpr int kX = 2 * kTileTT * 8 * kTileTok * kChunk, kW = kTileN * (BITS / 2) * kChunk;
    static constexpr int kStage = kX + kW;
};

template <int BITS>
__global__ __launch_bounds__(256, 2) void linear_tiles(LinearArgs a, TileArgs ta)
{
    using L = TileLds<BITS>;
    constexpr int TT = kTileTT, XB = L::kX, LPR = BITS / 2; /* 16-byte chunks of a row's step */
    constexpr int kWRuns = L::kW / 1024;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, wv = wave_of(), h = lane >> 5, col = lane & 31;
    const int wn = wv & 1, wt = wv >> 1;
    const int unit = (int)xcd_unit();
    if (unit >= ta.n_tiles * ta.t_tiles)
        return;
    const TileAt wg = tile_at<kTileN, 64 * TT>(unit, ta.n_tiles, ta.t_tiles);
    const TileAt at = {wg.n0 + wn * 64, wg.tok0 + wt * TT * kTileTok};
    const int64_t row_bytes = (int64_t)a.K * BITS / 8;
    const uint8_t* w = (const uint8_t*)a.w;
    /* Chunk c of row n of a stage lies in LDS slot c ^ f(n) of the row's LPR, so
     * that 16 rows' reads of one chunk fall into different banks. */
    constexpr int RPB = LPR >= 16 ? 1 : 16 / LPR;
    auto swz = [](int n) { return n / RPB % LPR; };

    /* where the weights are fewer runs than waves, waves load the same one */
    constexpr int kWMine = (kWRuns + 3) / 4;
    const uint32_t lds0 = lds_address(lds);
    const uint8_t* w0 = w + wg.n0 * row_bytes;
    uint32_t woff[kWMine];
#pragma unroll
    for (int i = 0; i < kWMine; ++i) {
        const int slot = (i * 4 + wv) % kWRuns * 64 + lane, n = slot / LPR, c = slot % LPR ^ swz(n);
        woff[i] = (uint32_t)(min(n, a.N - 1 - wg.n0) * (int)row_bytes + c * kChunk);
    }
    auto fetch = [&](int step) {
        const uint32_t buf = lds0 + (step & 1) * L::kStage;
        step = min(step, ta.stages - 1); /* past the end: loaded and not used */
        const uint8_t* x = ta.xh + ((int64_t)step * ta.tiles + wg.tok0 / kTileTok) * (8 * kTileTok * kChunk);
#pragma unroll
        for (int i = 0; i < XB / 4096; ++i) {
            const int o = (i * 4 + wv) * 1024;
            to_lds(x + o, lane * 16, buf + o);
        }
        const int64_t kb = (int64_t)min(step * kKB, a.K - kKB) * BITS / 8;
#pragma unroll
        for (int i = 0; i < kWMine; ++i)
            to_lds(w0 + kb, woff[i], buf + XB + (i * 4 + wv) % kWRuns * 1024);
    };

    v16f acc[2][TT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[r][t][i] = 0.0f;

    fetch(0);
    for (int step = 0; step < ta.stages; ++step) {
        arrive_all<0>();
        fetch(step + 1);
        const uint8_t* buf = lds + (step & 1) * L::kStage;
        /* Instruction i multiplies what was read two and unpacked one
         * instruction ago, so that reads and unpacking run in the shadow of the
         * matrix cores. */
        uint2 wraw[2][2];
        v8h xf[2][TT], wf[2][2];
        auto read_w = [&](int i) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int n = wn * 64 + r * 32 + col;
                const uint8_t* p = buf + XB + n * (LPR * kChunk);
                auto slot = [&](int c) { return (c ^ swz(n)) * kChunk; };
                if constexpr (BITS == 8)
                    wraw[i & 1][r] = *(const uint2*)(p + slot(i) + h * 8);
                else if constexpr (BITS == 4)
                    wraw[i & 1][r].x = *(const uint32_t*)(p + slot(i >> 1) + (i & 1) * 8 + h * 4);
                else
                    wraw[i & 1][r].x = *(const uint32_t*)(p + slot(0) + i * 4);
            }
        };
        auto read_x = [&](int i) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                xf[i & 1][t] = *(const v8h*)(buf + ((wt * TT + t) * 8 + 2 * i) * (kTileTok * kChunk) + lane * 16);
        };
        auto unpack = [&](int i) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint2 v = wraw[i & 1][r];
                if constexpr (BITS == 2)
                    wf[i & 1][r] = codes_f16<2>(__builtin_amdgcn_perm(0, v.x, h ? 0x0C030C02u : 0x0C010C00u), 0);
                else
                    wf[i & 1][r] = codes_f16<BITS>(v.x, v.y);
            }
        };
        read_w(0);
        read_x(0);
        read_w(1);
        unpack(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i + 1 < 4) {
                read_x(i + 1);
                unpack(i + 1);
            }
            if (i + 2 < 4)
                read_w(i + 2);
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wf[i & 1][r], xf[i & 1][t], acc[r][t], 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 2 * TT; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); /* a matrix instruction, */
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0); /* an LDS read and */
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0); /* four VALU under it */
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); /* no load outlives the workgroup's LDS */
    float v[2][TT][16], xscale[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        xscale[t] = ta.xs[min(at.tok0 + t * kTileTok + col, a.S - 1)];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = min(at.n0 + r * 32 + 8 * (i / 4) + 4 * h + i % 4, a.N - 1);
            const float ws = a.w_scale[n], bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
            for (int t = 0; t < TT; ++t)
                v[r][t][i] = __builtin_fmaf(acc[r][t][i], xscale[t] * ws, bias);
        }
    activate_all<2 * TT * 16>(&v[0][0][0], a.act);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store_rows<bf16>(a, at.tok0 + t * kTileTok + col, at.n0 + r * 32 + 8 * i + 4 * h, &v[r][t][4 * i]);
}

/*
 * The same product on the int8 matrix cores, exact up to the fp32 fold: one
 * v_mfma_i32_32x32x32_i8 is one 32-element block of 32 rows x 32 tokens, its
 * result times the token's scale is added in fp32 (with group scales, into the
 * group's sum).  A wave takes 32 RR rows x 32 TT tokens, the workgroup's four
 * waves WN x 4 / WN of these, in stages of four blocks; weights and codes
 * travel packed from memory to LDS one stage ahead.  Codes of fewer bits are
 * unpacked to the top of their bytes, 2^(8 - bits) times their value, which
 * the row's scale takes out again.  Measured: 2048 x 4096 x 4096 int4, fp32 out,
 * 88 us (780 TFLOP/s; the VALU's limit is 1.26 P), with groups of 128 112 us; 16 x
 * 10240 x 6144 int4 17 us with the weights in HBM (15 from the last-level cache), bound
 * by the latency of its stages.
 */
constexpr int kStageK = 128;

/* A lane's sixteen codes of a block as they lie in LDS, and as int8. */
template <int BITS>
struct RawCodes {
    uint32_t w[BITS / 2];
};

template <int BITS>
__device__ __forceinline__ RawCodes<BITS> read_codes(const uint8_t* p, int half, int h)
{
    RawCodes<BITS> r;
    if constexpr (BITS == 8) {
        const uint4 v = *(const uint4*)p;
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else if constexpr (BITS == 4) {
        const uint2 v = *(const uint2*)(p + h * 8);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
        r.w[0] = *(const uint32_t*)(p + half * 8 + h * 4);
    }
    return r;
}

template <int BITS>
__device__ __forceinline__ v4i codes_i8(const RawCodes<BITS>& r)
{
    if constexpr (BITS == 8) {
        return v4i{(int)r.w[0], (int)r.w[1], (int)r.w[2], (int)r.w[3]};
    } else if constexpr (BITS == 4) {
        const uint32_t e0 = r.w[0] & 0xF0F0F0F0u, o0 = (r.w[0] << 4) & 0xF0F0F0F0u;
        const uint32_t e1 = r.w[1] & 0xF0F0F0F0u, o1 = (r.w[1] << 4) & 0xF0F0F0F0u;
        return v4i{(int)__builtin_amdgcn_perm(o0, e0, 0x05010400u), (int)__builtin_amdgcn_perm(o0, e0, 0x07030602u),
                   (int)__builtin_amdgcn_perm(o1, e1, 0x05010400u), (int)__builtin_amdgcn_perm(o1, e1, 0x07030602u)};
    } else {
        /* byte j of the word holds elements 4 j .. 4 j + 3, the first in bits 7..6 */
        const uint32_t w = r.w[0];
        const uint32_t a = w & 0xC0C0C0C0u, b = (w << 2) & 0xC0C0C0C0u, c = (w << 4) & 0xC0C0C0C0u,
                       d = (w << 6) & 0xC0C0C0C0u;
        const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
        const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
        return v4i{(int)__builtin_amdgcn_perm(cd0, ab0, 0x05040100u), (int)__builtin_amdgcn_perm(cd0, ab0, 0x07060302u),
                   (int)__builtin_amdgcn_perm(cd1, ab1, 0x05040100u), (int)__builtin_amdgcn_perm(cd1, ab1, 0x07060302u)};
    }
}

template <int RR, int TT, int WN>
struct FoldShape {
    static constexpr int kRows = 32 * RR * WN, kTok = 32 * TT * (4 / WN);
};

/* LDS of a stage: codes, weights, the tokens' scales, the groups'; and the stages in flight, as many as
 * leave room for two workgroups in a CU's 160 KB. */
template <int BITS, int RR, int TT, int WN, int GROUPED>
struct FoldLds {
    using F = FoldShape<RR, TT, WN>;
    static constexpr int kX = F::kTok * kStageK, kW = F::kRows * kStageK * BITS / 8;
    static constexpr int kRunsD = (F::kTok * kChunk + 1023) / 1024;
    /* row scales of each block's group (GROUPED 1), or of the stage's (2) */
    static constexpr int kScales = GROUPED == 0 ? 0 : GROUPED == 1 ? 4 : 1, kS = kScales * WN * 256;
    static constexpr int kStage = kX + kW + kRunsD * 1024 + kS;
    static constexpr int kFit = 79 * 1024 / kStage;
    static constexpr int kStages = kFit < 2 ? 2 : kFit > 3 ? 3 : kFit;
    /* loads of a wave and stage; where there are fewer runs than waves, waves
     * load the same one, so that every wave counts alike */
    static constexpr int kLoads = kX / 4096 + (kW + 4095) / 4096 + 1 + kScales;
};

template <int BITS, int RR, int TT, int WN, int GROUPED, typename TO>
__global__ __launch_bounds__(256, 2) void linear_fold(LinearArgs a, TileArgs ta)
{
    constexpr int XC = kStageK / kChunk;       /* chunks of a token's stage */
    constexpr int WC = kStageK * BITS / 128;   /* chunks of a row's stage: 8, 4, 2 */
    using F = FoldShape<RR, TT, WN>;
    using L = FoldLds<BITS, RR, TT, WN, GROUPED>;
    constexpr int XB = L::kX, WB = L::kW, SB = L::kStage - L::kS, STAGES = L::kStages;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63, wv = wave_of(), h = lane >> 5, col = lane & 31;

    const int unit = (int)xcd_unit(), total = ta.n_tiles * ta.t_tiles;
    if (unit >= total * ta.splits)
        return;
    const int id = unit / ta.splits, split = unit % ta.splits;
    const TileAt wg = tile_at<F::kRows, F::kTok>(id, ta.n_tiles, ta.t_tiles);
    const TileAt at = {wg.n0 + wv % WN * 32 * RR, wg.tok0 + wv / WN * 32 * TT};
    const int share = (ta.stages + ta.splits - 1) / ta.splits;
    const int s0 = split * share, s1 = min(s0 + share, ta.stages);
    const int nb = a.K / 32, gpr = GROUPED ? a.K / a.group : 1, gb = GROUPED ? a.group / 32 : 1;
    const int64_t row_bytes = (int64_t)a.K * BITS / 8;

    /* Slot s of a token's or row's chunks holds chunk s ^ f, so that 16 of them
     * read at one chunk fall into different banks.  Chunks past the row's end
     * are its last one: their blocks' scales are taken as 0. */
    auto xswz = [](int t) { return t / 2 % 8; };
    auto wswz = [](int n) { return n / (16 / WC) % WC; };
    constexpr int kXMine = XB / 4096, kWMine = (WB + 4095) / 4096;
    const uint32_t lds0 = lds_address(lds);
    const uint8_t* w0 = (const uint8_t*)a.w + wg.n0 * row_bytes;
    const int8_t* x0 = a.xq + (int64_t)wg.tok0 * a.K;
    const float* d0 = a.xd + (int64_t)wg.tok0 * nb;
    const float* s_0 = a.w_scale + (int64_t)wg.n0 * gpr;
    /* this lane's row and chunk of each of its runs */
    int xrow[kXMine], xchunk[kXMine], wrow[kWMine], wchunk[kWMine];
#pragma unroll
    for (int i = 0; i < kXMine; ++i) {
        const int slot = (i * 4 + wv) * 64 + lane, t = slot / XC;
        xrow[i] = min(t, a.S - 1 - wg.tok0) * a.K;
        xchunk[i] = (slot % XC ^ xswz(t)) * kChunk;
    }
#pragma unroll
    for (int i = 0; i < kWMine; ++i) {
        const int slot = (i * 4 + wv) % (WB / 1024) * 64 + lane, n = slot / WC;
        wrow[i] = min(n, a.N - 1 - wg.n0) * (int)row_bytes;
        wchunk[i] = (slot % WC ^ wswz(n)) * kChunk;
    }
    const int drun = wv % L::kRunsD;
    const uint32_t doff = (uint32_t)min(drun * 64 + lane, a.S - 1 - wg.tok0) * nb * 4;
    const uint32_t soff = (uint32_t)(min(at.n0 + lane % (32 * RR), a.N - 1) - wg.n0) * gpr * 4;
    auto fetch = [&](int stage) {
        const uint32_t buf = lds0 + (stage - s0) % STAGES * L::kStage;
        stage = min(stage, ta.stages - 1); /* past the end: loaded and not used */
        const int xk = stage * kStageK, xb = min(xk, a.K - kChunk);
#pragma unroll
        for (int i = 0; i < kXMine; ++i)
            to_lds(x0 + xb, xrow[i] + min(xk + xchunk[i], a.K - kChunk) - xb, buf + (i * 4 + wv) * 1024);
        const int wk = stage * WC * kChunk, wlast = (int)row_bytes - kChunk, wb = min(wk, wlast);
#pragma unroll
        for (int i = 0; i < kWMine; ++i)
            to_lds(w0 + wb, wrow[i] + min(wk + wchunk[i], wlast) - wb, buf + XB + (i * 4 + wv) % (WB / 1024) * 1024);
        /* the four scales of each token's stage, at a row's end its last four */
        to_lds(d0 + min(stage * 4, nb - 4), doff, buf + XB + WB + drun * 1024);
        if constexpr (GROUPED) {
#pragma unroll
            for (int b = 0; b < L::kScales; ++b)
                word_to_lds(s_0 + min(stage * 4 + b, nb - 1) / gb, soff, buf + SB + (b * WN + wv % WN) * 256);
        }
    };

    float acc[RR][TT][16], part[GROUPED ? RR : 1][GROUPED ? TT : 1][16];
#pragma unroll
    for (int r = 0; r < RR; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[r][t][i] = 0.0f;
                if constexpr (GROUPED)
                    part[r][t][i] = 0.0f;
            }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        fetch(s0 + i);
    for (int stage = s0; stage < s1; ++stage) {
        /* all but the loads of the STAGES - 2 stages behind this one */
        arrive_all<L::kLoads*(STAGES - 2)>();
        fetch(stage + STAGES - 1);
        const uint8_t* buf = lds + (stage - s0) % STAGES * L::kStage;
        float d[TT][4];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float4 v = *(const float4*)(buf + XB + WB + (at.tok0 - wg.tok0 + t * 32 + col) * kChunk);
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int b = 0; b < 4; ++b)
                d[t][b] = e[b];
            const int over = stage * 4 + 4 - nb; /* blocks of the last stage past the row's end */
            if (over > 0) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    d[t][b] = b + over < 4 ? e[b + over < 4 ? b + over : 3] : 0.0f;
            }
        }
        /* the whole stage's operands are read ahead of its products */
        RawCodes<BITS> wr[4][RR];
        v4i xf[4][TT];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const int n = at.n0 - wg.n0 + r * 32 + col;
                const int c = BITS == 8 ? 2 * b + h : BITS == 4 ? b : b / 2;
                /* an odd last block of an int2 row was loaded with the block before it */
                const int half = BITS == 2 && stage * 4 + b == nb - 1 && (nb & 1) ? 1 : b & 1;
                wr[b][r] = read_codes<BITS>(buf + XB + (n * WC + (c ^ wswz(n))) * kChunk, half, h);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int tok = at.tok0 - wg.tok0 + t * 32 + col;
                xf[b][t] = *(const v4i*)(buf + (tok * XC + ((2 * b + h) ^ xswz(tok))) * kChunk);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        /* the product of one tile runs under the fold of the one before it */
        v16i z[2];
        auto fold = [&](int m) {
            const int b2 = m / (RR * TT), r = m / TT % RR, t = m % TT;
            float* o = GROUPED ? part[GROUPED ? r : 0][GROUPED ? t : 0] : acc[r][t];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = __builtin_fmaf((float)z[m & 1][i], d[t][b2], o[i]);
        };
        /* after block b: where its group ends (or the range does, which is no
         * harm inside a group) the group's sums take their rows' scales */
        auto close = [&](int b) {
            if (GROUPED == 2 && b < 3)
                return;
            const int blk = stage * 4 + b;
            if ((blk + 1) % gb && (b < 3 || stage + 1 < s1))
                return;
            const float* words = (const float*)(buf + SB + (b % (GROUPED == 1 ? 4 : 1) * WN + wv % WN) * 256);
#pragma unroll
            for (int r = 0; r < RR; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = *(const float4*)(words + r * 32 + 8 * q + 4 * h);
                    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            float& p = part[GROUPED ? r : 0][GROUPED ? t : 0][4 * q + j];
                            acc[r][t][4 * q + j] = __builtin_fmaf(p, e[j], acc[r][t][4 * q + j]);
                            p = 0.0f;
                        }
                }
        };
        v4i wf[RR];
#pragma unroll
        for (int m = 0; m < 4 * RR * TT; ++m) {
            const int b = m / (RR * TT), r = m / TT % RR, t = m % TT;
            if (t == 0)
                wf[r] = codes_i8<BITS>(wr[b][r]);
            const v16i zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
            z[m & 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[r], xf[b][t], zero, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (m)
                fold(m - 1);
            if constexpr (GROUPED)
                if (m && m % (RR * TT) == 0)
                    close(b - 1);
        }
        fold(4 * RR * TT - 1);
        if constexpr (GROUPED)
            close(3);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); /* no load outlives the workgroup's LDS */
    constexpr float unit_w = 1.0f / (float)(1 << (8 - BITS));
    if (ta.splits == 1) {
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int n = min(at.n0 + r * 32 + 8 * (i / 4) + 4 * h + i % 4, a.N - 1);
                const float ws = GROUPED ? unit_w : unit_w * a.w_scale[n], bias = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[r][t][i] = __builtin_fmaf(acc[r][t][i], ws, bias);
            }
        activate_all<RR * TT * 16>(&acc[0][0][0], a.act);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int r = 0; r < RR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_rows<TO>(a, at.tok0 + t * 32 + col, at.n0 + r * 32 + 8 * i + 4 * h, &acc[r][t][4 * i]);
        return;
    }
    float4* o = (float4*)ta.part + (((int64_t)split * total + id) * 4 + wv) * (RR * TT * 4 * 64) + lane;
#pragma unroll
    for (int r = 0; r < RR; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[((r * TT + t) * 4 + i) * 64] =
                    make_float4(acc[r][t][4 * i], acc[r][t][4 * i + 1], acc[r][t][4 * i + 2], acc[r][t][4 * i + 3]);
}

/* Adds the splits' sums in their order and finishes them: a workgroup takes
 * one of a tile's groups of four rows, in the fold kernel's layout. */
template <int RR, int TT, int WN, typename TO>
__global__ __launch_bounds__(256) void linear_join(LinearArgs a, TileArgs ta, float unit_w)
{
    using F = FoldShape<RR, TT, WN>;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, total = ta.n_tiles * ta.t_tiles;
    const int id = blockIdx.x, q = blockIdx.y, i = q & 3, t = (q >> 2) % TT, r = (q >> 2) / TT;
    const float4* o = (const float4*)ta.part + (((int64_t)id * 4 + wv) * (RR * TT * 4) + q) * 64 + lane;
    const int64_t step = (int64_t)total * 4 * (RR * TT * 4) * 64;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < ta.splits; ++s) {
        const float4 x = o[s * step];
        v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
    const TileAt wg = tile_at<F::kRows, F::kTok>(id, ta.n_tiles, ta.t_tiles);
    const int tok = wg.tok0 + wv / WN * 32 * TT + t * 32 + (lane & 31);
    const int n = wg.n0 + wv % WN * 32 * RR + r * 32 + 8 * i + 4 * (lane >> 5);
    float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int m = min(n + j, a.N - 1);
        e[j] = __builtin_fmaf(e[j], a.group ? unit_w : unit_w * a.w_scale[m], a.bias ? a.bias[m] : 0.0f);
    }
    activate_all<4>(e, a.act);
    store_rows<TO>(a, tok, n, e);
}

/* ---- which form, and its shape ------------------------------------------- */

int64_t n_tiles_of(int32_t S, int32_t N, int rows, int toks)
{
    return (int64_t)((N + rows - 1) / rows) * ((S + toks - 1) / toks);
}

/* linear_rows_kernel's weight reads are the whole cost up to four tokens (S = 4,
 * N = 10240, K = 6144, int4: 11.1 us against 15.7 on the matrix cores; S = 8:
 * 17.4 against 15.7); shorter rows than a stage of the fold stay with it. */
bool use_rows(int32_t S, int32_t K)
{
    return S <= 4 || K < kStageK;
}

/* linear_tiles pays for the expansion where every CU has two of its tiles or
 * more (int4, bf16: 4096 x 10240 x 6144 490 us against 586 on the int8 cores;
 * 2048 x 4096 x 4096, one tile a CU, 94 against 86 to 93). */
bool use_tiles(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type)
{
    return !use_rows(S, K) && out_type == COLI_BF16 && !group && n_tiles_of(S, N, kTileN, 64 * kTileTT) >= 512;
}

struct TilePlan {
    int tiles, n_tiles, t_tiles, stages;
    size_t x_bytes, total;
};

TilePlan tile_plan(int32_t S, int32_t N, int32_t K)
{
    TilePlan p;
    p.n_tiles = (N + kTileN - 1) / kTileN;
    p.t_tiles = (S + 64 * kTileTT - 1) / (64 * kTileTT);
    p.tiles = p.t_tiles * 2 * kTileTT;
    p.stages = (K + kKB - 1) / kKB;
    p.x_bytes = (size_t)p.stages * p.tiles * 8 * kTileTok * kChunk;
    p.total = (p.x_bytes + (size_t)S * 4 + 255) / 256 * 256;
    return p;
}

template <int BITS>
hipError_t launch_tiles(const LinearArgs& a, hipStream_t s)
{
    const TilePlan p = tile_plan(a.S, a.N, a.K);
    TileArgs ta = {};
    uint8_t* xh = (uint8_t*)a.ws;
    float* xs = (float*)(xh + p.x_bytes);
    ta.xh = xh;
    ta.xs = xs;
    ta.tiles = p.tiles;
    ta.n_tiles = p.n_tiles;
    ta.t_tiles = p.t_tiles;
    ta.stages = p.stages;
    const int per = std::max(1, std::min(8, p.tiles * p.stages / 512));
    hipLaunchKernelGGL((linear_expand<BITS>), dim3(p.tiles, (p.stages + per - 1) / per), dim3(256), 0, s, a, xh, xs,
                       p.tiles, p.stages, per);
    constexpr int bytes = 2 * TileLds<BITS>::kStage;
    const hipError_t e = hipFuncSetAttribute((const void*)linear_tiles<BITS>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((linear_tiles<BITS>), dim3((p.n_tiles * p.t_tiles + 7) / 8 * 8), dim3(256), bytes, s, a, ta);
    return hipGetLastError();
}

/* Shapes of the fold kernel, rows and tokens of a workgroup: 128 x 128 where
 * every CU gets one, else 64 x 64 (S = 512, N = K = 4096, int4: 33.4 us, 39.2 with
 * 128 x 128), for up to 32 tokens 128 x 32.  A scale group's own sums take as many
 * registers again, so 128 x 128 is 128 x 64 with groups.  With fewer tiles than 512 the
 * stages are shared out as well, two at least each, and linear_join adds the
 * parts (S = 64, N = 10240, K = 6144, int8: 21.4 us against 30.6 with one
 * workgroup per CU). */
struct FoldPlan {
    int shape, rows, toks, n_tiles, t_tiles, stages, splits;
    size_t total;
};

constexpr int kWantTiles = 512;

FoldPlan fold_plan(int32_t S, int32_t N, int32_t K, int32_t group)
{
    FoldPlan p;
    p.stages = (K + kStageK - 1) / kStageK;
    p.shape = S <= 32 ? 2 : n_tiles_of(S, N, 128, 128) >= 256 ? 0 : 1;
    p.rows = p.shape == 1 ? 64 : 128;
    p.toks = p.shape == 0 && !group ? 128 : p.shape <= 1 ? 64 : 32;
    p.n_tiles = (N + p.rows - 1) / p.rows;
    p.t_tiles = (S + p.toks - 1) / p.toks;
    const int total = p.n_tiles * p.t_tiles;
    p.splits = std::max(1, std::min(kWantTiles / total, p.stages / 2));
    p.total = p.splits > 1 ? (size_t)p.splits * total * p.rows * p.toks * 4 : 256;
    return p;
}

template <int BITS, int RR, int TT, int WN, int GROUPED, typename TO>
hipError_t launch_fold_g(const LinearArgs& a, const FoldPlan& p, hipStream_t s)
{
    TileArgs ta = {};
    ta.part = (float*)a.ws;
    ta.n_tiles = p.n_tiles;
    ta.t_tiles = p.t_tiles;
    ta.stages = p.stages;
    ta.splits = p.splits;
    constexpr int bytes = FoldLds<BITS, RR, TT, WN, GROUPED>::kStage * FoldLds<BITS, RR, TT, WN, GROUPED>::kStages;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)linear_fold<BITS, RR, TT, WN, GROUPED, TO>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess)
            return e;
    }
    const int total = p.n_tiles * p.t_tiles;
    hipLaunchKernelGGL((linear_fold<BITS, RR, TT, WN, GROUPED, TO>), dim3((total * p.splits + 7) / 8 * 8), dim3(256),
                       bytes, s, a, ta);
    if (p.splits > 1)
        hipLaunchKernelGGL((linear_join<RR, TT, WN, TO>), dim3(total, RR * TT * 4), dim3(256), 0, s, a, ta,
                           1.0f / (float)(1 << (8 - BITS)));
    return hipGetLastError();
}

template <int BITS, int RR, int TT, int WN, typename TO>
hipError_t launch_fold_shape(const LinearArgs& a, const FoldPlan& p, hipStream_t s)
{
    return a.group == 0             ? launch_fold_g<BITS, RR, TT, WN, 0, TO>(a, p, s)
           : a.group % kStageK == 0 ? launch_fold_g<BITS, RR, TT, WN, 2, TO>(a, p, s)
                                    : launch_fold_g<BITS, RR, TT, WN, 1, TO>(a, p, s);
}

template <int BITS, typename TO>
hipError_t launch_fold(const LinearArgs& a, hipStream_t s)
{
    const FoldPlan p = fold_plan(a.S, a.N, a.K, a.group);
    switch (p.shape) {
    case 0:
        return a.group == 0               ? launch_fold_g<BITS, 2, 2, 2, 0, TO>(a, p, s)
               : a.group % kStageK == 0 ? launch_fold_g<BITS, 2, 1, 2, 2, TO>(a, p, s)
                                        : launch_fold_g<BITS, 2, 1, 2, 1, TO>(a, p, s);
    case 1: return launch_fold_shape<BITS, 1, 1, 2, TO>(a, p, s);
    default: return launch_fold_shape<BITS, 1, 1, 4, TO>(a, p, s);
    }
}

template <int BITS>
hipError_t launch(const LinearArgs& a, hipStream_t s)
{
    const bool f32 = a.out_type == COLI_F32;
    if (use_rows(a.S, a.K))
        return f32 ? launch_rows<BITS, float>(a, s) : launch_rows<BITS, bf16>(a, s);
    if (use_tiles(a.S, a.N, a.K, a.group, a.out_type))
        return launch_tiles<BITS>(a, s);
    return f32 ? launch_fold<BITS, float>(a, s) : launch_fold<BITS, bf16>(a, s);
}

} // namespace

size_t linear_workspace_need(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type)
{
    if (use_rows(S, K))
        return 256;
    return use_tiles(S, N, K, group, out_type) ? tile_plan(S, N, K).total : fold_plan(S, N, K, group).total;
}

/* The largest need of 1 .. S tokens.  Fewer tokens are fewer tiles, whose split
 * sums can take more than the whole of a larger call; the fold's plan changes
 * with every 64 tokens (and at 32), and splits nothing past kWantTiles / 2 tiles. */
size_t linear_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t group, int32_t out_type)
{
    size_t most = linear_workspace_need(S, N, K, group, out_type);
    if (use_rows(S, K)) /* and so do fewer tokens */
        return most;
    const int ends = std::min((S + 63) / 64, kWantTiles / (int)n_tiles_of(1, N, 128, 1));
    for (int t = 0; t <= ends; ++t)
        most = std::max(most, linear_workspace_need(std::min(S, t ? 64 * t : 32), N, K, group, out_type));
    return most;
}

hipError_t launch_linear_q(const LinearArgs& a, hipStream_t s)
{
    return a.qtype == COLI_Q8 ? launch<8>(a, s) : a.qtype == COLI_Q4 ? launch<4>(a, s) : launch<2>(a, s);
}

} // namespace coli
