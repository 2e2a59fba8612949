/*
 * linear_device.h -- device helpers shared by the linear products (linear.hip,
 * linear_i8.hip): activations, weight codes as int8 operands, the order of
 * tiles, and the last step to the output.
 */
#ifndef COLI_LINEAR_DEVICE_H
#define COLI_LINEAR_DEVICE_H

#include "block_device.h"

namespace coli {

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

constexpr int kChunk = 16;    /* bytes that a lane loads at once */

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
template <typename TO, typename Args>
__device__ __forceinline__ void store_rows(const Args& a, int tok, int n, const float* v)
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

} // namespace coli

#endif
