/*
 * kv_attention.hip -- softmax attention over the paged int8 cache.
 *
 * For a query row q and its sequence's tokens j, t_j = scale log2(e) q.k_j,
 *   out = sum_j 2^(t_j - m) v_j / sum_j 2^(t_j - m)
 * in one pass over the cache: m and the two sums are carried per row and
 * rescaled when m grows.
 *
 * Scores on the int8 matrix cores.  A key is code * scale already, so q is
 * written once as a fixed-point number of int8 digits below its row's largest
 * value (two digits, 15 bits, for bf16 queries; three, 23 bits, for fp32).  That
 * rounds it by up to half a unit, amax / 65024 or amax / 16646144, whatever the
 * value's own size: a score is off by that times |scale| sum |k| at most, where
 * fp32 products of bf16 queries would be exact.  The product with each digit is
 * exact in int32, the codes enter the matrix cores as they lie in memory, and one
 * int32 -> fp32 conversion per score carries q's, the block's and the softmax
 * scale.  Values take the bf16 matrix cores: an int8 code is exact in bf16, p
 * times the block's value scale is rounded to bf16 (bf16 outputs) or split into
 * three bf16 terms (fp32).
 *
 * Tiles.  S^T = K Q^T with v_mfma_i32_32x32x32_i8 gives lane (row = l % 32,
 * h = l / 32) the scores of tokens 8 (i / 4) + 4 h + i % 4 of its query row.
 * Those are the lane's own operand of O^T = V^T P^T (v_mfma_f32_32x32x16_bf16),
 * the page layout of V putting the same tokens into the same lane: P never
 * leaves its lane, and a row's statistics need one exchange between lanes l
 * and l ^ 32.
 */
#include "block_device.h"

#include <algorithm>

namespace coli {

namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr int kBlk = COLI_KV_BLOCK;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.0f;

struct AttnArgs {
    coli_kv_cache c;
    coli_kv_batch b;
    coli_kv_attn a;
    float* part_o;  /* [nsplit][n_tokens][n_heads][D] */
    float* part_ml; /* [nsplit][n_tokens][n_heads][2]: m (log2) and the sum */
    int32_t nsplit, row_tiles, group; /* group: query heads per cache head */
    uint32_t units; /* under 2^31 */
};

/*
 * The two tile shapes.  Tile<R> has R query rows (its columns, lane l % R) and
 * 64 / R lane groups g = l / R; a lane holds R of a page's 64 scores of its
 * row.  What differs is the matrix instruction and which token a score
 * register stands for; both follow the page layout of V, so that eight
 * consecutive score registers are the lane's operand of the value product.
 */
template <int R>
struct Tile;

template <>
struct Tile<32> {
    static constexpr int kDims = 32; /* dims of a key operand */
    using Acc = v16f;
    using V = v4i;
    static constexpr int kAcc = 16;
    /* token (of 32) of score register i, dim (of 32) of accumulator register i */
    static __device__ __forceinline__ int token(int i, int g) { return 8 * (i / 4) + 4 * g + i % 4; }
    static __device__ __forceinline__ int dim(int i, int g) { return 8 * (i / 4) + 4 * g + i % 4; }
    template <int D, int ND>
    static __device__ __forceinline__ void scores(const v4i* k, const v4i (&dig)[ND][D / 32], int (&s)[ND][16])
    {
#pragma unroll
        for (int e = 0; e < ND; ++e) {
            v16i acc = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(k[x], dig[e][x], acc, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[e][i] = acc[i];
        }
    }
    /* keys: D / 32 operands; values: D / 32 operand pairs */
    template <int D>
    static __device__ __forceinline__ void load_k(const int8_t* p, int col, int g, v4i* k)
    {
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
            k[x] = *(const v4i*)(p + x * 1024 + g * 512 + col * 16);
    }
    template <int D>
    static __device__ __forceinline__ void load_v(const int8_t* p, int col, int g, V* v)
    {
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
            v[x] = *(const v4i*)(p + x * 1024 + col * 32 + g * 16);
    }
    static __device__ __forceinline__ Acc mfma(v8b a, v8b b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Tile<16> {
    static constexpr int kDims = 64;
    using Acc = v4f;
    using V = v2i;
    static constexpr int kAcc = 4;
    static __device__ __forceinline__ int token(int i, int g)
    {
        return 16 * (g >> 1) + 8 * (i / 4) + 4 * (g & 1) + i % 4;
    }
    static __device__ __forceinline__ int dim(int i, int g) { return 4 * g + i; }
    template <int D, int ND>
    static __device__ __forceinline__ void scores(const v4i* k, const v4i (&dig)[ND][D / 64], int (&s)[ND][8])
    {
#pragma unroll
        for (int e = 0; e < ND; ++e)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                v4i acc = {0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[j * (D / 64) + x], dig[e][x], acc, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[e][4 * j + i] = acc[i];
            }
    }
    /* row r of key operand j is token 16 (r / 8) + 8 j + r % 8 */
    template <int D>
    static __device__ __forceinline__ void load_k(const int8_t* p, int col, int g, v4i* k)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                k[j * (D / 64) + x] =
                    *(const v4i*)(p + (4 * x + g) * 512 + (16 * (col >> 3) + 8 * j + (col & 7)) * 16);
    }
    template <int D>
    static __device__ __forceinline__ void load_v(const int8_t* p, int col, int g, V* v)
    {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
            v[x] = *(const v2i*)(p + x * 512 + col * 32 + (g & 1) * 16 + (g >> 1) * 8);
    }
    static __device__ __forceinline__ Acc mfma(v8b a, v8b b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

/* The value of lane l ^ 32. */
__device__ __forceinline__ float other_half(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

/* The value of lane l ^ 16. */
__device__ __forceinline__ float other_quarter(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
}

/* Maximum and sum over a row's lanes. */
template <int R>
__device__ __forceinline__ float row_max(float v)
{
    if constexpr (R == 16)
        v = fmaxf(v, other_quarter(v));
    return fmaxf(v, other_half(v));
}

template <int R>
__device__ __forceinline__ float row_sum(float v)
{
    if constexpr (R == 16)
        v += other_quarter(v);
    return v + other_half(v);
}

/* A query row in int8 digits, most significant first, as operands of the key
 * product, negated for a negative softmax scale; returns the value of one unit
 * (not negative, NaN if the row holds a NaN or an infinity). */
template <typename T, int R, int D, int ND>
__device__ __forceinline__ float load_query(const T* row, bool live, bool negate, int g,
                                            v4i (&dig)[ND][D / Tile<R>::kDims])
{
    constexpr int KS = D / Tile<R>::kDims;
    float x[KS * 16];
    float amax = 0.0f, bad = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = load4(row + s * Tile<R>::kDims + g * 16 + 4 * j);
            float* o = x + s * 16 + 4 * j;
            o[0] = v.x;
            o[1] = v.y;
            o[2] = v.z;
            o[3] = v.w;
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            bad += (v.x - v.x) + (v.y - v.y) + (v.z - v.z) + (v.w - v.w);
        }
    amax = row_max<R>(amax);
    bad = row_sum<R>(bad);
    /* rows so small that the quotient below would overflow are lifted first */
    const float lift = amax < 0x1p-60f ? 0x1p64f : 1.0f;
    constexpr float top = ND == 2 ? 127.0f * 256 : 127.0f * 65536;
    const float up = amax * lift;
    const float f = up == 0.0f ? 0.0f : negate ? -top / up : top / up;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int w[ND];
#pragma unroll
            for (int e = 0; e < ND; ++e)
                w[e] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int v = live ? (int)__builtin_rintf(x[s * 16 + 4 * j + i] * lift * f) : 0;
#pragma unroll
                for (int e = ND - 1; e >= 0; --e) {
                    const int low = e ? (int)(int8_t)v : v;
                    w[e] |= (low & 0xFF) << (8 * i);
                    v = (v - low) >> 8;
                }
            }
#pragma unroll
            for (int e = 0; e < ND; ++e)
                dig[e][s][j] = w[e];
        }
    return (up / top) / lift + bad;
}

/* Eight int8 codes as bf16 (exact: the upper halves of their fp32 forms). */
__device__ __forceinline__ v8b codes_bf16(int w0, int w1)
{
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int w = j < 2 ? w0 : w1, o = (j & 1) * 16;
        const float a = (float)(int8_t)(w >> o), b = (float)(int8_t)(w >> (o + 8));
        r[j] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
    v8b v;
    __builtin_memcpy(&v, r, 16);
    return v;
}

/* Eight weights as NP bf16 terms. */
template <int NP>
__device__ __forceinline__ void split_bf16(const float* p, v8b (&term)[NP])
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = p[i];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
            if (e + 1 < NP) {
                x[2 * j] -= __uint_as_float(r[j] << 16);
                x[2 * j + 1] -= __uint_as_float(r[j] & 0xFFFF0000u);
            }
        }
        __builtin_memcpy(&term[e], r, 16);
    }
}

/* Scores of 32 tokens in units of q's and k's scales.  |digit sum| <= 127 *
 * 128 * 256 < 2^22, so a shift by 8 stays in int32. */
template <int R, int D, int ND>
__device__ __forceinline__ void score_half(const v4i* k, const v4i (&dig)[ND][D / Tile<R>::kDims], float* t)
{
    int s[ND][R / 2];
    Tile<R>::template scores<D, ND>(k, dig, s);
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
        if constexpr (ND == 2)
            t[i] = (float)((s[0][i] << 8) + s[1][i]);
        else
            t[i] = __builtin_fmaf((float)s[0][i], 65536.0f, (float)((s[1][i] << 8) + s[2][i]));
    }
}

/* The tokens that a tile's rows see: [begin, end) for the lane's own row, and
 * over the tile's rows the blocks that any sees and the tokens that all see. */
struct Span {
    int begin, end, all_begin, all_end, any_begin, any_end;
};

__device__ __forceinline__ Span row_span(const coli_kv_attn& a, const SeqBounds& q, int qi, int qi_lo, int qi_hi)
{
    Span s;
    s.end = s.all_end = s.any_end = q.kv_len;
    s.begin = s.all_begin = s.any_begin = 0;
    if (a.causal) {
        s.end = max(q.first + qi + 1, 0);
        s.all_end = max(q.first + qi_lo + 1, 0);
        s.any_end = max(q.first + qi_hi + 1, 0);
        if (a.window > 0) {
            s.begin = max(s.end - a.window, 0);
            s.any_begin = max(s.all_end - a.window, 0);
            s.all_begin = max(s.any_end - a.window, 0);
        }
    }
    return s;
}

/* Scores of the tokens that the lane's row does not see, in NU halves of a block
 * from token `base` on. */
template <int R, int NU>
__device__ __forceinline__ void mask_tile(float* t, int base, int end, int begin, int lg)
{
#pragma unroll
    for (int i = 0; i < NU * (R / 2); ++i) {
        const int j = base + i / (R / 2) * 32 + Tile<R>::token(i % (R / 2), lg);
        t[i] = j < end && j >= begin ? t[i] : -__builtin_inff();
    }
}

/* Scores t in units of c (c >= 0, one per row) become w 2^(t c - m), w being the
 * block's value scale, with m raised towards the largest; l, the lane's sum, takes
 * them up without w; returns the factor of what was summed before.  Both scales
 * go into the exponent's fma: the largest of t is the largest of t c, and w is
 * 2^log2(w), whose rounding (2^-21) weighs a block's sums and its share of l
 * alike.  A w that is not positive is multiplied in afterwards. */
template <int R, int N>
__device__ __forceinline__ float softmax_tile(float* t, float c, float w, float& m, float& l)
{
    float mx = t[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        mx = fmaxf(mx, t[i]);
    mx = row_max<R>(mx);
    /* m follows the largest only when that is 2^kSlack above it: until then the
     * powers stay below 2^kSlack and the sums need no factor.  A row that has
     * seen nothing keeps -inf (0 * -inf is no number). */
    const float mn = mx != -__builtin_inff() && mx * c > m + kSlack ? mx * c : m;
    const float mb = mn == -__builtin_inff() ? 0.0f : mn;
    const float cc = c == 0.0f ? 0x1p-126f : c; /* hidden tokens stay at -inf, the others at 0 */
    const float f = __builtin_amdgcn_exp2f(m - mb);
    const bool plus = w >= 0x1p-100f; /* uniform */
    const float off = (plus ? __builtin_amdgcn_logf(w) : 0.0f) - mb, back = plus ? 1.0f / w : 1.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(t[i], cc, off));
        sum += t[i];
    }
    l = __builtin_fmaf(l, f, sum * back);
    m = mn;
    if (!plus) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            t[i] *= w;
    }
    return f;
}

/*
 * Few query rows: a workgroup takes one tile of R rows of one (sequence, cache
 * head) and one of nsplit ranges of its blocks, its four waves the pieces of
 * that range in turn, each with its own statistics; they are joined through
 * LDS, the ranges by kv_attention_join.
 *
 * Keys and values go straight from memory to the matrix cores' registers (a
 * wave reads whole lines of a page).  The next piece's keys are in flight
 * under this piece's softmax and value product, its values under the next
 * scores.  Bound by the cache's bytes: 131071 tokens of 8 heads of 128 dims, fp32
 * queries, 48 us (5.6 TB/s); 32 sequences of up to 9000, 4 queries each, bf16, 95
 * us (4.6 TB/s; ranges are equal shares of a sequence, the longest end last).
 * Twice as many ranges cost 25 % (each loads its query digits and joins four
 * waves).  A piece is a block, or half a block where the registers hold no more.
 */
template <typename T, int R, int D>
__global__ __launch_bounds__(256, R == 32 && D > 128 ? 1 : 2) void kv_attention_split(AttnArgs g)
{
    using TL = Tile<R>;
    constexpr int ND = sizeof(T) == 4 ? 3 : 2, NP = sizeof(T) == 4 ? 3 : 1;
    constexpr int NU = D <= (R == 16 ? 128 : 64) ? 2 : 1; /* halves of a block in a piece */
    constexpr int HS = R / 2;            /* scores of a half in a lane */
    constexpr int KN = D / 32, VN = D / R, DT = D / R, NA = TL::kAcc;
    __shared__ float so[2][DT * NA][64];
    __shared__ float sm[4][R], sl[4][R];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lg = lane / R, col = lane % R;
    const int H = g.c.n_heads, G = g.group;

    /* Numbers of units and rows fit 31 bits, and so do the divisions: in 64 bits
     * one short sequence took 12.4 us in place of 11.8.  r0 < 2^31 and a stride of
     * at most 2^31 (R divides it) do not wrap. */
    for (uint32_t unit = blockIdx.x; unit < g.units; unit += gridDim.x) {
        const int split = (int)(unit % (uint32_t)g.nsplit);
        uint32_t r = unit / (uint32_t)g.nsplit;
        const int hk = (int)(r % (uint32_t)H);
        r /= (uint32_t)H;
        const int rt0 = (int)(r % (uint32_t)g.row_tiles), s = (int)(r / (uint32_t)g.row_tiles);
        const SeqBounds q = seq_bounds(g.b, s);
        const uint32_t n_rows = (uint32_t)q.q_len * G;
        for (uint32_t r0 = (uint32_t)rt0 * R; r0 < n_rows; r0 += (uint32_t)g.row_tiles * R) {
            const int live_rows = (int)min(n_rows - r0, (uint32_t)R);
            const uint32_t row = r0 + min(col, live_rows - 1);
            const int qi = (int)(row / (uint32_t)G), head = hk * G + (int)(row % (uint32_t)G);
            const bool live = col < live_rows;
            const int64_t tok = (int64_t)q.row0 + qi;
            v4i dig[ND][D / TL::kDims];
            const float unit_q =
                load_query<T, R, D, ND>((const T*)g.a.q + tok * g.a.q_stride + (int64_t)head * D, live,
                                        g.a.scale < 0.0f, lg, dig) *
                (fabsf(g.a.scale) * kLog2e);
            const Span sp = row_span(g.a, q, qi, (int)(r0 / (uint32_t)G), (int)((r0 + live_rows - 1) / (uint32_t)G));
            /* pieces of 32 NU tokens */
            constexpr int PT = 32 * NU;
            const int p_lo = sp.any_begin / PT, p_hi = (sp.any_end + PT - 1) / PT;
            const int per = (max(p_hi - p_lo, 0) + g.nsplit - 1) / g.nsplit;
            const int p0 = __builtin_amdgcn_readfirstlane(min(p_lo + split * per, p_hi));
            const int p1 = __builtin_amdgcn_readfirstlane(min(p0 + per, p_hi));

            float m = -__builtin_inff(), l = 0.0f;
            typename TL::Acc acc[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    acc[d][i] = 0.0f;

            /* a missing page reads page 0, whose scales may be anything: it is masked
             * as a whole and both its scales are taken as 0; pieces past the range
             * read its last one (loads are unconditional) */
            auto page_at = [&](int p) {
                return __builtin_amdgcn_readfirstlane(page_of(g.b, g.c.n_pages, s, min(p, p1 - 1) * PT / kBlk));
            };
            v4i kreg[NU][KN];
            typename TL::V vreg[NU][VN];
            auto at = [&](int page) { return (int64_t)max(page, 0) * H + hk; };
            auto half_of = [&](int p) { return NU == 2 ? 0 : (min(p, p1 - 1) & 1) * 32 * D; };
            auto load_k = [&](int page, int p) {
                const int8_t* b = g.c.k + at(page) * (kBlk * D) + half_of(p);
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    TL::template load_k<D>(b + u * 32 * D, col, lg, kreg[u]);
            };
            auto load_v = [&](int page, int p) {
                const int8_t* b = g.c.v + at(page) * (kBlk * D) + half_of(p);
#pragma unroll
                for (int u = 0; u < NU; ++u)
                    TL::template load_v<D>(b + u * 32 * D, col, lg, vreg[u]);
            };
            int p = __builtin_amdgcn_readfirstlane(p0 + wv);
            if (p < p1) {
                int page = page_at(p), next = page_at(p + 4);
                load_k(page, p);
                load_v(page, p);
                float ks = g.c.k_scale[at(page)], vs = g.c.v_scale[at(page)];
                for (; p < p1; p += 4) {
                    float t[NU * HS];
#pragma unroll
                    for (int u = 0; u < NU; ++u)
                        score_half<R, D, ND>(kreg[u], dig, t + u * HS);
                    const int after = page_at(p + 8);
                    load_k(next, p + 4);
                    const float ks_next = g.c.k_scale[at(next)], vs_next = g.c.v_scale[at(next)];
                    const bool missing = page < 0;
                    const float c = unit_q * (missing ? 0.0f : ks);
                    const int base = p * PT;
                    if (missing || base + PT > sp.all_end || base < sp.all_begin)
                        mask_tile<R, NU>(t, base, missing ? 0 : sp.end, sp.begin, lg);
                    const float f = softmax_tile<R, NU * HS>(t, c, missing ? 0.0f : vs, m, l);
                    if (__any(f != 1.0f)) {
#pragma unroll
                        for (int d = 0; d < DT; ++d)
#pragma unroll
                            for (int i = 0; i < NA; ++i)
                                acc[d][i] *= f;
                    }
#pragma unroll
                    for (int x = 0; x < NU * HS / 8; ++x) {
                        constexpr int per_half = HS / 8; /* value operands of a half */
                        v8b term[NP];
                        split_bf16<NP>(t + 8 * x, term);
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            const auto& vv = vreg[x / per_half][d];
                            const v8b a = codes_bf16(vv[2 * (x % per_half)], vv[2 * (x % per_half) + 1]);
#pragma unroll
                            for (int e = 0; e < NP; ++e)
                                acc[d] = TL::mfma(a, term[e], acc[d]);
                        }
                    }
                    load_v(next, p + 4);
                    page = next;
                    next = after;
                    ks = ks_next;
                    vs = vs_next;
                }
            }

            /* join the four waves: statistics first, then the sums two by two */
            l = row_sum<R>(l);
            __syncthreads();
            if (lg == 0) {
                sm[wv][col] = m;
                sl[wv][col] = l;
            }
            __syncthreads();
            const float wm = m;
            m = fmaxf(fmaxf(sm[0][col], sm[1][col]), fmaxf(sm[2][col], sm[3][col]));
            const float mb = m == -__builtin_inff() ? 0.0f : m;
            l = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                l += sl[w][col] * __builtin_amdgcn_exp2f(sm[w][col] - mb);
            const float f = __builtin_amdgcn_exp2f(wm - mb);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    acc[d][i] *= f;
#pragma unroll
            for (int half = 2; half >= 1; half >>= 1) {
                if (wv >= half && wv < 2 * half)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int i = 0; i < NA; ++i)
                            so[wv - half][d * NA + i][lane] = acc[d][i];
                __syncthreads();
                if (wv < half)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int i = 0; i < NA; ++i)
                            acc[d][i] += so[wv][d * NA + i][lane];
                __syncthreads();
            }
            if (wv == 0 && live) {
                const bool whole = g.nsplit == 1;
                const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                const int64_t o_at = ((int64_t)split * g.b.n_tokens + tok) * g.a.n_heads + head;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < NA; i += 4) {
                        const int dim = d * R + TL::dim(i, lg);
                        const float4 v = make_float4(acc[d][i] * inv, acc[d][i + 1] * inv, acc[d][i + 2] * inv,
                                                     acc[d][i + 3] * inv);
                        if (whole)
                            store4((T*)g.a.out + tok * g.a.out_stride + (int64_t)head * D + dim, v);
                        else
                            store4(g.part_o + o_at * D + dim, v);
                    }
                if (lg == 0) {
                    if (!whole)
                        *(float2*)(g.part_ml + 2 * o_at) = make_float2(m, l);
                    else if (g.a.lse)
                        g.a.lse[tok * g.a.n_heads + head] = l == 0.0f ? -__builtin_inff() : m * kLn2 + logf(l);
                }
            }
        }
    }
}

/*
 * Many query rows: a workgroup takes 128 rows of one (sequence, cache head), 32
 * to a wave, and a range of its blocks.  A block's codes travel to LDS under
 * the blocks before it, and its values are turned into bf16 there once for the
 * four waves, one block ahead; the waves read both as they lie (an operand is
 * one run of 1 KB).
 * Bound by the VALU: about 11 instructions per score and row, the exponential
 * four times the others, beside 33 + 32 cycles of the matrix cores for 64
 * scores.  Measured: 4 prompts of up to 2047 tokens over up to 4095, 64 / 8 heads
 * of 128 dims, bf16, 491 us = 0.79 PFLOP/s; a wave's matrix-core and VALU phases
 * follow each other, and two waves of a SIMD cover them in part.
 */
constexpr int kTileRows = 128;

template <typename T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void kv_attention_tile(AttnArgs g)
{
    using TL = Tile<32>;
    constexpr int ND = sizeof(T) == 4 ? 3 : 2, NP = sizeof(T) == 4 ? 3 : 1;
    constexpr int KS = D / 32, DT = D / 32, PB = kBlk * D; /* bytes of a block's keys, or values */
    extern __shared__ __align__(1024) uint8_t lds[];       /* of two blocks each: keys, values, values in bf16 */
    const int lane = threadIdx.x & 63, wv = wave_of(), lg = lane >> 5, col = lane & 31;
    const uint32_t lds0 = lds_address(lds);
    const int H = g.c.n_heads, G = g.group;
    for (uint32_t unit = (uint32_t)xcd_unit(); unit < g.units; unit += gridDim.x) {
        /* heads outermost (an XCD's share has every sequence), then sequences, the
         * longest row tiles first */
        const int split = (int)(unit % (uint32_t)g.nsplit);
        uint32_t r = unit / (uint32_t)g.nsplit;
        const int rt0 = g.row_tiles - 1 - (int)(r % (uint32_t)g.row_tiles);
        r /= (uint32_t)g.row_tiles;
        const int s = (int)(r % (uint32_t)g.b.n_seq), hk = (int)(r / (uint32_t)g.b.n_seq);
        const SeqBounds q = seq_bounds(g.b, s);
        const uint32_t n_rows = (uint32_t)q.q_len * G;
        for (uint32_t r0 = (uint32_t)rt0 * kTileRows; r0 < n_rows; r0 += (uint32_t)g.row_tiles * kTileRows) {
            const int live_rows = (int)min(n_rows - r0, (uint32_t)kTileRows);
            const int mine = wv * 32 + col;
            const uint32_t row = r0 + min(mine, live_rows - 1);
            const int qi = (int)(row / (uint32_t)G), head = hk * G + (int)(row % (uint32_t)G);
            const bool live = mine < live_rows;
            const int64_t tok = (int64_t)q.row0 + qi;
            v4i dig[ND][KS];
            const float unit_q = load_query<T, 32, D, ND>((const T*)g.a.q + tok * g.a.q_stride + (int64_t)head * D, live,
                                                          g.a.scale < 0.0f, lg, dig) *
                                 (fabsf(g.a.scale) * kLog2e);
            /* the workgroup's blocks, and what this wave's rows see of them */
            const Span wg = row_span(g.a, q, qi, (int)(r0 / (uint32_t)G), (int)((r0 + live_rows - 1) / (uint32_t)G));
            const uint32_t w0 = r0 + min(wv * 32, live_rows - 1), w1 = r0 + min(wv * 32 + 31, live_rows - 1);
            const Span sp = row_span(g.a, q, qi, (int)(w0 / (uint32_t)G), (int)(w1 / (uint32_t)G));
            const int p_lo = wg.any_begin / kBlk, p_hi = (wg.any_end + kBlk - 1) / kBlk;
            const int per = (max(p_hi - p_lo, 0) + g.nsplit - 1) / g.nsplit;
            const int p0 = __builtin_amdgcn_readfirstlane(min(p_lo + split * per, p_hi));
            const int p1 = __builtin_amdgcn_readfirstlane(min(p0 + per, p_hi));

            float m = -__builtin_inff(), l = 0.0f;
            v16f acc[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[d][i] = 0.0f;

            auto page_at = [&](int p) {
                return __builtin_amdgcn_readfirstlane(page_of(g.b, g.c.n_pages, s, min(p, p1 - 1)));
            };
            auto at = [&](int page) { return (int64_t)max(page, 0) * H + hk; };
            auto fetch = [&](const int8_t* from, uint32_t to) {
#pragma unroll
                for (int i = 0; i < PB / 4096; ++i) {
                    const int o = (i * 4 + wv) * 1024;
                    to_lds(from + o, lane * 16, lds0 + to + o);
                }
            };
            auto fetch_k = [&](int page, int p) { fetch(g.c.k + at(page) * PB, (p & 1) * PB); };
            auto fetch_v = [&](int page, int p) { fetch(g.c.v + at(page) * PB, (2 + (p & 1)) * PB); };
            /* values to bf16: sixteen tokens of a dim are two operands of it */
            auto convert = [&](int p) {
                const uint8_t* raw = lds + (2 + (p & 1)) * PB;
                uint8_t* vb = lds + (4 + 2 * (p & 1)) * PB;
#pragma unroll
                for (int i = 0; i < PB / 4096; ++i) {
                    const int u = i * 256 + threadIdx.x, half = u / (2 * D), c = u / 2 % D, hh = u & 1;
                    const v4i w = *(const v4i*)(raw + u * 16);
                    uint8_t* o = vb + (half * 2 * DT + c / 32) * 1024 + hh * 512 + c % 32 * 16;
                    *(v8b*)o = codes_bf16(w[0], w[1]);
                    *(v8b*)(o + DT * 1024) = codes_bf16(w[2], w[3]);
                }
            };
            if (p0 < p1) {
                int page = page_at(p0), page1 = page_at(p0 + 1), page2 = page_at(p0 + 2);
                fetch_k(page, p0);
                fetch_v(page, p0);
                float ks = g.c.k_scale[at(page)], vs = g.c.v_scale[at(page)];
                arrive_all<0>();
                fetch_v(page1, p0 + 1);
                convert(p0);
                for (int p = p0; p < p1; ++p) {
                    const int page3 = page_at(p + 3);
                    const float ks_next = g.c.k_scale[at(page1)], vs_next = g.c.v_scale[at(page1)];
                    /* this block's keys and the next one's values have arrived, this one's
                     * are converted; what is written next was left before this point */
                    arrive_all<0>();
                    fetch_k(page1, p + 1);
                    fetch_v(page2, p + 2);
                    convert(p + 1);
                    const uint8_t* buf = lds + (p & 1) * PB;
                    const uint8_t* vb = lds + (4 + 2 * (p & 1)) * PB;
                    const int base = p * kBlk;
                    if (page >= 0 && base < sp.any_end && base + kBlk > sp.any_begin) {
                        float t[32];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            v4i k[KS];
#pragma unroll
                            for (int x = 0; x < KS; ++x)
                                k[x] = *(const v4i*)(buf + (u * KS + x) * 1024 + lane * 16);
                            score_half<32, D, ND>(k, dig, t + 16 * u);
                        }
                        if (base + kBlk > sp.all_end || base < sp.all_begin)
                            mask_tile<32, 2>(t, base, sp.end, sp.begin, lg);
                        const float f = softmax_tile<32, 32>(t, unit_q * ks, vs, m, l);
                        if (__any(f != 1.0f)) {
#pragma unroll
                            for (int d = 0; d < DT; ++d)
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    acc[d][i] *= f;
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            v8b term[NP];
                            split_bf16<NP>(t + 8 * x, term);
#pragma unroll
                            for (int d = 0; d < DT; ++d) {
                                const v8b a = *(const v8b*)(vb + (x * DT + d) * 1024 + lane * 16);
#pragma unroll
                                for (int e = 0; e < NP; ++e)
                                    acc[d] = TL::mfma(a, term[e], acc[d]);
                            }
                        }
                    }
                    page = page1;
                    page1 = page2;
                    page2 = page3;
                    ks = ks_next;
                    vs = vs_next;
                }
                arrive_all<0>(); /* the buffers are free for the next tile of rows */
            }
            l = row_sum<32>(l);
            if (live) {
                const bool whole = g.nsplit == 1;
                const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                const int64_t o_at = ((int64_t)split * g.b.n_tokens + tok) * g.a.n_heads + head;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const int dim = d * 32 + TL::dim(i, lg);
                        const float4 v =
                            make_float4(acc[d][i] * inv, acc[d][i + 1] * inv, acc[d][i + 2] * inv, acc[d][i + 3] * inv);
                        if (whole)
                            store4((T*)g.a.out + tok * g.a.out_stride + (int64_t)head * D + dim, v);
                        else
                            store4(g.part_o + o_at * D + dim, v);
                    }
                if (lg == 0) {
                    if (!whole)
                        *(float2*)(g.part_ml + 2 * o_at) = make_float2(m, l);
                    else if (g.a.lse)
                        g.a.lse[tok * g.a.n_heads + head] = l == 0.0f ? -__builtin_inff() : m * kLn2 + logf(l);
                }
            }
        }
    }
}

/* Joins the ranges' partial sums, W waves per (token, head): wave w takes the
 * ranges w, w + W, ... in order, four rows of partial sums in flight, and the
 * waves' sums are added in wave order.  With many ranges four waves are worth
 * their exchange (64 rows of 128 ranges: 6.8 us, 40 with one wave). */
template <typename T, int D, int W>
__global__ __launch_bounds__(256) void kv_attention_join(AttnArgs g)
{
    constexpr int E = D / 64;
    __shared__ float so[4][D], sl[4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, part = wv % W;
    const int64_t n = (int64_t)g.b.n_tokens * g.a.n_heads;
    const int64_t want = (int64_t)blockIdx.x * (4 / W) + wv / W;
    const int64_t at = min(want, n - 1);
    const int64_t tok = (uint32_t)at / (uint32_t)g.a.n_heads; /* at < kMaxSplitRows */
    const int head = (int)((uint32_t)at % (uint32_t)g.a.n_heads);
    /* not a row of no sequence */
    const bool live = want < n && tok >= g.b.cu_q[0] && tok < g.b.cu_q[g.b.n_seq];
    const float2* ml = (const float2*)g.part_ml + at;
    float m = -__builtin_inff(), l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = 0.0f;
    if (live) {
        for (int i = lane; i < g.nsplit; i += 64)
            m = fmaxf(m, ml[i * n].x);
        for (int w = 32; w >= 1; w >>= 1)
            m = fmaxf(m, shfl_xor(m, w));
        const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll 4
        for (int i = part; i < g.nsplit; i += W) {
            const float2 v = ml[i * n];
            const float f = __builtin_amdgcn_exp2f(v.x - base);
            l = __builtin_fmaf(v.y, f, l);
            const float* p = g.part_o + (i * n + at) * D;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = __builtin_fmaf(p[lane + 64 * e], f, o[e]);
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            so[wv][lane + 64 * e] = o[e];
        if (lane == 0)
            sl[wv] = l;
        __syncthreads();
        if (part)
            return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            l += sl[wv + w];
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] += so[wv + w][lane + 64 * e];
        }
    }
    if (!live)
        return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        store1((T*)g.a.out + tok * g.a.out_stride + (int64_t)head * D + lane + 64 * e, o[e] * inv);
    if (g.a.lse && lane == 0)
        g.a.lse[at] = l == 0.0f ? -__builtin_inff() : m * kLn2 + logf(l);
}

constexpr size_t kPartAlign = 256;

/* How a call is cut: rows of a tile, tiles by the longest expected query run,
 * ranges so that about kTargetUnits workgroups run, each wave (kv_attention_tile:
 * each workgroup) with a few blocks at least. */
struct Plan {
    int rows, row_tiles, nsplit;
    int64_t units;
    size_t o_bytes, total;
};

constexpr int64_t kTargetUnits = 512;
constexpr int kMaxSplit = 256;
constexpr int64_t kMaxSplitRows = 1 << 22; /* bounds the workspace and the join's grid */

/* Bytes of n rows' partial sums, and with their statistics. */
size_t sums_bytes(size_t n, int32_t D)
{
    return (n * D * 4 + kPartAlign - 1) / kPartAlign * kPartAlign;
}

size_t part_bytes(size_t n, int32_t D)
{
    return n == 0 ? kPartAlign : sums_bytes(n, D) + (n * 8 + kPartAlign - 1) / kPartAlign * kPartAlign;
}

Plan plan_attention(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a)
{
    Plan p;
    const int G = a.n_heads / c.n_heads;
    const int64_t rows = (int64_t)std::max(1, std::min(b.max_q, b.n_tokens)) * G;
    p.rows = rows > 32 ? kTileRows : rows <= 16 || a.type == COLI_F32 ? 16 : 32;
    /* At most 2^27 units before the split, which adds none beyond kTargetUnits
     * twice over; a workgroup goes on to the row tiles that are left. */
    const int64_t pairs = (int64_t)std::max(b.n_seq, 1) * c.n_heads;
    p.row_tiles = (int)std::min((rows + p.rows - 1) / p.rows, std::max<int64_t>(1, ((int64_t)1 << 27) / pairs));
    /* An odd number where several sequences fill the chip: workgroups are dealt to
     * the CUs in turn, and a power of two would give the tiles that short sequences
     * do have to a few of them (one prompt of 900 among 63 decoding sequences: 334
     * us with 60 tiles each, 194 with 61; 2000 among 63: 375 with 64, 230 with 65). */
    if (p.rows == kTileRows && b.n_seq > 1 && pairs * p.row_tiles >= kTargetUnits)
        p.row_tiles |= 1;
    const int64_t units = pairs * p.row_tiles;
    const int64_t seen = a.window > 0 ? std::min<int64_t>(a.max_kv, (int64_t)a.window + b.max_q) : a.max_kv;
    const int64_t blocks = (seen + kBlk - 1) / kBlk, target = kTargetUnits;
    p.nsplit = (int)std::max<int64_t>(1, std::min({(target + units - 1) / units, (blocks + 3) / 4, (int64_t)kMaxSplit}));
    if (p.rows == kTileRows && units >= 256)
        p.nsplit = 1;
    if ((int64_t)b.n_tokens * a.n_heads > kMaxSplitRows)
        p.nsplit = 1;
    p.units = units * p.nsplit;
    const size_t n = p.nsplit == 1 ? 0 : (size_t)p.nsplit * b.n_tokens * a.n_heads;
    p.o_bytes = sums_bytes(n, c.head_dim);
    p.total = part_bytes(n, c.head_dim);
    return p;
}

/* The partial sums of any call with sizes up to these and no more rows than
 * n_seq * max_q.  A call that is split has u < kTargetUnits units (u < 256 of
 * kTileRows) of at most R rows each in at most (kTargetUnits + u - 1) / u ranges;
 * and it has no more rows than there are here, in no more ranges than its blocks
 * or one unit per cache head allow. */
size_t most_part_bytes(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a)
{
    const int64_t rows = (int64_t)std::max(1, std::min(b.max_q, b.n_tokens)) * (a.n_heads / c.n_heads);
    const int64_t R = rows > 32 ? kTileRows : rows <= 16 || a.type == COLI_F32 ? 16 : 32;
    const int64_t u = std::min(R == kTileRows ? 255 : kTargetUnits - 1,
                               (int64_t)std::max(b.n_seq, 1) * c.n_heads * ((rows + R - 1) / R));
    const int64_t splits = std::min({(kTargetUnits + c.n_heads - 1) / c.n_heads,
                                     ((int64_t)a.max_kv + 4 * kBlk - 1) / (4 * kBlk), (int64_t)kMaxSplit});
    const int64_t here = std::min((int64_t)b.n_tokens * a.n_heads, kMaxSplitRows) * splits;
    return part_bytes(splits < 2 ? 0 : (size_t)std::min(here, R * (kTargetUnits + u - 1)), c.head_dim);
}

template <typename T, int D>
hipError_t launch(const AttnArgs& g, int rows, hipStream_t s)
{
    if (rows == kTileRows) {
        constexpr int bytes = 8 * kBlk * D;
        if (bytes > 64 * 1024) {
            const hipError_t e = hipFuncSetAttribute((const void*)kv_attention_tile<T, D>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != hipSuccess)
                return e;
        }
        hipLaunchKernelGGL((kv_attention_tile<T, D>), dim3(std::min((g.units + 7) / 8 * 8, 1u << 20)), dim3(256), bytes, s,
                           g);
    } else {
        const uint32_t grid = std::min(g.units, 1u << 20);
        if (rows == 16)
            hipLaunchKernelGGL((kv_attention_split<T, 16, D>), dim3(grid), dim3(256), 0, s, g);
        else
            hipLaunchKernelGGL((kv_attention_split<bf16, 32, D>), dim3(grid), dim3(256), 0, s, g);
    }
    if (g.nsplit > 1) {
        const int64_t n = (int64_t)g.b.n_tokens * g.a.n_heads;
        if (g.nsplit <= 8)
            hipLaunchKernelGGL((kv_attention_join<T, D, 1>), dim3((uint32_t)((n + 3) / 4)), dim3(256), 0, s, g);
        else
            hipLaunchKernelGGL((kv_attention_join<T, D, 4>), dim3((uint32_t)n), dim3(256), 0, s, g);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const AttnArgs& g, int rows, hipStream_t s)
{
    switch (g.c.head_dim) {
    case 64: return launch<T, 64>(g, rows, s);
    case 128: return launch<T, 128>(g, rows, s);
    case 192: return launch<T, 192>(g, rows, s);
    default: return launch<T, 256>(g, rows, s);
    }
}

} // namespace

size_t kv_attention_workspace_need(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a)
{
    return plan_attention(c, b, a).total;
}

/* n_tokens may be above n_seq * max_q, which the second does not cover. */
size_t kv_attention_workspace_bytes(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a)
{
    return std::max(plan_attention(c, b, a).total, most_part_bytes(c, b, a));
}

hipError_t launch_kv_attention(const coli_kv_cache& c, const coli_kv_batch& b, const coli_kv_attn& a, void* ws,
                               hipStream_t s)
{
    const Plan p = plan_attention(c, b, a);
    AttnArgs g;
    g.c = c;
    g.b = b;
    g.a = a;
    g.nsplit = p.nsplit;
    g.row_tiles = p.row_tiles;
    g.group = a.n_heads / c.n_heads;
    g.units = (uint32_t)p.units;
    g.part_o = (float*)ws;
    g.part_ml = (float*)((uint8_t*)ws + p.o_bytes);
    return a.type == COLI_F32 ? launch_d<float>(g, p.rows, s) : launch_d<bf16>(g, p.rows, s);
}

} // namespace coli
