/*
 * block_api.hip -- the C ABI of the operators around the layer (declared in
 * include/colibri_block.h): argument validation on the host, then one launcher.
 * Nothing here synchronises or allocates.
 */
#include "block.h"
#include "layer.h"

#include <math.h>

using namespace coli;

namespace {

bool is_type(int32_t t)
{
    return t == COLI_F32 || t == COLI_BF16;
}

/* Alignment of pointers that are read and written four elements at a time. */
size_t align4(int32_t type)
{
    return type == COLI_F32 ? 16 : 8;
}

bool good_stride(int64_t stride, int64_t least, int64_t by)
{
    return stride >= least && stride % by == 0 && stride <= (int64_t)1 << 40;
}

int check_linear(const coli_qbank* W, int32_t S, int32_t out_type)
{
    if (!W || S < 0 || !W->data || !W->row_scale || W->n_mat != 1 || W->rows < 1 || W->K < 32 || W->K % 32)
        return COLI_E_INVAL;
    if (W->rows > COLI_MAX_LINEAR_ROWS || W->K > COLI_MAX_LINEAR_K || S > COLI_MAX_TOKENS || !is_type(out_type))
        return COLI_E_UNSUPPORTED;
    return check_bank(W, 1, W->rows, W->K);
}

int check_cache(const coli_kv_cache* c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->n_pages < 1 || c->n_heads < 1)
        return COLI_E_INVAL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256)
        return COLI_E_UNSUPPORTED;
    if (c->n_heads > COLI_MAX_KV_HEADS)
        return COLI_E_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return COLI_E_UNSUPPORTED;
    return COLI_OK;
}

int check_batch_sizes(const coli_kv_batch* b)
{
    if (!b || b->n_seq < 0 || b->max_pages < 0 || b->n_tokens < 0 || b->max_q < 0)
        return COLI_E_INVAL;
    if (b->n_seq > COLI_MAX_SEQS || b->max_pages > COLI_MAX_SEQ_PAGES)
        return COLI_E_UNSUPPORTED;
    return COLI_OK;
}

int check_batch(const coli_kv_batch* b)
{
    const int st = check_batch_sizes(b);
    if (st)
        return st;
    if (b->n_seq == 0 || b->n_tokens == 0)
        return COLI_OK;
    if (!b->cu_q || !b->kv_len || (b->max_pages > 0 && !b->page_table))
        return COLI_E_INVAL;
    if (!aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4))
        return COLI_E_UNSUPPORTED;
    return COLI_OK;
}

int check_attn_sizes(const coli_kv_cache* c, const coli_kv_batch* b, const coli_kv_attn* a)
{
    if (!a || a->n_heads < 1 || a->n_heads % c->n_heads || a->max_kv < 0 || a->window < 0 ||
        (a->window > 0 && !a->causal) || !isfinite(a->scale))
        return COLI_E_INVAL;
    if (!is_type(a->type) || a->n_heads > 8 * COLI_MAX_KV_HEADS ||
        (int64_t)b->n_tokens * (a->n_heads / c->n_heads) >= (int64_t)1 << 31)
        return COLI_E_UNSUPPORTED;
    return COLI_OK;
}

} // namespace

extern "C" {

int colibri_add_rms_norm(const coli_norm* n, coli_stream_t stream)
{
    if (!n || n->rows < 0 || n->K < 32 || n->K % 32 || !(n->eps >= 0.0f) || !isfinite(n->eps))
        return COLI_E_INVAL;
    if (n->K > COLI_MAX_DIM || !is_type(n->x_type) || !is_type(n->residual_type) || !is_type(n->y_type))
        return COLI_E_UNSUPPORTED;
    if (n->rows == 0)
        return COLI_OK;
    if (!n->x || !n->weight || !n->q != !n->d || (!n->sum && !n->y && !n->q))
        return COLI_E_INVAL;
    if (!aligned(n->x, align4(n->x_type)) || !aligned(n->residual, align4(n->residual_type)) ||
        !aligned(n->sum, align4(n->residual_type)) || !aligned(n->y, align4(n->y_type)) ||
        !aligned(n->weight, 16) || !aligned(n->q, 4) || !aligned(n->d, 4))
        return COLI_E_UNSUPPORTED;
    if (!good_stride(n->x_stride, n->K, 4) || (n->residual && !good_stride(n->residual_stride, n->K, 4)))
        return COLI_E_INVAL;
    return hip_status(launch_add_rms_norm(*n, (hipStream_t)stream));
}

size_t colibri_linear_workspace_bytes(const coli_qbank* W, int32_t S, int32_t out_type)
{
    if (check_linear(W, S, out_type))
        return 0;
    return linear_workspace_bytes(S, W->rows, W->K, W->group, out_type);
}

int colibri_linear_q(const coli_qbank* W, const int8_t* xq, const float* xd, int32_t S, const float* bias,
                     int32_t act, const void* residual, void* out, int32_t out_type, void* ws,
                     size_t ws_bytes, coli_stream_t stream)
{
    const int st = check_linear(W, S, out_type);
    if (st)
        return st;
    if (act < COLI_ACT_NONE || act > COLI_ACT_GELU)
        return COLI_E_INVAL;
    if (S == 0)
        return COLI_OK;
    if (!xq || !xd || !out || !ws)
        return COLI_E_INVAL;
    if (!aligned(xq, 16) || !aligned(xd, 4) || !aligned(bias, 4) || !aligned(residual, 4) || !aligned(out, 4) ||
        !aligned(ws, kAlign))
        return COLI_E_UNSUPPORTED;
    if (ws_bytes < linear_workspace_need(S, W->rows, W->K, W->group, out_type))
        return COLI_E_WORKSPACE;
    LinearArgs a;
    a.w = W->data;
    a.w_scale = W->row_scale;
    a.xq = xq;
    a.xd = xd;
    a.bias = bias;
    a.residual = residual;
    a.out = out;
    a.ws = ws;
    a.S = S;
    a.N = W->rows;
    a.K = W->K;
    a.qtype = W->qtype;
    a.group = W->group;
    a.act = act;
    a.out_type = out_type;
    return hip_status(launch_linear_q(a, (hipStream_t)stream));
}

int colibri_kv_append(const coli_kv_cache* cache, const coli_kv_batch* batch, const void* k, const void* v,
                      int32_t type, int64_t k_stride, int64_t v_stride, coli_stream_t stream)
{
    int st = check_cache(cache);
    if (st || (st = check_batch(batch)))
        return st;
    if (!is_type(type))
        return COLI_E_UNSUPPORTED;
    if (batch->n_seq == 0 || batch->n_tokens == 0 || batch->max_pages == 0)
        return COLI_OK;
    if (!k || !v)
        return COLI_E_INVAL;
    if (!aligned(k, align4(type)) || !aligned(v, align4(type)))
        return COLI_E_UNSUPPORTED;
    const int64_t least = (int64_t)cache->n_heads * cache->head_dim;
    if (!good_stride(k_stride, least, 4) || !good_stride(v_stride, least, 4))
        return COLI_E_INVAL;
    return hip_status(launch_kv_append(*cache, *batch, k, v, type, k_stride, v_stride, (hipStream_t)stream));
}

int colibri_kv_read(const coli_kv_cache* cache, const coli_kv_batch* batch, void* k, void* v, int32_t type,
                    coli_stream_t stream)
{
    int st = check_cache(cache);
    if (st || (st = check_batch(batch)))
        return st;
    if (!is_type(type))
        return COLI_E_UNSUPPORTED;
    if (!k && !v)
        return COLI_E_INVAL;
    if (!aligned(k, align4(type)) || !aligned(v, align4(type)))
        return COLI_E_UNSUPPORTED;
    if (batch->n_seq == 0 || batch->n_tokens == 0)
        return COLI_OK;
    return hip_status(launch_kv_read(*cache, *batch, k, v, type, (hipStream_t)stream));
}

size_t colibri_kv_attention_workspace_bytes(const coli_kv_cache* cache, const coli_kv_batch* batch,
                                            const coli_kv_attn* attn)
{
    if (check_cache(cache) || check_batch_sizes(batch) || check_attn_sizes(cache, batch, attn))
        return 0;
    return kv_attention_workspace_bytes(*cache, *batch, *attn);
}

int colibri_kv_attention(const coli_kv_cache* cache, const coli_kv_batch* batch, const coli_kv_attn* attn,
                         void* ws, size_t ws_bytes, coli_stream_t stream)
{
    int st = check_cache(cache);
    if (st || (st = check_batch(batch)) || (st = check_attn_sizes(cache, batch, attn)))
        return st;
    if (batch->n_seq == 0 || batch->n_tokens == 0)
        return COLI_OK;
    if (!attn->q || !attn->out || !ws)
        return COLI_E_INVAL;
    if (!aligned(attn->q, 16) || !aligned(attn->out, 16) || !aligned(attn->lse, 4) || !aligned(ws, kAlign))
        return COLI_E_UNSUPPORTED;
    const int64_t least = (int64_t)attn->n_heads * cache->head_dim;
    if (!good_stride(attn->q_stride, least, 8) || !good_stride(attn->out_stride, least, 8))
        return COLI_E_INVAL;
    if (ws_bytes < kv_attention_workspace_need(*cache, *batch, *attn))
        return COLI_E_WORKSPACE;
    return hip_status(launch_kv_attention(*cache, *batch, *attn, ws, (hipStream_t)stream));
}

} // extern "C"
