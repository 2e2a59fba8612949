"""What the operators around the layer refuse, on the host: the C ABI returns
an error before anything is enqueued (no GPU is needed), and the binding
raises on tensors that do not fit."""

import ctypes

import pytest
import torch

import quantized_routed_expert_sigmoid_amd as qre
from quantized_routed_expert_sigmoid_amd import block

P = 1 << 20  # a well aligned address that no call here may touch
OK, INVAL, UNSUP, WS = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    return block._f()


def norm(**kw):
    d = dict(x=P, residual=P, weight=P, sum=P, y=P, q=P, d=P, x_stride=64, residual_stride=64, rows=2, K=64, x_type=32,
             residual_type=32, y_type=32, eps=1e-6)
    d.update(kw)
    return block.NormDesc(**d)


@pytest.mark.parametrize("kw,st", [
    (dict(rows=-1), INVAL), (dict(K=0), INVAL), (dict(K=48), INVAL), (dict(K=8224, x_stride=8224), UNSUP),
    (dict(x=None), INVAL), (dict(weight=None), INVAL), (dict(q=None), INVAL), (dict(d=None), INVAL),
    (dict(sum=None, y=None, q=None, d=None), INVAL), (dict(x_type=8), UNSUP), (dict(residual_type=0), UNSUP),
    (dict(y_type=1), UNSUP), (dict(eps=-1.0), INVAL), (dict(eps=float("nan")), INVAL), (dict(eps=float("inf")), INVAL),
    (dict(x=P + 8), UNSUP), (dict(residual=P + 4), UNSUP), (dict(y=P + 8), UNSUP), (dict(q=P + 2), UNSUP),
    (dict(weight=P + 4), UNSUP), (dict(x_stride=60), INVAL), (dict(x_stride=66), INVAL),
    (dict(residual_stride=63), INVAL), (dict(rows=0, x=None), OK)])
def test_norm(L, kw, st):
    assert L.colibri_add_rms_norm(ctypes.byref(norm(**kw)), None) == st


def test_norm_null(L):
    assert L.colibri_add_rms_norm(None, None) == INVAL


def bank(**kw):
    d = dict(data=P, row_scale=P, n_mat=1, rows=5, K=64, qtype=4, group=0)
    d.update(kw)
    return qre.QBankDesc(**d)


@pytest.mark.parametrize("kw,st", [
    (dict(n_mat=2), INVAL), (dict(rows=0), INVAL), (dict(K=40), INVAL), (dict(K=0), INVAL), (dict(data=None), INVAL),
    (dict(row_scale=None), INVAL), (dict(qtype=5), UNSUP), (dict(group=48), INVAL), (dict(group=-32), INVAL),
    (dict(group=128), INVAL), (dict(rows=(1 << 20) + 1), UNSUP), (dict(K=(1 << 15) + 32), UNSUP), (dict(data=P + 4), UNSUP)])
def test_linear_bank(L, kw, st):
    w = bank(**kw)
    assert L.colibri_linear_q(ctypes.byref(w), P, P, 1, None, 0, None, P, 32, P, 1 << 40, None) == st
    assert L.colibri_linear_workspace_bytes(ctypes.byref(w), 1, 32) == 0


@pytest.mark.parametrize("args,st", [
    ((None, P, 1, P, 0, P, P, 32, P, 1 << 40), INVAL), ((P, None, 1, P, 0, P, P, 32, P, 1 << 40), INVAL),
    ((P, P, -1, P, 0, P, P, 32, P, 1 << 40), INVAL), ((P, P, 65537, P, 0, P, P, 32, P, 1 << 40), UNSUP),
    ((P, P, 1, P, 4, P, P, 32, P, 1 << 40), INVAL), ((P, P, 1, P, -1, P, P, 32, P, 1 << 40), INVAL),
    ((P, P, 1, P, 0, P, None, 32, P, 1 << 40), INVAL), ((P, P, 1, P, 0, P, P, 8, P, 1 << 40), UNSUP),
    ((P, P, 1, P, 0, P, P, 32, None, 1 << 40), INVAL), ((P, P, 1, P, 0, P, P, 32, P, 0), WS),
    ((P + 4, P, 1, P, 0, P, P, 32, P, 1 << 40), UNSUP), ((P, P + 2, 1, P, 0, P, P, 32, P, 1 << 40), UNSUP),
    ((P, P, 1, P + 1, 0, P, P, 32, P, 1 << 40), UNSUP), ((P, P, 1, P, 0, P + 2, P, 32, P, 1 << 40), UNSUP),
    ((P, P, 1, P, 0, P, P + 2, 32, P, 1 << 40), UNSUP), ((P, P, 1, P, 0, P, P, 32, P + 64, 1 << 40), UNSUP),
    ((None, None, 0, None, 0, None, None, 32, None, 0), OK)])
def test_linear(L, args, st):
    assert L.colibri_linear_q(ctypes.byref(bank()), *args, None) == st


def test_linear_null(L):
    assert L.colibri_linear_q(None, P, P, 1, None, 0, None, P, 32, P, 1 << 40, None) == INVAL
    assert L.colibri_linear_workspace_bytes(None, 1, 32) == 0
    assert L.colibri_linear_workspace_bytes(ctypes.byref(bank()), -1, 32) == 0
    assert L.colibri_linear_workspace_bytes(ctypes.byref(bank()), 0, 32) > 0


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=4, n_heads=2, head_dim=64)
    d.update(kw)
    return block.KVCacheDesc(**d)


def batch(**kw):
    d = dict(page_table=P, cu_q=P, kv_len=P, n_seq=2, max_pages=3, n_tokens=5, max_q=3)
    d.update(kw)
    return block.KVBatchDesc(**d)


def attn(**kw):
    d = dict(q=P, out=P, lse=P, q_stride=256, out_stride=256, type=32, n_heads=4, causal=1, window=0, max_kv=100, scale=1.0)
    d.update(kw)
    return block.KVAttnDesc(**d)


CACHE_BAD = [(dict(k=None), INVAL), (dict(v=None), INVAL), (dict(k_scale=None), INVAL), (dict(v_scale=None), INVAL),
             (dict(n_pages=0), INVAL), (dict(n_heads=0), INVAL), (dict(head_dim=96), UNSUP), (dict(head_dim=0), UNSUP),
             (dict(head_dim=320), UNSUP), (dict(n_heads=1025), UNSUP), (dict(k=P + 8), UNSUP), (dict(v_scale=P + 1), UNSUP)]
BATCH_BAD = [(dict(n_seq=-1), INVAL), (dict(max_pages=-1), INVAL), (dict(n_tokens=-1), INVAL), (dict(max_q=-1), INVAL),
             (dict(n_seq=65536), UNSUP), (dict(max_pages=(1 << 24) + 1), UNSUP), (dict(cu_q=None), INVAL),
             (dict(kv_len=None), INVAL), (dict(page_table=None), INVAL), (dict(cu_q=P + 2), UNSUP)]


def three(L, c, b, a):
    r = ctypes.byref
    return (L.colibri_kv_append(r(c), r(b), P, P, 32, 128, 128, None), L.colibri_kv_read(r(c), r(b), P, P, 32, None),
            L.colibri_kv_attention(r(c), r(b), r(a), P, 1 << 50, None))


@pytest.mark.parametrize("kw,st", CACHE_BAD)
def test_cache(L, kw, st):
    c = cache(**kw)
    assert three(L, c, batch(), attn()) == (st,) * 3
    assert L.colibri_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(batch()), ctypes.byref(attn())) == 0


@pytest.mark.parametrize("kw,st", BATCH_BAD)
def test_batch(L, kw, st):
    assert three(L, cache(), batch(**kw), attn()) == (st,) * 3


@pytest.mark.parametrize("kw", [dict(n_seq=0, cu_q=None, kv_len=None, page_table=None), dict(n_tokens=0)])
def test_empty_batch(L, kw):
    assert three(L, cache(), batch(**kw), attn()) == (OK,) * 3


@pytest.mark.parametrize("args,st", [
    ((None, P, 32, 128, 128), INVAL), ((P, None, 32, 128, 128), INVAL), ((P, P, 8, 128, 128), UNSUP),
    ((P + 8, P, 32, 128, 128), UNSUP), ((P + 8, P + 4, 16, 128, 128), UNSUP), ((P, P, 32, 127, 128), INVAL),
    ((P, P, 32, 130, 128), INVAL), ((P, P, 32, 128, 64), INVAL)])
def test_append(L, args, st):
    assert L.colibri_kv_append(ctypes.byref(cache()), ctypes.byref(batch()), *args, None) == st


@pytest.mark.parametrize("args,st", [((None, None, 32), INVAL), ((P, P, 8), UNSUP), ((P + 8, P, 32), UNSUP)])
def test_read(L, args, st):
    assert L.colibri_kv_read(ctypes.byref(cache()), ctypes.byref(batch()), *args, None) == st


@pytest.mark.parametrize("kw,st", [
    (dict(q=None), INVAL), (dict(out=None), INVAL), (dict(type=8), UNSUP), (dict(n_heads=3), INVAL), (dict(n_heads=0), INVAL),
    (dict(window=-1), INVAL), (dict(window=4, causal=0), INVAL), (dict(max_kv=-1), INVAL), (dict(scale=float("nan")), INVAL),
    (dict(scale=float("inf")), INVAL), (dict(q=P + 8), UNSUP), (dict(out=P + 8), UNSUP), (dict(lse=P + 2), UNSUP),
    (dict(q_stride=255), INVAL), (dict(q_stride=260), INVAL), (dict(out_stride=248), INVAL)])
def test_attention(L, kw, st):
    r = ctypes.byref
    assert L.colibri_kv_attention(r(cache()), r(batch()), r(attn(**kw)), P, 1 << 50, None) == st


def test_attention_workspace(L):
    r = ctypes.byref
    assert L.colibri_kv_attention(r(cache()), r(batch()), r(attn()), None, 1 << 50, None) == INVAL
    assert L.colibri_kv_attention(r(cache()), r(batch()), r(attn()), P + 64, 1 << 50, None) == UNSUP
    assert L.colibri_kv_attention(r(cache()), r(batch()), r(attn()), P, 0, None) == WS
    assert L.colibri_kv_attention(r(cache()), r(batch()), None, P, 1 << 50, None) == INVAL
    assert L.colibri_kv_attention_workspace_bytes(r(cache()), r(batch()), r(attn(n_heads=5))) == 0
    many = batch(n_tokens=1 << 30)
    assert L.colibri_kv_attention(r(cache()), r(many), r(attn()), P, 1 << 62, None) == UNSUP


def test_binding_refuses():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        qre.add_rms_norm(x, torch.ones(64))
    with pytest.raises(ValueError, match="device tensor"):
        qre.linear_q(None, torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="device tensor"):
        qre.KVCache.empty(2, 1, 64, device="cpu")
    with pytest.raises(TypeError):
        block._type(torch.float16)


def test_library_exports_every_declared_symbol(L):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "colibri_block.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(colibri_\w+)\s*\(", text))
    assert len(names) == 7
    for name in names:
        assert hasattr(L, name), name
