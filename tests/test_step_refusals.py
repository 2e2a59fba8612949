"""What the operators of a serving step refuse, on the host: the C ABI returns an
error before anything is enqueued (no GPU is needed), and the binding raises on
tensors that do not fit."""

import ctypes

import pytest
import torch

import quantized_routed_expert_sigmoid_amd as qre
from quantized_routed_expert_sigmoid_amd import block, step

P = 1 << 20  # a well aligned address that no call here may touch
OK, INVAL, UNSUP, WS = 0, 1, 2, 3
BIG = 1 << 50
r = ctypes.byref


@pytest.fixture(scope="module")
def L():
    block._f()
    return step._g()


def bank(**kw):
    d = dict(data=P, row_scale=P, n_mat=1, rows=5, K=64, qtype=4, group=0)
    d.update(kw)
    return qre.QBankDesc(**d)


BANK_BAD = [(dict(n_mat=2), INVAL), (dict(rows=0), INVAL), (dict(K=40), INVAL), (dict(K=0), INVAL), (dict(data=None), INVAL),
            (dict(row_scale=None), INVAL), (dict(qtype=5), UNSUP), (dict(rows=(1 << 20) + 1), UNSUP),
            (dict(K=(1 << 15) + 32), UNSUP), (dict(data=P + 4), UNSUP), (dict(row_scale=P + 2), UNSUP)]


@pytest.mark.parametrize("kw,st", BANK_BAD + [(dict(group=48), INVAL), (dict(group=-32), INVAL), (dict(group=128), INVAL)])
def test_embed_bank(L, kw, st):
    assert L.colibri_embed_q(r(bank(**kw)), P, 4, 1, 1.0, P, 32, None) == st


@pytest.mark.parametrize("args,st", [
    ((None, 4, 1, 1.0, P, 32), INVAL), ((P, 4, 1, 1.0, None, 32), INVAL), ((P, 4, -1, 1.0, P, 32), INVAL),
    ((P, 4, 1, float("nan"), P, 32), INVAL), ((P, 4, 1, float("inf"), P, 32), INVAL), ((P, 2, 1, 1.0, P, 32), UNSUP),
    ((P, 4, 1, 1.0, P, 8), UNSUP), ((P, 4, 65537, 1.0, P, 32), UNSUP), ((P + 2, 4, 1, 1.0, P, 32), UNSUP),
    ((P + 4, 8, 1, 1.0, P, 32), UNSUP), ((P, 4, 1, 1.0, P + 8, 16), UNSUP), ((None, 4, 0, 1.0, None, 32), OK)])
def test_embed(L, args, st):
    assert L.colibri_embed_q(r(bank()), *args, None) == st
    assert L.colibri_embed_q(None, P, 4, 1, 1.0, P, 32, None) == INVAL


def pages(**kw):
    d = dict(refs=P, page_table=P, kv_len=P, n_pages=9, n_seq=3, max_pages=4)
    d.update(kw)
    return step.KVPagesDesc(**d)


def five(L, p):
    return (L.colibri_kv_extend(r(p), P, P, P, P, P, BIG, None), L.colibri_kv_trim(r(p), P, None),
            L.colibri_kv_fork(r(p), P, P, 2, None), L.colibri_kv_compact(r(p), P, P, P, P, BIG, None))


@pytest.mark.parametrize("kw,st", [
    (dict(n_pages=0), INVAL), (dict(n_seq=-1), INVAL), (dict(max_pages=-1), INVAL), (dict(n_pages=(1 << 26) + 1), UNSUP),
    (dict(n_seq=65536), UNSUP), (dict(max_pages=(1 << 24) + 1), UNSUP), (dict(refs=None), INVAL), (dict(kv_len=None), INVAL),
    (dict(page_table=None), INVAL), (dict(refs=P + 2), UNSUP), (dict(kv_len=P + 1), UNSUP), (dict(page_table=P + 3), UNSUP)])
def test_pages(L, kw, st):
    assert five(L, pages(**kw)) == (st,) * 4


def test_pages_null_and_empty(L):
    assert L.colibri_kv_trim(None, P, None) == INVAL and L.colibri_kv_pages_workspace_bytes(None) == 0
    assert five(L, pages(n_seq=0, page_table=None, kv_len=None))[:3] == (OK,) * 3
    assert L.colibri_kv_fork(r(pages()), None, None, 0, None) == OK
    assert L.colibri_kv_pages_workspace_bytes(r(pages(n_pages=0))) == 0
    assert L.colibri_kv_pages_workspace_bytes(r(pages(refs=None))) >= 4 * (9 + 3)


@pytest.mark.parametrize("i", range(4))
def test_extend(L, i):
    def call(a, ws=P, n=BIG):
        return L.colibri_kv_extend(r(pages()), *a, ws, n, None)
    assert call([None if j == i else P for j in range(4)]) == INVAL
    assert call([P + 2 if j == i else P for j in range(4)]) == UNSUP
    assert call([P] * 4, None) == INVAL and call([P] * 4, P + 64) == UNSUP and call([P] * 4, P, 0) == WS


def test_trim_fork_compact(L):
    p = pages()
    assert L.colibri_kv_trim(r(p), None, None) == INVAL and L.colibri_kv_trim(r(p), P + 1, None) == UNSUP
    for a, st in [((None, P, 1), INVAL), ((P, None, 1), INVAL), ((P, P, -1), INVAL), ((P, P, 65536), UNSUP),
                  ((P + 2, P, 1), UNSUP), ((P, P + 2, 1), UNSUP)]:
        assert L.colibri_kv_fork(r(p), *a, None) == st
    for a, st in [((None, P, P, P, BIG), INVAL), ((P, None, P, P, BIG), INVAL), ((P, P, None, P, BIG), INVAL),
                  ((P, P, P, None, BIG), INVAL), ((P, P, P, P + 16, BIG), UNSUP), ((P, P, P, P, 16), WS),
                  ((P + 2, P, P, P, BIG), UNSUP), ((P, P, P + 2, P, BIG), UNSUP)]:
        assert L.colibri_kv_compact(r(p), *a, None) == st


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=4, n_heads=2, head_dim=64)
    d.update(kw)
    return block.KVCacheDesc(**d)


@pytest.mark.parametrize("kw,st", [
    (dict(k=None), INVAL), (dict(v=None), INVAL), (dict(k_scale=None), INVAL), (dict(v_scale=None), INVAL),
    (dict(n_pages=0), INVAL), (dict(n_heads=0), INVAL), (dict(head_dim=96), UNSUP), (dict(n_heads=1025), UNSUP),
    (dict(k=P + 8), UNSUP), (dict(v_scale=P + 1), UNSUP), (dict(n_heads=3), INVAL), (dict(head_dim=128), INVAL)])
def test_copy_caches(L, kw, st):
    assert L.colibri_kv_copy(r(cache(**kw)), r(cache()), P, P, 1, None) == st
    assert L.colibri_kv_copy(r(cache()), r(cache(**kw)), P, P, 1, None) == st


def test_copy(L):
    def call(*a):
        return L.colibri_kv_copy(r(cache()), r(cache()), *a, None)
    assert call(None, P, 1) == INVAL and call(P, None, 1) == INVAL and call(P, P, -1) == INVAL
    assert call(P + 2, P, 1) == UNSUP and call(P, P + 2, 1) == UNSUP and call(None, None, 0) == OK
    assert L.colibri_kv_copy(None, r(cache()), P, P, 1, None) == INVAL


def test_binding_refuses():
    with pytest.raises(ValueError, match="device tensor"):
        qre.embed_q(None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        qre.KVPages.empty(2, 3, 4, device="cpu")


def test_library_exports_every_declared_symbol(L):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "colibri_step.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(colibri_\w+)\s*\(", text))
    assert names
    for name in names:
        assert hasattr(L, name), name


def logits(**kw):
    d = dict({n: P for n in ("logits", "out", "token", "lse", "tokens", "spans", "penalties", "bias", "bias_ids", "cu_bias",
                             "mask", "mask_of")}, logits_stride=100, out_stride=100, mask_stride=4, type=32, rows=2,
             vocab=100, n_tokens=5, n_bias=5, n_masks=1)
    d.update(kw)
    return step.LogitsDesc(**d)


@pytest.mark.parametrize("kw,st", [
    (dict(rows=-1), INVAL), (dict(vocab=0), INVAL), (dict(rows=65536), UNSUP),
    (dict(vocab=(1 << 20) + 1, logits_stride=1 << 21, out_stride=1 << 21), UNSUP),
    (dict(type=8), UNSUP), (dict(n_tokens=-1), INVAL), (dict(n_bias=-1), INVAL), (dict(n_masks=-1), INVAL),
    (dict(n_bias=(1 << 30) + 1), UNSUP),
    (dict(logits=None), INVAL), (dict(out=None, token=None, lse=None), INVAL), (dict(spans=None), INVAL),
    (dict(tokens=None), INVAL), (dict(bias=None), INVAL), (dict(bias_ids=None), INVAL), (dict(mask_of=None), INVAL),
    (dict(mask_stride=3), INVAL), (dict(logits_stride=99), INVAL), (dict(out_stride=99, out=P + 4096), INVAL),
    (dict(out_stride=101), INVAL), (dict(logits_stride=1 << 41, out=P + 4096), UNSUP), (dict(logits=P + 2), UNSUP),
    (dict(out=P + 2), UNSUP), (dict(token=P + 2), UNSUP), (dict(lse=P + 1), UNSUP), (dict(tokens=P + 2), UNSUP),
    (dict(spans=P + 2), UNSUP), (dict(penalties=P + 2), UNSUP), (dict(bias=P + 2), UNSUP), (dict(bias_ids=P + 2), UNSUP),
    (dict(cu_bias=P + 2), UNSUP), (dict(mask=P + 2), UNSUP), (dict(mask_of=P + 2), UNSUP),
    (dict(logits=P + 1, type=16), UNSUP),
    (dict(rows=0, logits=None), OK)])
def test_logits(L, kw, st):
    assert L.colibri_adjust_logits(r(logits(**kw)), P, BIG, None) == st


def test_logits_workspace(L):
    assert L.colibri_adjust_logits(None, P, BIG, None) == INVAL
    assert L.colibri_adjust_logits(r(logits()), None, BIG, None) == INVAL
    assert L.colibri_adjust_logits(r(logits()), P + 64, BIG, None) == UNSUP
    assert L.colibri_adjust_logits(r(logits()), P, 0, None) == WS
    for rows, vocab in ((-1, 5), (65536, 5), (1, 0), (1, (1 << 20) + 1)):
        assert L.colibri_logits_workspace_bytes(rows, vocab) == 0
    sizes = [L.colibri_logits_workspace_bytes(rows, v) for rows in (0, 1, 7, 65535) for v in (1, 4096, 4097, 1 << 20)]
    assert all(sizes) and sizes == sorted(sizes[:4]) + sorted(sizes[4:8]) + sorted(sizes[8:12]) + sorted(sizes[12:])


def test_logits_binding_refuses():
    with pytest.raises(ValueError, match="device tensor"):
        qre.adjust_logits(torch.zeros(2, 5))


@pytest.mark.parametrize("a,st", [
    ((None, 32, 64, 2, 64, P, P), INVAL), ((P, 32, 64, 2, 64, None, P), INVAL), ((P, 32, 64, 2, 64, P, None), INVAL),
    ((P, 32, 64, -1, 64, P, P), INVAL), ((P, 32, 64, 2, 48, P, P), INVAL), ((P, 32, 64, 2, 0, P, P), INVAL),
    ((P, 32, 60, 2, 64, P, P), INVAL), ((P, 32, 66, 2, 64, P, P), INVAL), ((P, 8, 64, 2, 64, P, P), UNSUP),
    ((P, 32, 1 << 41, 2, 64, P, P), UNSUP), ((P, 32, 32800, 2, 32800, P, P), UNSUP), ((P, 32, 64, 65537, 64, P, P), UNSUP),
    ((P + 8, 32, 64, 2, 64, P, P), UNSUP), ((P + 4, 16, 64, 2, 64, P, P), UNSUP), ((P, 32, 64, 2, 64, P + 8, P), UNSUP),
    ((P, 32, 64, 2, 64, P, P + 2), UNSUP), ((None, 32, 64, 0, 64, None, None), OK)])
def test_quantize(L, a, st):
    assert L.colibri_quantize_i8(*a, None) == st


@pytest.mark.parametrize("kw,st", [
    (dict(rows=-1), INVAL), (dict(K=48), INVAL), (dict(K=8224, x_stride=8224), UNSUP), (dict(x=None), INVAL),
    (dict(q=None), INVAL), (dict(d=None), INVAL), (dict(sum=None, y=None, q=None, d=None), INVAL), (dict(x_type=8), UNSUP),
    (dict(eps=float("nan")), INVAL), (dict(x=P + 8), UNSUP), (dict(q=P + 2), UNSUP), (dict(x_stride=60), INVAL),
    (dict(residual_stride=63), INVAL), (dict(rows=0, x=None), OK)])
def test_norm(L, kw, st):
    d = dict(x=P, residual=P, weight=P, sum=P, y=P, q=P, d=P, x_stride=64, residual_stride=64, rows=2, K=64, x_type=32,
             residual_type=32, y_type=32, eps=1e-6)
    assert L.colibri_add_rms_norm_i8(r(block.NormDesc(**d | kw)), None) == st
    assert L.colibri_add_rms_norm_i8(None, None) == INVAL


@pytest.mark.parametrize("kw,st", BANK_BAD + [(dict(group=32), UNSUP), (dict(group=48), INVAL)])
def test_linear_bank(L, kw, st):
    w = bank(**kw)
    assert L.colibri_linear_i8(r(w), P, P, 1, None, 0, None, P, 32, P, BIG, None) == st
    assert L.colibri_linear_i8_workspace_bytes(r(w), 1, 32) == 0


@pytest.mark.parametrize("a,st", [
    ((None, P, 1, P, 0, P, P, 32, P, BIG), INVAL), ((P, None, 1, P, 0, P, P, 32, P, BIG), INVAL),
    ((P, P, -1, P, 0, P, P, 32, P, BIG), INVAL), ((P, P, 65537, P, 0, P, P, 32, P, BIG), UNSUP),
    ((P, P, 1, P, 4, P, P, 32, P, BIG), INVAL), ((P, P, 1, P, -1, P, P, 32, P, BIG), INVAL),
    ((P, P, 1, P, 0, P, None, 32, P, BIG), INVAL), ((P, P, 1, P, 0, P, P, 8, P, BIG), UNSUP),
    ((P, P, 1, P, 0, P, P, 32, None, BIG), INVAL), ((P, P, 1, P, 0, P, P, 32, P, 0), WS),
    ((P + 4, P, 1, P, 0, P, P, 32, P, BIG), UNSUP), ((P, P + 2, 1, P, 0, P, P, 32, P, BIG), UNSUP),
    ((P, P, 1, P + 1, 0, P, P, 32, P, BIG), UNSUP), ((P, P, 1, P, 0, P + 2, P, 32, P, BIG), UNSUP),
    ((P, P, 1, P, 0, P, P + 2, 32, P, BIG), UNSUP), ((P, P, 1, P, 0, P, P, 32, P + 64, BIG), UNSUP),
    ((None, None, 0, None, 0, None, None, 32, None, 0), OK)])
def test_linear(L, a, st):
    assert L.colibri_linear_i8(r(bank()), *a, None) == st


def test_linear_null(L):
    assert L.colibri_linear_i8(None, P, P, 1, None, 0, None, P, 32, P, BIG, None) == INVAL
    assert L.colibri_linear_i8_workspace_bytes(None, 1, 32) == 0
    assert L.colibri_linear_i8_workspace_bytes(r(bank()), -1, 32) == 0
    assert L.colibri_linear_i8_workspace_bytes(r(bank()), 0, 32) > 0


@pytest.mark.parametrize("N,K", [(10240, 6144), (4096, 4096), (130, 2080), (64, 512), (1, 32768), (32768, 2048), (2100, 224),
                                 (16, 128)])
@pytest.mark.parametrize("bits", [8, 4])
def test_linear_workspace_grows_with_the_batch(L, N, K, bits):
    """A workspace for S tokens serves every smaller batch: its size never falls."""
    w = bank(rows=N, K=K, qtype=bits)
    sizes = sorted(set(range(1, 1300, 7)) | {64, 65, 128, 129, 256, 257, 2047, 2048, 2049, 4096, 8192, 16384,
                                            32767, 32768, 65536})
    most = [L.colibri_linear_i8_workspace_bytes(r(w), S, 32) for S in sizes]
    assert all(a <= b for a, b in zip(most, most[1:])), list(zip(sizes, most))
