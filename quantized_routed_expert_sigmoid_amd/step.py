"""Python binding of the operators of a serving step (include/colibri_step.h):
embedding lookup, the sequences of a paged cache from step to step, the linear
product with one activation scale per token, and what is done to logits.

Argument marshalling only, as in block.py: tensors are on one GPU, work is
enqueued on that GPU's current stream, nothing synchronises, and a refused call
raises before anything is enqueued.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

import quantized_routed_expert_sigmoid_amd as _qre

from .block import KVCache, _at, _call, _dev, _f32, _flat, _i32, _i64, _on, _room, _type, _vp

_IDS = {torch.int32: 4, torch.int64: 8}


class KVPagesDesc(ctypes.Structure):
    """coli_kv_pages"""
    _fields_ = [("refs", _vp), ("page_table", _vp), ("kv_len", _vp), ("n_pages", _i32), ("n_seq", _i32),
                ("max_pages", _i32)]


_fns = None  # (the library,)


def _g():
    """The library, with the argument types of these entry points set."""
    global _fns
    L = _qre._lib or _qre.lib()
    if _fns is None or _fns[0] is not L:
        sz, ci = ctypes.c_size_t, ctypes.c_int
        for name, res, args in [
                ("colibri_embed_q", ci, [_vp, _vp, _i32, _i32, _f32, _vp, _i32, _vp]),
                ("colibri_kv_pages_workspace_bytes", sz, [_vp]),
                ("colibri_kv_extend", ci, [_vp, _vp, _vp, _vp, _vp, _vp, sz, _vp]),
                ("colibri_kv_trim", ci, [_vp, _vp, _vp]),
                ("colibri_kv_fork", ci, [_vp, _vp, _vp, _i32, _vp]),
                ("colibri_kv_compact", ci, [_vp, _vp, _vp, _vp, _vp, sz, _vp]),
                ("colibri_kv_copy", ci, [_vp, _vp, _vp, _vp, _i32, _vp])]:
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _fns = (L,)
    return L


def _do(dev: torch.device, name: str, *args):
    _g()
    _call(dev, name, *args)


def _bank_scales(bank, w):
    if bank.scale.dtype != torch.float32 or (
            bank.scale.numel() != w.n_mat * w.rows * (w.K // w.group if w.group else 1)):
        raise ValueError("bank: one fp32 scale per row, or per group, expected")


# ---------------------------------------------------------------------------


def embed_q(bank, ids: torch.Tensor, scale: float = 1.0, *, dtype: Optional[torch.dtype] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[i] = row ids[i] of the bank times scale, [n][K] of `dtype` (default: out's, or fp32).

    bank: a QBank of one matrix [1][rows][K] (int8, int4 or int2, scales per row
    or per group); ids int32 or int64 [n], one outside [0, rows) gives zeros."""
    dev = _dev(ids)
    if ids.dtype not in _IDS:
        raise TypeError(f"ids: int32 or int64 expected, got {ids.dtype}")
    if ids.dim() != 1:
        raise ValueError("ids: [n] expected")
    w, n = bank.desc(), ids.shape[0]
    dtype = dtype or (out.dtype if out is not None else torch.float32)
    t = _type(dtype)
    _on(dev, bank.data, bank.scale, out)
    _bank_scales(bank, w)
    _flat(ids, ids.dtype, (n,), "ids")
    _flat(out, dtype, (n, w.K), "out")
    if out is None:
        out = torch.empty(n, w.K, dtype=dtype, device=dev)
    _do(dev, "colibri_embed_q", ctypes.byref(w), ids.data_ptr(), _IDS[ids.dtype], n, scale, out.data_ptr(), t)
    return out


# ---------------------------------------------------------------------------


class KVPages:
    """The sequences of a paged cache: page_table int32 [n_seq][max_pages] and
    kv_len int32 [n_seq] (what kv_append and kv_attention take) with refs int32
    [n_pages], the number of entries that hold each page.  The caches of all layers
    share one."""

    def __init__(self, page_table: torch.Tensor, kv_len: torch.Tensor, refs: torch.Tensor):
        dev = _dev(page_table)
        _on(dev, kv_len, refs)
        if page_table.dim() != 2:
            raise ValueError("page_table: [n_seq][max_pages] expected")
        n, mp = page_table.shape
        _flat(page_table, torch.int32, (n, mp), "page_table")
        _flat(kv_len, torch.int32, (n,), "kv_len")
        if refs.dim() != 1:
            raise ValueError("refs: [n_pages] expected")
        _flat(refs, torch.int32, refs.shape, "refs")
        self.page_table, self.kv_len, self.refs = page_table, kv_len, refs
        self.n_seq, self.max_pages, self.n_pages = n, mp, refs.shape[0]
        self.desc = KVPagesDesc(refs.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(), self.n_pages, n, mp)

    @classmethod
    def empty(cls, n_seq: int, max_pages: int, n_pages: int, device="cuda") -> "KVPages":
        """n_seq empty sequences of at most max_pages pages of a pool of n_pages."""
        table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=device)
        kv_len, refs = (torch.zeros(n, dtype=torch.int32, device=device) for n in (n_seq, n_pages))
        return cls(table, kv_len, refs)


class KVExtend(NamedTuple):
    """granted, src and dst int32 [n_seq]: the tokens that each sequence got, and the copies to make."""
    granted: torch.Tensor
    src: torch.Tensor
    dst: torch.Tensor


class KVMoves(NamedTuple):
    """src and dst int32 [n_pages // 2], -1 behind the last move; n_live int32 [1]."""
    src: torch.Tensor
    dst: torch.Tensor
    n_live: torch.Tensor


def kv_pages_workspace(pages: KVPages) -> torch.Tensor:
    """Workspace of kv_extend and kv_compact; calls that may overlap need one each."""
    n = _g().colibri_kv_pages_workspace_bytes(ctypes.byref(pages.desc))
    if n == 0:
        raise _qre.ColibriError(_qre.COLI_E_INVAL, "colibri_kv_pages_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=pages.refs.device)


def kv_extend(pages: KVPages, add: torch.Tensor, *, ws: Optional[torch.Tensor] = None) -> KVExtend:
    """Room for add[s] (int32 [n_seq]) more tokens of each sequence, as kv_append needs
    it: kv_len grows and new blocks get free pages.  Where the last block's page
    is shared the sequence gets one of its own: run kv_copy(cache, src, dst) on
    every layer's cache before pages change again.  A sequence whose table or
    whose share of the free pages (given out in sequence order) does not suffice
    stays as it is, granted[s] = 0."""
    dev = pages.refs.device
    _on(dev, add, ws)
    _flat(add, torch.int32, (pages.n_seq,), "add")
    ws = kv_pages_workspace(pages) if ws is None else ws
    r = KVExtend(*torch.empty(3, pages.n_seq, dtype=torch.int32, device=dev).unbind(0))
    _do(dev, "colibri_kv_extend", ctypes.byref(pages.desc), add.data_ptr(), r.granted.data_ptr(), r.src.data_ptr(),
        r.dst.data_ptr(), *_room(ws))
    return r


def kv_trim(pages: KVPages, new_len: torch.Tensor):
    """Shortens each sequence to new_len[s] (int32 [n_seq]) tokens and frees the
    pages that no sequence holds any more; 0 frees the sequence, a negative number
    or one that is not below kv_len[s] leaves it as it is."""
    _on(pages.refs.device, new_len)
    _flat(new_len, torch.int32, (pages.n_seq,), "new_len")
    _do(pages.refs.device, "colibri_kv_trim", ctypes.byref(pages.desc), new_len.data_ptr())


def kv_fork(pages: KVPages, parent: torch.Tensor, child: torch.Tensor):
    """Makes the empty sequences child[i] equal to parent[i] (int32 [n] each) by
    sharing their pages; kv_extend gives them pages of their own as they grow.
    Skipped are pairs with a number outside the sequences, with a child that is
    not empty or that an earlier pair names, and with a parent that is a child too."""
    _on(pages.refs.device, parent, child)
    if parent.dim() != 1:
        raise ValueError("parent: [n] expected")
    _flat(parent, torch.int32, parent.shape, "parent")
    _flat(child, torch.int32, parent.shape, "child")
    _do(pages.refs.device, "colibri_kv_fork", ctypes.byref(pages.desc), parent.data_ptr(), child.data_ptr(),
        parent.shape[0])


def kv_compact(pages: KVPages, *, ws: Optional[torch.Tensor] = None) -> KVMoves:
    """Moves the used pages to the front: used pages from n_live on take the places
    of the free ones below it.  Run kv_copy(cache, src, dst) on every layer's cache."""
    dev = pages.refs.device
    _on(dev, ws)
    ws = kv_pages_workspace(pages) if ws is None else ws
    r = KVMoves(*torch.empty(2, pages.n_pages // 2, dtype=torch.int32, device=dev).unbind(0),
                torch.empty(1, dtype=torch.int32, device=dev))
    _do(dev, "colibri_kv_compact", ctypes.byref(pages.desc), r.src.data_ptr(), r.dst.data_ptr(), r.n_live.data_ptr(),
        *_room(ws))
    return r


def kv_copy(cache: KVCache, src: torch.Tensor, dst: torch.Tensor, *, to: Optional[KVCache] = None):
    """Copies page src[i] (int32 [n]) of the cache, with its scales, to page dst[i] of `to`
    (default: of the same cache).  Pairs with a number outside their cache are skipped; no
    page is written twice, and none that is read."""
    to = cache if to is None else to
    dev = cache.k.device
    _on(dev, to.k, src, dst)
    if src.dim() != 1:
        raise ValueError("src: [n] expected")
    _flat(src, torch.int32, src.shape, "src")
    _flat(dst, torch.int32, src.shape, "dst")
    _do(dev, "colibri_kv_copy", ctypes.byref(cache.desc), ctypes.byref(to.desc), src.data_ptr(), dst.data_ptr(),
        src.shape[0])
