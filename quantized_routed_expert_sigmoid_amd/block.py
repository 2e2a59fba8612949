"""Python binding of the operators around the layer (include/colibri_block.h): the
residual addition with root-mean-square norm and Q8_0, the quantised matrix
product with its epilogue, and attention over a paged int8 cache.

Argument marshalling only, as in the package itself: tensors are on one GPU,
work is enqueued on that GPU's current stream, nothing synchronises, and a
refused call raises before anything is enqueued.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

import quantized_routed_expert_sigmoid_amd as _qre

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_TYPES = {torch.float32: 32, torch.bfloat16: 16}
_ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
KV_BLOCK = 64


class NormDesc(ctypes.Structure):
    """coli_norm"""
    _fields_ = [("x", _vp), ("residual", _vp), ("weight", _vp), ("sum", _vp), ("y", _vp), ("q", _vp), ("d", _vp),
                ("x_stride", _i64), ("residual_stride", _i64), ("rows", _i32), ("K", _i32), ("x_type", _i32),
                ("residual_type", _i32), ("y_type", _i32), ("eps", _f32)]


class KVCacheDesc(ctypes.Structure):
    """coli_kv_cache"""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("n_pages", _i32), ("n_heads", _i32),
                ("head_dim", _i32)]


class KVBatchDesc(ctypes.Structure):
    """coli_kv_batch"""
    _fields_ = [("page_table", _vp), ("cu_q", _vp), ("kv_len", _vp), ("n_seq", _i32), ("max_pages", _i32),
                ("n_tokens", _i32), ("max_q", _i32)]


class KVAttnDesc(ctypes.Structure):
    """coli_kv_attn"""
    _fields_ = [("q", _vp), ("out", _vp), ("lse", _vp), ("q_stride", _i64), ("out_stride", _i64), ("type", _i32),
                ("n_heads", _i32), ("causal", _i32), ("window", _i32), ("max_kv", _i32), ("scale", _f32)]


# the current stream's handle and the current device's number, without the
# objects that torch.cuda builds around them (a few microseconds a call) where
# this torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

_fns = None  # (the library, its entry points)


def _f():
    """The library's entry points with their argument types."""
    global _fns
    L = _qre._lib or _qre.lib()
    if _fns is None or _fns[0] is not L:
        sz, ci = ctypes.c_size_t, ctypes.c_int
        for name, res, args in [
                ("colibri_add_rms_norm", ci, [_vp, _vp]),
                ("colibri_linear_workspace_bytes", sz, [_vp, _i32, _i32]),
                ("colibri_linear_q", ci, [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, sz, _vp]),
                ("colibri_kv_append", ci, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _vp]),
                ("colibri_kv_read", ci, [_vp, _vp, _vp, _vp, _i32, _vp]),
                ("colibri_kv_attention_workspace_bytes", sz, [_vp, _vp, _vp]),
                ("colibri_kv_attention", ci, [_vp, _vp, _vp, _vp, sz, _vp])]:
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _fns = (L,)
    return L


def _type(dtype: torch.dtype) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"float32 or bfloat16 expected, got {dtype}")
    return t


def _on(dev: torch.device, *tensors: Optional[torch.Tensor]):
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on one device expected: {t.device} beside {dev}")


def _dev(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    return t.device


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _flat(t: Optional[torch.Tensor], dtype: torch.dtype, shape: tuple, what: str):
    """t is contiguous, of this type and shape (or None)."""
    if t is None or (t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    raise ValueError(f"{what}: contiguous tensor expected")


def _room(ws: torch.Tensor):
    """Address and bytes of a workspace."""
    if not ws.is_contiguous():
        raise ValueError("ws: contiguous tensor expected")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _call(dev: torch.device, name: str, *args):
    """Enqueues on the current stream of the tensors' device, which may not be the current one."""
    fn, index = getattr(_f(), name), dev.index
    stream = _raw_stream(index)
    if index == _current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        raise _qre.ColibriError(st, name)


# ---------------------------------------------------------------------------


class NormResult(NamedTuple):
    """sum [rows][K], y [rows][K], q int8 [rows][K] and d fp32 [rows][K/32]; None where not asked for."""
    sum: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    d: Optional[torch.Tensor]


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                 residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                 y_dtype: Optional[torch.dtype] = None, q8: bool = True) -> NormResult:
    """t = x + residual, y = t / sqrt(mean(t^2) + eps) * weight, and Q8_0 of y.

    x and residual: [rows][K] fp32 or bf16, rows may be strided; weight fp32
    [K].  With a residual the sum is returned in its type, in sum_out if given
    (which may be residual or x itself, to update the stream in place).  y is
    returned in y_dtype if that is given (the layer takes fp32), the Q8_0 codes
    and scales (what linear_q takes) unless q8 is False."""
    dev = _dev(x)
    if not (x.dim() == 2):
        raise ValueError("x: [rows][K] expected")
    rows, K = x.shape
    xt = _type(x.dtype)
    _on(dev, weight, residual, sum_out)
    _flat(weight, torch.float32, (K,), "weight")
    if not (rows <= 1 or x.stride(0) >= K):
        raise ValueError("x: rows that do not overlap expected")
    if not (K == 0 or x.stride(1) == 1):
        raise ValueError("x: contiguous rows expected")
    rt, rs = xt, K
    if residual is not None:
        if not (residual.shape == x.shape):
            raise ValueError("residual: the shape of x expected")
        if not (residual.stride(1) == 1):
            raise ValueError("residual: contiguous rows expected")
        rt, rs = _type(residual.dtype), residual.stride(0) if rows > 1 else K
        if sum_out is None:
            sum_out = torch.empty(rows, K, dtype=residual.dtype, device=dev)
    elif sum_out is not None:
        rt = _type(sum_out.dtype)
    if sum_out is not None:
        _flat(sum_out, residual.dtype if residual is not None else sum_out.dtype, (rows, K), "sum_out")
    y = None if y_dtype is None else torch.empty(rows, K, dtype=y_dtype, device=dev)
    q = d = None
    if q8:
        q = torch.empty(rows, K, dtype=torch.int8, device=dev)
        d = torch.empty(rows, K // 32, dtype=torch.float32, device=dev)
    n = NormDesc(x.data_ptr(), _at(residual), weight.data_ptr(), _at(sum_out), _at(y), _at(q), _at(d),
                 x.stride(0) if rows > 1 else K, rs, rows, K, xt, rt, xt if y is None else _type(y_dtype), eps)
    _call(dev, "colibri_add_rms_norm", ctypes.byref(n))
    return NormResult(sum_out, y, q, d)


def linear_workspace(bank, S: int, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Workspace of linear_q for any number of tokens up to S and outputs of this type; calls that may overlap need
    one each."""
    return _linear_ws(bank.desc(), _length(S), _type(dtype), bank.data.device)


def _linear_ws(w, S: int, t: int, dev: torch.device) -> torch.Tensor:
    n = _f().colibri_linear_workspace_bytes(ctypes.byref(w), S, t)
    if n == 0:
        raise _qre.ColibriError(_qre.COLI_E_INVAL, "colibri_linear_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=dev)


def linear_q(bank, xq: torch.Tensor, xd: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
             activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
             dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t][r] = act(sum_k W[r][k] x[t][k] + bias[r]) + residual[t][r].

    bank: a QBank of one matrix [1][rows][K]; xq int8 [S][K] and xd fp32
    [S][K/32] are the activations' Q8_0 form (add_rms_norm, quantize_q8_0);
    bias fp32 [rows]; activation None, "relu", "silu" or "gelu"; residual and
    out [S][rows] of `dtype` (default: theirs, or fp32); out may be residual."""
    dev = _dev(xq)
    if activation not in _ACTS:
        raise ValueError(f"activation: one of {[a for a in _ACTS if a]} expected, got {activation!r}")
    w = bank.desc()
    if not (xq.dim() == 2 and xq.shape[1] == w.K):
        raise ValueError(f"xq: [S][{w.K}] expected, got {tuple(xq.shape)}")
    S = xq.shape[0]
    given = out if out is not None else residual
    dtype = dtype or (given.dtype if given is not None else torch.float32)
    t = _type(dtype)
    _on(dev, xd, bias, residual, out, ws, bank.data, bank.scale)
    _flat(xq, torch.int8, (S, w.K), "xq")
    _flat(xd, torch.float32, (S, w.K // 32), "xd")
    _flat(bias, torch.float32, (w.rows,), "bias")
    _flat(residual, dtype, (S, w.rows), "residual")
    _flat(out, dtype, (S, w.rows), "out")
    if bank.scale.dtype != torch.float32 or (
            bank.scale.numel() != w.n_mat * w.rows * (w.K // w.group if w.group else 1)):
        raise ValueError("bank: one fp32 scale per row, or per group, expected")
    if out is None:
        out = torch.empty(S, w.rows, dtype=dtype, device=dev)
    if ws is None:
        ws = _linear_ws(w, S, t, dev)
        room = ws.data_ptr(), ws.numel()
    else:
        room = _room(ws)
    _call(dev, "colibri_linear_q", ctypes.byref(w), xq.data_ptr(), xd.data_ptr(), S, _at(bias), _ACTS[activation],
          _at(residual), out.data_ptr(), t, *room)
    return out


# ---------------------------------------------------------------------------


def kv_page_shape(n_pages: int, n_heads: int, head_dim: int) -> Tuple[int, int, int]:
    """Shape of KVCache.k and .v."""
    return (n_pages, n_heads, KV_BLOCK * head_dim)


class KVCache:
    """A paged int8 cache of keys and values: k, v int8 [n_pages][n_heads][64 * head_dim]
    (the codes of one block of 64 tokens and head in the order given in
    include/colibri_block.h), k_scale, v_scale fp32 [n_pages][n_heads]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 head_dim: int):
        dev = _dev(k)
        _on(dev, v, k_scale, v_scale)
        if not (k.dim() == 3 and k.shape[2] == KV_BLOCK * head_dim):
            raise ValueError(f"k: [n_pages][n_heads][{KV_BLOCK * head_dim}] expected, got {tuple(k.shape)}")
        _flat(k, torch.int8, k.shape, "k")
        _flat(v, torch.int8, k.shape, "v")
        _flat(k_scale, torch.float32, k.shape[:2], "k_scale")
        _flat(v_scale, torch.float32, k.shape[:2], "v_scale")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_heads, self.head_dim = k.shape[0], k.shape[1], head_dim
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.n_pages,
                                self.n_heads, head_dim)

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of n_pages unwritten pages."""
        shape = kv_page_shape(n_pages, n_heads, head_dim)
        k, v = (torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2))
        ks, vs = (torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs, head_dim)


_MOST = 0x7FFFFFFF


def _length(n: int) -> int:
    """n in 32 bits: beyond them the largest number there is, below zero -1 (which the library refuses)."""
    return -1 if n < 0 else min(n, _MOST)


def _longest(n_tokens: int, n_seq: int, least: int) -> int:
    """The longest run of rows to expect of a batch of which nothing else is known.

    Decode and verify steps have equal or nearly equal runs.  Otherwise one sequence may hold most of the rows, and
    `least` is the run that fills the chip by itself: a longer one takes several turns there, where the shape for it
    would start workgroups for every sequence as if each were as long (attention, 64 / 8 heads: 200 prompts of 40 rows
    444 us, 1522 with all rows as the longest run; one prompt of 900 rows among 63 decoding sequences 197 us, 2388 with
    the rows evenly shared out)."""
    if n_seq == 0 or n_tokens == 0:
        return n_tokens
    even = -(-n_tokens // n_seq)
    if n_tokens <= 4 * n_seq or (n_tokens <= 16 * n_seq and n_tokens % n_seq == 0):
        return even
    return min(n_tokens, max(2 * even, least))


def _batch(cache: KVCache, page_table, cu_q, kv_len, n_tokens: int, max_q: Optional[int], least: int) -> KVBatchDesc:
    dev = cache.k.device
    _on(dev, page_table, cu_q, kv_len)
    if not (page_table.dim() == 2):
        raise ValueError("page_table: [n_seq][max_pages] expected")
    n, mp = page_table.shape
    _flat(page_table, torch.int32, (n, mp), "page_table")
    _flat(cu_q, torch.int32, (n + 1,), "cu_q")
    _flat(kv_len, torch.int32, (n,), "kv_len")
    if max_q is None:
        max_q = _longest(n_tokens, n, least)
    elif not 0 <= max_q <= _MOST:
        max_q = _length(max_q)
    return KVBatchDesc(page_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), n, mp, n_tokens, max_q)


def _rows(t: torch.Tensor, n_heads: int, D: int, what: str) -> int:
    """Stride between the tokens of t [n_tokens][n_heads][D], whose heads lie together."""
    if not (t.dim() == 3 and t.shape[1] == n_heads and t.shape[2] == D):
        raise ValueError(f"{what}: [n_tokens][{n_heads}][{D}] expected, got {tuple(t.shape)}")
    if not (t.stride(2) == 1 and (n_heads == 1 or t.stride(1) == D)):
        raise ValueError(f"{what}: contiguous heads expected")
    return t.stride(0) if t.shape[0] > 1 else n_heads * D


def kv_append(cache: KVCache, page_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, k: torch.Tensor,
              v: torch.Tensor, *, max_q: Optional[int] = None):
    """Writes new keys and values [n_tokens][n_heads][head_dim] (fp32 or bf16,
    tokens may be strided) to the last places of their sequences: rows cu_q[s]
    .. cu_q[s+1]-1 are the tokens kv_len[s] - q_len .. kv_len[s]-1 of sequence
    s, whose token j lies in page page_table[s][j // 64].  A touched block's
    scale grows with its largest value and what it held is requantised."""
    H, D = cache.n_heads, cache.head_dim
    _on(cache.k.device, k, v)
    ks, vs = _rows(k, H, D, "k"), _rows(v, H, D, "v")
    if not (k.shape[0] == v.shape[0] and k.dtype == v.dtype):
        raise ValueError("k and v: one length and type expected")
    b = _batch(cache, page_table, cu_q, kv_len, k.shape[0], max_q, 8192 // H)
    _call(cache.k.device, "colibri_kv_append", ctypes.byref(cache.desc), ctypes.byref(b), k.data_ptr(),
          v.data_ptr(), _type(k.dtype), ks, vs)


def kv_read(cache: KVCache, page_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, n_tokens: int, *,
            dtype: torch.dtype = torch.float32, max_q: Optional[int] = None,
            k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """-> (k, v) [n_tokens][n_heads][head_dim]: the values of each sequence's last
    cu_q[s+1] - cu_q[s] tokens (in k and v if given; rows that belong to no
    sequence are left as they are)."""
    dev, shape = cache.k.device, (n_tokens, cache.n_heads, cache.head_dim)
    _on(dev, k, v)
    _flat(k, dtype, shape, "k")
    _flat(v, dtype, shape, "v")
    k = torch.empty(shape, dtype=dtype, device=dev) if k is None else k
    v = torch.empty(shape, dtype=dtype, device=dev) if v is None else v
    b = _batch(cache, page_table, cu_q, kv_len, n_tokens, max_q, 8192 // cache.n_heads)
    if n_tokens:
        _call(dev, "colibri_kv_read", ctypes.byref(cache.desc), ctypes.byref(b), k.data_ptr(), v.data_ptr(),
              _type(dtype))
    return k, v


def kv_attention_workspace(cache: KVCache, n_seq: int, n_tokens: int, n_heads: int, max_q: int, max_kv: int,
                           dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Workspace of kv_attention for these sizes and for smaller ones of n_tokens <= n_seq * max_q; calls that may
    overlap need one each."""
    b = KVBatchDesc(None, None, None, _length(n_seq), 0, _length(n_tokens), _length(max_q))
    a = KVAttnDesc(None, None, None, 0, 0, _type(dtype), _length(n_heads), 1, 0, _length(max_kv), 1.0)
    n = _f().colibri_kv_attention_workspace_bytes(ctypes.byref(cache.desc), ctypes.byref(b), ctypes.byref(a))
    if n == 0:
        raise _qre.ColibriError(_qre.COLI_E_INVAL, "colibri_kv_attention_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=cache.k.device)


def kv_attention(cache: KVCache, page_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor,
                 q: torch.Tensor, *, scale: Optional[float] = None, causal: bool = True, window: int = 0,
                 max_q: Optional[int] = None, max_kv: Optional[int] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [n_tokens][n_heads][head_dim] = softmax(scale q.k) v over the cached tokens of each row's sequence.

    q: [n_tokens][n_heads][head_dim] fp32 or bf16, tokens may be strided;
    scale defaults to head_dim ** -0.5; causal: row i of sequence s sees the
    tokens up to its own, kv_len[s] - q_len + i, with window > 0 the last
    `window` of them.  lse fp32 [n_tokens][n_heads] receives the log of each
    row's sum.  max_q and max_kv are the expected longest lengths: they shape
    the launch, not the result (by default what the numbers of rows and
    sequences suggest, and the table's capacity; a max_kv far above the lengths
    costs time, and so does a max_q far from them).  A score is off by up to the
    row's largest |q| / 65024 (bf16; fp32: / 2^24) times |scale| sum |k|.  ws: see
    kv_attention_workspace."""
    dev, D = cache.k.device, cache.head_dim
    if not (q.dim() == 3):
        raise ValueError("q: [n_tokens][n_heads][head_dim] expected")
    T, H = q.shape[0], q.shape[1]
    qs = _rows(q, H, D, "q")
    _on(dev, q, out, lse, ws)
    if out is None:
        out = torch.empty(T, H, D, dtype=q.dtype, device=dev)
    if not (out.shape == q.shape and out.dtype == q.dtype):
        raise ValueError("out: the shape and type of q expected")
    os = _rows(out, H, D, "out")
    _flat(lse, torch.float32, (T, H), "lse")
    b = _batch(cache, page_table, cu_q, kv_len, T, max_q, 65536 // H)
    most = page_table.shape[1] * KV_BLOCK if max_kv is None else max_kv
    if ws is None:
        ws = kv_attention_workspace(cache, b.n_seq, T, H, b.max_q, most, q.dtype)
    if not (0 <= window <= _MOST and 0 <= most <= _MOST):
        window, most = _length(window), _length(most)
    a = KVAttnDesc(q.data_ptr(), out.data_ptr(), _at(lse), qs, os, _type(q.dtype), H, 1 if causal else 0, window, most,
                   D ** -0.5 if scale is None else scale)
    _call(dev, "colibri_kv_attention", ctypes.byref(cache.desc), ctypes.byref(b), ctypes.byref(a), *_room(ws))
    return out
