"""Plain forms of the operators of a serving step, for their tests, and the
bounds that the tests hold the kernels to.  Written from the definitions in
include/colibri_step.h; numbers in 64 bits on the CPU, pages by plain loops."""

import math

import torch

from tests.block_ref import U, round_half_away, weight_codes  # noqa: F401

BLOCK = 64


# ---- embedding ------------------------------------------------------------


def embed(data, scale, bits, group, ids, mul):
    rows, K = data.shape[0], data.shape[1] * 8 // bits
    w = weight_codes(data, bits).double() * scale.double().view(rows, -1).repeat_interleave(group or K, 1)
    ok = (ids >= 0) & (ids < rows)
    return torch.where(ok[:, None], w[ids.clamp(0, rows - 1).long()] * mul, 0.0)


def embed_tol(want, dtype):
    """The scales' two products are rounded to fp32 each, the result to its type."""
    return (2 * U[torch.float32] * (1 + U[torch.float32]) + U[dtype] * 1.001 * (dtype != torch.float32)) * want.abs() + 1e-37


# ---- linear product -------------------------------------------------------


def quantize(x):
    """Codes and scales of [rows][K] by the rule's fp32 operations."""
    x = x.float()
    d = x.abs().amax(1) / 127.0
    v = x * torch.where(d > 0, 1.0 / d, torch.zeros(()))[:, None]
    return round_half_away(v).clamp(-127, 127).to(torch.int8), d


def linear(data, scale, bits, xq, xd, bias, act, residual):
    """-> (out, the value before the bias, before the activation)."""
    z = (xq.double() @ weight_codes(data, bits).double().t()) * scale.double() * xd.double()[:, None]
    y = u = z + bias.double() if bias is not None else z
    if act == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif act == "silu":
        y = y * torch.special.expit(y)
    elif act == "gelu":
        y = y * torch.special.ndtr(y)
    return (y + residual.double() if residual is not None else y), z, u


def linear_tol(y, z, u, act, dtype):
    """The sum (exact in whole numbers) and the scales' product are rounded, their product with the bias
    once; an activation's slope is under 1.2, its own error as in include/colibri_block.h; the residual's sum and
    the result are rounded."""
    e = 1.2 * (2.01 * U[torch.float32] * z.abs() + U[torch.float32] * u.abs())
    if act == "silu":
        e = e + 2.0 ** -23 * (u.abs() + 8)
    elif act == "gelu":
        e = e + 2.0 ** -22 * (1 + u.abs())
    return e + U[torch.float32] * y.abs() * 1.01 + U[dtype] * 1.001 * (dtype != torch.float32) * y.abs() + 1e-37


# ---- pages ----------------------------------------------------------------


class Pages:
    """The state of coli_kv_pages as lists, and the calls on it."""

    def __init__(self, table, kv_len, refs):
        self.table, self.kv_len, self.refs = [list(r) for r in table], list(kv_len), list(refs)
        self.cap = (len(self.table[0]) if self.table else 0) * BLOCK

    def len_of(self, s):
        return min(max(self.kv_len[s], 0), self.cap)

    @staticmethod
    def blocks(n):
        return -(-n // BLOCK)

    def held(self, p):
        return 0 <= p < len(self.refs)

    def extend(self, add):
        n = len(self.kv_len)
        granted, src, dst = [0] * n, [-1] * n, [-1] * n
        before = list(self.refs)
        free = [p for p, r in enumerate(before) if r <= 0]
        used = 0
        for s in range(n):
            ln, a = self.len_of(s), add[s]
            if a <= 0 or ln + a > self.cap:
                continue
            have, want, last = self.blocks(ln), self.blocks(ln + a), ln // BLOCK
            shared = ln % BLOCK != 0 and self.held(self.table[s][last]) and before[self.table[s][last]] > 1
            need = want - have + shared
            used += need
            if need and used > len(free):
                continue
            mine = free[used - need:used]
            if shared:
                src[s], dst[s] = self.table[s][last], mine[0]
                self.refs[src[s]] -= 1
                self.refs[dst[s]] = 1
                self.table[s][last] = dst[s]
                mine = mine[1:]
            for b, p in zip(range(have, want), mine):
                self.table[s][b] = p
                self.refs[p] = 1
            self.kv_len[s] = ln + a
            granted[s] = a
        return granted, src, dst

    def trim(self, to):
        for s, t in enumerate(to):
            ln = self.len_of(s)
            if 0 <= t < ln:
                for b in range(self.blocks(t), self.blocks(ln)):
                    if self.held(self.table[s][b]):
                        self.refs[self.table[s][b]] -= 1
                    self.table[s][b] = -1
                self.kv_len[s] = t

    def fork(self, parent, child):
        n, empty = len(self.kv_len), [k <= 0 for k in self.kv_len]
        for i, (p, c) in enumerate(zip(parent, child)):
            if not (0 <= p < n and 0 <= c < n) or not empty[c] or c in child[:i] or p in child:
                continue
            ln = self.len_of(p)
            for b in range(self.blocks(ln)):
                self.table[c][b] = self.table[p][b]
                if self.held(self.table[p][b]):
                    self.refs[self.table[p][b]] += 1
            self.kv_len[c] = ln

    def compact(self):
        n = len(self.refs)
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, n) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for s in range(len(self.kv_len)):
            for b in range(self.blocks(self.len_of(s))):
                self.table[s][b] = to.get(self.table[s][b], self.table[s][b])
        for a, b in to.items():
            self.refs[a], self.refs[b] = 0, self.refs[a]
        pad = [-1] * (n // 2 - len(src))
        return src + pad, dst + pad, [live]


# ---- logits ---------------------------------------------------------------


def adjust_row(x, tokens, span, penalties, ids, bias, words, dtype):
    """One row's adjusted logits in `dtype`, and the sum of the magnitudes that were rounded."""
    x = x.to(dtype)
    V, A = x.numel(), x.abs().double()
    if penalties is not None:
        rep, freq, pres = (float(v) for v in penalties)
        first, made, end = max(int(span[0]), 0), int(span[1]), min(int(span[2]), len(tokens))
        part = tokens[first:max(end, first)]
        inside = (part >= 0) & (part < V)
        late = torch.arange(first, max(end, first)) >= made
        seen = torch.bincount(part[inside].long(), minlength=V) > 0
        count = torch.bincount(part[inside & late].long(), minlength=V)
        rep, freq, pres = (torch.tensor(v, dtype=dtype) for v in (rep, freq, pres))
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        A = A + x.abs().double()
        less = freq * count.to(dtype) + pres
        x = torch.where(count > 0, x - less, x)
        A = A + (count > 0) * (x.abs() + (freq * count).abs() + less.abs()).double()
    if ids is not None:
        x = x.clone()
        for t, b in zip(ids.tolist(), bias):
            if 0 <= t < V:
                x[t] = x[t] + b.to(dtype)
                A[t] += x[t].abs().double()
    if words is not None:
        t = torch.arange(V)
        ok = (words.long()[t // 32] >> (t % 32)) & 1
        x = torch.where(ok > 0, x, torch.tensor(-math.inf, dtype=dtype))
    return x, A


def best(x):
    """Lowest index of the largest value (the first NaN's, -1 where all is -inf)."""
    nan = torch.isnan(x).nonzero()
    if len(nan):
        return int(nan[0])
    top = x.max()
    return -1 if top == -math.inf else int((x == top).nonzero()[0])


def logits_tol(x, A, dtype):
    """Every operation is rounded once, by at most 2^-24 of its result; A holds their magnitudes."""
    return U[torch.float32] * A.nan_to_num(posinf=0.0) + U[dtype] * 1.001 * (dtype != torch.float32) * x.abs().nan_to_num(
        posinf=0.0) + 1e-37


def lse_tol(x, A, lse):
    """Sums pass through at most 40 additions of positive numbers; a term's exponent is off by three roundings
    of d = v - largest, and d exp(-d) < 0.37; the exponential by 2^-22: together under 2^-18.  The values' own errors
    and the result's three roundings come on top."""
    own = (U[torch.float32] * A)[torch.isfinite(x)]
    return 2.0 ** -18 + (float(own.max()) if len(own) else 0.0) + 3 * 2.0 ** -24 * (abs(lse) if math.isfinite(lse) else 0.0)
