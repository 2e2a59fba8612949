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
