"""The operators of a serving step in a run, as they are used: prompts and decode steps of a small
block with an embedding and a vocabulary, beams that fork, drafts that are taken back and a compacted pool,
against the same steps in plain form (64 bits) on caches that hold the same pages."""

import math

import pytest
import torch

from tests import block_ref, step_ref as ref
from tests.gpu_common import say
from tests.test_gpu_block import gen, within
from tests.test_gpu_step import codes, ints

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
V, K, HQ, H, D, N_SEQ, PAGES, MAX_PAGES = 1003, 256, 4, 2, 64, 6, 40, 6


@pytest.fixture(scope="module")
def qre():
    import quantized_routed_expert_sigmoid_amd as m
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m.lib()
    return m


class Model:
    def __init__(self, qre):
        g = gen("step run")
        self.qre = qre
        self.w = {n: (codes(g, rows, k, bits), 0.02 * torch.rand(rows, generator=g) + 0.01, bits)
                  for n, rows, k, bits in [("embed", V, K, 4), ("qkv", (HQ + 2 * H) * D, K, 8), ("o", K, HQ * D, 4),
                                           ("head", V, K, 8)]}
        self.bank = {n: qre.QBank(d.unsqueeze(0).cuda(), s.unsqueeze(0).cuda(), b) for n, (d, s, b) in self.w.items()}
        self.norm = 1 + 0.2 * torch.rand(K, generator=g)
        self.cache = qre.KVCache.empty(PAGES, H, D)
        self.cache.k.zero_(), self.cache.v.zero_(), self.cache.k_scale.zero_(), self.cache.v_scale.zero_()
        self.pages = qre.KVPages.empty(N_SEQ, MAX_PAGES, PAGES)

    def linear(self, name, x, **kw):
        q, d = self.qre.quantize_i8(x)
        return self.qre.linear_i8(self.bank[name], q, d, **kw)

    def step(self, ids, cu, spans, tokens, penalties, mask, mask_of):
        """Hidden states, logits and the best tokens of the rows' last places; the cache has room for them."""
        q, p = self.qre, self.pages
        h = q.embed_q(self.bank["embed"], ids, math.sqrt(K))
        n = q.add_rms_norm_i8(h, self.norm.cuda(), 1e-5)
        qkv = q.linear_i8(self.bank["qkv"], n.q, n.d).view(ids.numel(), -1, D)
        a, k, v = qkv.split([HQ, H, H], 1)
        q.kv_append(self.cache, p.page_table, cu, p.kv_len, k, v)
        a = q.kv_attention(self.cache, p.page_table, cu, p.kv_len, a)
        s = self.linear("o", a.view(ids.numel(), -1), residual=h)
        n = q.add_rms_norm_i8(s, self.norm.cuda(), 1e-5)
        logits = q.linear_i8(self.bank["head"], n.q, n.d)
        return h, qkv, a, s, logits, q.adjust_logits(logits, tokens=tokens, spans=spans, penalties=penalties, mask=mask,
                                                     mask_of=mask_of)

    def check(self, got, before, ids, cu, lens, spans, tokens, penalties, mask, mask_of):
        """Each operator's output against its plain form on the inputs that it had."""
        h, qkv, a, s, logits, adjusted = (x if isinstance(x, tuple) else x.cpu() for x in got)

        def lin(name, x, res=None):
            q, d = ref.quantize(x)
            y, z, u = ref.linear(*self.w[name], q, d, None, "none", res)
            return y, ref.linear_tol(y, z, u, "none", F32)
        want = ref.embed(*self.w["embed"], 0, ids.cpu(), math.sqrt(K))
        within(h, want, ref.embed_tol(want, F32), "embed")
        y = self.qre.add_rms_norm(h.cuda(), self.norm.cuda(), 1e-5, y_dtype=F32, q8=False).y.cpu()
        w, tol = lin("qkv", y)
        within(qkv.flatten(1), w, tol, "qkv")
        seqs = block_ref.Seqs([(int(cu[i + 1] - cu[i]), n) for i, n in enumerate(lens)], self.pages.page_table.cpu())
        at = block_ref.page_bytes(D)
        new = qkv.split([HQ, H, H], 1)
        now = []
        for c, sc, x, i in ((before[0], before[2], new[1], 0), (before[1], before[3], new[2], 1)):
            now.append(block_ref.append(c, sc, at[i], seqs, x))
        for (c, sc), mine, ms in zip(now, (self.cache.k, self.cache.v), (self.cache.k_scale, self.cache.v_scale)):
            assert torch.equal(mine.cpu(), c) and torch.equal(ms.cpu(), sc)
        out, _, sb, vb = block_ref.attention(block_ref.page_values(*now[0], at[0]), block_ref.page_values(*now[1], at[1]),
                                             seqs, new[0], D ** -0.5)
        within(a, out, block_ref.attention_tol(out, sb, vb, F32), "attention")
        w, tol = lin("o", a.flatten(1), h)
        within(s, w, tol, "o")
        y = self.qre.add_rms_norm(s.cuda(), self.norm.cuda(), 1e-5, y_dtype=F32, q8=False).y.cpu()
        w, tol = lin("head", y)
        within(logits, w, tol, "head")
        for r in range(logits.shape[0]):
            m = int(mask_of[r])
            x, A = ref.adjust_row(logits[r], tokens.cpu(), spans[r].cpu(), penalties[r].cpu(), None, None,
                                  mask[m].cpu() if m >= 0 else None, torch.float64)
            within(adjusted.logits[r], x, ref.logits_tol(x, A, F32), "adjusted")
            x32, _ = ref.adjust_row(logits[r], tokens.cpu(), spans[r].cpu(), penalties[r].cpu(), None, None,
                                    mask[m].cpu() if m >= 0 else None, F32)
            assert int(adjusted.token[r]) == ref.best(x32)


def test_a_run_of_steps(qre):
    say("run of steps")
    m = Model(qre)
    g = gen("step run inputs")
    plain = ref.Pages(m.pages.page_table.tolist(), m.pages.kv_len.tolist(), m.pages.refs.tolist())
    text = [[] for _ in range(N_SEQ)]
    room = 200  # of a sequence's tokens in the history
    mask = torch.randint(-2 ** 31, 2 ** 31, (2, (V + 31) // 32), generator=g).to(torch.int32).cuda()

    def contents():
        return [t.cpu().clone() for t in (m.cache.k, m.cache.v, m.cache.k_scale, m.cache.v_scale)]

    def move(src, dst):
        """The copies in plain form, then on the GPU; both caches are the same."""
        want = contents()
        for t in want:
            for a, b in zip(src.tolist(), dst.tolist()):
                if a >= 0:
                    t[b] = t[a]
        qre.kv_copy(m.cache, src, dst)
        for x, y in zip(contents(), want):
            assert torch.equal(x, y)

    def run(new):
        """new[s]: the tokens that sequence s gets."""
        add = [len(x) for x in new]
        r = qre.kv_extend(m.pages, ints(add))
        want = plain.extend(add)
        assert [t.tolist() for t in r] == list(want) and want[0] == add
        move(r.src, r.dst)
        rows = [(s, i) for s in range(N_SEQ) for i in range(len(new[s]))]
        for s in range(N_SEQ):
            text[s] = text[s] + new[s]
        flat = torch.zeros(N_SEQ, room, dtype=torch.int32)
        for s in range(N_SEQ):
            flat[s, :len(text[s])] = torch.tensor(text[s], dtype=torch.int32)
        spans = ints([[s * room, s * room + 3, s * room + len(text[s]) - len(new[s]) + i + 1] for s, i in rows])
        pen = torch.tensor([[1.3, 0.2, 0.1]]).repeat(len(rows), 1).cuda()
        cu = ints([sum(add[:s]) for s in range(N_SEQ + 1)])
        ids = ints([t for x in new for t in x])
        mask_of = ints([s % 3 - 1 for s, _ in rows])
        before = contents()
        got = m.step(ids, cu, spans, flat.view(-1).cuda(), pen, mask, mask_of)
        m.check(got, before, ids, cu.cpu(), list(plain.kv_len), spans, flat.view(-1), pen, mask, mask_of.cpu())
        best = got[-1].token.tolist()
        last = {s: best[i] for i, (s, _) in enumerate(rows)}
        return [last.get(s, -1) for s in range(N_SEQ)]

    def trim(to):
        qre.kv_trim(m.pages, ints(to))
        plain.trim(to)
        for s, t in enumerate(to):
            if 0 <= t < len(text[s]):
                text[s] = text[s][:t]

    def same():
        assert m.pages.kv_len.tolist() == plain.kv_len == [len(x) for x in text]
        assert m.pages.refs.tolist() == plain.refs and m.pages.page_table.tolist() == plain.table

    prompts = [[int(t) for t in torch.randint(0, V, (n,), generator=g)] if n else [] for n in (70, 5, 64, 0, 0, 0)]
    best = run(prompts)  # ragged prompts
    qre.kv_fork(m.pages, ints([0, 0, 1]), ints([3, 4, 5]))
    plain.fork([0, 0, 1], [3, 4, 5])
    for p, c in ((0, 3), (0, 4), (1, 5)):
        text[c] = list(text[p])
        best[c] = (best[p] + c) % V
    same()
    best = run([[best[s]] for s in range(N_SEQ)])  # beams part: the shared last pages are copied
    same()
    best = run([[best[s]] + [int(t) for t in torch.randint(0, V, (3,), generator=g)] for s in range(N_SEQ)])  # drafts
    trim([len(text[0]) - 3, len(text[1]) - 1, -1, 0, len(text[4]) - 2, 0])  # taken back; two beams end
    same()
    mv = qre.kv_compact(m.pages)
    want = plain.compact()
    assert [t.tolist() for t in mv] == list(want) and any(a >= 0 for a in want[0])
    move(mv.src, mv.dst)
    same()
    run([[7], [8], [9], [], [11], []])
    same()
