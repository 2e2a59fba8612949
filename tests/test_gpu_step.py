"""The operators of a serving step on the GPU against plain forms
(tests/step_ref.py): the embedding lookup and the paged cache's sequences from
step to step."""

import random

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_common import say
from tests.test_gpu_block import gen, within

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qre():
    import quantized_routed_expert_sigmoid_amd as m
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m.lib()
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def side_stream(f):
    """f() on a stream of its own, ordered behind and before the current one."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = f()
    torch.cuda.current_stream().wait_stream(s)
    return r


def codes(g, n, K, bits):
    """Random packed codes [n][K * bits / 8]; int8 ones in [-127, 127]."""
    if bits == 8:
        return torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).view(torch.uint8)
    return torch.randint(0, 256, (n, K * bits // 8), generator=g, dtype=torch.uint8)


# ---- embedding ------------------------------------------------------------

EMBED = [(1, 7, 32, 8, 0, F32), (5, 100, 96, 4, 32, BF16), (3, 1, 2080, 2, 0, F32), (33, 513, 6144, 4, 128, BF16),
         (2, 64, 8224, 2, 32, BF16), (1, 9, 32768, 8, 64, F32), (300, 1000, 256, 8, 0, BF16), (17, 31, 2048, 4, 0, F32)]


@pytest.mark.parametrize("n,rows,K,bits,group,dtype", EMBED)
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_embed(qre, n, rows, K, bits, group, dtype, id_type):
    say(f"embed {n} of {rows} x {K} int{bits} / {group} {dtype} {id_type}")
    g = gen("embed", n, rows, K, bits)
    data = codes(g, rows, K, bits)
    scale = 0.02 * torch.randn(rows * (K // group if group else 1), generator=g)
    ids = torch.randint(0, rows, (n,), generator=g).to(id_type)
    if n > 2:
        ids[0], ids[1], ids[2] = -1, rows, ids[n - 1]  # padding, past the end, twice the same
    if n > 4 and id_type == torch.int64:
        ids[3] = 1 << 32  # no id in 32 bits either
    bank = qre.QBank(data.unsqueeze(0).cuda(), scale.unsqueeze(0).cuda(), bits, group)
    want = ref.embed(data, scale, bits, group, ids, 78.5)
    within(qre.embed_q(bank, ids.cuda(), 78.5, dtype=dtype), want, ref.embed_tol(want, dtype), "embed")
    out = torch.full((n, K), 7.0, dtype=dtype, device="cuda")
    assert qre.embed_q(bank, ids.cuda(), -78.5, out=out) is out
    within(out, -want, ref.embed_tol(want, dtype), "embed into out")


def test_embed_no_tokens_and_far_rows(qre):
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, K = 1 << 20, 4096  # rows past 2^31 bytes
    data = torch.randint(0, 256, (1, rows, K), generator=g, device="cuda", dtype=torch.uint8)
    bank = qre.QBank(data, torch.ones(1, rows, device="cuda"), 8)
    assert qre.embed_q(bank, ints([])).shape == (0, K)
    ids = [rows - 1, 0, 600000, 524289]
    assert torch.equal(qre.embed_q(bank, ints(ids)), data[0, ids].view(torch.int8).float())


# ---- pages ----------------------------------------------------------------


class Both:
    """One state on the GPU and in plain Python; each call goes to both and they are compared."""

    def __init__(self, qre, n_seq, max_pages, n_pages):
        self.qre = qre
        self.dev = qre.KVPages.empty(n_seq, max_pages, n_pages)
        self.plain = ref.Pages(self.dev.page_table.tolist(), self.dev.kv_len.tolist(), self.dev.refs.tolist())

    def set(self, table=None, kv_len=None, refs=None):
        """Sets a part of both states to a list."""
        for name, v in (("table", table), ("kv_len", kv_len), ("refs", refs)):
            if v is not None:
                setattr(self.plain, name, [list(r) for r in v] if name == "table" else list(v))
                (self.dev.page_table if name == "table" else getattr(self.dev, name)).copy_(ints(v))

    def same(self, what):
        assert self.dev.kv_len.tolist() == self.plain.kv_len, f"{what}: kv_len"
        assert self.dev.refs.tolist() == self.plain.refs, f"{what}: refs"
        assert self.dev.page_table.tolist() == self.plain.table, f"{what}: page_table"

    def extend(self, add):
        r = self.qre.kv_extend(self.dev, ints(add))
        granted, src, dst = self.plain.extend(add)
        assert r.granted.tolist() == granted and r.src.tolist() == src and r.dst.tolist() == dst, "extend"
        self.same("extend")
        return granted, src, dst

    def trim(self, to):
        self.qre.kv_trim(self.dev, ints(to))
        self.plain.trim(to)
        self.same("trim")

    def fork(self, parent, child):
        self.qre.kv_fork(self.dev, ints(parent), ints(child))
        self.plain.fork(parent, child)
        self.same("fork")

    def compact(self):
        r = self.qre.kv_compact(self.dev)
        src, dst, live = self.plain.compact()
        assert r.src.tolist() == src and r.dst.tolist() == dst and r.n_live.tolist() == live, "compact"
        self.same("compact")


# the last three are past what one workgroup takes: sequences, pages, both
SIZES = [(1, 1, 1), (3, 4, 9), (7, 5, 16), (40, 33, 700), (64, 9, 4097), (1024, 3, 2000), (1025, 3, 2000), (20, 300, 33000),
         (1500, 40, 40001)]


@pytest.mark.parametrize("n_seq,max_pages,n_pages", SIZES)
def test_pages_of_many_steps(qre, n_seq, max_pages, n_pages):
    """Steps of every kind in turn, with shortage, sequences that outgrow their tables and forks of forks."""
    say(f"pages {n_seq} x {max_pages} of {n_pages}")
    r = random.Random(n_seq * 31 + n_pages)
    b = Both(qre, n_seq, max_pages, n_pages)
    cap = max_pages * 64
    for step in range(12 if n_seq < 100 else 5):
        most = r.choice((1, 70, cap // 3 + 1, cap + 10))
        b.extend([r.choice((0, -3, 1, 64, r.randint(1, most), r.randint(1, most))) for _ in range(n_seq)])
        used = [s for s in range(n_seq) if b.plain.kv_len[s]]
        b.trim([r.choice((-1, -7, 0, 63, 64, r.randint(0, cap), cap + 5, 0x7FFFFFFF)) for _ in range(n_seq)])
        free = [s for s in range(n_seq) if not b.plain.kv_len[s]]
        pairs = r.randint(1, max(1, min(len(free), 50)))
        b.fork([r.choice(used or [0]) for _ in range(pairs)], [r.choice(free or [0]) for _ in range(pairs)])
        b.extend([r.choice((0, 1, 5)) for _ in range(n_seq)])
        if step % 3 == 2:
            b.compact()
    b.trim([0] * n_seq)
    assert not any(b.plain.refs)
    b.extend([cap] * n_seq)
    b.compact()


def test_extend_in_order_when_pages_run_out(qre):
    """The first sequence that finds too few pages and all behind it that need any stay as they are."""
    b = Both(qre, 5, 4, 6)
    granted, _, _ = b.extend([100, 200, 65, 0, 1])  # 2 + 4 pages, then none
    assert granted == [100, 200, 0, 0, 0]
    granted, _, _ = b.extend([28, 56, 1, 1, 300])  # inside their blocks
    assert granted == [28, 56, 0, 0, 0]
    assert b.extend([1, 1, -5, 0x7FFFFFFF, -0x80000000])[0] == [0, 0, 0, 0, 0]


@pytest.mark.parametrize("n_pages", [50, 33000])
def test_shared_last_pages(qre, n_pages):
    """Every holder of a shared, partly filled page that grows leaves it; whole pages stay shared."""
    b = Both(qre, 6, 4, n_pages)
    b.extend([130, 0, 0, 128, 0, 0])
    b.fork([0, 0, 3], [1, 2, 4])
    granted, src, dst = b.extend([1, 2, 0, 1, 1, 0])
    assert granted == [1, 2, 0, 1, 1, 0] and src[:3] == [2, 2, -1] and src[3:] == [-1] * 3
    granted, src, dst = b.extend([1, 1, 1, 1, 1, 1])  # sequence 2 holds it alone now
    assert src == [-1] * 6
    b.trim([5, -1, 5, -1, -1, -1])  # into a whole page that is shared
    granted, src, dst = b.extend([1, 0, 1, 0, 0, 0])
    assert src == [0, -1, 0, -1, -1, -1]


@pytest.mark.parametrize("n_pages", [40, 33000])
def test_pages_with_holes_and_bad_lengths(qre, n_pages):
    """Entries that hold no page, lengths out of bounds, entries behind the length that mean nothing."""
    b = Both(qre, 4, 3, n_pages)
    b.set(table=[[5, -1, 7], [n_pages, 6, 0x7FFFFFFF], [-9, 3, 3], [1, 2, 4]], kv_len=[130, 70, -4, 1000],
          refs=[1 if p in (1, 2, 4, 5, 6, 7) else 0 for p in range(n_pages)])
    b.extend([10, 10, 10, 1])
    b.fork([0, 3, 1], [2, 2, 9])
    b.extend([1, 200, 0, 0])
    b.trim([64, 1, -1, 64])
    b.fork([1, 0], [2, 1])
    b.compact()
    b.trim([0, 0, 0, 0])


def test_fork_pairs_that_are_skipped(qre):
    b = Both(qre, 8, 2, 30)
    b.extend([70, 5, 0, 0, 0, 0, 0, 64])
    #  out of range (4), taken twice, a child that lives, a parent that is a child, itself
    b.fork([0, 8, 0, -1, 1, 0, 2, 3, 0x7FFFFFFF], [2, 3, 8, 3, 2, 1, 4, 3, -0x80000000])
    assert b.plain.kv_len == [70, 5, 70, 0, 0, 0, 0, 64]
    b.fork([], [])
    n = 3000
    b.fork([0] * n, [5] * n)
    assert b.plain.kv_len[5] == 70 and b.plain.refs[b.plain.table[0][0]] == 3


def test_no_sequences_and_no_pages_in_a_table(qre):
    for n_seq, max_pages in ((0, 4), (3, 0)):
        b = Both(qre, n_seq, max_pages, 5)
        b.extend([1] * n_seq)
        b.trim([0] * n_seq)
        b.compact()


def filled_cache(qre, n_pages, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randint(-127, 128, (n_pages, H, 64 * D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(n_pages, H, generator=g, device="cuda") for _ in range(2))
    return qre.KVCache(k, v, ks, vs, D)


def contents(c):
    return [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


@pytest.mark.parametrize("H,D,n_pages", [(1, 64, 3), (8, 128, 20), (3, 192, 11), (300, 64, 7), (2, 256, 70)])
def test_copy(qre, H, D, n_pages):
    say(f"copy {n_pages} pages of {H} x {D}")
    a, b = filled_cache(qre, n_pages, H, D, 1), filled_cache(qre, n_pages + 2, H, D, 2)
    src, dst = [0, -1, 1, n_pages, 0], [n_pages - 1, 1, -1, 0, n_pages]
    want = contents(a)
    for t in want:
        t[n_pages - 1] = t[0]
    qre.kv_copy(a, ints(src), ints(dst))
    for x, y in zip(contents(a), want):
        assert torch.equal(x, y)
    here = contents(a)
    want = contents(b)
    for t, s in zip(want, here):
        t[n_pages - 1], t[n_pages] = s[0], s[0]
    qre.kv_copy(a, ints(src), ints(dst), to=b)
    for x, y in zip(contents(b) + contents(a), want + here):
        assert torch.equal(x, y)
    qre.kv_copy(a, ints([]), ints([]))


def test_copy_of_pages_far_behind(qre):
    """Pages past 2^31 bytes of a cache, and more pairs than a launch has rows."""
    c = filled_cache(qre, 17000, 8, 256, 3)
    want = [t[[16999, 2]] for t in contents(c)]
    src, dst = [-1] * 70000, [-1] * 70000
    src[3], dst[3] = 16999, 16500
    src[69999], dst[69999] = 2, 16998
    qre.kv_copy(c, ints(src), ints(dst))
    for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), want):
        assert torch.equal(x[[16500, 16998]], y)


@pytest.mark.parametrize("n_pages", [60, 33000])
def test_pages_captured_and_on_another_stream(qre, n_pages):
    """A step of every call captured once and replayed on a changing state equals the plain calls."""
    n, ref_of = 6, lambda p: ref.Pages(p.page_table.tolist(), p.kv_len.tolist(), p.refs.tolist())
    p, c = qre.KVPages.empty(n, 4, n_pages), filled_cache(qre, n_pages, 1, 64, 4)
    add, keep, parent, child = ints([70, 3, 0, 0, 64, 0]), ints([-1] * n), ints([0, 4]), ints([2, 3])
    ws = qre.kv_pages_workspace(p)

    def step():
        qre.kv_trim(p, keep)
        qre.kv_fork(p, parent, child)
        r = qre.kv_extend(p, add, ws=ws)
        qre.kv_copy(c, r.src, r.dst)
        m = qre.kv_compact(p, ws=ws)
        qre.kv_copy(c, m.src, m.dst)
        return r, m

    side_stream(step)  # warm, and on a stream that is not the default one
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, m = step()
    for t in range(5):
        plain, held = ref_of(p), contents(c)
        keep.copy_(ints([[-1, 0, 10][(s + t) % 3] if t else -1 for s in range(n)]))
        parent.copy_(ints([t % n, 4]))
        child.copy_(ints([(t + 1) % n, 3]))
        plain.trim(keep.tolist())
        plain.fork(parent.tolist(), child.tolist())
        want = plain.extend(add.tolist())
        moves = plain.compact()
        graph.replay()
        torch.cuda.synchronize()
        assert [x.tolist() for x in r] == list(want) and [x.tolist() for x in m] == list(moves)
        assert ref_of(p).table == plain.table and ref_of(p).refs == plain.refs and ref_of(p).kv_len == plain.kv_len
        for src, dst in (want[1:], moves[:2]):
            for x in held:
                taken = [(a, b, x[a].clone()) for a, b in zip(src, dst) if a >= 0]
                for _, b, y in taken:
                    x[b] = y
        for x, y in zip(contents(c), held):
            assert torch.equal(x, y)
