"""Penalties, biases and masks on logits, the best token and the log of the sum on the GPU against
plain forms (tests/step_ref.py): values against 64 bits, tokens against the same steps in 32 bits."""

import math

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
    return torch.tensor(v, dtype=torch.int32)


def make(rows, V, hist, n_bias, masks, dtype, *labels):
    """Inputs on the CPU, with what goes wrong easily among them."""
    g = gen("logits", rows, V, hist, n_bias, *labels)
    i = {"logits": (3 * torch.randn(rows, V, generator=g)).to(dtype)}
    if hist is not None:
        n = hist + rows
        i["tokens"] = (torch.rand(n, generator=g) ** 4 * V).to(torch.int32)
        i["tokens"][::17] = -1  # padding
        i["tokens"][5::29] = V + 3
        first = torch.randint(0, n // 3 + 1, (rows,), generator=g)
        end = torch.clamp(first + torch.randint(0, n + 1, (rows,), generator=g), max=n)
        made = first + ((end - first) * torch.rand(rows, generator=g)).long()
        i["spans"] = torch.stack([first, made, end], 1).to(torch.int32)
        i["penalties"] = torch.stack([0.5 + torch.rand(rows, generator=g), torch.randn(rows, generator=g),
                                      torch.randn(rows, generator=g)], 1)
        if rows > 3:
            i["spans"][1] = ints([-5, -2, n + 9])  # taken inside the list
            i["spans"][2] = ints([7, 2, 3])  # no tokens
            i["spans"][3, 1] = i["spans"][3, 2] + 4  # none generated
            i["penalties"][3] = torch.tensor([1.0, 0.0, 0.0])
    if n_bias is not None:
        lens = [int(v) for v in torch.randint(0, n_bias + 1, (rows,), generator=g)]
        lens[0] = n_bias
        i["cu_bias"] = ints([sum(lens[:j]) for j in range(rows + 1)])
        i["bias_ids"] = torch.randint(-2, V + 2, (sum(lens),), generator=g).to(torch.int32)
        i["bias_ids"][1:sum(lens):3] = i["bias_ids"][0:sum(lens) - 1:3]  # the same token twice
        i["bias"] = 4 * torch.randn(sum(lens), generator=g)
        if rows > 2:
            i["cu_bias"][-1] += 100  # past the list
    if masks:
        words = (V + 31) // 32
        m = torch.randint(-2 ** 31, 2 ** 31, (masks, words + 1), generator=g).to(torch.int32)
        m[0] = 0
        m[-1, 1:] = 0
        i["mask"], i["mask_of"] = m, torch.randint(-1, masks + 1, (rows,), generator=g).to(torch.int32)
        i["mask_of"][0] = 0
        if rows > 1:
            i["mask_of"][1] = masks - 1
    return i


def call(qre, i, **kw):
    return qre.adjust_logits(**{k: v.cuda() for k, v in i.items()}, **kw)


def check(i, got, dtype):
    rows, V = i["logits"].shape
    for r in range(rows):
        def row(dt):
            lo, hi = (int(v) for v in i["cu_bias"][r:r + 2].clamp(0, len(i["bias"]))) if "bias" in i else (0, 0)
            m = int(i["mask_of"][r]) if "mask" in i else -1
            return ref.adjust_row(
                i["logits"][r].float(), i.get("tokens"), i["spans"][r] if "spans" in i else None,
                i["penalties"][r] if "penalties" in i else None, i["bias_ids"][lo:hi] if "bias" in i else None,
                i["bias"][lo:hi] if "bias" in i else None, i["mask"][m] if 0 <= m < len(i.get("mask", ())) else None, dt)
        want, A = row(torch.float64)
        if got.logits is not None:
            within(got.logits[r], want, ref.logits_tol(want, A, dtype), f"logits of row {r}")
        if got.token is not None:
            assert int(got.token[r]) == ref.best(row(torch.float32)[0]), f"token of row {r}"
            lse = float(torch.logsumexp(want, 0))
            mine = float(got.lse[r])
            assert mine == lse or abs(mine - lse) <= ref.lse_tol(want, A, lse), f"lse of row {r}: {mine} for {lse}"


CASES = [(1, 1, None, None, 0, F32), (1, 5, 3, 2, 1, BF16), (4, 31, 40, None, 2, F32), (5, 4096, 300, 7, 3, F32),
         (3, 4097, None, 600, 2, BF16), (2, 8190, 9000, 40, 0, BF16), (9, 20011, 70, 30, 4, F32),
         (2, 151003, 5000, 300, 2, BF16),
         (6, 1000, 1, 1, 0, F32), (7, 12289, 2500, None, 0, BF16), (2, 1048576, 100, 20, 1, F32)]


@pytest.mark.parametrize("rows,V,hist,n_bias,masks,dtype", CASES)
def test_adjust(qre, rows, V, hist, n_bias, masks, dtype):
    say(f"logits {rows} x {V} history {hist} biases {n_bias} masks {masks} {dtype}")
    i = make(rows, V, hist, n_bias, masks, dtype)
    got = call(qre, i)
    check(i, got, dtype)
    only = call(qre, i, write=False)
    assert only.logits is None and torch.equal(only.token, got.token) and torch.equal(only.lse, got.lse)
    plain = call(qre, i, best=False)
    assert plain.token is None and torch.equal(plain.logits, got.logits)


@pytest.mark.parametrize("hist", [60000, 200000])
def test_long_histories(qre, hist):
    i = make(3, 9001, hist, 2500, 0, F32, "long")
    i["spans"][0] = ints([0, 0, hist])
    check(i, call(qre, i), F32)


@pytest.mark.parametrize("n", range(6))
def test_few_tokens_in_all(qre, n):
    i = make(3, 40, 4, None, 0, F32, "few")
    i["tokens"] = ints([7, 7, 3, 39, 0][:n])
    i["spans"] = ints([[0, 1, n], [0, 0, n], [1, n, n]])
    check(i, call(qre, i), F32)


def test_drafts_share_their_sequence(qre):
    """Row i of a verify step sees the sequence and the first i drafts."""
    i = make(5, 700, 50, None, 0, F32, "drafts")
    i["spans"] = ints([[3, 20, 40 + d] for d in range(5)])
    check(i, call(qre, i), F32)


def test_strided_rows_in_place_and_around(qre):
    i = make(4, 5003, 200, 9, 2, F32, "strides")
    want = call(qre, i)
    wide = torch.full((4, 5011), 99.0, device="cuda")
    wide[:, 3:5006] = i["logits"].cuda()
    view = wide[:, 3:5006]
    rest = {k: v.cuda() for k, v in i.items() if k != "logits"}
    got = qre.adjust_logits(view, out=view, **rest)
    assert got.logits.data_ptr() == view.data_ptr() and torch.equal(view, want.logits)
    assert torch.equal(got.token, want.token) and torch.equal(got.lse, want.lse)
    assert bool((wide[:, :3] == 99).all()) and bool((wide[:, 5006:] == 99).all())
    apart = torch.full((4, 6000), 5.0, device="cuda")
    qre.adjust_logits(i["logits"].cuda(), out=apart[:, 1:5004], **rest)
    assert torch.equal(apart[:, 1:5004], want.logits) and bool((apart[:, 5004:] == 5).all())


def test_ties_zeros_infinities_and_nan(qre):
    inf, nan = math.inf, math.nan
    V = 9000
    x = torch.zeros(9, V)
    x[0, 4000:] = -0.0  # one value: the first
    x[1, 5000], x[1, 8999] = 2.0, 2.0
    x[2], x[2, 7000] = -inf, -3.0
    x[3] = -inf
    x[4, 6000], x[4, 70] = inf, 5.0
    x[5, 8000], x[5, 4096], x[5, 3] = nan, nan, inf
    x[6], x[6, 17] = -1e30, 1e30
    x[7, 100] = nan  # behind the mask
    x[8, 100] = inf  # behind the mask
    mask = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32)
    mask[0, 100 // 32] = ~(1 << 100 % 32)
    i = {"logits": x, "mask": mask, "mask_of": ints([-1] * 7 + [0, 0])}
    got = call(qre, i)
    assert got.token.tolist() == [0, 5000, 7000, -1, 6000, 4096, 17, 0, 0]
    lse = got.lse.tolist()
    assert lse[2] == -3.0 and lse[3] == -inf and lse[4] == inf and math.isnan(lse[5]) and lse[6] == float(x[6, 17])
    assert abs(lse[7] - math.log(V - 1)) < 1e-5 and lse[8] == lse[7]
    y = x.clone()
    y[7, 100] = y[8, 100] = -inf
    assert torch.equal(got.logits.cpu().nan_to_num(nan=7.5), y.nan_to_num(nan=7.5))
    for row in range(9):  # a row by itself
        one = qre.adjust_logits(x[row:row + 1].cuda(), mask=mask.cuda(), mask_of=ints([-1 if row < 7 else 0]).cuda(),
                                write=False)
        assert one.token.tolist() == got.token[row:row + 1].tolist()


def test_a_token_listed_many_times(qre):
    """Biases of one token are added in the list's order, in fp32."""
    n = 1500
    g = gen("many biases")
    b = torch.randn(n, generator=g) * 10 ** (6 * torch.rand(n, generator=g) - 3)
    ids = torch.full((n,), 77, dtype=torch.int32)
    ids[::3] = 4500
    i = {"logits": torch.zeros(1, 5000), "bias": b, "bias_ids": ids, "cu_bias": ints([0, n])}
    got = call(qre, i)
    for t in (77, 4500):
        s = torch.tensor(0.0)
        for v in b[ids == t]:
            s = s + v
        assert float(got.logits[0, t]) == float(s)
    assert int((got.logits != 0).sum()) == 2


def test_biases_of_infinity_ban_and_force(qre):
    i = {"logits": torch.randn(1, 300), "bias": torch.tensor([-math.inf, math.inf]), "bias_ids": ints([int(3), 9]),
         "cu_bias": ints([0, 2])}
    got = call(qre, i)
    assert got.token.tolist() == [9] and float(got.logits[0, 3]) == -math.inf


def test_rows_past_2_31_elements(qre):
    V, rows = 200003, 11000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, V, dtype=BF16, device="cuda")
    tail = torch.randn(3, V, generator=g, device="cuda").to(BF16)
    x.fill_(-1.0)
    x[-3:] = tail
    got, want = qre.adjust_logits(x, out=x), qre.adjust_logits(tail)
    assert torch.equal(got.token[-3:], want.token) and torch.equal(got.lse[-3:], want.lse)
    assert torch.equal(x[-3:], tail) and int(got.token[0]) == 0


def test_no_rows(qre):
    got = qre.adjust_logits(torch.empty(0, 50, device="cuda"))
    assert got.logits.shape == (0, 50) and got.token.numel() == 0


def test_captured_and_on_two_streams(qre):
    i = make(6, 30011, 900, 20, 3, BF16, "graph")
    d = {k: v.cuda() for k, v in i.items()}
    out, ws = torch.empty_like(d["logits"]), qre.logits_workspace(6, 30011)

    def step():
        return qre.adjust_logits(**d, out=out, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    for n in range(4):
        j = make(6, 30011, 900, 20, 3, BF16, "graph", n)
        for k in d:
            if j[k].shape == d[k].shape:
                d[k].copy_(j[k])
        want = qre.adjust_logits(**d)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.token, want.token) and torch.equal(r.lse, want.lse)
        assert torch.equal(r.logits.nan_to_num(neginf=-7), want.logits.nan_to_num(neginf=-7))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(qre.adjust_logits(**d))
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x.token, want.token) and torch.equal(x.lse, want.lse)
