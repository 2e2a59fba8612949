"""The linear product with one activation scale per token, and the quantisation before
it, on the GPU against plain forms (tests/step_ref.py)."""

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_common import say
from tests.test_gpu_block import NORM, gen, within
from tests.test_gpu_step import codes

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def qre():
    import quantized_routed_expert_sigmoid_amd as m
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m.lib()
    return m


# ---- quantisation ---------------------------------------------------------


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 1024), (2, 1056), (70, 2080), (3, 6144), (2, 8192), (3, 8224),
                                    (1, 32768)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize(qre, rows, K, dtype):
    g = gen("quantize", rows, K)
    x = (torch.randn(rows, K, generator=g) * 10 ** (4 * torch.rand(rows, 1, generator=g) - 2)).to(dtype)
    if rows > 2:
        x[0] = 0  # scale 0
        x[1, 1:] = 0  # one value
        x[2, -1] = 1e30  # far above the rest
    q, d = qre.quantize_i8(x.cuda())
    want_q, want_d = ref.quantize(x)
    assert torch.equal(q.cpu(), want_q) and torch.equal(d.cpu(), want_d)
    wide = torch.full((rows, K + 8), 9.0, dtype=dtype, device="cuda")
    wide[:, 4:4 + K] = x.cuda()
    q, d = qre.quantize_i8(wide[:, 4:4 + K])
    assert torch.equal(q.cpu(), want_q) and torch.equal(d.cpu(), want_d)


def test_quantize_of_halves(qre):
    """Halves go away from zero."""
    x = torch.zeros(2, 64)
    x[:, 0], x[0, 1:5], x[1, 1:5] = 127.0, torch.tensor([0.5, -0.5, 2.5, -2.5]), torch.tensor([0.49, -0.49, 126.5, -126.5])
    q, d = qre.quantize_i8(x.cuda())
    assert d.tolist() == [1.0, 1.0] and q[:, :5].tolist() == [[127, 1, -1, 3, -3], [127, 0, 0, 127, -127]]


@pytest.mark.parametrize("rows,K,xt,rt,yt", NORM)
def test_norm_with_one_scale_per_row(qre, rows, K, xt, rt, yt):
    """The sum and y of add_rms_norm, and the codes that quantize_i8 gives the unrounded y."""
    g = gen("norm i8", rows, K)
    x = torch.randn(rows, K, generator=g).mul(3).to(xt).cuda()
    r = None if rt is None else torch.randn(rows, K, generator=g).to(rt).cuda()
    w = (1 + 0.3 * torch.randn(K, generator=g)).cuda()
    if rows > 2:
        x[1] = 0  # a row of zeros, where there is no residual
        x[2, 0] = 1e4  # one value far above the rest
    want = qre.add_rms_norm(x, w, 1e-5, residual=r, y_dtype=F32, q8=False)
    q, d = qre.quantize_i8(want.y)
    got = qre.add_rms_norm_i8(x, w, 1e-5, residual=r, y_dtype=yt)
    assert torch.equal(got.q, q) and torch.equal(got.d, d) and got.d.shape == (rows,)
    assert torch.equal(got.y, want.y.to(yt)) and (r is None or torch.equal(got.sum, want.sum))
    only = qre.add_rms_norm_i8(x, w, 1e-5, residual=r)
    assert only.y is None and torch.equal(only.q, q) and torch.equal(only.d, d)
    if r is not None:
        stream = r.clone()
        assert qre.add_rms_norm_i8(x, w, 1e-5, residual=stream, sum_out=stream).sum is stream
        assert torch.equal(stream, want.sum)


# ---- product --------------------------------------------------------------


def make(qre, S, N, K, bits, *labels):
    g = gen("linear i8", S, N, K, bits, *labels)
    data = codes(g, N, K, bits)
    scale = 0.02 * torch.randn(N, generator=g)
    xq, xd = ref.quantize(torch.randn(S, K, generator=g))
    return g, data, scale, xq, xd, qre.QBank(data.unsqueeze(0).cuda(), scale.unsqueeze(0).cuda(), bits)


# every form and tile, with and without splits; K below, at and past the steps of both forms; odd last depths
SHAPES = [(1, 1, 32), (1, 100, 6144), (2, 16, 64), (5, 15, 96), (16, 257, 160), (17, 33, 2080), (32, 100, 128), (33, 40, 224),
          (64, 70, 320), (13, 16401, 96), (200, 50, 96), (65, 20, 128), (70, 130, 160), (100, 1, 2080), (130, 257, 192),
          (120, 2600, 3232), (20, 30000, 96), (7, 25000, 224), (333, 4101, 224), (256, 64, 32768),
          (90, 4099, 2080), (33, 9001, 1184), (300, 1100, 6176), (64, 6001, 4128), (20, 9001, 3104), (129, 5003, 1120),
          (128, 10111, 6176), (1, 9, 32768), (2000, 2101, 160), (4101, 4357, 160), (4096, 4096, 128)]


@pytest.mark.parametrize("S,N,K", SHAPES)
@pytest.mark.parametrize("bits", [8, 4, 2])
def test_linear(qre, S, N, K, bits):
    dtype = (F32, BF16)[(S + bits // 2) % 2]
    act = ACTS[(S + N + bits) % 4]
    say(f"linear {S} x {N} x {K} int{bits} {act} {dtype}")
    g, data, scale, xq, xd, bank = make(qre, S, N, K, bits)
    bias = torch.randn(N, generator=g) if (N + K // 32) % 2 else None
    res = torch.randn(S, N, generator=g).to(dtype) if S % 3 else None
    want, z, u = ref.linear(data, scale, bits, xq, xd, bias, act, res)
    got = qre.linear_i8(bank, xq.cuda(), xd.cuda(), bias=None if bias is None else bias.cuda(), activation=act,
                        residual=None if res is None else res.cuda(), dtype=dtype)
    within(got, want, ref.linear_tol(want, z, u, act, dtype), "linear")


@pytest.mark.parametrize("bits", [8, 4, 2])
@pytest.mark.parametrize("S,N,K", [(3, 40, 128), (300, 130, 416), (4200, 4200, 160), (50, 33, 32768)])
def test_largest_codes(qre, S, N, K, bits):
    """Sums at their bounds are exact: every code at an end of its range."""
    top = {8: 0x7F, 4: 0x88, 2: 0xAA}[bits]
    value = {8: 127, 4: -8, 2: -2}[bits]
    bank = qre.QBank(torch.full((1, N, K * bits // 8), top, dtype=torch.uint8, device="cuda"),
                     torch.ones(1, N, device="cuda"), bits)
    xq = torch.full((S, K), -127, dtype=torch.int8, device="cuda")
    xd = torch.ones(S, device="cuda")
    want = torch.tensor(-127.0 * value * K, dtype=torch.float64).float()
    assert bool((qre.linear_i8(bank, xq, xd) == want.cuda()).all())


@pytest.mark.parametrize("bits", [8, 4, 2])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_token_is_the_same_in_any_batch(qre, bits, dtype):
    S, N, K = 4099, 4101, 416
    g, data, scale, xq, xd, bank = make(qre, S, N, K, bits, "batch")
    bias, xq, xd = torch.randn(N, generator=g).cuda(), xq.cuda(), xd.cuda()
    whole = qre.linear_i8(bank, xq, xd, bias=bias, activation="gelu", dtype=dtype)
    for n in (1, 3, 16, 17, 33, 64, 65, 129, 300, 1100, 2500):
        part = qre.linear_i8(bank, xq[:n].contiguous(), xd[:n].contiguous(), bias=bias, activation="gelu", dtype=dtype)
        assert torch.equal(part, whole[:n]), n


@pytest.mark.parametrize("S", [1, 20, 100, 700, 4200])
def test_in_place_on_the_residual_and_a_large_workspace(qre, S):
    N, K = 4133, 256
    g, data, scale, xq, xd, bank = make(qre, S, N, K, 8, "in place")
    res = torch.randn(S, N, generator=g).to(BF16).cuda()
    ws = qre.linear_i8_workspace(bank, 8192, BF16)
    want = qre.linear_i8(bank, xq.cuda(), xd.cuda(), residual=res)
    out = res.clone()
    assert qre.linear_i8(bank, xq.cuda(), xd.cuda(), residual=out, out=out, ws=ws) is out
    assert torch.equal(out, want)


@pytest.mark.parametrize("S", [2, 40, 90, 4200])
def test_nan_and_infinity_in_a_scale_stay_in_their_row(qre, S):
    g, data, scale, xq, xd, bank = make(qre, S, 4100, 160, 4, "nan")
    want = qre.linear_i8(bank, xq.cuda(), xd.cuda(), activation="silu")
    xd[1] = float("nan")
    got = qre.linear_i8(bank, xq.cuda(), xd.cuda(), activation="silu")
    assert bool(torch.isnan(got[1]).all())
    keep = torch.arange(S) != 1
    assert torch.equal(got[keep], want[keep])


def test_no_tokens(qre):
    _, _, _, _, _, bank = make(qre, 1, 5, 64, 8, "none")
    out = qre.linear_i8(bank, torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert out.shape == (0, 5)
    q, d = qre.quantize_i8(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and d.shape == (0,)


def test_bank_and_output_past_2_31(qre):
    """Rows of the bank behind 2^31 bytes, and outputs behind 2^31 elements."""
    N, K = 300000, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    data = torch.randint(-127, 128, (1, N, K), generator=g, device="cuda", dtype=torch.int8).view(torch.uint8)
    bank = qre.QBank(data, torch.ones(1, N, device="cuda"), 8)
    for S in (2, 100):
        xq = torch.randint(-127, 128, (S, K), generator=g, device="cuda", dtype=torch.int8)
        got = qre.linear_i8(bank, xq, torch.ones(S, device="cuda"))
        rows = [0, 262143, 262144, N - 1]
        want = xq.double() @ data[0, rows].view(torch.int8).double().t().contiguous()
        assert torch.equal(got[:, rows], want.float())
    small = qre.QBank(data[:, :, :128].contiguous(), torch.ones(1, N, device="cuda"), 8)
    S = 8192
    xq = torch.randint(-127, 128, (S, 128), generator=g, device="cuda", dtype=torch.int8)
    got = qre.linear_i8(small, xq, torch.ones(S, device="cuda"), dtype=BF16)
    toks, rows = [0, 7158, 7159, S - 1], [0, 150000, N - 1]
    want = xq[toks].double() @ small.data[0, rows].view(torch.int8).double().t().contiguous()
    assert torch.equal(got[toks][:, rows], want.float().to(BF16))


@pytest.mark.parametrize("S", [1, 30, 200, 4200])
def test_captured_and_on_two_streams(qre, S):
    N, K = 4100, 288
    g, data, scale, _, _, bank = make(qre, S, N, K, 4, "graph")
    x = torch.randn(S, K, generator=g).to(BF16).cuda()
    ws = qre.linear_i8_workspace(bank, S, BF16)

    def step():
        return qre.linear_i8(bank, *qre.quantize_i8(x), dtype=BF16, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(3):
        x.copy_(torch.randn(S, K, generator=g))
        want = qre.linear_i8(bank, *qre.quantize_i8(x), dtype=BF16)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(qre.linear_i8(bank, *qre.quantize_i8(x), dtype=BF16))
    torch.cuda.synchronize()
    for z in got:
        assert torch.equal(z, want)
