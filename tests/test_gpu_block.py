"""The operators around the layer on the GPU against plain 64-bit forms
(tests/block_ref.py): norm with Q8_0, the quantised linear product, the int8
cache's append and read-back, attention over it, and a whole block of them
around the layer."""

import math

import pytest
import torch

import synth
from tests import block_ref as ref
from tests.gpu_common import say, to_device

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qre():
    import quantized_routed_expert_sigmoid_amd as m
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m.lib()
    return m


def gen(*labels):
    g = torch.Generator()
    g.manual_seed(synth.stream_key(*labels) & 0x7FFFFFFF)
    return g


def within(got, want, tol, what):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    bad = (got - want).abs() > tol
    bad &= ~torch.isnan(want) & (got != want)
    if bool(bad.any()):
        i = int(((got - want).abs() / tol.clamp(min=1e-300)).nan_to_num().flatten().argmax())
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst at {i}: "
                    f"{got.flatten()[i]} for {want.flatten()[i]}, bound {tol.expand_as(want).flatten()[i]:.3e}")


# ---- norm -----------------------------------------------------------------

NORM = [(1, 32, F32, None, F32), (3, 96, BF16, BF16, BF16), (5, 6144, F32, F32, F32), (2, 8192, BF16, F32, F32),
        (130, 2080, F32, BF16, BF16), (7, 1056, BF16, None, BF16), (300, 64, BF16, BF16, F32), (1, 4096, F32, F32, BF16),
        (67, 512, F32, F32, F32), (9, 2048, BF16, F32, BF16)]


@pytest.mark.parametrize("rows,K,xt,rt,yt", NORM)
def test_norm(qre, rows, K, xt, rt, yt):
    say(f"norm {rows} x {K} {xt} {rt} {yt}")
    g = gen("norm", rows, K)
    x = torch.randn(rows, K, generator=g).mul(3).to(xt)
    r = None if rt is None else torch.randn(rows, K, generator=g).to(rt)
    w = 1 + 0.3 * torch.randn(K, generator=g)
    if rows > 2:
        x[1] = 0
        if r is not None:
            r[1] = 0
        x[2, 0] = 3000.0  # one large value: the other codes of its block go to zero
    t, y = ref.add_rms_norm(x, r, w, 1e-5)
    res = qre.add_rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), y_dtype=yt)
    if r is None:
        assert res.sum is None
    else:
        within(res.sum, t, (ref.U[rt] + 2.0 ** -24) * t.abs(), "sum")
    # the sum of squares passes through fewer than 64 additions, its error is halved by the root
    within(res.y, y, (2.0 ** -18 + ref.U[yt]) * y.abs(), "y")
    yb = y.view(rows, K // 32, 32)
    d = yb.abs().amax(-1) / 127
    within(res.d, d, 2.0 ** -17 * d, "d")
    v = res.q.cpu().double().view(rows, K // 32, 32) * res.d.cpu().double()[..., None]
    within(v, yb, 0.5 * d[..., None] * (1 + 2.0 ** -10) + 2.0 ** -17 * yb.abs(), "codes")
    # the codes are those of the library's quantiser on the same y
    full = qre.add_rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), y_dtype=F32)
    q, dd = qre.quantize_q8_0(full.y)
    assert torch.equal(q, full.q) and torch.equal(dd, full.d)
    assert torch.equal(full.q, res.q) and torch.equal(full.d, res.d)


def test_norm_strided_in_place_and_parts(qre):
    g = gen("norm in place")
    K = 1504
    wide = torch.randn(6, 2 * K, generator=g).cuda()
    x, r0 = wide[:, K:], torch.randn(6, K, generator=g).cuda()
    w = torch.rand(K, generator=g).cuda()
    want = qre.add_rms_norm(x.contiguous(), w, 1e-6, residual=r0, y_dtype=F32)
    r = r0.clone()
    got = qre.add_rms_norm(x, w, 1e-6, residual=r, sum_out=r, y_dtype=F32)
    assert got.sum.data_ptr() == r.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    only = qre.add_rms_norm(x, w, 1e-6, residual=r0, y_dtype=F32, q8=False)
    assert only.q is None and only.d is None and torch.equal(only.y, want.y)
    codes = qre.add_rms_norm(x, w, 1e-6, residual=r0)
    assert codes.y is None and torch.equal(codes.q, want.q)
    cast = torch.empty(6, K, dtype=BF16, device="cuda")
    alone = qre.add_rms_norm(x, w, 1e-6, sum_out=cast, y_dtype=F32)
    assert torch.equal(cast, x.to(BF16)) and alone.sum is cast
    empty = qre.add_rms_norm(x[:0], w, 1e-6, residual=r0[:0], y_dtype=F32)
    assert empty.q.shape == (0, K)
    wide_r = torch.randn(6, 2 * K, generator=g).to(BF16).cuda()[:, :K]
    a = qre.add_rms_norm(x, w, 1e-6, residual=wide_r)
    b = qre.add_rms_norm(x, w, 1e-6, residual=wide_r.contiguous())
    assert torch.equal(a.q, b.q) and torch.equal(a.sum, b.sum)


def test_norm_many_rows(qre):
    """More rows than any launch has workgroups at once."""
    x = torch.randn(70001, 32, generator=gen("norm rows")).cuda()
    w = torch.ones(32, device="cuda")
    got = qre.add_rms_norm(x, w, 1e-6, y_dtype=F32)
    _, y = ref.add_rms_norm(x.cpu(), None, w.cpu(), 1e-6)
    within(got.y, y, 2.0 ** -18 * y.abs() + 1e-30, "y")


# ---- linear ---------------------------------------------------------------


def make_linear(qre, S, N, K, bits, group, *labels):
    g = gen("linear", S, N, K, bits, group, *labels)
    if bits == 8:
        w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).view(torch.uint8)
    else:
        w = torch.randint(0, 256, (N, K * bits // 8), generator=g).to(torch.uint8)
    sc = torch.randn(N, K // group if group else 1, generator=g).abs() * 0.02
    x = torch.randn(S, K // 32, 32, generator=g) * torch.exp(2 * torch.randn(S, K // 32, 1, generator=g))
    if S > 1:
        x[S // 2] = 0
    d = x.abs().amax(-1) / 127
    q = ref.round_half_away(x / d.clamp(min=1e-30)[..., None]).clamp(-127, 127).to(torch.int8).view(S, K)
    bank = qre.QBank(w[None].cuda(), sc.view(1, -1).cuda(), bits, group)
    return w, sc, q, d, bank, g


LINEAR = [(1, 64, 32, 8, 0), (1, 10, 6144, 4, 0), (2, 33, 2080, 2, 0), (3, 130, 256, 4, 64), (4, 257, 8192, 8, 128),
          (5, 17, 64, 4, 32), (8, 1000, 1056, 2, 0), (9, 64, 512, 8, 0), (16, 129, 96, 4, 0), (17, 300, 2080, 4, 0),
          (31, 31, 768, 2, 256), (33, 127, 1024, 8, 32), (64, 260, 1536, 4, 0), (100, 513, 2080, 2, 0),
          (129, 256, 4096, 4, 0), (200, 384, 160, 8, 0), (257, 1029, 640, 4, 128), (1, 1, 32, 2, 32),
          (300, 3, 32, 4, 0), (1, 2049, 16384, 4, 0), (6, 40, 12288, 8, 0)]


@pytest.mark.parametrize("S,N,K,bits,group", LINEAR)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_linear(qre, S, N, K, bits, group, dtype):
    say(f"linear {S} x {N} x {K} int{bits} group {group} {dtype}")
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, bits, group)
    bias, res = torch.randn(N, generator=g), torch.randn(S, N, generator=g).to(dtype)
    act = ["none", "silu", "gelu", "relu"][(S + N) % 4]
    for b, r, a in ((None, None, None), (bias, res, act)):
        y, A = ref.linear(w, sc, bits, group, q, d, b, a, r)
        got = qre.linear_q(bank, q.cuda(), d.cuda(), bias=None if b is None else b.cuda(), activation=a,
                           residual=None if r is None else r.cuda(), dtype=dtype)
        within(got, y, ref.linear_tol(y, A, K, dtype), f"{a}")


@pytest.mark.parametrize("S,N,K,bits,group", [
    (7700, 2100, 224, 4, 0), (7690, 2179, 160, 2, 0), (7681, 2177, 416, 8, 0), (2100, 2050, 288, 4, 0),
    (2060, 2113, 160, 2, 32), (2049, 2050, 416, 8, 0), (2049, 2177, 640, 4, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_linear_many_tokens(qre, S, N, K, bits, group, dtype):
    """Tiles for every compute unit, with ragged edges, a last step of half its length and an epilogue."""
    say(f"linear {S} x {N} x {K} int{bits} group {group} {dtype}")
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, bits, group)
    bias, res = torch.randn(N, generator=g), torch.randn(S, N, generator=g).to(dtype)
    y, A = ref.linear(w, sc, bits, group, q, d, bias, "silu", res)
    got = qre.linear_q(bank, q.cuda(), d.cuda(), bias=bias.cuda(), activation="silu", residual=res.cuda())
    within(got, y, ref.linear_tol(y, A, K, dtype), "many")


@pytest.mark.parametrize("S", [1, 40])
def test_linear_in_place_and_guard(qre, S):
    """out as its own residual; nothing is written behind the result; equal calls give equal bits."""
    w, sc, q, d, bank, g = make_linear(qre, S, 77, 416, 4, 32)
    r = torch.randn(S, 77, generator=g)
    buf = torch.full((S * 77 + 64,), 7.0, device="cuda")
    out = buf[:S * 77].view(S, 77)
    out.copy_(r)
    ws = qre.linear_workspace(bank, S)
    qre.linear_q(bank, q.cuda(), d.cuda(), residual=out, out=out, ws=ws)
    want = qre.linear_q(bank, q.cuda(), d.cuda(), residual=r.cuda())
    assert torch.equal(out, want) and bool((buf[S * 77:] == 7.0).all())


@pytest.mark.parametrize("S", [1, 4, 16, 64])
def test_linear_extreme_scales(qre, S):
    """Activations far apart in size: zero blocks, one outlier block 2^60 above the rest of its row, tiny rows."""
    N, K = 48, 256
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, 8, 0, "extreme")
    d[:, 0] *= 2.0 ** 60
    d[:, 3] = 0
    d[S // 2] = 2.0 ** -100
    y, A = ref.linear(w, sc, 8, 0, q, d, None, None, None)
    for dtype in (F32, BF16):
        got = qre.linear_q(bank, q.cuda(), d.cuda(), dtype=dtype)
        within(got, y, ref.linear_tol(y, A, K, dtype), str(dtype))


# ---- cache ----------------------------------------------------------------


def make_cache(qre, lens, H, D, *labels, spare=2, extra_pages=1, v_spread=1.0):
    """A cache of random codes and scales, shuffled pages, and the batch's host and device forms."""
    g = gen("cache", H, D, str(lens), *labels)
    need = [max(-(-n // 64), 0) for _, n in lens]
    n_pages, most = sum(need) + spare, max(need + [1]) + extra_pages
    codes = [torch.randint(-127, 128, (n_pages, H, 64 * D), generator=g).to(torch.int8) for _ in range(2)]
    scales = [(0.3 + torch.rand(n_pages, H, generator=g)) * torch.exp(v_spread * torch.randn(n_pages, H, generator=g))
              / 60 for _ in range(2)]
    scales[0] = (0.3 + torch.rand(n_pages, H, generator=g)) / 60
    order = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for s, p in enumerate(need):
        table[s, :p] = order[at:at + p].int()
        at += p
    seqs = ref.Seqs(lens, table)
    cache = qre.KVCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda(), D)
    return g, codes, scales, seqs, cache


def dev(seqs):
    return (seqs.table.cuda(), torch.tensor(seqs.cu, dtype=torch.int32).cuda(),
            torch.tensor([n for _, n in seqs.lens], dtype=torch.int32).cuda())


APPEND = [([(1, 1)], 1, 64), ([(1, 64), (1, 65), (1, 66)], 2, 128), ([(5, 70), (0, 33), (130, 200), (64, 64)], 3, 64),
          ([(200, 200), (1, 2)], 1, 192), ([(3, 67), (66, 131)], 2, 256), ([(70, 65), (1, 0)], 1, 64)]


@pytest.mark.parametrize("lens,H,D", APPEND)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("max_q", [None, 1])
def test_append_and_read(qre, lens, H, D, dtype, max_q):
    say(f"append {lens} {H} {D} {dtype} max_q {max_q}")
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, str(dtype))
    T = seqs.rows
    k = (torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))).to(dtype)
    v = torch.randn(T, H, D, generator=g).to(dtype)
    if T > 2:
        k[1:3] = 0
    both = torch.cat([k, v], 1).cuda()  # strided views of one tensor
    qre.kv_append(cache, *dev(seqs), both[:, :H], both[:, H:], max_q=max_q)
    for at, was, sc, new, now, now_sc in zip(ref.page_bytes(D), codes, scales, (k, v), (cache.k, cache.v),
                                             (cache.k_scale, cache.v_scale)):
        want, want_sc = ref.append(was, sc, at, seqs, new)
        assert torch.equal(now_sc.cpu(), want_sc)
        assert torch.equal(now.cpu(), want)
    # read back what was appended, and everything
    for rows in (lens, [(max(n, 0), n) for _, n in lens]):
        sq = ref.Seqs(rows, seqs.table)
        for rt in (F32, BF16):
            got = qre.kv_read(cache, *dev(sq), sq.rows, dtype=rt, max_q=max_q)
            for at, c, sc, x in zip(ref.page_bytes(D), (cache.k, cache.v), (cache.k_scale, cache.v_scale), got):
                vals = ref.page_values(c.cpu(), sc.cpu(), at)
                for s, (q, n) in enumerate(rows):
                    all_, _ = ref.tokens(vals, seqs.table[s], max(n, 0), c.shape[0])
                    w = torch.zeros(q, H, D, dtype=torch.float64)
                    have = min(q, max(n, 0))
                    if have:
                        w[q - have:] = all_[-have:]
                    within(x[sq.cu[s]:sq.cu[s + 1]], w, ref.U[rt] * w.abs(), "read")


def test_append_twice_gives_the_same(qre):
    """The same rows again change nothing: the scale already covers them."""
    g, _, _, seqs, cache = make_cache(qre, [(3, 40), (100, 190)], 2, 64, "twice")
    k, v = torch.randn(103, 2, 64, generator=g).cuda(), torch.randn(103, 2, 64, generator=g).cuda()
    qre.kv_append(cache, *dev(seqs), k, v)
    one = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    qre.kv_append(cache, *dev(seqs), k, v)
    assert all(torch.equal(a, b) for a, b in zip(one, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def test_append_missing_and_foreign_pages(qre):
    """Entries outside the cache are skipped; pages of nobody keep their bytes, stale scales (NaN) of fresh pages
    are not read; rows behind the last sequence are not written by the read-back."""
    g, codes, scales, seqs, cache = make_cache(qre, [(130, 130), (70, 130)], 2, 64, "missing", spare=3)
    seqs.table[0, 1] = -1
    seqs.table[1, 1] = cache.n_pages
    cache.k_scale[seqs.table[0, 0].item()] = float("nan")
    scales[0][seqs.table[0, 0].item()] = float("nan")
    k, v = torch.randn(210, 2, 64, generator=g), torch.randn(210, 2, 64, generator=g)
    qre.kv_append(cache, *dev(seqs), k.cuda(), v.cuda())
    for at, was, sc, new, now, now_sc in zip(ref.page_bytes(64), codes, scales, (k, v), (cache.k, cache.v),
                                             (cache.k_scale, cache.v_scale)):
        want, want_sc = ref.append(was, sc, at, seqs, new)
        assert torch.equal(now.cpu(), want) and torch.equal(now_sc.cpu(), want_sc)
    kk, vv = torch.full((210, 2, 64), 9.0, device="cuda"), torch.full((210, 2, 64), 9.0, device="cuda")
    qre.kv_read(cache, *dev(seqs), 210, k=kk, v=vv)
    assert bool((kk[200:] == 9.0).all()) and bool((vv[200:] == 9.0).all())
    assert bool((kk[64:128] == 0).all()) and bool((kk[130 + 4:130 + 68] == 0).all())
    assert bool((kk[:64] != 9.0).all())


# ---- attention ------------------------------------------------------------

ATTN = [([(1, 1)], 1, 1, 64), ([(1, 64)], 4, 2, 64), ([(1, 65), (1, 63), (1, 500)], 8, 1, 128),
        ([(1, 130), (0, 40), (1, 0), (1, 7)], 6, 2, 128), ([(4, 300), (4, 4), (4, 68)], 16, 2, 128),
        ([(8, 100), (3, 3), (1, 257)], 3, 1, 192), ([(5, 129), (7, 700)], 8, 2, 256), ([(9, 9), (40, 200)], 8, 1, 64),
        ([(130, 130)], 4, 2, 128), ([(77, 300), (1, 90), (200, 201), (0, 0)], 5, 1, 64), ([(150, 260)], 2, 2, 256),
        ([(33, 500), (64, 64)], 12, 2, 192), ([(1, 4100)], 24, 3, 64), ([(2, 3000), (2, 2)], 64, 1, 128),
        ([(10, 4)], 2, 1, 64)]


@pytest.mark.parametrize("lens,Hq,H,D", ATTN)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention(qre, lens, Hq, H, D, dtype):
    say(f"attention {lens} {Hq}/{H} {D} {dtype}")
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, Hq)
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    q = torch.randn(seqs.rows, Hq, D, generator=g).to(dtype)
    most_q, most_kv = max(x for x, _ in lens), max(n for _, n in lens)
    for causal, window in ((True, 0), (True, 1), (True, 100), (False, 0)):
        want, lse, sb, vb = ref.attention(kval, vval, seqs, q, D ** -0.5, causal, window)
        got_lse = torch.full((seqs.rows, Hq), 3.0, device="cuda")
        for mq, mkv in ((most_q, most_kv), (None, None), (1, 1)):
            got = qre.kv_attention(cache, *dev(seqs), q.cuda(), causal=causal, window=window, max_q=mq, max_kv=mkv,
                                   lse=got_lse)
            what = f"causal {causal} window {window} max_q {mq} max_kv {mkv}"
            within(got, want, ref.attention_tol(want, sb, vb, dtype), what)
            within(got_lse, lse, ref.lse_tol(sb, lse, dtype), what + " lse")


@pytest.mark.parametrize("q_len", [1, 50])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_sharp_scores_and_zero_blocks(qre, q_len, dtype):
    """One key far above the rest, blocks of scale zero, value scales 2^12 apart."""
    D, H, Hq = 128, 2, 4
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 400)], H, D, "sharp", v_spread=4.0)
    scales[0][seqs.table[0, 2].item()] = 0
    scales[1][seqs.table[0, 3].item()] = 0
    cache.k_scale.copy_(scales[0])
    cache.v_scale.copy_(scales[1])
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    q = (30 * torch.randn(q_len, Hq, D, generator=g)).to(dtype)
    want, lse, sb, vb = ref.attention(kval, vval, seqs, q, 0.3)
    got = qre.kv_attention(cache, *dev(seqs), q.cuda(), scale=0.3)
    within(got, want, ref.attention_tol(want, sb, vb, dtype), "sharp")


@pytest.mark.parametrize("q_len", [1, 6, 80])
def test_attention_missing_pages_and_rows_behind(qre, q_len):
    """Missing pages are seen by nobody (a sequence of only missing pages gives zeros), garbage behind a sequence's
    end stays out, rows behind the last sequence stay as they were."""
    D, H, Hq = 64, 2, 8
    lens = [(q_len, 400), (q_len, 120), (q_len, 100)]
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, "holes")
    seqs.table[0, 0] = -5
    seqs.table[0, 3] = 2 ** 30
    seqs.table[1, :] = -1
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    rows = seqs.rows + 3
    q = torch.randn(rows, Hq, D, generator=g)
    q[-1] = float("nan")
    want, lse, sb, vb = ref.attention(kval, vval, seqs, q, D ** -0.5)
    out, ol = torch.full((rows, Hq, D), 5.0, device="cuda"), torch.full((rows, Hq), 5.0, device="cuda")
    qre.kv_attention(cache, *dev(seqs), q.cuda(), out=out, lse=ol)
    n = seqs.rows
    within(out[:n], want[:n], ref.attention_tol(want, sb, vb, F32)[:n], "holes")
    within(ol[:n], lse[:n], ref.lse_tol(sb, lse, F32)[:n], "lse")
    assert bool((out[n:] == 5.0).all()) and bool((ol[n:] == 5.0).all())
    assert bool((out[q_len:2 * q_len] == 0).all())


@pytest.mark.parametrize("q_len", [2, 60])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_bad_query_stays_alone(qre, q_len, dtype):
    """A NaN or an infinity in one query gives NaN there and nowhere else; the order of rows in memory is free."""
    D, H, Hq = 128, 1, 8
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 90)], H, D, "nan")
    q = torch.randn(q_len, Hq, D, generator=g).to(dtype)
    clean = qre.kv_attention(cache, *dev(seqs), q.cuda())
    q[1, 3, 5] = float("nan")
    q[0, 6, 7] = float("inf")
    q[0, 7, 0] = float("-inf")
    wide = torch.zeros(q_len, Hq + 2, D, dtype=dtype, device="cuda")
    wide[:, 1:-1] = q.cuda()
    lse = torch.zeros(q_len, Hq, device="cuda")
    out = torch.zeros(q_len, 2 * Hq, D, dtype=dtype, device="cuda")
    qre.kv_attention(cache, *dev(seqs), wide[:, 1:-1], out=out[:, Hq:], lse=lse)
    bad = torch.zeros(q_len, Hq, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[0, 6] = bad[0, 7] = True
    assert bool(torch.isnan(out[:, Hq:][bad]).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(out[:, Hq:][~bad], clean[~bad]) and bool((out[:, :Hq] == 0).all())


@pytest.mark.parametrize("q_len", [1, 4, 40])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_attention_scale_of_any_sign(qre, q_len, scale):
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 150), (q_len, q_len)], 1, 64, "sign")
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(64)))
    for dtype in (F32, BF16):
        q = torch.randn(seqs.rows, 8, 64, generator=g).to(dtype)
        want, lse, sb, vb = ref.attention(kval, vval, seqs, q, scale)
        got_lse = torch.zeros(seqs.rows, 8, device="cuda")
        got = qre.kv_attention(cache, *dev(seqs), q.cuda(), scale=scale, lse=got_lse)
        within(got, want, ref.attention_tol(want, sb, vb, dtype), "out")
        within(got_lse, lse, ref.lse_tol(sb, lse, dtype), "lse")


@pytest.mark.parametrize("q_len", [2, 50])
def test_lengths_beyond_their_bounds(qre, q_len):
    """kv_len above the table's capacity counts as the capacity, below zero as zero; cu_q above the rows is cut;
    rows before the first sequence stay as they were."""
    D, H, Hq = 64, 1, 8
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 192), (q_len, 100)], H, D, "bounds", extra_pages=0)
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    rows = 2 * q_len
    q = torch.randn(rows + 1, Hq, D, generator=g)
    table = seqs.table.cuda()
    cu = torch.tensor([1, q_len + 1, 10 ** 6], dtype=torch.int32).cuda()
    kv = torch.tensor([10 ** 9, -7], dtype=torch.int32).cuda()
    out = torch.full((rows + 1, Hq, D), 5.0, device="cuda")
    for max_kv in (192, 1, None):
        qre.kv_attention(cache, table, cu, kv, q.cuda(), out=out, max_kv=max_kv)
        s2 = ref.Seqs([(q_len, 192), (q_len, 0)], seqs.table)
        want, _, sb, vb = ref.attention(kval, vval, s2, q[1:], D ** -0.5)
        within(out[1:], want, ref.attention_tol(want, sb, vb, F32), "cut")
        assert bool((out[0] == 5.0).all())
    k, v = qre.kv_read(cache, table, cu, kv, rows + 1)
    assert bool((k[q_len + 1:] == 0).all())
    before = cache.k.clone()
    qre.kv_append(cache, table, torch.tensor([0, 0, q_len], dtype=torch.int32).cuda(), kv,
                  torch.randn(rows + 1, H, D).cuda(), torch.randn(rows + 1, H, D).cuda())
    assert torch.equal(cache.k, before)  # no token number that is not negative


def test_attention_long_offsets(qre):
    """A page beyond 2^31 bytes of the pool: offsets in 64 bits."""
    D, H = 256, 8
    n_pages = (1 << 31) // (H * 64 * D) + 4
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * (n_pages * H * 64 * D):
        pytest.skip("not enough device memory")
    cache = qre.KVCache.empty(n_pages, H, D)
    g = gen("far")
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32)
    seqs = ref.Seqs([(100, 100)], table)
    k, v = torch.randn(100, H, D, generator=g), torch.randn(100, H, D, generator=g)
    qre.kv_append(cache, *dev(seqs), k.cuda(), v.cuda())
    last = qre.KVCache(cache.k[-2:].clone(), cache.v[-2:].clone(), cache.k_scale[-2:].clone(),
                       cache.v_scale[-2:].clone(), D)
    near = ref.Seqs([(100, 100)], torch.tensor([[1, 0]], dtype=torch.int32))
    q = torch.randn(100, H, D, generator=g).cuda()
    for x, y in ((seqs, near), (ref.Seqs([(1, 100)], table), ref.Seqs([(1, 100)], near.table))):
        n = x.rows
        assert torch.equal(qre.kv_attention(cache, *dev(x), q[:n]), qre.kv_attention(last, *dev(y), q[:n]))
    a, b = qre.kv_read(cache, *dev(seqs), 100), qre.kv_read(last, *dev(near), 100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    d = k.abs().amax() / 127
    assert float((a[0].cpu() - k).abs().max()) <= float(d) * 0.51


def test_attention_many_sequences(qre):
    """A batch of 300 sequences of one token each over pages they share."""
    D, H, Hq, n = 64, 1, 4, 300
    g, codes, scales, seqs, cache = make_cache(qre, [(1, 200)], H, D, "many")
    r = torch.randint(1, 201, (n,), generator=g)
    many = ref.Seqs([(1, int(x)) for x in r], seqs.table.expand(n, -1).contiguous())
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    q = torch.randn(n, Hq, D, generator=g)
    want, _, sb, vb = ref.attention(kval, vval, many, q, D ** -0.5)
    within(qre.kv_attention(cache, *dev(many), q.cuda(), max_q=1), want, ref.attention_tol(want, sb, vb, F32), "many")


# ---- as they are used -----------------------------------------------------


def make_block(qre, hidden=256, heads=4, kv_heads=2, D=64):
    """Weights of one block: norms, quantised projections, the layer."""
    w = synth.scaled(synth.WORKLOADS["tiny"], name="block", layer="block", hidden=hidden, inter=64, n_experts=8,
                     top_k=2, bits=4, has_shared=True, rsf=2.5, var_router=1.0 / hidden)
    L = synth.make_layer(w)
    g = gen("block")

    def bank(n, k, bits):
        d = torch.randint(0, 256, (1, n, k * bits // 8), generator=g).to(torch.uint8)
        if bits == 8:
            d[d == 128] = 0
        return qre.QBank(d.cuda(), (torch.rand(1, n, generator=g) * 0.3 / math.sqrt(k)).cuda(), bits)
    return {"w": w, "layer": to_device(L), "n1": torch.rand(hidden, generator=g).cuda() + 0.5,
            "n2": torch.rand(hidden, generator=g).cuda() + 0.5, "qkv": bank((heads + 2 * kv_heads) * D, hidden, 4),
            "bias": torch.randn((heads + 2 * kv_heads) * D, generator=g).cuda() * 0.1, "o": bank(hidden, heads * D, 8),
            "heads": heads, "kv": kv_heads, "D": D, "cache": qre.KVCache.empty(12, kv_heads, D)}


def block_forward(qre, B, h, delta, table, cu, kv_len, max_q=None):
    """The residual stream h and the last block's output delta through one block; returns (stream, output)."""
    n = qre.add_rms_norm(delta, B["n1"], 1e-5, residual=h)
    qkv = qre.linear_q(B["qkv"], n.q, n.d, bias=B["bias"]).view(h.shape[0], -1, B["D"])
    q, k, v = qkv.split([B["heads"], B["kv"], B["kv"]], dim=1)
    qre.kv_append(B["cache"], table, cu, kv_len, k, v, max_q=max_q)
    a = qre.kv_attention(B["cache"], table, cu, kv_len, q, max_q=max_q).view(h.shape[0], -1)
    s = qre.linear_q(B["o"], *qre.quantize_q8_0(a), residual=n.sum)
    m = qre.add_rms_norm(s, B["n2"], 1e-5, y_dtype=F32, q8=False)
    return s, qre.moe_layer_forward(B["layer"], m.y)


def test_block_prompt_then_decode(qre):
    """Two sequences: a prompt, then token by token, against the same tokens in one prompt and against the plain
    forms step by step (each on the previous kernel's own output)."""
    B = make_block(qre)
    hid, D, nh, nk = 256, B["D"], B["heads"], B["kv"]
    g = gen("block run")
    table = torch.randperm(12, generator=g).view(2, 6).int()
    lens = [(70, 70), (33, 33)]
    seqs = ref.Seqs(lens, table)
    h, delta = torch.randn(seqs.rows, hid, generator=g).cuda(), torch.randn(seqs.rows, hid, generator=g).cuda()
    args = dev(seqs)

    n = qre.add_rms_norm(delta, B["n1"], 1e-5, residual=h, y_dtype=F32)
    t, y = ref.add_rms_norm(delta.cpu(), h.cpu(), B["n1"].cpu(), 1e-5)
    within(n.y, y, 2.0 ** -17 * y.abs(), "norm")
    qkv = qre.linear_q(B["qkv"], n.q, n.d, bias=B["bias"])
    w, A = ref.linear(B["qkv"].data[0].cpu(), B["qkv"].scale[0].cpu(), 4, 0, n.q.cpu(), n.d.cpu(), B["bias"].cpu(), None,
                      None)
    within(qkv, w, ref.linear_tol(w, A, hid, F32), "qkv")
    q, k, v = qkv.view(-1, nh + 2 * nk, D).split([nh, nk, nk], dim=1)
    qre.kv_append(B["cache"], *args, k, v)
    kval, vval = (ref.page_values(c.cpu(), s.cpu(), at) for c, s, at in zip(
        (B["cache"].k, B["cache"].v), (B["cache"].k_scale, B["cache"].v_scale), ref.page_bytes(D)))
    a = qre.kv_attention(B["cache"], *args, q)
    want, _, sb, vb = ref.attention(kval, vval, seqs, q.cpu().contiguous(), D ** -0.5)
    within(a, want, ref.attention_tol(want, sb, vb, F32), "attention")
    s, out = block_forward(qre, B, h, delta, *args)
    assert bool(torch.isfinite(out).all())

    # the next tokens one by one, with lengths in device memory
    for step in range(3):
        lens2 = [(1, 71 + step), (1, 34 + step)]
        sq = ref.Seqs(lens2, table)
        h1, d1 = torch.randn(2, hid, generator=g).cuda(), torch.randn(2, hid, generator=g).cuda()
        s1, o1 = block_forward(qre, B, h1, d1, *dev(sq), max_q=1)
        assert bool(torch.isfinite(o1).all()) and s1.shape == (2, hid)


def test_block_captured_and_replayed(qre):
    """A decode step captured into a graph and replayed on growing lengths equals the eager steps."""
    B = make_block(qre)
    g = gen("block graph")
    table = torch.randperm(12, generator=g).view(2, 6).int().cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    kv = torch.tensor([60, 3], dtype=torch.int32).cuda()
    xs = [(torch.randn(2, 256, generator=g).cuda(), torch.randn(2, 256, generator=g).cuda()) for _ in range(6)]
    B["cache"].k.zero_()
    B["cache"].v.zero_()
    B["cache"].k_scale.fill_(0.01)
    B["cache"].v_scale.fill_(0.01)
    start = [t.clone() for t in (B["cache"].k, B["cache"].v, B["cache"].k_scale, B["cache"].v_scale)]

    def reset():
        for t, c in zip((B["cache"].k, B["cache"].v, B["cache"].k_scale, B["cache"].v_scale), start):
            t.copy_(c)
        kv.copy_(torch.tensor([60, 3], dtype=torch.int32))

    eager = []
    for h, d in xs:
        kv += 1
        eager.append([t.clone() for t in block_forward(qre, B, h, d, table, cu, kv, max_q=1)])
    reset()
    h, d = xs[0][0].clone(), xs[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_forward(qre, B, h, d, table, cu, kv, max_q=1)
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block_forward(qre, B, h, d, table, cu, kv, max_q=1)
    reset()
    for i, (hh, dd) in enumerate(xs):
        kv += 1
        h.copy_(hh)
        d.copy_(dd)
        graph.replay()
        junk = torch.randn(1000, device="cuda").sum().item()  # eager work and a synchronisation between the replays
        assert math.isfinite(junk)
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), f"replay {i}"


def test_prompt_kernels_captured_and_replayed(qre):
    """The forms for many tokens (LDS of more than 64 KB among them) inside one graph, replayed with other inputs."""
    D, H, Hq = 128, 2, 8
    g, codes, scales, seqs, cache = make_cache(qre, [(90, 300), (40, 700)], H, D, "graph")
    args = dev(seqs)
    w, sc, xq, xd, bank, _ = make_linear(qre, 130, 2100, 384, 4, 128, "graph")
    _, _, xq2, xd2, bank2, _ = make_linear(qre, 7700, 2100, 128, 2, 0, "graph")
    ins = [(torch.randn(130, Hq, D, generator=g).to(BF16).cuda(), torch.randn(130, H, D, generator=g).to(BF16).cuda(),
            torch.roll(xq.cuda(), i, 0), torch.roll(xd.cuda(), i, 0), torch.roll(xq2.cuda(), i, 0),
            torch.roll(xd2.cuda(), i, 0)) for i in range(4)]
    start = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]

    def step(q, k, a, b, c, d):
        qre.kv_append(cache, *args, k, k, max_q=90)
        return (qre.kv_attention(cache, *args, q), qre.linear_q(bank, a, b, dtype=F32),
                qre.linear_q(bank2, c, d, dtype=BF16, activation="gelu"), *qre.kv_read(cache, *args, 130))

    def reset():
        for t, c in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), start):
            t.copy_(c)
    eager = []
    for x in ins:
        reset()
        eager.append([t.clone() for t in step(*x)])
    buf = [t.clone() for t in ins[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*buf)
    for i in (1, 3, 0, 2, 1):
        reset()
        for b, x in zip(buf, ins[i]):
            b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager[i]):
            assert torch.equal(a, b), f"inputs {i}"


def test_two_streams_at_once(qre):
    """Calls that overlap on two streams, each with its own workspace and outputs."""
    g, codes, scales, seqs, cache = make_cache(qre, [(1, 2000), (1, 900)], 2, 128, "streams")
    q = torch.randn(2, 16, 128, generator=g).cuda()
    w, sc, xq, xd, bank, _ = make_linear(qre, 3, 500, 1024, 4, 0)
    xq, xd, args = xq.cuda(), xd.cuda(), dev(seqs)
    want, lin = qre.kv_attention(cache, *args, q), qre.linear_q(bank, xq, xd)
    torch.cuda.synchronize()
    _, _, _, long_seqs, long_cache = make_cache(qre, [(60, 500), (200, 900)], 2, 128, "streams")
    long_q, long_args = torch.randn(260, 8, 128, generator=g).cuda(), dev(long_seqs)
    _, _, xq2, xd2, bank2, _ = make_linear(qre, 300, 500, 1024, 8, 0)
    xq2, xd2 = xq2.cuda(), xd2.cuda()
    want2, lin2 = qre.kv_attention(long_cache, *long_args, long_q), qre.linear_q(bank2, xq2, xd2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append((qre.kv_attention(cache, *args, q), qre.linear_q(bank, xq, xd),
                         qre.kv_attention(long_cache, *long_args, long_q), qre.linear_q(bank2, xq2, xd2)))
    torch.cuda.synchronize()
    for got in outs:
        for a, b in zip(got, (want, lin, want2, lin2)):
            assert torch.equal(a, b)
