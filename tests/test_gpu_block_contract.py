"""What the contract of the operators around the layer promises at its edges, on
the GPU."""

import math

import pytest
import torch

from tests import block_ref as ref
from tests.gpu_common import say
from tests.test_gpu_block import BF16, F32, block_forward, dev, gen, make_block, make_cache, make_linear, qre, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- missing pages --------------------------------------------------------


@pytest.mark.parametrize("bad", [float("nan"), -1.0, float("inf"), float("-inf")])
@pytest.mark.parametrize("q_len", [1, 6, 80])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_missing_page_takes_no_part(qre, dtype, q_len, bad):
    """A missing page is seen by no query, whatever stands in the pool's first page (which need not be written)."""
    D, H, Hq = 64, 2, 8
    lens = [(q_len, 400), (q_len, 120), (q_len, 100)]
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, "first page")
    used = set(seqs.table[seqs.table >= 0].tolist())
    free = next(p for p in range(1, cache.n_pages) if p not in used)
    seqs.table[seqs.table == 0] = free
    seqs.table[0, 0] = -1
    seqs.table[0, 4] = cache.n_pages
    seqs.table[1, :] = -7
    q = torch.randn(seqs.rows, Hq, D, generator=g).to(dtype)
    results = []
    for value in (1.0, bad):
        cache.k_scale[0] = value
        cache.v_scale[0] = value
        lse = torch.full((seqs.rows, Hq), 3.0, device="cuda")
        results.append((qre.kv_attention(cache, *dev(seqs), q.cuda(), max_q=q_len, max_kv=400, lse=lse), lse))
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    want, lse64, sb, vb = ref.attention(kval, vval, seqs, q, D ** -0.5)
    for out, lse in results:
        within(out, want, ref.attention_tol(want, sb, vb, dtype), "out")
        within(lse, lse64, ref.lse_tol(sb, lse64, dtype), "lse")
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


# ---- NaN through the activations ------------------------------------------


@pytest.mark.parametrize("S,N,K,dtype", [(1, 70, 256, F32), (4, 70, 256, BF16), (9, 70, 512, F32), (70, 70, 256, BF16),
                                         (2049, 2050, 128, F32), (7700, 2100, 128, BF16)])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_linear_keeps_nan(qre, S, N, K, dtype, act):
    """A NaN in a bias, a row's scale or a token's scale comes out as NaN, and nowhere else."""
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, 8, 0, "nan")
    bias = torch.randn(N, generator=g)
    clean = qre.linear_q(bank, q.cuda(), d.cuda(), bias=bias.cuda(), activation=act, dtype=dtype)
    bias[3] = float("nan")
    bank.scale[0, 5] = float("nan")
    d[S // 2, 1] = float("nan")
    got = qre.linear_q(bank, q.cuda(), d.cuda(), bias=bias.cuda(), activation=act, dtype=dtype)
    bad = torch.zeros(S, N, dtype=torch.bool, device="cuda")
    bad[:, 3] = bad[:, 5] = True
    bad[S // 2] = True
    assert bool(torch.isnan(got[bad]).all())
    assert torch.equal(got[~bad], clean[~bad])


# ---- workspaces of larger batches -----------------------------------------


@pytest.mark.parametrize("N,K,bits,dtype", [(10240, 1024, 4, F32), (4096, 4096, 2, BF16), (130, 2080, 8, F32)])
def test_linear_workspace_serves_smaller_batches(qre, N, K, bits, dtype):
    """One workspace for the largest batch, calls of every smaller size in it; the same bits as with their own."""
    most = 1024
    w, sc, q, d, bank, g = make_linear(qre, most, N, K, bits, 0, "ws")
    q, d = q.cuda(), d.cuda()
    ws = qre.linear_workspace(bank, most, dtype)
    for S in (1, 4, 5, 32, 33, 64, 65, 257, 512, most):
        got = qre.linear_q(bank, q[:S], d[:S], dtype=dtype, ws=ws)
        assert torch.equal(got, qre.linear_q(bank, q[:S], d[:S], dtype=dtype)), S


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_workspace_serves_smaller_batches(qre, dtype):
    """One workspace for the largest batch; fewer sequences, shorter runs and shorter caches in it."""
    D, H, Hq, n = 64, 2, 8, 80
    g, codes, scales, seqs, cache = make_cache(qre, [(40, 700)] * n, H, D, "ws")
    ws = qre.kv_attention_workspace(cache, n, n * 40, Hq, 40, 700, dtype)
    q = torch.randn(n * 40, Hq, D, generator=g).to(dtype).cuda()
    for m, ql, kv in ((80, 40, 700), (80, 1, 700), (16, 1, 700), (1, 1, 700), (1, 40, 700), (3, 7, 500), (1, 1, 30)):
        s = ref.Seqs([(ql, kv)] * m, seqs.table[:m].contiguous())
        x = q[:m * ql]
        got = qre.kv_attention(cache, *dev(s), x, max_q=ql, max_kv=kv, ws=ws)
        assert torch.equal(got, qre.kv_attention(cache, *dev(s), x, max_q=ql, max_kv=kv)), (m, ql, kv)


def test_workspace_with_gaps_is_refused(qre):
    w, sc, q, d, bank, g = make_linear(qre, 40, 77, 416, 4, 32, "gaps")
    n = qre.linear_workspace(bank, 40).numel()
    for ws in (torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(256, dtype=torch.uint8, device="cuda")[:1].expand(n)):
        with pytest.raises(ValueError, match="ws: contiguous"):
            qre.linear_q(bank, q.cuda(), d.cuda(), ws=ws)
    g, codes, scales, seqs, cache = make_cache(qre, [(1, 900)], 1, 64, "gaps")
    n = qre.kv_attention_workspace(cache, 1, 1, 8, 1, 900).numel()
    with pytest.raises(ValueError, match="ws: contiguous"):
        qre.kv_attention(cache, *dev(seqs), torch.randn(1, 8, 64).cuda(), max_kv=900,
                         ws=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])


@pytest.mark.parametrize("q_len", [1, 40])
def test_window_beyond_32_bits_is_no_window(qre, q_len):
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 300)], 2, 64, "wide window")
    q = torch.randn(q_len, 8, 64, generator=g).cuda()
    want = qre.kv_attention(cache, *dev(seqs), q)
    for window in (300, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        assert torch.equal(qre.kv_attention(cache, *dev(seqs), q, window=window), want), window
    for window in (-1, 5 - 2 ** 32):
        with pytest.raises(qre.ColibriError):
            qre.kv_attention(cache, *dev(seqs), q, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_mixed_batch_without_hints(qre, dtype):
    """A long prompt among decoding sequences and short runs, no lengths given: append, read-back and attention."""
    D, H, Hq = 64, 2, 8
    lens = [(1, 200)] * 20 + [(700, 800)] + [(1, 90)] * 20 + [(0, 64), (30, 30)]
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, "mixed", str(dtype))
    k, v = torch.randn(seqs.rows, H, D, generator=g).to(dtype), torch.randn(seqs.rows, H, D, generator=g).to(dtype)
    qre.kv_append(cache, *dev(seqs), k.cuda(), v.cuda())
    for at, was, sc, new, now, now_sc in zip(ref.page_bytes(D), codes, scales, (k, v), (cache.k, cache.v),
                                             (cache.k_scale, cache.v_scale)):
        want, want_sc = ref.append(was, sc, at, seqs, new)
        assert torch.equal(now.cpu(), want) and torch.equal(now_sc.cpu(), want_sc)
    kval, vval = (ref.page_values(c.cpu(), s.cpu(), at) for c, s, at in zip(
        (cache.k, cache.v), (cache.k_scale, cache.v_scale), ref.page_bytes(D)))
    got_k, got_v = qre.kv_read(cache, *dev(seqs), seqs.rows)
    for got, val in ((got_k, kval), (got_v, vval)):
        for s, (q, n) in enumerate(lens):
            if q:
                want = ref.tokens(val, seqs.table[s], n, cache.n_pages)[0][n - q:]
                within(got[seqs.cu[s]:seqs.cu[s + 1]], want, ref.U[F32] * want.abs(), "read")
    q = torch.randn(seqs.rows, Hq, D, generator=g).to(dtype)
    want, lse64, sb, vb = ref.attention(kval, vval, seqs, q, D ** -0.5)
    lse = torch.zeros(seqs.rows, Hq, device="cuda")
    within(qre.kv_attention(cache, *dev(seqs), q.cuda(), lse=lse), want, ref.attention_tol(want, sb, vb, dtype), "out")
    within(lse, lse64, ref.lse_tol(sb, lse64, dtype), "lse")


# ---- attention held to the queries that the kernel uses --------------------


def fixed_point(q, dtype):
    """The queries as the kernel takes them: integers of a row's unit, amax / (127 * 256) for bf16 and amax / (127 *
    65536) for fp32 (fp32 arithmetic step by step). -> integers, units (float64)."""
    x = q.float()
    top = torch.tensor(127.0 * (65536 if dtype == F32 else 256))
    amax = x.abs().amax(-1, keepdim=True)
    up = amax * torch.where(amax < 2.0 ** -60, 2.0 ** 64, 1.0)
    lift = torch.where(amax < 2.0 ** -60, torch.tensor(2.0 ** 64), torch.tensor(1.0))
    f = torch.where(up == 0, torch.tensor(0.0), torch.div(top.expand_as(up), up))
    n = torch.round(x * lift * f)
    return n.double(), torch.div(torch.div(up, top), lift).double()


def attention_bounds(codes, scales, seqs, q, scale, dtype):
    """Causal attention in 64 bits on the kernel's fixed-point queries -> out, its bound, lse, its bound.

    With T2 the largest |score| of a row in units of log 2 and W the largest |log2| of a value scale, an exponent
    passes through five roundings of the score (log2 e, its product with the scale and the unit, the key scale, the
    conversion), one of log2(w) - m, one of the fma and two of the waves' and ranges' factors: under 2^-24 (10 T2 +
    8 (T2 + W + 8)), with 128 units for the low digits of fp32 queries; the exponentials' and the logarithm's own
    errors are under 2^-20 together.  A weight enters the value product rounded once (bf16: 2^-8, three terms for
    fp32: 2^-23); sums in fp32 pass through fewer than n / 8 + 128 additions."""
    n_pages, H = codes[0].shape[:2]
    T, Hq, D = q.shape
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    ints, unit = fixed_point(q, dtype)
    out, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, lse_tol = torch.zeros(T, Hq, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    p_err = 2.0 ** -23 if dtype == F32 else 2.0 ** -8
    for s, (ql, n) in enumerate(seqs.lens):
        k, _ = ref.tokens(kval, seqs.table[s], n, n_pages)
        v, _ = ref.tokens(vval, seqs.table[s], n, n_pages)
        pages = seqs.table[s, :-(-n // ref.BLOCK)].long()
        hidden = torch.arange(n)[None] > torch.arange(n - ql, n)[:, None]
        rows = slice(seqs.cu[s], seqs.cu[s] + ql)
        for h in range(Hq):
            hk = h // (Hq // H)
            z = scale * unit[rows, h] * (ints[rows, h] @ k[:, hk].t())
            t2 = (z.abs().masked_fill(hidden, 0.0).amax(1, keepdim=True)) / math.log(2)
            z = z.masked_fill(hidden, -math.inf)
            W = scales[1][pages, hk].double().log2().abs().amax()
            low = 128 * abs(scale) * unit[rows, h] * scales[0][pages, hk].double().amax() / math.log(2)
            e = 2.0 ** -24 * (18 * t2 + 8 * (W + 8)) + low + 2.0 ** -20
            m = z.amax(1, keepdim=True)
            p = torch.exp(z - m)
            l = p.sum(1, keepdim=True)
            p = p / l
            sums = (n / 8 + 128) * 2.0 ** -24
            out[rows, h] = p @ v[:, hk]
            tol[rows, h] = (2 * e + p_err + 2 * sums) * (p @ v[:, hk].abs()) + ref.U[dtype] * out[rows, h].abs() + 1e-30
            lse[rows, h] = (m + torch.log(l)).squeeze(1)
            lse_tol[rows, h] = (e + sums).squeeze(1) + 2.0 ** -22 * (1 + lse[rows, h].abs())
    return out, tol, lse, lse_tol


@pytest.mark.parametrize("lens,Hq,H,D", [([(1, 4100)], 8, 1, 128), ([(3, 3000), (3, 130)], 8, 2, 64), ([(6, 4000)], 8, 1, 128),
                                         ([(70, 3900)], 4, 1, 64), ([(40, 1500), (1, 64)], 8, 2, 192), ([(2, 2500)], 2, 1, 256)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_every_page_counts(qre, lens, Hq, H, D, dtype):
    """Each page of a long context has a value dim of its own: a page left out, or counted twice, is out of bounds."""
    say(f"pages {lens} {Hq}/{H} {D} {dtype}")
    g, codes, scales, seqs, cache = make_cache(qre, lens, H, D, "own dim")
    scales[1] = (0.5 + torch.rand(cache.n_pages, H, generator=g)) / 60
    codes[1].zero_()
    at = ref.page_bytes(D)[1]
    for s, (_, n) in enumerate(lens):
        for b in range(-(-n // ref.BLOCK)):
            page = int(seqs.table[s, b])
            codes[1][page][:, at[:, b % D]] = torch.randint(1, 128, (H, ref.BLOCK), generator=g).to(torch.int8)
    cache.v.copy_(codes[1])
    cache.v_scale.copy_(scales[1])
    q = torch.randn(seqs.rows, Hq, D, generator=g).to(dtype)
    want, tol, lse, ltol = attention_bounds(codes, scales, seqs, q, D ** -0.5, dtype)
    assert bool((tol < 0.05 * want)[want > 0].all())  # zeros, or a page twice, would be found
    got_lse = torch.zeros(seqs.rows, Hq, device="cuda")
    for mq, mkv in ((max(x for x, _ in lens), max(n for _, n in lens)), (None, None), (1, 1)):
        got = qre.kv_attention(cache, *dev(seqs), q.cuda(), max_q=mq, max_kv=mkv, lse=got_lse)
        within(got, want, tol, f"max_q {mq} max_kv {mkv}")
        within(got_lse, lse, ltol, "lse")


@pytest.mark.parametrize("q_len", [1, 5, 50])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_of_sharp_scores(qre, q_len, dtype):
    """One key far above the rest, value scales 2^12 apart: the result is that key's value, zeros are out of bounds."""
    D, H, Hq = 128, 2, 4
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 400)], H, D, "sharp scores", v_spread=2.0)
    q = (30 * torch.randn(q_len, Hq, D, generator=g)).to(dtype)
    want, tol, lse, ltol = attention_bounds(codes, scales, seqs, q, 0.3, dtype)
    assert float((tol < 0.1 * want.abs()).double().mean()) > 0.9
    got_lse = torch.zeros(q_len, Hq, device="cuda")
    within(qre.kv_attention(cache, *dev(seqs), q.cuda(), scale=0.3, lse=got_lse), want, tol, "sharp")
    within(got_lse, lse, ltol, "lse")


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_of_an_outlier_channel(qre, q_len, dtype):
    """One query channel 2000 times the others: a score is off by at most half a unit of the row, amax / 65024 (bf16)
    or amax / 16646144 (fp32), times scale * sum |k|, and on the unit's integers the bounds are the usual ones."""
    D, H, Hq = 128, 1, 8
    g, codes, scales, seqs, cache = make_cache(qre, [(q_len, 300)], H, D, "outlier")
    codes[0][:, :, ref.page_bytes(D)[0][:, 5]] = 0
    cache.k.copy_(codes[0])
    q = torch.randn(q_len, Hq, D, generator=g)
    q[..., 5] = 2000.0
    q = q.to(dtype)
    want, tol, lse, ltol = attention_bounds(codes, scales, seqs, q, D ** -0.5, dtype)
    got_lse = torch.zeros(q_len, Hq, device="cuda")
    within(qre.kv_attention(cache, *dev(seqs), q.cuda(), lse=got_lse), want, tol, "outlier")
    within(got_lse, lse, ltol, "lse")
    kval, vval = (ref.page_values(c, s, at) for c, s, at in zip(codes, scales, ref.page_bytes(D)))
    _, exact, _, _ = ref.attention(kval, vval, seqs, q, D ** -0.5)
    pages = seqs.table[0, :5].long()
    k_sum = kval[pages].abs().sum(-1).amax()
    half = 2000.0 / (65024 if dtype == BF16 else 16646144) * (1 + 2.0 ** -20)
    within(got_lse, exact, half * k_sum * D ** -0.5 + ltol, "lse of the queries themselves")


# ---- linear: plans and ranges ---------------------------------------------


def linear_bound(y, A, K, dtype, half_prec=None):
    """fp32 sums of K products (K / 16 + 40 roundings at most: blocks of 16 and more are summed by one instruction),
    the scales' product by two roundings and, with half_prec = (|W|, largest scale of each token), activations in
    fp16: half a step is 2^-11 of a value, or of the token's largest scale 2^-31 where the value leaves fp16's normal
    range (the power of two puts 127 times that scale above 2^13.98, a subnormal's half step is 2^-25)."""
    tol = ((K / 16 + 40) * 2.0 ** -24 + 2.0 ** -22) * A + ref.U[dtype] * y.abs() + 1e-36
    if half_prec is not None:
        w_sum, top = half_prec
        tol = tol + 2.0 ** -11 * A + 2.0 ** -31 * top[:, None] * w_sum[None]
    return tol


@pytest.mark.parametrize("S,N,K,bits,group", [
    (64, 200, 960, 8, 96), (40, 130, 960, 4, 160), (33, 70, 1920, 2, 96), (300, 257, 480, 4, 160), (70, 300, 640, 8, 64),
    (20, 130, 1280, 4, 64), (9, 4101, 1120, 2, 160), (129, 64, 288, 8, 96), (2049, 2050, 480, 4, 96), (2049, 2050, 320, 2, 160),
    (2049, 2050, 320, 8, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_linear_groups_across_stages(qre, S, N, K, bits, group, dtype):
    """Scale groups that neither divide a stage of 128 nor are multiples of it end inside stages and run across them."""
    say(f"linear {S} x {N} x {K} int{bits} group {group} {dtype}")
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, bits, group, "groups")
    y, A = ref.linear(w, sc, bits, group, q, d, None, None, None)
    within(qre.linear_q(bank, q.cuda(), d.cuda(), dtype=dtype), y, linear_bound(y, A, K, dtype), "groups")


@pytest.mark.parametrize("bits", [8, 4, 2])
def test_linear_half_precision_range(qre, bits):
    """Blocks of a token 2^10 to 2^28 apart in the form that holds activations in fp16; each weight row sees one of
    them only, so that what a small block loses shows."""
    S, N, K = 7700, 2100, 128
    w, sc, q, d, bank, g = make_linear(qre, S, N, K, bits, 0, "half")
    by = 32 * bits // 8
    rows = torch.arange(N)
    for b in range(4):
        w[rows % 4 != b, by * b:by * (b + 1)] = 0
    bank.data.copy_(w[None])
    d = torch.rand(S, 1, generator=g) + 0.5
    d = d * torch.tensor([1.0, 2.0 ** -24, 2.0 ** -28, 2.0 ** -10])
    y, A = ref.linear(w, sc, bits, 0, q, d, None, None, None)
    codes = ref.weight_codes(w, bits).double().abs().sum(1) * sc.double().abs()[:, 0]
    tol = linear_bound(y, A, K, BF16, (codes, d.amax(1).double()))
    assert float((tol < 0.1 * A)[:, 1::4].double().mean()) > 0.9
    within(qre.linear_q(bank, q.cuda(), d.cuda(), dtype=BF16), y, tol, "range")


@pytest.mark.parametrize("S", [1, 8])
def test_linear_activations_over_their_range(qre, S):
    """SiLU within 2^-23 (|v| + 8) of its value (the exponent's rounding grows with |v|), GELU within 2^-22 of 1 + |v|;
    v is the bias."""
    N, K = 4096, 128
    v = torch.linspace(-86, 86, N)
    bank = qre.QBank(torch.zeros(1, N, K, dtype=torch.uint8, device="cuda"), torch.ones(1, N, device="cuda"), 8)
    q, d = torch.ones(S, K, dtype=torch.int8, device="cuda"), torch.ones(S, K // 32, device="cuda")
    x = v.double()
    silu, gelu = x * torch.special.expit(x), x * torch.special.ndtr(x)
    for act, want, tol in (("silu", silu, 2.0 ** -23 * (x.abs() + 8) * silu.abs() + 1e-37),
                           ("gelu", gelu, 2.0 ** -22 * (1 + x.abs())), ("relu", x.clamp(min=0), torch.zeros(N).double())):
        got = qre.linear_q(bank, q, d, bias=v.cuda(), activation=act)
        within(got, want.expand(S, N), tol.expand(S, N), act)


# ---- as they are used -----------------------------------------------------


def test_decode_steps_against_plain_forms(qre):
    """A prompt, then token by token: every operator of every step against its plain form on the kernels' own inputs,
    and the steps' parts together give what the block gives."""
    B = make_block(qre)
    hid, D, nh, nk = 256, B["D"], B["heads"], B["kv"]
    g = gen("decode steps")
    table = torch.randperm(12, generator=g).view(2, 6).int()
    cache = B["cache"]
    at = ref.page_bytes(D)
    for t in (cache.k, cache.v):
        t.zero_()
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))  # pages that no token was written to
    for lens in ([(62, 62), (33, 33)], [(1, 63), (1, 34)], [(1, 64), (1, 35)], [(1, 65), (1, 36)], [(3, 68), (3, 39)]):
        sq = ref.Seqs(lens, table)
        args, mq = dev(sq), max(q for q, _ in lens)
        h, delta = torch.randn(sq.rows, hid, generator=g).cuda(), torch.randn(sq.rows, hid, generator=g).cuda()
        held = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        whole = [t.clone() for t in block_forward(qre, B, h, delta, *args, max_q=mq)]
        after = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        for t, x in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), held):
            t.copy_(x)

        n = qre.add_rms_norm(delta, B["n1"], 1e-5, residual=h, y_dtype=F32)
        t, y = ref.add_rms_norm(delta.cpu(), h.cpu(), B["n1"].cpu(), 1e-5)
        within(n.sum, t, 2.0 ** -23 * t.abs(), "sum")
        within(n.y, y, 2.0 ** -17 * y.abs(), "norm")
        qkv = qre.linear_q(B["qkv"], n.q, n.d, bias=B["bias"])
        w, A = ref.linear(B["qkv"].data[0].cpu(), B["qkv"].scale[0].cpu(), 4, 0, n.q.cpu(), n.d.cpu(), B["bias"].cpu(),
                          None, None)
        within(qkv, w, linear_bound(w, A, hid, F32), "qkv")
        q, k, v = qkv.view(-1, nh + 2 * nk, D).split([nh, nk, nk], dim=1)
        qre.kv_append(cache, *args, k, v, max_q=mq)
        for a, was, sc, new, now, now_sc in zip(at, held[:2], held[2:], (k, v), (cache.k, cache.v),
                                                (cache.k_scale, cache.v_scale)):
            want, want_sc = ref.append(was.cpu(), sc.cpu(), a, sq, new.cpu())
            fresh = ~torch.isnan(want_sc)
            assert torch.equal(now_sc.cpu()[fresh], want_sc[fresh]) and bool(torch.isnan(now_sc.cpu()[~fresh]).all())
            assert torch.equal(now.cpu(), want)
        a = qre.kv_attention(cache, *args, q, max_q=mq)
        codes = [cache.k.cpu(), cache.v.cpu()]
        scales = [cache.k_scale.cpu().nan_to_num(1.0), cache.v_scale.cpu().nan_to_num(1.0)]
        want, tol, _, _ = attention_bounds(codes, scales, sq, q.cpu().contiguous(), D ** -0.5, F32)
        assert bool((tol < 0.01 * want.abs().amax()).all())
        within(a, want, tol, "attention")
        oq, od = qre.quantize_q8_0(a.view(sq.rows, -1))
        s = qre.linear_q(B["o"], oq, od, residual=n.sum)
        w, A = ref.linear(B["o"].data[0].cpu(), B["o"].scale[0].cpu(), 8, 0, oq.cpu(), od.cpu(), None, None, n.sum.cpu())
        within(s, w, linear_bound(w, A, nh * D, F32), "output projection")
        m = qre.add_rms_norm(s, B["n2"], 1e-5, y_dtype=F32, q8=False)
        _, y = ref.add_rms_norm(s.cpu(), None, B["n2"].cpu(), 1e-5)
        within(m.y, y, 2.0 ** -17 * y.abs(), "second norm")
        assert torch.equal(s, whole[0]) and torch.equal(qre.moe_layer_forward(B["layer"], m.y), whole[1])
        for t, x in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), after):
            assert torch.equal(t.nan_to_num(0.0) if t.is_floating_point() else t,
                               x.nan_to_num(0.0) if x.is_floating_point() else x)
