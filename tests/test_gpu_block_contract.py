"""What the contract of the operators around the layer promises at its edges, on
the GPU."""

import pytest
import torch

from tests import block_ref as ref
from tests.test_gpu_block import BF16, F32, dev, make_cache, make_linear, qre, within  # noqa: F401

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
