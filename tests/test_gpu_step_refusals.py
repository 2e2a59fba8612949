"""What the binding of the operators of a serving step refuses on GPU tensors, before anything is enqueued."""

import pytest
import torch

from tests.test_gpu_step import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qre():
    import quantized_routed_expert_sigmoid_amd as m
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m.lib()
    return m


def bank(qre, rows=7, K=64, bits=8, group=0):
    return qre.QBank(torch.zeros(1, rows, K * bits // 8, dtype=torch.uint8, device="cuda"),
                     torch.ones(1, rows * (K // group if group else 1), device="cuda"), bits, group)


def test_embed(qre):
    b, ids = bank(qre), ints([0, 1])
    for bad, error in [(dict(ids=ids.float()), TypeError), (dict(ids=ids.view(1, 2)), ValueError),
                       (dict(ids=ints([0, 1, 2, 3])[::2]), ValueError), (dict(dtype=torch.float16), TypeError),
                       (dict(out=torch.empty(2, 63, device="cuda")), ValueError),
                       (dict(out=torch.empty(2, 64, device="cuda"), dtype=torch.bfloat16), TypeError),
                       (dict(out=torch.empty(2, 64)), ValueError), (dict(scale=float("nan")), qre.ColibriError)]:
        kw = dict(ids=ids) | bad
        with pytest.raises(error):
            qre.embed_q(b, **kw)
    with pytest.raises(ValueError):
        qre.embed_q(qre.QBank(b.data, b.scale[:, :3].contiguous(), 8), ids)


def test_linear(qre):
    b, x = bank(qre), torch.ones(3, 64, device="cuda")
    q, d = qre.quantize_i8(x)
    for bad, error in [(dict(xq=q[:, :32]), ValueError), (dict(xq=q.float()), TypeError), (dict(xd=d[:2]), ValueError),
                       (dict(xd=d.view(3, 1)), ValueError), (dict(bias=torch.ones(6, device="cuda")), ValueError),
                       (dict(residual=torch.ones(3, 8, device="cuda")), ValueError), (dict(activation="tanh"), ValueError),
                       (dict(out=torch.empty(3, 7, device="cuda"), dtype=torch.bfloat16), TypeError),
                       (dict(xd=d.cpu()), ValueError),
                       (dict(ws=torch.empty(8, dtype=torch.uint8, device="cuda")), qre.ColibriError),
                       (dict(bank=bank(qre, group=32)), qre.ColibriError)]:
        kw = dict(bank=b, xq=q, xd=d) | bad
        with pytest.raises(error):
            qre.linear_i8(**kw)
    with pytest.raises(ValueError):
        qre.quantize_i8(x.t())
    with pytest.raises(TypeError):
        qre.quantize_i8(x.half())
    with pytest.raises(qre.ColibriError):
        qre.quantize_i8(torch.ones(2, 48, device="cuda"))
    with pytest.raises(qre.ColibriError):
        qre.quantize_i8(torch.ones(2, 65, device="cuda")[:, 1:])


def test_norm(qre):
    x, w = torch.ones(3, 64, device="cuda"), torch.ones(64, device="cuda")
    for a, kw, error in [((x.t(), w), {}, ValueError), ((x, w[:32]), {}, ValueError), ((x, w.cpu()), {}, ValueError),
                         ((x.half(), w), {}, TypeError), ((x, w), dict(residual=x[:2]), ValueError),
                         ((x, w), dict(eps=float("inf")), qre.ColibriError), ((x, w), dict(y_dtype=torch.float16), TypeError)]:
        with pytest.raises(error):
            qre.add_rms_norm_i8(*a, **kw)


def test_logits(qre):
    x = torch.zeros(2, 40, device="cuda")
    good = dict(tokens=ints([1]), spans=ints([[0, 0, 1]] * 2), penalties=torch.ones(2, 3, device="cuda"),
                bias=torch.ones(1, device="cuda"), bias_ids=ints([0]), cu_bias=ints([0, 1, 1]), mask=ints([[0, 0]]),
                mask_of=ints([0, -1]))
    qre.adjust_logits(x, **good)
    for name in good:
        with pytest.raises(ValueError):
            qre.adjust_logits(x, **{k: v for k, v in good.items() if k != name})
        with pytest.raises((TypeError, ValueError)):
            qre.adjust_logits(x, **good | {name: good[name].double()})
        with pytest.raises(ValueError):
            qre.adjust_logits(x, **good | {name: good[name].cpu()})
    for bad, error in [(dict(spans=ints([[0, 0, 1]])), ValueError), (dict(mask=ints([[0]])), ValueError),
                       (dict(cu_bias=ints([0, 1])), ValueError), (dict(out=x, write=False), ValueError),
                       (dict(out=x.bfloat16()), TypeError), (dict(out=x[:, :39]), ValueError),
                       (dict(out=torch.zeros(40, 2, device="cuda").t()), ValueError),
                       (dict(write=False, best=False), qre.ColibriError),
                       (dict(ws=torch.empty(8, dtype=torch.uint8, device="cuda")), qre.ColibriError)]:
        with pytest.raises(error):
            qre.adjust_logits(x, **good | bad)
    with pytest.raises(ValueError):
        qre.adjust_logits(x.t())
    with pytest.raises(qre.ColibriError):
        qre.adjust_logits(x[:1].expand(2, 40))
    with pytest.raises(TypeError):
        qre.adjust_logits(x.half())


def test_pages(qre):
    p = qre.KVPages.empty(3, 2, 5)
    for bad in (ints([1, 2]), torch.zeros(3, device="cuda"), torch.zeros(3, dtype=torch.int32), ints([0] * 6)[::2]):
        with pytest.raises((TypeError, ValueError)):
            qre.kv_extend(p, bad)
        with pytest.raises((TypeError, ValueError)):
            qre.kv_trim(p, bad)
    for a, b in ((ints([0]), ints([1, 2])), (ints([[0]]), ints([[1]])), (ints([0]), torch.ones(1, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            qre.kv_fork(p, a, b)
    small = torch.empty(4, dtype=torch.uint8, device="cuda")
    with pytest.raises(qre.ColibriError):
        qre.kv_extend(p, ints([0, 0, 0]), ws=small)
    with pytest.raises(qre.ColibriError):
        qre.kv_compact(p, ws=small)
    with pytest.raises(ValueError):
        qre.KVPages(p.page_table, p.kv_len[:2], p.refs)
    with pytest.raises(TypeError):
        qre.KVPages(p.page_table, p.kv_len, p.refs.long())
    a, b = qre.KVCache.empty(2, 1, 64), qre.KVCache.empty(2, 2, 64)
    with pytest.raises(qre.ColibriError):
        qre.kv_copy(a, ints([0]), ints([1]), to=b)
    with pytest.raises(ValueError):
        qre.kv_copy(a, ints([0]), ints([1, 0]))
    assert not bool(p.refs.any()) and not bool(p.kv_len.any())
