"""Cases of the operators around the mixture-of-experts layer, for measuring.

Four operators, each in its plain form (elementary torch operations in fp32)
and, where `own` is true, through the package's calls:

  norm       residual addition, root-mean-square norm, Q8_0 of the result
  linear     Q8_0 activations times a quantised matrix, with bias, activation
             and residual
  append     new keys and values into a paged int8 cache with one scale per
             block of 64 tokens and head
  attention  softmax attention of queries over that cache
"""

import math
import random

import torch

own = False

BLOCK = 64  # tokens of a cache page
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one decode step's token before the layer: latency
        {"name": "norm, one token", "op": "norm", "rows": 1, "k": 6144, "dtype": "f32"},
        # a prompt's tokens, bf16 activations, an odd number of rows
        {"name": "norm, prompt", "op": "norm", "rows": 8191, "k": 6144, "dtype": "bf16"},
        # query, key and value projection of one decoded token
        {"name": "linear, one token", "op": "linear", "s": 1, "n": 10240, "k": 6144, "bits": 4, "group": 0,
         "act": "none", "bias": True, "residual": False, "dtype": "bf16"},
        # output projection of a verify step, added to the residual stream
        {"name": "linear, verify step", "op": "linear", "s": 4, "n": 6144, "k": 8192, "bits": 8, "group": 128,
         "act": "none", "bias": False, "residual": True, "dtype": "f32"},
        # a short ragged prompt, two-bit weights, odd sizes
        {"name": "linear, odd sizes", "op": "linear", "s": 333, "n": 4101, "k": 2080, "bits": 2, "group": 0,
         "act": "silu", "bias": True, "residual": True, "dtype": "f32"},
        # query, key and value projection of a long prompt
        {"name": "linear, prompt", "op": "linear", "s": 4096, "n": 10240, "k": 6144, "bits": 4, "group": 0,
         "act": "none", "bias": True, "residual": False, "dtype": "bf16"},
        # the new token of every sequence of a serving batch
        {"name": "append, decode batch", "op": "append", "n_seq": 64, "max_q": 1, "max_kv": 700, "hkv": 8,
         "d": 128, "dtype": "f32"},
        # ragged prompts written into their pages
        {"name": "append, prompts", "op": "append", "n_seq": 5, "max_q": 3001, "max_kv": 4001, "hkv": 8,
         "d": 128, "dtype": "bf16"},
        # one token of a short chat: latency
        {"name": "attention, one short", "op": "attention", "n_seq": 1, "max_q": 1, "max_kv": 501, "hq": 64,
         "hkv": 8, "d": 128, "window": 0, "dtype": "f32"},
        # one token of one long sequence
        {"name": "attention, one long", "op": "attention", "n_seq": 1, "max_q": 1, "max_kv": 131071, "hq": 64,
         "hkv": 8, "d": 128, "window": 0, "dtype": "f32"},
        # a verify step of a ragged serving batch
        {"name": "attention, verify batch", "op": "attention", "n_seq": 32, "max_q": 4, "max_kv": 9000, "hq": 64,
         "hkv": 8, "d": 128, "window": 0, "dtype": "bf16"},
        # ragged prompts behind cached prefixes
        {"name": "attention, prompts", "op": "attention", "n_seq": 4, "max_q": 2047, "max_kv": 4095, "hq": 64,
         "hkv": 8, "d": 128, "window": 0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "append", "attention"))
    dtype = rng.choice(("f32", "bf16"))
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8191), "k": 32 * _log(rng, 1, 192), "dtype": dtype}
    if op == "linear":
        bits = rng.choice((8, 4, 2))
        group = rng.choice((0, 0, 32, 128))
        k = group * _log(rng, 1, 6144 // group) if group else 32 * _log(rng, 4, 192)
        return {"op": op, "s": _log(rng, 1, 4096), "n": _log(rng, 16, 10240), "k": k, "bits": bits, "group": group,
                "act": rng.choice(("none", "relu", "silu", "gelu")), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "dtype": dtype}
    d = rng.choice((64, 128, 128, 192, 256))
    hkv = rng.choice((1, 2, 4, 8))
    n_seq = _log(rng, 1, 64)
    if op == "append":
        max_q = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 4096 // n_seq))
        return {"op": op, "n_seq": n_seq, "max_q": max_q, "max_kv": max_q + _log(rng, 1, 2048), "hkv": hkv, "d": d,
                "dtype": dtype}
    hq = hkv * rng.choice((1, 3, 4, 8))
    kind = rng.random()
    if kind < 0.6:  # decode and verify steps
        max_q = rng.choice((1, 1, 2, 5, 8))
        max_kv = max_q + _log(rng, 1, max(2, 131072 // n_seq))
    else:  # prompts
        n_seq = _log(rng, 1, 6)
        max_q = _log(rng, 9, 2048 // n_seq)
        max_kv = max_q + _log(rng, 1, 2048)
    return {"op": op, "n_seq": n_seq, "max_q": max_q, "max_kv": max_kv, "hq": hq, "hkv": hkv, "d": d,
            "window": 0 if rng.random() < 0.7 else _log(rng, 1, max_kv), "dtype": dtype}


def _lens(case):
    """(new tokens, cached tokens with them) of each sequence: ragged, the first the largest."""
    r = random.Random(case["n_seq"] * 1000003 + case["max_q"] * 1009 + case["max_kv"])
    out = [(case["max_q"], case["max_kv"])]
    for _ in range(case["n_seq"] - 1):
        q = case["max_q"] if case["max_q"] <= 8 else r.randint(1, case["max_q"])
        out.append((q, r.randint(max(q, case["max_kv"] // 4), case["max_kv"])))
    return out


def _bytes_of(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    b = _bytes_of(case["dtype"])
    if case["op"] == "norm":
        n = case["rows"] * case["k"]
        # x and the residual in; the sum, the norm and its codes out
        return {"bytes": n * (4 * b + 1) + n // 32 * 4 + case["k"] * 4, "flops": 8 * n}
    if case["op"] == "linear":
        s, n, k = case["s"], case["n"], case["k"]
        scales = n * (k // case["group"] if case["group"] else 1)
        return {"bytes": n * k * case["bits"] // 8 + 4 * scales + s * k + s * k // 8 + s * n * b * (1 + case["residual"])
                + 4 * n * case["bias"], "flops": 2 * s * n * k}
    lens, hkv, d = _lens(case), case["hkv"], case["d"]
    if case["op"] == "append":
        new = sum(q for q, _ in lens)
        touched = sum(_span(q, n) for q, n in lens)
        # the new values in, the codes of the touched blocks out, their values read back
        return {"bytes": 2 * hkv * d * (new * b + touched * (1 + 1 + 2)), "flops": 4 * new * hkv * d}
    hq, w = case["hq"], case["window"]
    pairs = kv = q_rows = 0
    for q, n in lens:
        first = n - q + 1  # keys of the first new token
        q_rows += q
        if w:
            pairs += sum(min(w, first + i) for i in range(q))
            kv += min(n, w + q - 1)
        else:
            pairs += q * first + q * (q - 1) // 2
            kv += n
    return {"bytes": 2 * kv * hkv * d + 2 * q_rows * hq * d * b, "flops": 4 * pairs * hq * d}


def _span(q, n):
    """Tokens from the start of the first page that q new tokens of n touch."""
    return q + (n - q) % BLOCK


# ---------------------------------------------------------------------------
# Inputs


def _cache(case, g, lens):
    """Random cache pages in a shuffled order, and the page table (a page more than is needed in the pool)."""
    hkv, d = case["hkv"], case["d"]
    per = [-(-n // BLOCK) for _, n in lens]
    pages, most = sum(per) + 1, max(per)
    order = torch.randperm(pages, generator=g, device=DEV)[: sum(per)].to(torch.int32)
    table = torch.zeros(len(lens), most, dtype=torch.int32, device=DEV)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    codes = [torch.randint(-127, 128, (pages, hkv, BLOCK * d), generator=g, device=DEV, dtype=torch.int8)
             for _ in range(2)]
    scales = [(0.5 + torch.rand(pages, hkv, generator=g, device=DEV)) * 2.5 / 127 for _ in range(2)]
    return codes, scales, table


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": case}
    if case["op"] == "norm":
        s |= {"x": normal(case["rows"], case["k"]).to(dt), "residual": (2 * normal(case["rows"], case["k"])).to(dt),
              "weight": 1 + 0.2 * normal(case["k"]), "eps": 1e-5}
        s["values"] = torch.empty(case["rows"], case["k"] // 32, 32, dtype=torch.bfloat16, device=DEV)
        return s
    if case["op"] == "linear":
        S, n, k, bits, group = (case[x] for x in ("s", "n", "k", "bits", "group"))
        x = normal(S, k // 32, 32)
        d = x.abs().amax(-1) / 127
        s["xq"] = (x / d[..., None]).round().to(torch.int8).view(S, k)
        s["xd"] = d.contiguous()
        if bits == 8:
            w = torch.randint(-127, 128, (1, n, k), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)
            s["w"] = w.view(torch.uint8)
        else:
            s["w"] = torch.randint(0, 256, (1, n, k * bits // 8), generator=g, device=DEV, dtype=torch.uint8)
        s["w_scale"] = (0.02 * normal(1, n * (k // group if group else 1))).abs()
        s["bias"] = normal(n) if case["bias"] else None
        s["residual"] = normal(S, n).to(dt) if case["residual"] else None
        if own:
            import quantized_routed_expert_sigmoid_amd as qre
            s["bank"] = qre.QBank(s["w"], s["w_scale"], bits, group)
        return s
    lens = _lens(case)
    hkv, d = case["hkv"], case["d"]
    (s["k"], s["v"]), (s["k_scale"], s["v_scale"]), s["table"] = _cache(case, g, lens)
    new = [q for q, _ in lens]
    s["cu_q"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    s["kv_len"] = _ints([n for _, n in lens])
    total = sum(new)
    if case["op"] == "append":
        s["new_k"] = normal(total, hkv, d).to(dt)
        s["new_v"] = normal(total, hkv, d).to(dt)
        spans = [_span(q, n) for q, n in lens]
        s["cu_span"] = _ints([sum(spans[:i]) for i in range(len(spans) + 1)])
        s["spans"] = sum(spans)
        s["max_span"] = max(spans)
        # where each touched token lies: its page, its place there, and its row among the new ones or -1
        page, place, row, at = [], [], [], 0
        for i, (q, n) in enumerate(lens):
            first = (n - q) // BLOCK * BLOCK
            t = torch.arange(first, n, device=DEV)
            page.append(s["table"][i].long()[t // BLOCK])
            place.append(t % BLOCK)
            row.append(torch.where(t >= n - q, t - (n - q) + at, -1))
            at += q
        s["page"], s["place"], s["row"] = torch.cat(page), torch.cat(place), torch.cat(row)
    else:
        s["q"] = (normal(total, case["hq"], d) * 0.5).to(dt)
        # where the queries of the padded batch come from
        i = torch.arange(case["max_q"], device=DEV)
        lq = s["cu_q"].diff().long()
        s["pad"] = (s["cu_q"][:-1].long()[:, None] + i).clamp(max=total - 1)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lq)
        s["unpad"] = seq * case["max_q"] + torch.arange(total, device=DEV) - s["cu_q"].long()[seq]
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        s["cache"] = qre.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], d)
        if case["op"] == "attention":
            s["ws"] = qre.kv_attention_workspace(s["cache"], len(lens), total, case["hq"], case["max_q"],
                                                 case["max_kv"], s["q"].dtype)
    return s


# ---------------------------------------------------------------------------
# One pass


def run(state):
    case = state["case"]
    return {"norm": _norm, "linear": _linear, "append": _append, "attention": _attention}[case["op"]](state, case)


def _norm(s, case):
    rows, k = s["x"].shape
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        r = qre.add_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"], y_dtype=s["x"].dtype)
        torch.mul(r.q.view(rows, k // 32, 32), r.d.unsqueeze(-1), out=s["values"])
        return {"sum": r.sum, "y": r.y, "values": s["values"]}
    t = s["x"].float() + s["residual"].float()
    y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    b = y.view(rows, k // 32, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    v = b * torch.where(d > 0, 1 / d, 0.0)
    q = torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).clamp(-127, 127)
    return {"sum": t.to(s["x"].dtype), "y": y.to(s["x"].dtype), "values": (q * d).to(torch.bfloat16)}


def _codes(w, n, k, bits):
    """The weight codes [n][k] of a packed matrix."""
    w = w.view(n, -1)
    if bits == 8:
        return w.view(torch.int8).float()
    per = 8 // bits
    shift = torch.arange(per - 1, -1, -1, device=w.device, dtype=torch.uint8) * bits
    f = ((w[..., None] >> shift) & (2 ** bits - 1)).float()
    return (f - (f >= 2 ** (bits - 1)) * float(2 ** bits)).view(n, k)


def _linear(s, case):
    n, k, group = case["n"], case["k"], case["group"]
    dt = DTYPES[case["dtype"]]
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        return qre.linear_q(s["bank"], s["xq"], s["xd"], bias=s["bias"], activation=case["act"],
                            residual=s["residual"], dtype=dt)
    x = (s["xq"].view(-1, k // 32, 32) * s["xd"][..., None]).view(-1, k)
    w = _codes(s["w"], n, k, case["bits"])
    w = (w.view(n, -1, group or k) * s["w_scale"].view(n, -1, 1)).view(n, k)
    y = torch.matmul(x, w.t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] == "relu":
        y = torch.clamp(y, min=0)
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt)


def _k_of(pages, d):
    """Codes of K pages [...][64 * d] as [...][64][d]: halves of 32 tokens, 16 dims of each token together."""
    lead = pages.shape[:-1]
    return pages.view(*lead, 2, d // 16, 32, 16).transpose(-3, -2).reshape(*lead, BLOCK, d)


def _k_to(values, d):
    lead = values.shape[:-2]
    return values.reshape(*lead, 2, 32, d // 16, 16).transpose(-3, -2).reshape(*lead, BLOCK * d)


def _v_of(pages, d):
    """Codes of V pages [...][64 * d] as [...][64][d]: halves of 32 tokens; of each dim the tokens whose number has
    bit 2 clear, then the others."""
    lead = pages.shape[:-1]
    x = pages.view(*lead, 2, d, 2, 4, 4)  # half, dim, bit 2, bits 3 and 4, bits 0 and 1
    n = len(lead)
    return x.permute(*range(n), n, n + 3, n + 2, n + 4, n + 1).reshape(*lead, BLOCK, d)


def _v_to(values, d):
    lead = values.shape[:-2]
    x = values.reshape(*lead, 2, 4, 2, 4, d)  # half, bits 3 and 4, bit 2, bits 0 and 1, dim
    n = len(lead)
    return x.permute(*range(n), n, n + 4, n + 2, n + 1, n + 3).reshape(*lead, BLOCK * d)


def _append_plain(s, codes, scale, new, of, to):
    """New values into the pages they belong to; returns the touched tokens' values."""
    d = new.shape[-1]
    page, place, row = s["page"], s["place"], s["row"]
    fresh = (row >= 0)[:, None, None]
    x = torch.where(fresh, new.float()[row.clamp(min=0)], 0.0)
    # a block's scale: of what it held before, where a kept token is among the touched, and of the new tokens
    old = torch.zeros_like(scale)
    old[page[row < 0]] = scale[page[row < 0]]
    d_new = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax") / 127
    now = torch.maximum(old, d_new)
    held = of(codes[page], d)[torch.arange(page.numel(), device=page.device), :, place].float()
    inv = torch.where(now > 0, 1 / now, 0.0)[page][..., None]
    v = torch.where(fresh, x * inv, held * (old[page][..., None] * inv))
    q = torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).clamp(-127, 127)
    whole = of(codes, d)
    whole[page, :, place] = q.to(torch.int8)
    codes.copy_(to(whole, d))
    scale[page] = now[page]
    return (q * now[page][..., None]).to(torch.bfloat16)


def _append(s, case):
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        qre.kv_append(s["cache"], s["table"], s["cu_q"], s["kv_len"], s["new_k"], s["new_v"], max_q=case["max_q"])
        return qre.kv_read(s["cache"], s["table"], s["cu_span"], s["kv_len"], s["spans"], dtype=torch.bfloat16,
                           max_q=s["max_span"])
    return (_append_plain(s, s["k"], s["k_scale"], s["new_k"], _k_of, _k_to),
            _append_plain(s, s["v"], s["v_scale"], s["new_v"], _v_of, _v_to))


def _attention(s, case):
    hq, hkv, d, window = (case[x] for x in ("hq", "hkv", "d", "window"))
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        return qre.kv_attention(s["cache"], s["table"], s["cu_q"], s["kv_len"], s["q"], causal=True, window=window,
                                max_q=case["max_q"], max_kv=case["max_kv"], ws=s["ws"])
    n, most = s["table"].shape
    table, g, mq = s["table"].long(), hq // hkv, case["max_q"]

    def tokens(codes, scale, of):  # [n][hkv][most * 64][d]
        x = of(codes[table], d) * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(n, hkv, most * BLOCK, d)

    q = s["q"][s["pad"]].float().view(n, mq, hkv, g, d).transpose(1, 2).reshape(n, hkv, mq * g, d)
    p = torch.matmul(q, tokens(s["k"], s["k_scale"], _k_of).transpose(-1, -2).contiguous()) * d ** -0.5
    kv, lq = s["kv_len"].long(), s["cu_q"].diff().long()
    key = torch.arange(most * BLOCK, device=DEV)
    at = (kv - lq)[:, None] + torch.arange(mq, device=DEV)  # [n][mq]: each query's own place
    seen = (key <= at[..., None]) & (key < kv[:, None, None])
    if window:
        seen = seen & (key > at[..., None] - window)
    p = p.view(n, hkv, mq, g, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(n, hkv, mq * g, -1)
    o = torch.matmul(p, tokens(s["v"], s["v_scale"], _v_of)).view(n, hkv, mq, g, d).transpose(1, 2)
    return o.reshape(n * mq, hq, d)[s["unpad"]].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm": _norm64, "linear": _linear64, "append": _append64, "attention": _attention64}[case["op"]](s, case)


def _norm64(s, case):
    t = s["x"].double() + s["residual"].double()
    ms = torch.linalg.vector_norm(t, dim=-1, keepdim=True) ** 2 / case["k"]
    y = t / torch.sqrt(ms + s["eps"]) * s["weight"].double()
    d = (y.abs().unflatten(-1, (-1, 32)).max(-1, keepdim=True).values.float() / 127).double()
    v = y.unflatten(-1, (-1, 32)) / torch.where(d == 0, 1.0, d)
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)
    return {"sum": t, "y": y, "values": q.clamp(-127, 127) * d}


def _linear64(s, case):
    n, k, bits, group = (case[x] for x in ("n", "k", "bits", "group"))
    by = s["w"].view(n, -1).to(torch.int64)
    w = torch.empty(n, k, dtype=torch.float64, device=DEV)
    per = 8 // bits
    for j in range(per):
        f = (by >> (8 - bits * (j + 1))) % (1 << bits)
        w[:, j::per] = (f - (f >> (bits - 1)) * (1 << bits)).double()
    w *= s["w_scale"].double().view(n, -1).repeat_interleave(group or k, dim=1)
    x = s["xq"].double() * s["xd"].double().repeat_interleave(32, dim=1)
    y = x @ w.t().contiguous()
    if case["bias"]:
        y += s["bias"].double()
    if case["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif case["act"] == "silu":
        y = y * torch.special.expit(y)
    elif case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    if case["residual"]:
        y += s["residual"].double()
    return y


def _k_index(d):
    """Byte of (token, dim) in a K page, and in a V page."""
    t, c = torch.arange(BLOCK, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    k = t // 32 * (32 * d) + c // 16 * 512 + t % 32 * 16 + c % 16
    v = t // 32 * (32 * d) + c * 32 + t // 4 % 2 * 16 + t % 32 // 8 * 4 + t % 4
    return k, v


def _tokens64(s, i, n, d):
    """K and V of the first n tokens of sequence i: [n][hkv][d]."""
    pages = s["table"][i, : -(-n // BLOCK)].long()
    out = []
    for codes, scale, at in zip((s["k"], s["v"]), (s["k_scale"], s["v_scale"]), _k_index(d)):
        x = codes[pages][:, :, at].double() * scale[pages].double()[..., None, None]
        out.append(x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], d)[:n])
    return out


def _append64(s, case):
    d, outs = case["d"], ([], [])
    at = 0
    for i, (q, n) in enumerate(_lens(case)):
        first = (n - q) // BLOCK * BLOCK
        held = _tokens64(s, i, n - q, d)
        pages = s["table"][i].long()
        for held_x, new, scale, out in zip(held, (s["new_k"], s["new_v"]), (s["k_scale"], s["v_scale"]), outs):
            for b in range(first, n, BLOCK):
                keep, upto = held_x[b:b + BLOCK], min(n, b + BLOCK)
                x = new[at + max(b - (n - q), 0): at + upto - (n - q)].double()
                now = (x.abs().amax((0, 2)).float() / 127).double()
                if keep.shape[0]:
                    now = torch.maximum(now, scale[pages[b // BLOCK]].double())
                v = torch.cat([keep, x]) / now[:, None]
                out.append((torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp(-127, 127) * now[:, None])
        at += q
    return tuple(torch.cat(o) for o in outs)


def _attention64(s, case):
    if work(case)["flops"] > 2e13:
        return None
    hq, hkv, d, window = (case[x] for x in ("hq", "hkv", "d", "window"))
    g, at, out = hq // hkv, 0, []
    for i, (q, n) in enumerate(_lens(case)):
        k, v = _tokens64(s, i, n, d)
        x = s["q"][at:at + q].double()
        o = torch.zeros(q, hq, d, dtype=torch.float64, device=DEV)
        pos, key = torch.arange(n - q, n, device=DEV)[:, None], torch.arange(n, device=DEV)
        hidden = key > pos
        if window:
            hidden |= key <= pos - window
        for h in range(hq):
            z = x[:, h].contiguous() @ k[:, h // g].t().contiguous() / math.sqrt(d)
            z = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
            o[:, h] = z @ v[:, h // g].contiguous()
        out.append(o)
        at += q
    return torch.cat(out)
