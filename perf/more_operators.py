"""Cases of the operators of a serving step, for measuring.

A serving step goes from token ids to the next token ids.  Four operators, each
in its plain form (elementary torch operations) and, where `own` is true,
through the package's calls:

  embed    rows of a quantised embedding table, scaled
  linear   activations to 8 bits with one scale per token, times a quantised
           matrix with one scale per channel; bias, activation, residual
  logits   penalties for repeated tokens, biases and grammar masks on logits,
           the best token and the log of the sum
  pages    extending, trimming (freeing), forking and compacting the sequences
           of a paged cache, and the copies of pages that follow
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
        # the token of one decode step: latency
        {"name": "embed one token", "op": "embed", "n": 1, "rows": 131071, "k": 6144, "bits": 4, "group": 0,
         "dtype": "f32"},
        # a prompt's tokens from a table with group scales
        {"name": "embed prompt", "op": "embed", "n": 8191, "rows": 131071, "k": 6144, "bits": 8, "group": 128,
         "dtype": "bf16"},
        # query, key and value projection of one decoded token
        {"name": "linear one token", "op": "linear", "s": 1, "n": 10240, "k": 6144, "bits": 4, "act": "none",
         "bias": True, "residual": False, "dtype": "bf16"},
        # the vocabulary's projection of a decode batch: one large bank read once
        {"name": "linear vocabulary", "op": "linear", "s": 13, "n": 131071, "k": 6144, "bits": 8, "act": "none",
         "bias": False, "residual": False, "dtype": "f32"},
        # a short ragged prompt, two-bit weights, odd sizes
        {"name": "linear odd sizes", "op": "linear", "s": 333, "n": 4101, "k": 2080, "bits": 2, "act": "silu",
         "bias": True, "residual": True, "dtype": "f32"},
        # query, key and value projection of a long prompt
        {"name": "linear prompt", "op": "linear", "s": 4096, "n": 10240, "k": 6144, "bits": 8, "act": "none",
         "bias": True, "residual": False, "dtype": "bf16"},
        # one chat's next token: latency
        {"name": "logits one row", "op": "logits", "n_seq": 1, "drafts": 1, "v": 131071, "history": 701, "bias": 20,
         "masked": True, "write": False, "dtype": "f32"},
        # a verify step of a serving batch, all adjusted logits wanted
        {"name": "logits verify batch", "op": "logits", "n_seq": 32, "drafts": 4, "v": 151003, "history": 4001,
         "bias": 300, "masked": True, "write": True, "dtype": "bf16"},
        # a decode step of long contexts
        {"name": "logits long contexts", "op": "logits", "n_seq": 48, "drafts": 1, "v": 200001, "history": 131072,
         "bias": 0, "masked": False, "write": True, "dtype": "f32"},
        # a verify step's pages: four tokens more for each sequence, the rejected ones taken back: latency
        {"name": "pages verify step", "op": "pages", "kind": "verify", "n_seq": 64, "max_kv": 9000, "hkv": 8, "d": 128},
        # a step of a beam search: the losing half freed, the other forked, one token each, the shared last pages copied
        {"name": "pages beams", "op": "pages", "kind": "beams", "n_seq": 256, "max_kv": 4001, "hkv": 8, "d": 128},
        # half of the sequences end and the rest move together
        {"name": "pages compact", "op": "pages", "kind": "compact", "n_seq": 96, "max_kv": 9000, "hkv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("embed", "linear", "logits", "pages"))
    dtype = rng.choice(("f32", "bf16"))
    if op == "embed":
        group = rng.choice((0, 0, 32, 128))
        k = group * _log(rng, 1, 6144 // group) if group else 32 * _log(rng, 2, 192)
        return {"op": op, "n": _log(rng, 1, 8191), "rows": _log(rng, 100, 131071), "k": k, "bits": rng.choice((8, 4, 2)),
                "group": group, "dtype": dtype}
    if op == "linear":
        head = rng.random() < 0.2
        return {"op": op, "s": _log(rng, 1, 32 if head else 4096), "n": _log(rng, 16384 if head else 16, 131071 if head else 10240),
                "k": 32 * _log(rng, 4, 192), "bits": rng.choice((8, 4, 2)),
                "act": rng.choice(("none", "relu", "silu", "gelu")), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "dtype": dtype}
    if op == "logits":
        n_seq, drafts = _log(rng, 1, 48), rng.choice((1, 1, 1, 4, 5))
        n_seq = max(1, n_seq // drafts)
        return {"op": op, "n_seq": n_seq, "drafts": drafts, "v": _log(rng, 1000, 200001), "history": _log(rng, 1, 131072),
                "bias": rng.choice((0, 0, 20, 300)), "masked": rng.random() < 0.5, "write": rng.random() < 0.6,
                "dtype": dtype}
    kind = rng.choice(("verify", "beams", "compact"))
    n_seq = 2 * _log(rng, 1, 48)
    return {"op": op, "kind": kind, "n_seq": n_seq, "max_kv": _log(rng, 10, 600000 // n_seq), "hkv": rng.choice((1, 2, 4, 8)),
            "d": rng.choice((64, 128, 128, 192, 256)) if n_seq < 40 else rng.choice((64, 128))}


def _bytes_of(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    if case["op"] == "embed":
        n, k = case["n"], case["k"]
        scales = k // case["group"] if case["group"] else 1
        return {"bytes": n * (4 + k * case["bits"] // 8 + 4 * scales + k * _bytes_of(case["dtype"])), "flops": 2 * n * k}
    if case["op"] == "linear":
        s, n, k, b = case["s"], case["n"], case["k"], _bytes_of(case["dtype"])
        return {"bytes": n * k * case["bits"] // 8 + 4 * n * (1 + case["bias"]) + s * k * b + s * n * b * (1 + case["residual"]),
                "flops": 2 * s * n * k}
    if case["op"] == "logits":
        rows, v = case["n_seq"] * case["drafts"], case["v"]
        b = _bytes_of(case["dtype"])
        return {"bytes": rows * v * b * (1 + case["write"]) + 4 * sum(_histories(case)) + 8 * rows * case["bias"]
                + (rows + 1) // 2 * (v // 8) * case["masked"], "flops": 4 * rows * v}
    m = _model(case)
    page = 2 * case["hkv"] * (BLOCK * case["d"] + 4)  # keys and values of a page, with their scales
    return {"bytes": 2 * page * m["copies"] + 4 * m["ints"], "flops": m["ints"]}


# ---------------------------------------------------------------------------
# Inputs


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _codes_in(g, rows, k, bits):
    """A packed matrix of random codes."""
    if bits == 8:
        w = torch.randint(-127, 128, (1, rows, k), generator=g, device=DEV, dtype=torch.int8)
        return w.view(torch.uint8)
    return torch.randint(0, 256, (1, rows, k * bits // 8), generator=g, device=DEV, dtype=torch.uint8)


def _histories(case):
    """Tokens of each sequence so far: ragged, the first the longest."""
    r = random.Random(case["n_seq"] * 7919 + case["history"])
    return [case["history"]] + [r.randint(case["history"] // 4, case["history"]) for _ in range(case["n_seq"] - 1)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6007 + 29)
    s = {"case": case}
    {"embed": _prepare_embed, "linear": _prepare_linear, "logits": _prepare_logits, "pages": _prepare_pages}[case["op"]](
        case, s, g)
    return s


def _prepare_embed(case, s, g):
    rows, k, group = case["rows"], case["k"], case["group"]
    s["w"] = _codes_in(g, rows, k, case["bits"])
    s["w_scale"] = (0.01 * torch.randn(1, rows * (k // group if group else 1), generator=g, device=DEV)).abs()
    s["ids"] = torch.randint(0, rows, (case["n"],), generator=g, device=DEV, dtype=torch.int32)
    s["scale"] = math.sqrt(k)
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        s["bank"] = qre.QBank(s["w"], s["w_scale"], case["bits"], group)


def _prepare_linear(case, s, g):
    S, n, k, dt = case["s"], case["n"], case["k"], DTYPES[case["dtype"]]
    s["x"] = (torch.randn(S, k, generator=g, device=DEV) * (0.5 + torch.rand(S, 1, generator=g, device=DEV))).to(dt)
    s["w"] = _codes_in(g, n, k, case["bits"])
    s["w_scale"] = (0.02 * torch.randn(1, n, generator=g, device=DEV)).abs()
    s["bias"] = torch.randn(n, generator=g, device=DEV) if case["bias"] else None
    s["residual"] = torch.randn(S, n, generator=g, device=DEV).to(dt) if case["residual"] else None
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        s["bank"] = qre.QBank(s["w"], s["w_scale"], case["bits"])
        s["ws"] = qre.linear_i8_workspace(s["bank"], S, dt)


def _prepare_logits(case, s, g):
    n_seq, drafts, v = case["n_seq"], case["drafts"], case["v"]
    rows, hist = n_seq * drafts, _histories(case)
    s["logits"] = (2.5 * torch.randn(rows, v, generator=g, device=DEV)).to(DTYPES[case["dtype"]])
    # few tokens make up most of a text; the last ones are the sequence's draft
    total = sum(hist) + n_seq * (drafts - 1)
    u = torch.rand(total, generator=g, device=DEV, dtype=torch.float64)
    s["tokens"] = ((u ** 6 * v).long() * 7919 % v).to(torch.int32)
    spans, at = [], 0
    for h in hist:
        for i in range(drafts):
            spans.append((at, at + h // 2, at + h + i))  # first token, first generated one, end
        at += h + drafts - 1
    s["spans"] = _ints(spans)
    s["longest"] = max(hist) + drafts - 1
    # repetition, frequency, presence; the first row of eight takes none
    p = torch.stack([1 + 0.3 * torch.rand(rows, generator=g, device=DEV), torch.rand(rows, generator=g, device=DEV) - 0.2,
                     torch.rand(rows, generator=g, device=DEV) - 0.2], 1)
    p[1::8] = torch.tensor([1.0, 0.0, 0.0], device=DEV)
    s["penalties"] = p.contiguous()
    s["bias_ids"] = s["bias"] = s["cu_bias"] = s["mask"] = s["mask_of"] = None
    if case["bias"]:
        nb = min(case["bias"], v)
        s["bias_ids"] = torch.rand(rows, v, generator=g, device=DEV).topk(nb, -1).indices.to(torch.int32).view(-1)
        s["bias"] = 3 * torch.randn(rows * nb, generator=g, device=DEV)
        s["cu_bias"] = _ints([nb * i for i in range(rows + 1)])
    if case["masked"]:
        # every other row follows a grammar; one state of it allows nothing
        n_masks, words = (rows + 1) // 2, (v + 31) // 32
        m = torch.randint(-2 ** 31, 2 ** 31, (n_masks, words), generator=g, device=DEV, dtype=torch.int64)
        keep = torch.rand(n_masks, words, generator=g, device=DEV) < torch.rand(n_masks, 1, generator=g, device=DEV)
        s["mask"] = torch.where(keep, m, 0).to(torch.int32)
        if n_masks > 2:
            s["mask"][2] = 0
        s["mask_of"] = _ints([i // 2 if i % 2 == 0 else -1 for i in range(rows)])
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        s["ws"] = qre.logits_workspace(rows, v)
        s["out"] = torch.empty_like(s["logits"]) if case["write"] else None


def _model(case):
    """The sequences' lengths, what each step asks of them, and counts for `work`."""
    n, kind = case["n_seq"], case["kind"]
    r = random.Random(n * 1000003 + case["max_kv"])
    lens = [case["max_kv"]] + [r.randint(max(1, case["max_kv"] // 4), case["max_kv"]) for _ in range(n - 1)]
    blocks = [-(-x // BLOCK) for x in lens]
    m = {"lens": lens, "blocks": blocks, "add": [0] * n, "keep": [-1] * n, "parent": [], "child": [], "copies": 0}
    if kind == "verify":
        m["add"] = [4] * n
        m["back"] = [r.randint(0, 4) for _ in range(n)]
        m["ints"] = 8 * n
    else:
        gone = r.sample(range(n), n // 2)
        for i in gone:
            m["keep"][i] = 0
        left = [i for i in range(n) if m["keep"][i] < 0]
        m["ints"] = 2 * sum(blocks[i] for i in gone) + 4 * n
        if kind == "beams":
            m["child"] = sorted(gone)
            m["parent"] = [r.choice(left) for _ in m["child"]]
            m["add"] = [1] * n
            m["ints"] += 2 * sum(blocks[i] for i in m["parent"])
            m["copies"] = sum((m["parent"].count(i) + 1) for i in set(m["parent"]) if lens[i] % BLOCK)
        else:
            m["ints"] += 2 * sum(blocks[i] for i in left)
            # the expected number of moved pages, for pages handed out in any order
            live = sum(blocks[i] for i in left)
            m["copies"] = live * (_pool(m) - live) // _pool(m)
    return m


def _pool(m):
    return sum(m["blocks"]) + 2 * len(m["blocks"]) + len(m["blocks"]) // 2


def _prepare_pages(case, s, g):
    m = s["model"] = _model(case)
    n, hkv, d = case["n_seq"], case["hkv"], case["d"]
    pages, most = _pool(m), max(m["blocks"]) + 1
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    # one tensor holds the state, so that a pass begins by setting it back
    s["start"] = torch.full((n * most + n + pages,), -1, dtype=torch.int32, device=DEV)
    s["work"] = s["start"].clone()
    s["table"], s["kv_len"], s["refs"] = _state(s["work"], n, most, pages)
    table, kv_len, refs = _state(s["start"], n, most, pages)
    at = 0
    for i, b in enumerate(m["blocks"]):
        table[i, :b] = order[at:at + b]
        at += b
    kv_len.copy_(_ints(m["lens"]))
    refs.zero_()
    refs[order[:at].long()] = 1
    shape = (pages, hkv, BLOCK * d)
    s["k"], s["v"] = (torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8) for _ in range(2))
    s["k_scale"], s["v_scale"] = ((0.5 + torch.rand(pages, hkv, generator=g, device=DEV)) / 127 for _ in range(2))
    s["add"], s["keep"], s["parent"], s["child"] = (_ints(m[x]) for x in ("add", "keep", "parent", "child"))
    if case["kind"] == "verify":
        s["back_to"] = _ints([x + a - b for x, a, b in zip(m["lens"], m["add"], m["back"])])
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        s["cache"] = qre.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], d)
        s["pages"] = qre.KVPages(s["table"], s["kv_len"], s["refs"])
        s["ws"] = qre.kv_pages_workspace(s["pages"])


def _state(flat, n, most, pages):
    return flat[:n * most].view(n, most), flat[n * most:n * most + n], flat[n * most + n:]


# ---------------------------------------------------------------------------
# One pass


def run(state):
    case = state["case"]
    return {"embed": _embed, "linear": _linear, "logits": _logits, "pages": _pages}[case["op"]](state, case)


def _codes(w, n, k, bits):
    """The weight codes [n][k] of a packed matrix."""
    w = w.reshape(n, -1)
    if bits == 8:
        return w.view(torch.int8).float()
    per = 8 // bits
    shift = torch.arange(per - 1, -1, -1, device=w.device, dtype=torch.uint8) * bits
    f = ((w[..., None] >> shift) & (2 ** bits - 1)).float()
    return (f - (f >= 2 ** (bits - 1)) * float(2 ** bits)).view(n, k)


def _embed(s, case):
    n, k, group, dt = case["n"], case["k"], case["group"], DTYPES[case["dtype"]]
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        return qre.embed_q(s["bank"], s["ids"], s["scale"], dtype=dt)
    ids = s["ids"].long()
    w = _codes(s["w"][0][ids], n, k, case["bits"]).view(n, -1, group or k)
    scale = s["w_scale"].view(case["rows"], -1)[ids]
    return (w * scale[..., None] * s["scale"]).view(n, k).to(dt)


def _linear(s, case):
    n, k, dt = case["n"], case["k"], DTYPES[case["dtype"]]
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        xq, xd = qre.quantize_i8(s["x"])
        return qre.linear_i8(s["bank"], xq, xd, bias=s["bias"], activation=case["act"], residual=s["residual"],
                             dtype=dt, ws=s["ws"])
    x = s["x"].float()
    d = x.abs().amax(-1, keepdim=True) / 127
    v = x * torch.where(d > 0, 1 / d, 0.0)
    q = torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).clamp(-127, 127)
    y = torch.matmul(q, _codes(s["w"], n, k, case["bits"]).t()) * (d * s["w_scale"])
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


def _logits(s, case):
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        r = qre.adjust_logits(s["logits"], tokens=s["tokens"], spans=s["spans"], penalties=s["penalties"],
                              bias=s["bias"], bias_ids=s["bias_ids"], cu_bias=s["cu_bias"], mask=s["mask"],
                              mask_of=s["mask_of"], write=case["write"], out=s["out"], ws=s["ws"])
        return {"token": r.token, "lse": r.lse} | ({"logits": r.logits} if case["write"] else {})
    rows, v = s["logits"].shape
    first, made, end = s["spans"].long().unbind(1)
    at = first[:, None] + torch.arange(s["longest"], device=DEV)
    tok = s["tokens"].long()[at.clamp(max=s["tokens"].numel() - 1)]
    zero = torch.zeros(rows, v, dtype=torch.int32, device=DEV)
    seen = zero.scatter_add(1, tok, (at < end[:, None]).to(torch.int32))
    count = zero.scatter_add(1, tok, ((at < end[:, None]) & (at >= made[:, None])).to(torch.int32))
    rep, freq, pres = (x[:, None] for x in s["penalties"].unbind(1))
    x = s["logits"].float()
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - (freq * count + pres), x)
    if s["bias"] is not None:
        row = torch.repeat_interleave(torch.arange(rows, device=DEV), s["bias"].numel() // rows)
        x = x.index_put((row, s["bias_ids"].long()), s["bias"], accumulate=True)
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        ok = bits.view(s["mask"].shape[0], -1)[:, :v][s["mask_of"].clamp(min=0).long()] > 0
        x = x.masked_fill(~ok & (s["mask_of"] >= 0)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    here = torch.where(x == top, torch.arange(v, device=DEV, dtype=torch.int32), v)
    token = torch.where(top[:, 0] > -math.inf, here.amin(-1), -1)
    m = top.clamp(min=-1e30)
    lse = (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True)))[:, 0]
    return {"token": token.to(torch.int32), "lse": lse} | ({"logits": x.to(s["logits"].dtype)} if case["write"] else {})


def _entries(s):
    """Which entries of the page table hold a page."""
    return torch.arange(s["table"].shape[1], device=DEV) < ((s["kv_len"] + 63) // 64)[:, None]


def _count(s, held, by):
    """Adds `by` to the counts of the pages in the entries `held`."""
    s["refs"].scatter_add_(0, s["table"].clamp(min=0).long().view(-1), torch.where(held, by, 0).view(-1).to(torch.int32))


def _trim(s, to):
    cut = (to >= 0) & (to < s["kv_len"])
    gone = _entries(s) & cut[:, None] & (torch.arange(s["table"].shape[1], device=DEV) >= ((to + 63) // 64)[:, None])
    _count(s, gone, -1)
    s["table"].masked_fill_(gone, -1)
    s["kv_len"].copy_(torch.where(cut, to, s["kv_len"]))


def _fork(s, parent, child):
    p, c = parent.long(), child.long()
    s["table"][c] = torch.where(_entries(s)[p], s["table"][p], s["table"][c])
    s["kv_len"][c] = s["kv_len"][p]
    forked = torch.zeros_like(s["kv_len"], dtype=torch.bool)
    forked[c] = True
    _count(s, _entries(s) & forked[:, None], 1)


def _free_pages(s):
    """The free pages in ascending order in front, and their number."""
    free = s["refs"] == 0
    n = free.numel()
    place = torch.where(free, torch.cumsum(free, 0) - 1, n)
    out = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    out.scatter_(0, place, torch.arange(n, dtype=torch.int32, device=DEV))
    return out, free.sum()


def _extend(s, add):
    table, kv_len, refs = s["table"], s["kv_len"], s["refs"]
    n, most = table.shape
    seq = torch.arange(n, device=DEV)
    last = (kv_len // BLOCK).clamp(max=most - 1).long()
    old = table[seq, last]
    fits = (add > 0) & (kv_len + add <= most * BLOCK)
    shared = fits & (kv_len % BLOCK != 0) & (refs[old.clamp(min=0).long()] > 1)
    have, want = (kv_len + 63) // 64, (kv_len + add + 63) // 64
    need = torch.where(fits, want - have + shared.int(), 0)
    before = torch.cumsum(need, 0) - need
    pages, n_free = _free_pages(s)
    ok = fits & (before + need <= n_free)
    shared = shared & ok
    src = torch.where(shared, old, -1)
    dst = torch.where(shared, pages[before.clamp(max=pages.numel() - 1)], -1)
    refs.scatter_add_(0, old.clamp(min=0).long(), -shared.int())
    table[seq, last] = torch.where(shared, dst, old)
    b = torch.arange(most, device=DEV)
    new = ok[:, None] & (b >= have[:, None]) & (b < want[:, None])
    place = (before + shared)[:, None] + b - have[:, None]
    table.copy_(torch.where(new, pages[place.clamp(0, pages.numel() - 1)], table))
    _count(s, new, 1)
    refs.scatter_add_(0, dst.clamp(min=0).long(), shared.int())
    kv_len.add_(torch.where(ok, add, 0))
    return torch.where(ok, add, 0), src, dst


def _compact(s):
    refs, n = s["refs"], s["refs"].numel()
    live = refs > 0
    n_live = live.sum()
    page = torch.arange(n, dtype=torch.int32, device=DEV)
    moves, holes = live & (page >= n_live), ~live & (page < n_live)
    lists = []
    for which in (moves, holes):
        place = torch.where(which, torch.cumsum(which, 0) - 1, n)
        out = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
        out.scatter_(0, place, page)
        out[n] = -1
        lists.append(out[:n // 2])
    src, dst = lists
    to = torch.where(moves, dst[(torch.cumsum(moves, 0) - 1).clamp(0, n // 2 - 1)], page)
    s["table"].copy_(torch.where(_entries(s), to[s["table"].clamp(min=0).long()], s["table"]))
    kept = torch.zeros_like(refs)
    kept.scatter_add_(0, to.long(), refs)
    refs.copy_(kept)
    return src, dst, n_live.to(torch.int32).view(1)


def _copy(s, src, dst):
    page = torch.arange(s["refs"].numel(), device=DEV)
    take = page.clone()
    put = torch.where(dst >= 0, dst, page.numel()).long()
    take = torch.cat([take, take[:1]]).scatter_(0, put, src.long())[:-1]
    moved = take != page
    for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        x.copy_(torch.where(moved.view(-1, *[1] * (x.dim() - 1)), x[take], x))


def _pages(s, case):
    s["work"].copy_(s["start"])
    out = {"table": s["table"], "kv_len": s["kv_len"], "refs": s["refs"]}
    if own:
        import quantized_routed_expert_sigmoid_amd as qre
        p, ws = s["pages"], s["ws"]
        trim, fork = (lambda to: qre.kv_trim(p, to)), (lambda a, b: qre.kv_fork(p, a, b))
        extend, compact = (lambda add: qre.kv_extend(p, add, ws=ws)), (lambda: qre.kv_compact(p, ws=ws))
        copy = (lambda a, b: qre.kv_copy(s["cache"], a, b))
    else:
        trim, fork = (lambda to: _trim(s, to)), (lambda a, b: _fork(s, a, b))
        extend, compact = (lambda add: _extend(s, add)), (lambda: _compact(s))
        copy = (lambda a, b: _copy(s, a, b))
    if case["kind"] == "verify":
        granted, src, dst = extend(s["add"])
        trim(s["back_to"])
        return out | {"granted": granted, "src": src, "dst": dst}
    trim(s["keep"])
    if case["kind"] == "beams":
        fork(s["parent"], s["child"])
        granted, src, dst = extend(s["add"])
        out |= {"granted": granted}
    else:
        src, dst, n_live = compact()
        out |= {"n_live": n_live}
    copy(src, dst)
    return out | {"src": src, "dst": dst, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------------------
# The same from the definitions: numbers in 64 bits, pages by plain loops


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"embed": _embed64, "linear": _linear64, "logits": _logits64, "pages": _pages64}[case["op"]](s, case)


def _codes64(w, n, k, bits):
    by = w.reshape(n, -1).to(torch.int16)
    out = torch.empty(n, k, dtype=torch.float64, device=DEV)
    per = 8 // bits
    for j in range(per):
        f = (by >> (8 - bits * (j + 1))) % (1 << bits)
        out[:, j::per] = (f - (f >> (bits - 1)) * (1 << bits)).double()
    return out


def _embed64(s, case):
    n, k, ids = case["n"], case["k"], s["ids"].long()
    w = _codes64(s["w"][0, ids], n, k, case["bits"])
    per_row = s["w_scale"].double().view(case["rows"], -1)[ids]
    return w * per_row.repeat_interleave(case["group"] or k, dim=1) * s["scale"]


def _linear64(s, case):
    n, k = case["n"], case["k"]
    # the codes are defined by operations in 32 bits: d = amax / 127, v * (1 / d), half away from zero
    x = s["x"].float()
    d = torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True) / 127.0
    v = (x * d.reciprocal()).double()
    q = (torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp(-127, 127)
    out = []
    for lo in range(0, n, 16384):
        w = _codes64(s["w"][0, lo:lo + 16384], min(n, lo + 16384) - lo, k, case["bits"])
        out.append(q @ w.t().contiguous())
    y = torch.cat(out, 1) * d.double() * s["w_scale"].double()
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


def _logits64(s, case):
    rows, v = s["logits"].shape
    token, lse, out = [], [], []
    mask_of = s["mask_of"].tolist() if case["masked"] else [-1] * rows
    for r, (first, made, end) in enumerate(s["spans"].tolist()):
        rep, freq, pres = s["penalties"][r].double()
        x = s["logits"][r].double()
        seen = torch.bincount(s["tokens"][first:end].long(), minlength=v)
        count = torch.bincount(s["tokens"][made:end].long(), minlength=v)
        x = torch.where((seen > 0) & (x > 0), x / rep, torch.where(seen > 0, x * rep, x))
        x = x - (freq * count + pres * (count > 0))
        if case["bias"]:
            nb = s["bias"].numel() // rows
            x[s["bias_ids"][r * nb:(r + 1) * nb].long()] += s["bias"][r * nb:(r + 1) * nb].double()
        if mask_of[r] >= 0:
            word = s["mask"][mask_of[r]].long()[torch.arange(v, device=DEV) // 32]
            allowed = (word >> (torch.arange(v, device=DEV) % 32)) % 2 == 1
            x = torch.where(allowed, x, -math.inf)
        token.append(torch.where(x.max() > -math.inf, x.argmax(), -1))
        lse.append(torch.logsumexp(x, 0))
        out.append(x)
    r = {"token": torch.stack(token).to(torch.int32), "lse": torch.stack(lse)}
    return r | ({"logits": torch.stack(out)} if case["write"] else {})


def _pages64(s, case):
    m, kind = s["model"], case["kind"]
    n, most = s["table"].shape
    start = s["start"].tolist()
    table = [start[i * most:(i + 1) * most] for i in range(n)]
    kv, refs = start[n * most:n * most + n], start[n * most + n:]

    def shorten(i, to):
        for b in range(-(-to // BLOCK), -(-kv[i] // BLOCK)):
            refs[table[i][b]] -= 1
            table[i][b] = -1
        kv[i] = to

    for i, to in enumerate(m["keep"]):
        if 0 <= to < kv[i]:
            shorten(i, to)
    src = dst = granted = None
    for p, c in zip(m["parent"], m["child"]):
        for b in range(-(-kv[p] // BLOCK)):
            table[c][b] = table[p][b]
            refs[table[p][b]] += 1
        kv[c] = kv[p]
    if kind != "compact":
        free = [p for p, c in enumerate(refs) if c == 0]
        before = list(refs)
        src, dst, granted, at = [-1] * n, [-1] * n, [0] * n, 0
        for i, a in enumerate(m["add"]):
            if a <= 0 or kv[i] + a > most * BLOCK:
                continue
            b0, b1 = -(-kv[i] // BLOCK), -(-(kv[i] + a) // BLOCK)
            last = kv[i] // BLOCK
            copy = kv[i] % BLOCK != 0 and before[table[i][last]] > 1
            got, at = free[at:at + b1 - b0 + copy], at + b1 - b0 + copy
            if at > len(free):
                continue
            if copy:
                src[i], dst[i] = table[i][last], got.pop(0)
                refs[src[i]] -= 1
                refs[dst[i]] = 1
                table[i][last] = dst[i]
            for b in range(b0, b1):
                table[i][b] = got.pop(0)
                refs[table[i][b]] = 1
            kv[i] += a
            granted[i] = a
    out = {}
    if kind == "verify":
        for i in range(n):
            if m["back"][i]:
                shorten(i, m["lens"][i] + m["add"][i] - m["back"][i])
    if kind == "compact":
        live = sum(c > 0 for c in refs)
        src = [p for p in range(live, len(refs)) if refs[p] > 0]
        dst = [p for p in range(live) if refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            refs[a], refs[b] = 0, refs[a]
        for i in range(n):
            for b in range(-(-kv[i] // BLOCK)):
                table[i][b] = to.get(table[i][b], table[i][b])
        pad = [-1] * (len(refs) // 2 - len(src))
        src, dst = src + pad, dst + pad
        out["n_live"] = _ints([live])
    else:
        out["granted"] = _ints(granted)
    out |= {"table": _ints(table), "kv_len": _ints(kv), "refs": _ints(refs), "src": _ints(src), "dst": _ints(dst)}
    if kind != "verify":
        moved = [(a, b) for a, b in zip(src, dst) if a >= 0]
        for name in ("k", "v", "k_scale", "v_scale"):
            x = s[name].clone()
            if moved:
                a, b = (torch.tensor(t, device=DEV) for t in zip(*moved))
                x[b] = s[name][a]
            out[name] = x
    return out
