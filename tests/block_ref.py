"""Plain 64-bit forms of the operators around the layer, for their tests, and
the bounds that the tests hold the kernels to.  Written from the definitions
in include/colibri_block.h; CPU tensors in, CPU float64 tensors out."""

import math

import torch

BLOCK = 64
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of a rounding, relative


def round_half_away(v):
    return torch.sign(v) * torch.floor(v.abs() + 0.5)


# ---- norm -----------------------------------------------------------------


def add_rms_norm(x, residual, weight, eps):
    t = x.double() + (residual.double() if residual is not None else 0.0)
    return t, t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * weight.double()


# ---- linear ---------------------------------------------------------------


def weight_codes(data, bits):
    """[rows][K * bits / 8] uint8 -> codes [rows][K] (first element in the most significant field)."""
    by = data.to(torch.int64)
    per = 8 // bits
    out = torch.empty(by.shape[0], by.shape[1] * per, dtype=torch.int64)
    for j in range(per):
        f = (by >> (8 - bits * (j + 1))) & ((1 << bits) - 1)
        out[:, j::per] = torch.where(f >= 1 << (bits - 1), f - (1 << bits), f)
    return out


def linear(data, scale, bits, group, xq, xd, bias, act, residual):
    """-> (out, A): A[t][r] = sum_k |w x| + |bias| bounds the rounding of the sums."""
    K = xq.shape[1]
    w = weight_codes(data, bits).double() * scale.double().view(data.shape[0], -1).repeat_interleave(group or K, 1)
    x = xq.double() * xd.double().repeat_interleave(32, 1)
    y, A = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        y, A = y + bias.double(), A + bias.double().abs()
    if act == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif act == "silu":
        y = y * torch.special.expit(y)
    elif act == "gelu":
        y = y * torch.special.ndtr(y)
    if residual is not None:
        y = y + residual.double()
    return y, A


def linear_tol(y, A, K, dtype):
    """fp32 sums of K products: blocks of 16 and more are summed by one
    instruction, so no value passes through more than K / 16 + 32 additions.
    The activations are off by 2^-22 (fp32) or 2^-12 (bf16) of their value, the
    scales' product by two roundings.  The activations' slopes stay under 1.2,
    their own error under 2^-19 of the value; one rounding of the result."""
    sums = (K / 16 + 40) * 2.0 ** -24 + (2.0 ** -22 if dtype == torch.float32 else 2.0 ** -12)
    return 1.2 * sums * A + 2.0 ** -19 * A.clamp(max=y.abs() + 1.0) + U[dtype] * y.abs() + 1e-30


# ---- cache ----------------------------------------------------------------


def page_bytes(D):
    """Byte of (token, dim) in a page of keys, and of values."""
    t, c = torch.arange(BLOCK)[:, None], torch.arange(D)[None]
    k = t // 32 * (32 * D) + c // 16 * 512 + t % 32 * 16 + c % 16
    v = t // 32 * (32 * D) + c * 32 + t // 4 % 2 * 16 + t % 32 // 8 * 4 + t % 4
    return k, v


def page_values(codes, scale, at):
    """[n_pages][H][64 D] codes -> values [n_pages][H][64][D]."""
    return codes[:, :, at].double() * scale.double()[..., None, None]


class Seqs:
    """Host copy of a batch: lists of (q_len, kv_len) and the page table."""

    def __init__(self, lens, table, rows=None):
        self.lens, self.table = lens, table
        cu = [0]
        for q, _ in lens:
            cu.append(cu[-1] + q)
        self.cu, self.rows = cu, cu[-1] if rows is None else rows


def tokens(values, table_row, n, n_pages):
    """Values [n][H][D] of a sequence's first n tokens, and which of them exist."""
    blocks = -(-n // BLOCK)
    page = table_row[:blocks].long()
    ok = (page >= 0) & (page < n_pages)
    x = values[page.clamp(0, n_pages - 1)].permute(0, 2, 1, 3).reshape(blocks * BLOCK, *values.shape[1:2],
                                                                      values.shape[3])[:n]
    ok = ok.repeat_interleave(BLOCK)[:n]
    return torch.where(ok[:, None, None], x, 0.0), ok


def append(codes, scale, at, seqs, new):
    """One of K and V: the codes and scales after the append (copies), in float32
    arithmetic step by step as the header gives it."""
    codes, scale, n_pages = codes.clone(), scale.clone(), codes.shape[0]
    for s, (q, n) in enumerate(seqs.lens):
        first = n - q
        lo = max(first, 0)
        for b in range(lo // BLOCK, -(-n // BLOCK)):
            p = int(seqs.table[s, b]) if b < seqs.table.shape[1] else -1
            if not 0 <= p < n_pages or n <= lo:
                continue
            t0, t1 = max(lo - b * BLOCK, 0), min(n - b * BLOCK, BLOCK)
            r0 = seqs.cu[s] + b * BLOCK + t0 - first
            x = new[r0:r0 + t1 - t0].float()  # [t][H][D]
            was = scale[p].clone() if t0 > 0 else torch.zeros_like(scale[p])
            now = torch.maximum(was, x.abs().amax((0, 2)) / 127.0)
            inv = torch.where(now == 0, 0.0, 1.0 / now)
            for h in range(codes.shape[1]):
                if t0 and now[h] != was[h]:
                    old = codes[p, h][at[:t0]].float()
                    codes[p, h][at[:t0]] = round_half_away(old * (was[h] * inv[h])).clamp(-127, 127).to(torch.int8)
                codes[p, h][at[t0:t1]] = round_half_away(x[:, h] * inv[h]).clamp(-127, 127).to(torch.int8)
            scale[p] = now
    return codes, scale


def attention(kval, vval, seqs, q, scale, causal=True, window=0):
    """-> out, lse, and per row the bounds (score bound, largest |v|): float64."""
    T, Hq, D = q.shape
    n_pages, H = kval.shape[:2]
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    sb, vb = torch.zeros(T, Hq, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    cap = seqs.table.shape[1] * BLOCK
    for s, (ql, n) in enumerate(seqs.lens):
        n = max(0, min(n, cap))
        if ql == 0 or n == 0:
            continue
        k, ok = tokens(kval, seqs.table[s], n, n_pages)
        v, _ = tokens(vval, seqs.table[s], n, n_pages)
        pos = torch.arange(n - ql, n)[:, None]
        key = torch.arange(n)[None]
        seen = ok[None].expand(ql, n).clone()
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        for h in range(Hq):
            x = q[seqs.cu[s]:seqs.cu[s] + ql, h].double()
            kk, vv = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
            z = torch.where(seen, scale * (x @ kk.t()), -math.inf)
            rows = slice(seqs.cu[s], seqs.cu[s] + ql)
            m = z.amax(1, keepdim=True).clamp(min=-1e300)
            p = torch.exp(z - m)
            l = p.sum(1, keepdim=True)
            out[rows, h] = torch.where(l > 0, p / l.clamp(min=1e-300), 0.0) @ vv
            lse[rows, h] = (m + torch.log(l)).squeeze(1)
            sb[rows, h] = (abs(scale) * x.abs().amax(1, keepdim=True) * kk.abs().sum(1)[None] * seen).amax(1)
            vb[rows, h] = (vv.abs().amax(1)[None] * seen).amax(1)
    return out, lse, sb, vb


def attention_tol(out, sb, vb, dtype):
    """The queries enter as fixed-point numbers of at least 22 bits (fp32) or 15
    bits (bf16) below the row's largest: a score is off by e <= 2^-22 or 2^-15 of
    qmax * sum|k| * scale, plus its fp32 roundings and the exponential's (under
    2^-20 of 1 + the score's bound).  A weight is then off by at most 2 e + that
    (both numerator and sum), and by the rounding of p for the product
    (bf16: 2^-8; fp32: three bf16 terms, 2^-23); sums in fp32 of positive weights."""
    q, p = (2.0 ** -22, 2.0 ** -23) if dtype == torch.float32 else (2.0 ** -15, 2.0 ** -8)
    e = 2 * (q * sb + 2.0 ** -20 * (1 + sb)) + p + 2.0 ** -19
    return (e * vb)[..., None] + U[dtype] * out.abs()


def lse_tol(sb, lse, dtype):
    """As attention_tol: the largest score's error, and the fp32 sums'."""
    q = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -15
    return q * sb + 2.0 ** -20 * (1 + sb) + 2.0 ** -19 + 2.0 ** -22 * lse.abs().clamp(max=1e30)
