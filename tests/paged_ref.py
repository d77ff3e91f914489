"""Plain implementations of the paged 8-bit cache's operators in 64 bits, and builders of test problems.

Everything here is elementary torch on small tensors; it shares no code with the library."""
import math

import torch

E4M3_TINY = 2.0 ** -9   # the smallest e4m3 step
SLACK = 1.0 + 2.0 ** -20


def e8m0(exponents):
    """Scale tensor 2^e of integer exponents."""
    return (torch.as_tensor(exponents) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def scale_values(scale):
    """float64 values of an e8m0 tensor."""
    e = scale.view(torch.uint8).double()
    return torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))


def code_values(codes):
    return codes.float().double()


def needed_scale(amax):
    """The smallest power of two, 2^-63 at least, with amax <= 448 * scale (amax a Python float)."""
    e = -63
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def cos_sin_table(positions, rot, device="cpu", base=10000.0):
    half = rot // 2
    freq = torch.pow(base, -torch.arange(half, dtype=torch.float64) / max(half, 1))
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def rotate(x, cos_sin, rot, interleaved):
    """x [tokens, heads, d] in any precision, cos_sin [tokens, rot] of the tokens' positions: one operation at a time."""
    if rot == 0:
        return x.clone()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    cos, sin = cos_sin[:, None, :rot // 2].to(x.dtype), cos_sin[:, None, rot // 2:].to(x.dtype)
    y = x.clone()
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


class Cache:
    """A cache of random content with its block table, on the CPU; `to_device` moves it."""

    def __init__(self, lens, heads, page, d_qk, d_v, seed=0, spare=3, width=None, layout="heads", tail=0x7F):
        g = torch.Generator().manual_seed(seed)
        counts = [-(-n // page) for n in lens]
        self.width = max(counts + [1]) if width is None else width
        self.num_pages = sum(counts) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        held = [0] * self.num_pages
        for b, n in enumerate(lens):
            for j in range(counts[b]):
                table[b, j] = order.pop()
                held[table[b, j]] = min(page, n - j * page)
        self.lens, self.heads, self.page, self.d_qk, self.d_v, self.layout = list(lens), heads, page, d_qk, d_v, layout
        self.table = table
        self.seqlens = torch.tensor(lens, dtype=torch.int32)
        for name, d in (("k", d_qk), ("v", d_v)):
            x = torch.randn(self.num_pages, heads, page, d, generator=g).clamp(-4, 4) * 60
            codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
            for p in range(self.num_pages):
                codes[p, :, held[p]:] = tail  # behind the last token: codes that are no number
            exps = torch.randint(-8, -4, (self.num_pages, heads), generator=g)
            setattr(self, name, codes.view(torch.float8_e4m3fn))
            setattr(self, name + "_scale", e8m0(exps))

    def to_device(self, device):
        """(k_cache, v_cache, k_scale, v_scale, block_table, seqlens): codes stored as `layout` says."""
        out = []
        for t in (self.k, self.v):
            u = t.view(torch.uint8).to(device)
            if self.layout == "tokens":      # [pages, page, heads, d] in memory
                u = u.transpose(1, 2).contiguous().transpose(1, 2)
            elif self.layout == "apart":     # pages inside a larger allocation
                big = torch.zeros(u.shape[0], 2, *u.shape[1:], dtype=torch.uint8, device=device)
                big[:, 1] = u
                u = big[:, 1]
            out.append(u.view(torch.float8_e4m3fn))
        return (*out, self.k_scale.to(device), self.v_scale.to(device), self.table.to(device), self.seqlens.to(device))


def dense(codes, scale, table_row, length, page):
    """[heads, length, d] float64 values of one sequence."""
    heads, d = codes.shape[1], codes.shape[3]
    if length == 0:
        return torch.zeros(heads, 0, d, dtype=torch.float64)
    pages = table_row[:-(-length // page)].long()
    u = codes.view(torch.uint8).cpu()[pages].view(torch.float8_e4m3fn)
    x = code_values(u) * scale_values(scale.cpu())[pages][..., None, None]
    return x.transpose(0, 1).reshape(heads, -1, d)[:, :length]


def attention(q, codes_k, codes_v, scale_k, scale_v, table, lens, cu, page, causal, scale=None):
    """O, LSE in 64 bits and the bounds a computed pair has to keep, all on the CPU.

    q [total, heads_q, d] (any device).  The bounds follow the arithmetic: scores are fp32 sums of d exact products (delta
    each: d + 8 roundings of 2^-24 of sum |q||k|), which moves a weight by 2 delta relatively; a weight is rounded once more
    to `eps_p` (f16: 2^-11, bf16: 2^-8) and its exponential is off by 2^-21; sums over n tokens add n 2^-24; weights below
    2^-31 of the largest may vanish (n 2^-31); O is rounded to bf16 (2^-8)."""
    q = q.double().cpu()
    total, heads_q, d = q.shape
    heads = codes_k.shape[1]
    ratio = heads_q // heads
    dv = codes_v.shape[3]
    s = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.zeros(total, heads_q, dv, dtype=torch.float64)
    lse = torch.full((heads_q, total), -math.inf, dtype=torch.float64)
    weight = torch.zeros(total, heads_q, dv, dtype=torch.float64)  # sum p |v|
    delta = torch.zeros(total, heads_q, dtype=torch.float64)
    count = torch.zeros(total, dtype=torch.float64)
    table = table.cpu()
    for b, length in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        n = hi - lo
        if n == 0 or length == 0:
            continue
        k, v = dense(codes_k, scale_k, table[b], length, page), dense(codes_v, scale_v, table[b], length, page)
        seen = torch.ones(n, length, dtype=torch.bool)
        if causal:
            seen = torch.arange(length)[None] <= torch.arange(n)[:, None] + length - n
        count[lo:hi] = length
        for h in range(heads):
            for r in range(h * ratio, (h + 1) * ratio):
                sc = (q[lo:hi, r] @ k[h].t()) * s
                sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
                l = torch.logsumexp(sc, 1)
                p = torch.where(torch.isinf(l)[:, None], torch.zeros_like(sc), torch.exp(sc - l[:, None]))
                o[lo:hi, r] = p @ v[h]
                weight[lo:hi, r] = p @ v[h].abs()
                lse[r, lo:hi] = l
                size = (q[lo:hi, r].abs() @ k[h].abs().t()) * s
                delta[lo:hi, r] = torch.where(seen, size, torch.zeros_like(size)).amax(1) * (d + 8) * 2.0 ** -24
    return o, lse, weight, delta, count


def check_attention(got_o, got_lse, ref, eps_p, what=""):
    o, lse, weight, delta, count = ref
    got_o, got_lse = got_o.double().cpu(), got_lse.double().cpu()
    rel = eps_p + 2.0 ** -20 + 2 * delta[..., None] + count[:, None, None] * (2.0 ** -24 + 2.0 ** -31)
    bound = (2.0 ** -8 * o.abs() + weight * rel * (1 + 2.0 ** -8)) * SLACK + 1e-30
    err = (got_o - o).abs()
    assert torch.isfinite(got_o).all(), f"{what}: O is not finite"
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: O off by {worst:.3f} of its bound"
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(got_lse), empty), f"{what}: rows without a key differ"
    assert (got_o.permute(1, 0, 2)[empty] == 0).all(), f"{what}: O of rows without a key"
    lb = delta.t() + 2.0 ** -20 + count * 2.0 ** -24 + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -22
    lerr = torch.where(empty, torch.zeros_like(lse), (got_lse - lse).abs())
    worst_l = (lerr / lb)[~empty].max().item() if (~empty).any() else 0.0
    assert worst_l <= 1.0, f"{what}: LSE off by {worst_l:.3f} of its bound"
    return worst, worst_l
