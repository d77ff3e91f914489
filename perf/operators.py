"""Measured cases of the paged 8-bit key/value cache: the append and the attention that reads it.

The cache holds keys and values as e4m3 codes in pages of ``page`` tokens, ``[num_pages, heads_kv, page, d]``, with one
power-of-two scale (e8m0) for each page and head: a stored code stands for code * scale.  Two operators:

* ``append``: the new tokens' queries and keys are rotated by their positions, the queries come back in bf16, the keys
  and values are quantised into the pages that the block table gives.  The scale of a page and head is the smallest
  power of two (2^-63 at least) with max|x| <= 448 * scale over its tokens; where a new token makes it grow, the codes
  that are there are rounded again under the new scale.
* ``attend``: softmax attention of the new tokens (packed, ``cu_seqlens``) over each sequence's cached tokens, the new
  ones among them; causal is bottom-right aligned.  Returns O in bf16 and the log-sum-exp in fp32.

``own`` False computes both with elementary torch operations in fp32, True calls the package.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -63  # smallest scale 2^-63
DEVICE = "cuda"
HEAD_DIMS = [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)]


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    gqa = {"heads_q": 32, "heads_kv": 8, "d_qk": 128, "d_v": 128}
    append = {"op": "append", "rot": 128, "interleaved": False}
    attend = {"op": "attend", "causal": True}
    return [
        # one user's next token: the launch and the chain of dependent loads are all there is
        dict(append, name="append_one", batch=1, **gqa, page=64, new_min=1, new_max=1, ctx_min=1000, ctx_max=1000, salt=1),
        # a serving step: one token for each of many sequences of all ages
        dict(append, name="append_step", batch=128, **gqa, page=64, new_min=1, new_max=1, ctx_min=1, ctx_max=4000, salt=2),
        # a whole prompt at once, its length not a multiple of the page
        dict(append, name="append_prompt", batch=1, **gqa, page=64, new_min=8191, new_max=8191, ctx_min=0, ctx_max=0, salt=3),
        # a ragged batch of prompts behind cached prefixes; keys wider than values, part of the key rotated, in pairs
        {"op": "append", "name": "append_ragged", "batch": 24, "heads_q": 16, "heads_kv": 16, "d_qk": 192, "d_v": 128,
         "rot": 64, "interleaved": True, "page": 32, "new_min": 1, "new_max": 900, "ctx_min": 0, "ctx_max": 700, "salt": 4},
        # one user's next token over a short context
        dict(attend, name="attend_one", batch=1, **gqa, page=64, new_min=1, new_max=1, ctx_min=1026, ctx_max=1026, salt=5),
        # decode over long contexts, the sizes of this repository's decode benchmark
        dict(attend, name="attend_long", batch=8, **gqa, page=64, new_min=1, new_max=1, ctx_min=32767, ctx_max=32767, salt=6),
        # decode of many sequences of very different lengths, every query head with its own keys, small pages
        dict(attend, name="attend_ragged", batch=64, heads_q=16, heads_kv=16, d_qk=64, d_v=64, page=16, new_min=1, new_max=1,
             ctx_min=1, ctx_max=8000, salt=7),
        # decode with one key/value head for all query heads, large pages
        dict(attend, name="attend_shared", batch=32, heads_q=32, heads_kv=1, d_qk=128, d_v=128, page=128, new_min=1, new_max=1,
             ctx_min=3000, ctx_max=9000, salt=8),
        # decode with keys wider than values
        dict(attend, name="attend_wide", batch=16, heads_q=16, heads_kv=16, d_qk=192, d_v=128, page=64, new_min=1, new_max=1,
             ctx_min=2000, ctx_max=6000, salt=9),
        # a few drafted tokens for each sequence, checked in one call
        dict(attend, name="attend_draft", batch=16, **gqa, page=32, new_min=5, new_max=5, ctx_min=500, ctx_max=8000, salt=10),
        # a chunk of a prompt behind a cached prefix
        dict(attend, name="attend_chunk", batch=2, **gqa, page=64, new_min=2048, new_max=2048, ctx_min=5000, ctx_max=7001, salt=11),
        # prompts and single tokens in one batch
        dict(attend, name="attend_mixed", batch=10, heads_q=16, heads_kv=4, d_qk=64, d_v=64, page=32, new_min=1, new_max=1200,
             ctx_min=0, ctx_max=2500, salt=12),
    ]


def lengths(case):
    """(new tokens, tokens before them) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["salt"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["batch"])]
    return new, ctx


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        d_qk, d_v = rng.choice(HEAD_DIMS)
        heads_kv = rng.choice([1, 2, 3, 4, 8, 16])
        heads_q = heads_kv * rng.choice([1, 2, 3, 4, 5, 8, 16])
        case = {"op": rng.choice(["append", "attend", "attend"]), "batch": _log_int(rng, 1, 96), "heads_q": heads_q,
                "heads_kv": heads_kv, "d_qk": d_qk, "d_v": d_v, "page": rng.choice([16, 32, 64, 128])}
        kind = rng.choice(["token", "token", "few", "prompt"])
        case["new_min"] = 1
        case["new_max"] = 1 if kind == "token" else rng.randint(2, 16) if kind == "few" else _log_int(rng, 17, 4096)
        case["ctx_max"] = _log_int(rng, 1, 32767)
        case["ctx_min"] = rng.choice([0, case["ctx_max"] // 2, case["ctx_max"]])
        case["salt"] = rng.randrange(1 << 20)
        if case["op"] == "append":
            case["rot"] = rng.choice([0, 16, 32, d_qk // 2, d_qk])
            case["interleaved"] = rng.choice([False, True])
        else:
            case["causal"] = rng.choice([True, True, False])
        new, ctx = lengths(case)
        total = sum(new) + sum(ctx)
        cached = total * heads_kv * (d_qk + d_v)
        if max(heads_q // heads_kv, 1) > 32 or sum(new) * heads_q * d_qk > 64e6:
            continue
        if case["op"] == "append":
            if cached <= 200e6 and sum(new) <= 8000:
                return case
        else:
            flops = work(case)["flops"]
            padded = case["batch"] * max(new) * heads_q * (max(new) + max(ctx))
            values = case["batch"] * (max(new) + max(ctx)) * heads_kv * (d_qk + d_v)
            if cached <= 400e6 and flops <= 400e9 and padded <= 1.2e9 and values <= 600e6:
                return case


def work(case):
    new, ctx = lengths(case)
    hq, hkv, dq, dv, page = case["heads_q"], case["heads_kv"], case["d_qk"], case["d_v"], case["page"]
    tokens = sum(new)
    index = 4 * (2 * case["batch"] + 1)
    if case["op"] == "append":
        pages = sum((c + n - 1) // page - c // page + 1 for n, c in zip(new, ctx))
        read = tokens * (2 * hq * dq + 2 * hkv * (dq + dv) + 4 * case["rot"]) + 4 * pages + index
        written = tokens * (2 * hq * dq + hkv * (dq + dv)) + 2 * pages * hkv
        # three operations for each rotated value, three to find a scale and round each stored one
        flops = tokens * (3 * case["rot"] * (hq + hkv) + 3 * hkv * (dq + dv))
        return {"bytes": read + written, "flops": flops}
    lens = [n + c for n, c in zip(new, ctx)]
    pages = sum(-(-n // page) for n in lens)
    if case["causal"]:
        pairs = sum(n * (n + c) - n * (n - 1) // 2 for n, c in zip(new, ctx))
    else:
        pairs = sum(n * (n + c) for n, c in zip(new, ctx))
    read = sum(lens) * hkv * (dq + dv) + pages * (2 * hkv + 4) + index + tokens * hq * dq * 2
    written = tokens * hq * (2 * dv + 4)
    return {"bytes": read + written, "flops": 2 * hq * pairs * (dq + dv)}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _scales_of(amax):
    """The smallest powers of two, 2^-63 at least, with amax <= 448 * scale: their exponents (int32)."""
    mant, expo = torch.frexp(amax)  # amax = mant * 2^expo, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(mant <= 0.875, expo - 9, expo - 8)
    return torch.where(amax > 0, e.clamp(min=MIN_EXP), torch.full_like(e, MIN_EXP)).to(torch.int32)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _fill(gen, pages, heads, page, d, filled, spread):
    """Pages of normal values whose size differs between heads and channels, quantised; `filled` tokens hold something."""
    codes = torch.empty(pages, heads, page, d, dtype=torch.uint8, device=DEVICE)
    expo = torch.empty(pages, heads, dtype=torch.int32, device=DEVICE)
    size = torch.exp2(torch.randint(-2, 3, (1, heads, 1, d), generator=gen, device=DEVICE).float() * spread)
    at = torch.arange(page, device=DEVICE)
    step = max(1, (64 << 20) // max(1, heads * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn(n, heads, page, d, generator=gen, device=DEVICE) * size
        used = (at[None] < filled[i:i + n, None])[:, None, :, None]
        x = torch.where(used, x, torch.zeros((), device=DEVICE))
        e = _scales_of(x.abs().amax((2, 3)))
        codes[i:i + n] = (x / _pow2(e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        expo[i:i + n] = e
    return codes, expo


def prepare(case, seed):
    """A server's state before the call: the pages, the block table, the lengths and the new tokens' projections."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    new, ctx = lengths(case)
    hq, hkv, dq, dv, page, batch = (case[k] for k in ("heads_q", "heads_kv", "d_qk", "d_v", "page", "batch"))
    attend = case["op"] == "attend"
    lens = [n + c for n, c in zip(new, ctx)]
    counts = [-(-n // page) for n in lens]
    width, num_pages = max(counts), sum(counts) + 3
    order = torch.randperm(num_pages, generator=gen, device=DEVICE)
    # unused entries of the table are -1, pages are in no order
    cols = torch.arange(width, device=DEVICE)[None]
    counts_t = torch.tensor(counts, device=DEVICE)[:, None]
    first = torch.cumsum(counts_t, 0) - counts_t
    table = torch.where(cols < counts_t, order[(first + cols).clamp(max=num_pages - 1)], torch.full((), -1, device=DEVICE))
    # tokens that a page holds before the call
    held = torch.tensor(lens if attend else ctx, device=DEVICE)[:, None] - cols * page
    filled = torch.zeros(num_pages + 1, dtype=torch.int64, device=DEVICE)
    filled[torch.where(table >= 0, table, num_pages)] = held.clamp(0, page)
    filled = filled[:num_pages]
    k_codes, k_exp = _fill(gen, num_pages, hkv, page, dq, filled, 0.5)
    v_codes, v_exp = _fill(gen, num_pages, hkv, page, dv, filled, 0.25)
    if attend:  # behind the last token of a sequence a page holds anything, codes that are no number among it
        behind = (torch.arange(page, device=DEVICE)[None] >= filled[:, None])[:, None, :, None]
        k_codes.masked_fill_(behind, 0x7F)
        v_codes.masked_fill_(behind, 0xFF)
    tokens = sum(new)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE).to(torch.bfloat16)

    state = {"case": dict(case), "k_cache": k_codes.view(torch.float8_e4m3fn), "v_cache": v_codes.view(torch.float8_e4m3fn),
             "k_scale": (k_exp + 127).to(torch.uint8).view(torch.float8_e8m0fnu),
             "v_scale": (v_exp + 127).to(torch.uint8).view(torch.float8_e8m0fnu),
             "block_table": table.to(torch.int32).contiguous(),
             "seqlens_k": torch.tensor(lens, dtype=torch.int32, device=DEVICE),
             "cu_seqlens": torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEVICE),
             "max_new": max(new), "total_k": sum(lens)}
    if attend:
        state["q"] = normal(tokens, hq, dq)
        state["out"] = torch.empty(tokens, hq, dv, dtype=torch.bfloat16, device=DEVICE)
        state["lse"] = torch.empty(hq, tokens, dtype=torch.float32, device=DEVICE)
    else:
        # views of one projection's output, as a model has them
        qkv = normal(tokens, hq * dq + hkv * dq + hkv * dv)
        q, k, v = qkv.split([hq * dq, hkv * dq, hkv * dv], dim=1)
        state["q"], state["k"], state["v"] = q.view(tokens, hq, dq), k.view(tokens, hkv, dq), v.view(tokens, hkv, dv)
        state["q_out"] = torch.empty(tokens, hq, dq, dtype=torch.bfloat16, device=DEVICE)
        state["cos_sin"] = None
        if case["rot"]:
            half = case["rot"] // 2
            freq = torch.pow(10000.0, -torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
            angle = torch.arange(max(lens), dtype=torch.float64, device=DEVICE)[:, None] * freq
            state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return state


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attend(state) if own else _plain_attend(state)


def _cache_of(s):
    return {name: s[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _own_append(s):
    import exact_attention_forward_08_gb300 as fa

    fa.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["seqlens_k"],
                 s["cu_seqlens"], q=s["q"], cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], q_out=s["q_out"])
    return {"q": s["q_out"], **_cache_of(s)}


def _own_attend(s):
    import exact_attention_forward_08_gb300 as fa

    out, lse = fa.attention_forward_paged(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                          s["seqlens_k"], s["cu_seqlens"], s["max_new"], causal=s["case"]["causal"],
                                          total_k=s["total_k"], out=s["out"], lse=s["lse"])
    return {"o": out, "lse": lse}


def _token_places(s):
    """For each new token its sequence and its index among that sequence's new tokens."""
    cu = s["cu_seqlens"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return t, cu, seq, t - cu[seq]


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if rot == 0:
        return x
    head, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _plain_append(s):
    case = s["case"]
    page, rot = case["page"], case["rot"]
    t, cu, seq, at = _token_places(s)
    lens, table = s["seqlens_k"].long(), s["block_table"].long()
    start = lens - (cu[1:] - cu[:-1])  # tokens before the new ones
    pos = start[seq] + at
    pid, slot = table[seq, pos // page], pos % page
    q, k = s["q"].float(), s["k"].float()
    if rot:
        cos, sin = s["cos_sin"][pos].chunk(2, 1)
        q, k = (_rotate(x, cos, sin, rot, case["interleaved"]) for x in (q, k))
    # the page that a sequence's first new token goes to may hold older tokens
    old_pid, old_count = table[torch.arange(len(lens), device=lens.device), start.clamp(min=0) // page], start % page
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"], s["v_scale"])):
        codes, expo = cache.view(torch.uint8), scale.view(torch.uint8)
        amax = torch.zeros(expo.shape, device=x.device)
        amax.scatter_reduce_(0, pid[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        need = _scales_of(amax) + 127
        old = expo.int()
        held = torch.zeros(expo.shape[0], dtype=torch.bool, device=x.device)
        held[old_pid] = old_count > 0
        touched = torch.zeros(expo.shape[0], dtype=torch.bool, device=x.device)
        touched[pid] = True
        grown = torch.where(held[:, None], torch.maximum(need, old), need)
        expo.copy_(torch.where(touched[:, None], grown, old))
        # older codes of the pages whose scale grew
        before = codes[old_pid]
        shrink = _pow2(old[old_pid] - grown[old_pid])[..., None, None]
        again = (before.view(torch.float8_e4m3fn).float() * shrink).to(torch.float8_e4m3fn).view(torch.uint8)
        keep = torch.arange(page, device=x.device)[None] < old_count[:, None]
        codes[old_pid] = torch.where(keep[:, None, :, None], again, before)
        codes[pid, :, slot] = (x / _pow2(grown[pid] - 127)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["q_out"].copy_(q)
    return {"q": s["q_out"], **_cache_of(s)}


def _plain_attend(s):
    case = s["case"]
    hq, hkv, page = case["heads_q"], case["heads_kv"], case["page"]
    t, cu, seq, at = _token_places(s)
    batch, n = len(cu) - 1, s["max_new"]
    lens, new = s["seqlens_k"].long(), cu[1:] - cu[:-1]
    table = s["block_table"].long().clamp(min=0)
    length = table.shape[1] * page
    cols = torch.arange(length, device=cu.device)
    inside = cols[None] < lens[:, None]

    def dense(cache, scale):  # [batch, heads_kv, length, d]
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x *= _pow2(scale.view(torch.uint8)[table].int() - 127)[..., None, None]
        return x.transpose(1, 2).reshape(batch, hkv, length, -1)

    k, v = dense(s["k_cache"], s["k_scale"]), dense(s["v_cache"], s["v_scale"])
    v = torch.where(inside[:, None, :, None], v, torch.zeros((), device=v.device))
    rows = torch.arange(n, device=cu.device)
    q = s["q"][(cu[:-1, None] + rows).clamp(max=len(t) - 1)].float()  # [batch, n, heads_q, d]
    q = q.view(batch, n, hkv, hq // hkv, -1).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, q.shape[-1])
    scores = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(case["d_qk"]))
    scores = scores.view(batch, hkv, hq // hkv, n, length)
    seen = inside[:, None].expand(-1, n, -1)
    if case["causal"]:
        seen = seen & (cols[None, None] <= (rows[None] + (lens - new)[:, None])[..., None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros((), device=top.device), top)
    scores -= top
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]  # log 0 = -inf where a row sees nothing
    o = torch.matmul(scores.view(batch, hkv, -1, length), v).view(batch, hkv, hq // hkv, n, -1)
    o = torch.where(total > 0, o / total, torch.zeros((), device=o.device))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, -1)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, n, hq)
    return {"o": o[seq, at].to(torch.bfloat16), "lse": lse[seq, at].t().contiguous()}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, one sequence after the other
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    case = s["case"]
    new, ctx = lengths(case)
    page, rot = case["page"], case["rot"]
    table = s["block_table"].tolist()
    q_out = s["q"].double()
    out = {}
    done = 0
    k = s["k"].double()
    for n, c in zip(new, ctx):
        if rot:
            cs = s["cos_sin"][c:c + n].double()
            cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
            first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
            second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
            for x in (q_out, k):
                y = x[done:done + n]
                a, b = y[..., first].clone(), y[..., second].clone()
                y[..., first] = a * cos - b * sin
                y[..., second] = b * cos + a * sin
        done += n
    out["q"] = q_out
    for name, x in (("k", k), ("v", s["v"].double())):
        codes = s[name + "_cache"].float().double()
        scale = s[name + "_scale"].float().double()
        done = 0
        for b, (n, c) in enumerate(zip(new, ctx)):
            for j in range(c // page, (c + n - 1) // page + 1):
                p, lo, hi = table[b][j], max(c, j * page), min(c + n, (j + 1) * page)
                part = x[done + lo - c:done + hi - c].transpose(0, 1)  # [heads, tokens, d]
                want = torch.exp2(torch.ceil(torch.log2(part.abs().amax((1, 2)) / E4M3_MAX)).clamp(min=MIN_EXP))
                if lo > j * page:
                    want = torch.maximum(want, scale[p])
                    old = codes[p, :, :lo - j * page] * (scale[p] / want)[:, None, None]
                    codes[p, :, :lo - j * page] = old.to(torch.float8_e4m3fn).double()
                codes[p, :, lo - j * page:hi - j * page] = (part / want[:, None, None]).to(torch.float8_e4m3fn).double()
                scale[p] = want
            done += n
        out[name + "_cache"], out[name + "_scale"] = codes, scale
    return out


def _exact_attend(s):
    case = s["case"]
    new, ctx = lengths(case)
    hq, hkv, page = case["heads_q"], case["heads_kv"], case["page"]
    ratio = hq // hkv
    table = s["block_table"].tolist()
    q = s["q"].double() / math.sqrt(case["d_qk"])
    o = torch.empty(q.shape[0], hq, case["d_v"], dtype=torch.float64, device=q.device)
    lse = torch.empty(hq, q.shape[0], dtype=torch.float64, device=q.device)
    done = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        length = n + c
        pages = torch.tensor(table[b][:-(-length // page)], device=q.device)

        def dense(name):
            x = s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float().double()
            x = x * s[name + "_scale"].float().double()[pages][..., None, None]
            return x.transpose(0, 1).flatten(1, 2)[:, :length]

        k, v = dense("k"), dense("v")
        hidden = None
        if case["causal"]:
            i = torch.arange(n, device=q.device)[:, None]
            hidden = (torch.arange(length, device=q.device)[None] > i + c).repeat(ratio, 1)
        for h in range(hkv):
            mine = q[done:done + n, h * ratio:(h + 1) * ratio].transpose(0, 1).reshape(ratio * n, -1)
            scores = mine @ k[h].t()
            if hidden is not None:
                scores.masked_fill_(hidden, -math.inf)
            l = torch.logsumexp(scores, 1)
            got = torch.exp(scores - l[:, None]) @ v[h]
            o[done:done + n, h * ratio:(h + 1) * ratio] = got.view(ratio, n, -1).transpose(0, 1)
            lse[h * ratio:(h + 1) * ratio, done:done + n] = l.view(ratio, n)
        done += n
    return {"o": o, "lse": lse}
