"""Measured cases of long contexts over the paged 8-bit cache: rotary positions, sparse attention over selected pages, and
the pages' bookkeeping.

The cache is the package's own: e4m3 codes in pages of ``page`` tokens, ``[num_pages, heads_kv, page, d]``, one power-of-two
scale (e8m0) for each page and head.  Six operators:

* ``table``: cosines and sines of positions 0 .. n-1, the frequencies scaled for contexts beyond the trained length.
* ``rotate``: queries and keys turned by their positions (or their gradients by the transposed rotation), half or
  interleaved pairs, all or part of a head.
* ``select``: a decoding step's choice of pages.  The largest and smallest code of each channel are kept for each page and
  key head; those of the pages that hold the step's new tokens are found anew, then each new token and key head takes the
  ``top`` pages with the largest bound on the sum of its query heads' scores, the first and the last pages always.
* ``lists``: attention of each new token and key head over its own list of pages.
* ``fork``: rows of the block table taken over by others (beams, requests that end), with pages for new tokens; full pages
  are shared and counted, a page that is partly filled is copied for all but the first heir.
* ``compact``: pages in use moved to the lowest indices, the block table following.

``own`` False computes them with elementary torch operations, True calls the package.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
HEAD_DIMS = [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)]


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    gqa = {"heads_q": 32, "heads_kv": 8, "d_qk": 128, "d_v": 128}
    return [
        # the table of a model that was trained on 8192 positions and serves 16 times as many
        {"op": "table", "name": "table_long", "positions": 131072, "rot": 128, "scaling": "by_parts", "factor": 16.0,
         "original": 8192, "low": 1.0, "high": 32.0, "magnitude": 1.2772588722239782},
        # a short table, positions squeezed four to one
        {"op": "table", "name": "table_short", "positions": 4099, "rot": 64, "scaling": "linear", "factor": 4.0,
         "original": 0, "low": 1.0, "high": 2.0, "magnitude": 1.0},
        # one user's next token
        {"op": "rotate", "name": "rotate_one", "batch": 1, "new_min": 1, "new_max": 1, **gqa, "rot": 128,
         "interleaved": False, "backward": False, "explicit": True, "salt": 1},
        # gradients of a ragged training batch; part of each head turned, in pairs
        {"op": "rotate", "name": "rotate_gradient", "batch": 16, "new_min": 100, "new_max": 2500, "heads_q": 16,
         "heads_kv": 16, "d_qk": 192, "d_v": 128, "rot": 64, "interleaved": True, "backward": True, "explicit": False,
         "salt": 2},
        # one user's next token over a long context
        {"op": "select", "name": "select_one", "batch": 1, "new": 1, "ctx_min": 131000, "ctx_max": 131000, **gqa,
         "page": 64, "top": 32, "first": 1, "last": 2, "salt": 3},
        # a serving step of sequences of all ages, a few drafted tokens each
        {"op": "select", "name": "select_drafts", "batch": 24, "new": 3, "ctx_min": 100, "ctx_max": 131000, **gqa,
         "page": 64, "top": 48, "first": 1, "last": 1, "salt": 4},
        # the attention of one token over its selected pages
        {"op": "lists", "name": "lists_one", "tokens": 1, **gqa, "page": 64, "top": 32, "full": True, "pool": 3000,
         "salt": 5},
        # that of a serving step, some sequences still shorter than their lists
        {"op": "lists", "name": "lists_step", "tokens": 64, **gqa, "page": 64, "top": 64, "full": False, "pool": 6000,
         "salt": 6},
        # beam search: 16 requests of 4 beams take over one another's rows and get room for a token
        {"op": "fork", "name": "fork_beams", "groups": 16, "beams": 4, "shared_min": 500, "shared_max": 2000, "own_min": 1,
         "own_max": 900, **gqa, "page": 64, "serve": False, "salt": 7},
        # a server's step: some requests end, others begin with their prompts, the rest go on
        {"op": "fork", "name": "fork_serve", "groups": 256, "beams": 1, "shared_min": 0, "shared_max": 0, "own_min": 1,
         "own_max": 3000, "heads_q": 16, "heads_kv": 4, "d_qk": 64, "d_v": 64, "page": 32, "serve": True, "salt": 8},
        # a small pool with few holes
        {"op": "compact", "name": "compact_few", "rows": 20, "own_min": 1, "own_max": 1500, "heads_q": 16, "heads_kv": 4,
         "d_qk": 64, "d_v": 64, "page": 16, "spare": 0.1, "salt": 9},
        # a large pool, half of it free
        {"op": "compact", "name": "compact_half", "rows": 64, "own_min": 100, "own_max": 4000, **gqa, "page": 64,
         "spare": 1.0, "salt": 10},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    d_qk, d_v = rng.choice(HEAD_DIMS)
    heads_kv = rng.choice([1, 2, 3, 4, 8, 16])
    return {"heads_q": heads_kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), "heads_kv": heads_kv, "d_qk": d_qk, "d_v": d_v}


def _draw_table(rng):
    low = rng.choice([1.0, 2.0])
    return {"op": "table", "positions": _log_int(rng, 1, 131072), "rot": 16 * rng.randint(1, 8),
            "scaling": rng.choice(["none", "linear", "base", "by_parts"]), "factor": rng.choice([1.0, 2.0, 4.0, 10.5, 32.0]),
            "original": rng.choice([2048, 4096, 8192]), "low": low, "high": low * rng.choice([2.0, 4.0, 16.0]),
            "magnitude": rng.choice([1.0, 1.25])}


def _draw_rotate(rng):
    case = {"op": "rotate", "batch": _log_int(rng, 1, 64), **_heads(rng)}
    case["new_max"] = _log_int(rng, 1, 4096)
    case["new_min"] = rng.choice([1, case["new_max"]])
    case["rot"] = rng.choice([16, 32, case["d_qk"] // 2, case["d_qk"]])
    for name in ("interleaved", "backward", "explicit"):
        case[name] = rng.choice([False, True])
    case["salt"] = rng.randrange(1 << 20)
    values = sum(_new_tokens(case)) * (case["heads_q"] + case["heads_kv"]) * case["d_qk"]
    return case if values <= 100e6 else None


def _draw_select(rng):
    case = {"op": "select", "batch": _log_int(rng, 1, 96), "new": rng.choice([1, 1, 1, 2, 4, 7]), **_heads(rng)}
    case["ctx_max"] = _log_int(rng, 1, 131071)
    case["ctx_min"] = rng.choice([0, case["ctx_max"] // 2, case["ctx_max"]])
    case["page"] = rng.choice([16, 32, 64, 128])
    case["first"], case["last"] = rng.choice([0, 1, 2]), rng.choice([1, 1, 2, 4])
    case["top"] = case["first"] + case["last"] + _log_int(rng, 1, 128)
    case["salt"] = rng.randrange(1 << 20)
    tokens = sum(_contexts(case)) + case["batch"] * case["new"]
    widest = -(-(max(_contexts(case)) + case["new"]) // case["page"])
    scores = case["batch"] * case["new"] * case["heads_q"] * widest * case["d_qk"]
    small = tokens * case["heads_kv"] * case["d_qk"] <= 600e6 and scores <= 2e9
    return case if small and case["batch"] * widest * case["heads_kv"] * case["d_qk"] <= 50e6 else None


def _draw_lists(rng):
    case = {"op": "lists", "tokens": _log_int(rng, 1, 512), **_heads(rng), "page": rng.choice([16, 32, 64, 128]),
            "top": _log_int(rng, 1, 256), "full": rng.choice([False, True])}
    case["pool"] = case["top"] * rng.randint(2, 4) + _log_int(rng, 8, 2000)
    case["salt"] = rng.randrange(1 << 20)
    per_page = case["heads_kv"] * case["page"] * (case["d_qk"] + case["d_v"])
    values = case["tokens"] * case["top"] * per_page
    pairs = case["tokens"] * case["heads_q"] * case["top"] * case["page"]
    return case if values <= 500e6 and pairs <= 400e6 and case["pool"] * per_page <= 800e6 else None


def _draw_fork(rng):
    case = {"op": "fork", **_heads(rng), "page": rng.choice([16, 32, 64, 128]), "serve": rng.choice([False, True])}
    case["groups"], case["beams"] = _log_int(rng, 1, 256), 1
    if not case["serve"]:
        case["groups"], case["beams"] = _log_int(rng, 1, 32), rng.randint(2, 12)
    case["shared_max"] = 0 if case["serve"] else _log_int(rng, 1, 4000)
    case["shared_min"] = case["shared_max"] // 2
    case["own_max"], case["own_min"] = _log_int(rng, 1, 4000), 1
    case["salt"] = rng.randrange(1 << 20)
    return case if _pool_bytes(case) <= 600e6 else None


def _draw_compact(rng):
    case = {"op": "compact", "rows": _log_int(rng, 1, 256), **_heads(rng), "page": rng.choice([16, 32, 64, 128])}
    case["own_max"] = _log_int(rng, 1, 8000)
    case["own_min"] = rng.choice([0, 1, case["own_max"] // 2])
    case["spare"] = rng.choice([0.02, 0.1, 0.5, 1.0, 2.0])
    case["salt"] = rng.randrange(1 << 20)
    return case if _pool_bytes(case) <= 1.2e9 else None


def draw(rng):
    make = rng.choice([_draw_table, _draw_rotate, _draw_select, _draw_select, _draw_lists, _draw_lists, _draw_fork,
                       _draw_compact])
    while True:
        case = make(rng)
        if case is not None:
            return case


# What a case's own numbers fix, apart from the seed: lengths, rows and pages.

def _new_tokens(case):
    r = random.Random(case["salt"])
    return [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]


def _contexts(case):
    r = random.Random(case["salt"])
    return [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["batch"])]


def _list_lengths(case):
    """Tokens that each new token sees of its list of pages."""
    r = random.Random(case["salt"])
    page, top = case["page"], case["top"]
    return [(top - 1) * page + r.randint(1, page) if case["full"] or r.random() < 0.6 else r.randint(1, top * page)
            for _ in range(case["tokens"])]


def _rows(case):
    """(table rows as lists of pages, lengths, number of pages, parents, new tokens) of a fork's or a compaction's pool."""
    r = random.Random(case["salt"])
    page = case["page"]
    lens, shared = [], []
    if case["op"] == "compact":
        lens = [r.randint(case["own_min"], case["own_max"]) for _ in range(case["rows"])]
        shared = [(None, 0)] * len(lens)
    else:
        for g in range(case["groups"]):
            common = r.randint(case["shared_min"], case["shared_max"]) // page  # full pages of the prompt
            for _ in range(case["beams"]):
                lens.append(common * page + r.randint(case["own_min"], case["own_max"]))
                shared.append((g, common))
    batch = len(lens)
    if case["op"] == "compact":
        parents, grow = list(range(batch)), [0] * batch
    elif case["serve"]:
        parents = [b if r.random() < 0.9 else -1 for b in range(batch)]
        grow = [1 if p >= 0 else r.randint(0, case["own_max"]) for p in parents]
    else:
        beams = case["beams"]
        parents = [b - b % beams + r.randrange(beams) for b in range(batch)]
        grow = [1] * batch
    counts = [-(-n // page) for n in lens]
    unique = sum(c - s[1] for c, s in zip(counts, shared)) + sum(dict(s for s in shared if s[0] is not None).values())
    most = unique + sum(-(-g // page) + 1 for g in grow)  # enough for every copy and every new token
    num_pages = max(most + 1, int(unique * (1 + case["spare"])) + 1) if case["op"] == "compact" else most + 1
    order = list(range(num_pages))
    r.shuffle(order)
    prompts, table = {}, []
    for n, (g, common) in zip(counts, shared):
        if g is not None and g not in prompts:
            prompts[g] = [order.pop() for _ in range(common)]
        head = prompts[g] if g is not None else []
        table.append(head + [order.pop() for _ in range(n - len(head))])
    return table, lens, num_pages, parents, grow


def _pool_bytes(case):
    _, _, num_pages, _, _ = _rows(case)
    return num_pages * case["heads_kv"] * case["page"] * (case["d_qk"] + case["d_v"])


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["positions"] * case["rot"], "flops": 2 * case["positions"] * case["rot"]}
    hq, hkv, dq = case["heads_q"], case["heads_kv"], case["d_qk"]
    if op == "rotate":
        tokens = sum(_new_tokens(case))
        index = 4 * (tokens if case["explicit"] else case["batch"] + 1)
        return {"bytes": tokens * (4 * (hq + hkv) * dq + 4 * case["rot"]) + index,
                "flops": 3 * tokens * (hq + hkv) * case["rot"]}
    page, dv = case["page"], case.get("d_v", 0)
    if op == "select":
        batch, new, top = case["batch"], case["new"], case["top"]
        touched = pages = scored = 0
        for c in _contexts(case):
            last = (c + new - 1) // page
            touched += last - c // page + 1
            pages += last + 1
            scored += new * (last + 1)
        # touched pages' codes, all pages' bounds, scales and table entries, queries; bounds and lists written
        read = hkv * (touched * page * dq + (pages - touched) * 2 * dq + pages) + 4 * pages + batch * new * hq * dq * 2
        written = hkv * touched * 2 * dq + batch * new * (4 * hkv * top + 4)
        return {"bytes": read + written, "flops": hkv * (4 * scored * dq + touched * page * dq * 2)}
    if op == "lists":
        seen = _list_lengths(case)
        pages = sum(-(-n // page) for n in seen)
        tokens = case["tokens"]
        read = hkv * (sum(seen) * (dq + dv) + pages * 6) + tokens * (2 * hq * dq + 4)
        return {"bytes": read + tokens * hq * (2 * dv + 4), "flops": 2 * hq * sum(seen) * (dq + dv)}
    table, lens, num_pages, parents, grow = _rows(case)
    token = hkv * (dq + dv)
    entries = sum(len(row) for row in table)
    if op == "fork":
        copied = pages = out = 0
        heirs = set()
        for p, g in zip(parents, grow):
            part = lens[p] % page if p >= 0 else 0
            out += -(-((lens[p] if p >= 0 else 0) + g) // page)
            if part and p in heirs:
                copied, pages = copied + part, pages + 1
            heirs.add(p)
        moved = 2 * (copied * token + pages * hkv * (2 + 2 * dq))
        return {"bytes": moved + 4 * (entries + out + 2 * num_pages + 4 * len(lens)), "flops": num_pages + out}
    used = sorted({p for row in table for p in row})
    moves = sum(p >= len(used) for p in used)
    moved = 2 * moves * (token * page + hkv * (2 + 2 * dq))
    return {"bytes": moved + 4 * (2 * entries + 3 * num_pages + len(lens)), "flops": num_pages + entries}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _codes(gen, pages, heads, page, d):
    """e4m3 codes of pages whose channels have their own size and drift from page to page."""
    size = torch.exp2(torch.randint(-2, 3, (1, heads, 1, d), generator=gen, device=DEVICE).float() * 0.5)
    codes = torch.empty(pages, heads, page, d, dtype=torch.float8_e4m3fn, device=DEVICE)
    step = max(1, (64 << 20) // (heads * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn(n, heads, page, d, generator=gen, device=DEVICE)
        x += torch.randn(n, heads, 1, d, generator=gen, device=DEVICE)
        codes[i:i + n] = (x * size * 20).to(torch.float8_e4m3fn)
    return codes


def _scales(gen, pages, heads):
    e = torch.randint(120, 122, (pages, heads), generator=gen, device=DEVICE)
    return e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _bounds_of(codes):
    """[pages, heads, 2, d]: the largest and the smallest code of each channel."""
    x = codes.float()
    return torch.stack([x.amax(2), x.amin(2)], 2)


def _all_bounds(codes):
    bounds = torch.empty(codes.shape[0], codes.shape[1], 2, codes.shape[3], dtype=torch.float8_e4m3fn, device=DEVICE)
    step = max(1, (256 << 20) // codes[0].numel())
    for i in range(0, codes.shape[0], step):
        bounds[i:i + step] = _bounds_of(codes[i:i + step]).to(torch.float8_e4m3fn)
    return bounds


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE).to(torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    """What a program holds before the call: the cache and its tables, the projections, buffers for the results."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    state = {"case": dict(case)}
    make = {"table": _prepare_table, "rotate": _prepare_rotate, "select": _prepare_select, "lists": _prepare_lists,
            "fork": _prepare_pool, "compact": _prepare_pool}
    make[case["op"]](case, gen, state)
    return state


def _prepare_table(case, gen, s):
    # the base differs from model to model
    s["base"] = 10000.0 + float(torch.rand((), generator=gen, device=DEVICE)) * 490000.0
    s["out"] = torch.empty(case["positions"], case["rot"], dtype=torch.float32, device=DEVICE)


def _prepare_rotate(case, gen, s):
    new = _new_tokens(case)
    tokens, hq, hkv, d = sum(new), case["heads_q"], case["heads_kv"], case["d_qk"]
    if case["backward"]:
        s["q"], s["k"] = _normal(gen, tokens, hq, d), _normal(gen, tokens, hkv, d)
    else:  # views of one projection's output, as a model has them
        both = _normal(gen, tokens, (hq + 2 * hkv) * d)
        s["q"] = both[:, :hq * d].view(tokens, hq, d)
        s["k"] = both[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
    longest = 8192
    s["cu_seqlens"] = s["positions"] = None
    if case["explicit"]:
        s["positions"] = torch.randint(0, longest, (tokens,), generator=gen, device=DEVICE).to(torch.int32)
    else:
        s["cu_seqlens"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEVICE)
    half = case["rot"] // 2
    freq = torch.pow(10000.0, -torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
    angle = torch.arange(longest, dtype=torch.float64, device=DEVICE)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["q_out"] = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device=DEVICE)
    s["k_out"] = torch.empty(tokens, hkv, d, dtype=torch.bfloat16, device=DEVICE)


def _prepare_select(case, gen, s):
    ctx, new, page = _contexts(case), case["new"], case["page"]
    batch, hq, hkv, d = case["batch"], case["heads_q"], case["heads_kv"], case["d_qk"]
    counts = [-(-(c + new) // page) for c in ctx]
    num_pages, width = sum(counts) + 3, max(counts)
    order = torch.randperm(num_pages, generator=gen, device=DEVICE)
    cols = torch.arange(width, device=DEVICE)[None]
    counts_t = torch.tensor(counts, device=DEVICE)[:, None]
    first = torch.cumsum(counts_t, 0) - counts_t
    table = torch.where(cols < counts_t, order[(first + cols).clamp(max=num_pages - 1)], torch.full((), -1, device=DEVICE))
    s["block_table"] = table.to(torch.int32).contiguous()
    s["seqlens_k"] = _int32([c + new for c in ctx])
    s["cu_seqlens"] = _int32([i * new for i in range(batch + 1)])
    s["k_cache"] = _codes(gen, num_pages, hkv, page, d)
    s["k_scale"] = _scales(gen, num_pages, hkv)
    s["k_bounds"] = _all_bounds(s["k_cache"])
    # the pages that receive the new tokens still have the bounds of the step before: of none here
    at = torch.arange(width, device=DEVICE)[None]
    old = torch.tensor(ctx, device=DEVICE)[:, None] // page
    stale = table[(at >= old) & (at < counts_t)]
    s["k_bounds"].view(torch.uint8)[stale] = 0
    s["q"] = _normal(gen, batch * new, hq, d)
    s["lists"] = torch.empty(batch * new, hkv, case["top"], dtype=torch.int32, device=DEVICE)
    s["list_lens"] = torch.empty(batch * new, dtype=torch.int32, device=DEVICE)


def _prepare_lists(case, gen, s):
    page, top, pool, tokens = case["page"], case["top"], case["pool"], case["tokens"]
    hq, hkv, dq, dv = case["heads_q"], case["heads_kv"], case["d_qk"], case["d_v"]
    s["k_cache"], s["v_cache"] = _codes(gen, pool, hkv, page, dq), _codes(gen, pool, hkv, page, dv)
    s["k_scale"], s["v_scale"] = _scales(gen, pool, hkv), _scales(gen, pool, hkv)
    lens = _list_lengths(case)
    s["list_lens"] = _int32(lens)
    lists = torch.rand(tokens * hkv, pool, generator=gen, device=DEVICE).argsort(1)[:, :top].view(tokens, hkv, top)
    used = (s["list_lens"].long() + page - 1) // page
    keep = torch.arange(top, device=DEVICE)[None] < used[:, None]
    s["lists"] = torch.where(keep[:, None], lists, torch.full((), -1, device=DEVICE)).to(torch.int32).contiguous()
    s["q"] = _normal(gen, tokens, hq, dq)
    s["out"] = torch.empty(tokens, hq, dv, dtype=torch.bfloat16, device=DEVICE)
    s["lse"] = torch.empty(hq, tokens, dtype=torch.float32, device=DEVICE)


def _prepare_pool(case, gen, s):
    table, lens, num_pages, parents, grow = _rows(case)
    page, hkv, batch = case["page"], case["heads_kv"], len(lens)
    width = max([1] + [-(-(n + max(grow)) // page) for n in lens] + [-(-g // page) for g in grow])
    # which page is which differs from run to run
    name = torch.randperm(num_pages, generator=gen, device=DEVICE)
    rows = torch.tensor([row + [-1] * (width - len(row)) for row in table], device=DEVICE).view(batch, width)
    rows = torch.where(rows >= 0, name[rows.clamp(min=0)], rows)
    s["block_table"] = rows.to(torch.int32)
    s["seqlens_k"] = _int32(lens)
    s["page_refs"] = torch.bincount(rows[rows >= 0], minlength=num_pages).to(torch.int32)
    s["k_cache"] = _codes(gen, num_pages, hkv, page, case["d_qk"])
    s["v_cache"] = _codes(gen, num_pages, hkv, page, case["d_v"])
    s["k_scale"], s["v_scale"] = _scales(gen, num_pages, hkv), _scales(gen, num_pages, hkv)
    s["k_bounds"] = _all_bounds(s["k_cache"])
    s["parents"], s["new_tokens"] = _int32(parents), _int32(grow)
    s["table_out"] = torch.empty_like(s["block_table"])
    s["seqlens_out"] = torch.empty_like(s["seqlens_k"])
    s["refs_out"], s["page_map"] = torch.empty_like(s["page_refs"]), torch.empty_like(s["page_refs"])
    s["used"] = torch.empty(1, dtype=torch.int32, device=DEVICE)


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"table": _own_table, "rotate": _own_rotate, "select": _own_select, "lists": _own_lists, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"table": _plain_table, "rotate": _plain_rotate, "select": _plain_select, "lists": _plain_lists,
            "fork": _plain_fork, "compact": _plain_compact}[op](state)


def _pool(s):
    return {name: s[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale", "k_bounds")}


def _own_table(s):
    import exact_attention_forward_08_gb300 as fa

    c = s["case"]
    return fa.rotary_table(c["positions"], c["rot"], base=s["base"], scaling=c["scaling"], factor=c["factor"],
                           original=c["original"], low=c["low"], high=c["high"], magnitude=c["magnitude"], out=s["out"])


def _own_rotate(s):
    import exact_attention_forward_08_gb300 as fa

    call = fa.rotary_backward if s["case"]["backward"] else fa.rotary
    q, k = call(s["q"], s["k"], s["cos_sin"], positions=s["positions"], cu_seqlens=s["cu_seqlens"],
                interleaved=s["case"]["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": q, "k": k}


def _own_select(s):
    import exact_attention_forward_08_gb300 as fa

    c = s["case"]
    fa.kv_bounds(s["k_cache"], s["k_bounds"], s["block_table"], s["seqlens_k"], s["cu_seqlens"],
                 s["q"].shape[0])
    lists, lens = fa.kv_select(s["q"], s["k_bounds"], s["k_scale"], s["block_table"], s["seqlens_k"], s["cu_seqlens"],
                               c["new"], c["page"], c["top"], keep_first=c["first"], keep_last=c["last"],
                               lists=s["lists"], list_lens=s["list_lens"])
    return {"lists": lists, "list_lens": lens, "k_bounds": s["k_bounds"]}


def _own_lists(s):
    import exact_attention_forward_08_gb300 as fa

    o, lse = fa.attention_forward_lists(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["lists"],
                                        s["list_lens"], out=s["out"], lse=s["lse"])
    return {"o": o, "lse": lse}


def _own_fork(s):
    import exact_attention_forward_08_gb300 as fa

    table, lens, refs = fa.kv_fork(s["parents"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                   s["seqlens_k"], s["page_refs"], new_tokens=s["new_tokens"], k_bounds=s["k_bounds"],
                                   table_out=s["table_out"], seqlens_out=s["seqlens_out"], refs_out=s["refs_out"])
    return {"table": table, "seqlens": lens, "refs": refs, **_pool(s)}


def _own_compact(s):
    import exact_attention_forward_08_gb300 as fa

    table, refs, page_map, used = fa.kv_compact(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                                s["seqlens_k"], s["page_refs"], k_bounds=s["k_bounds"],
                                                table_out=s["table_out"], refs_out=s["refs_out"], page_map=s["page_map"],
                                                used=s["used"])
    return {"table": table, "refs": refs, "page_map": page_map, "used": used, **_pool(s)}


def _plain_table(s):
    c = s["case"]
    rot, factor, base = c["rot"], c["factor"], s["base"]
    if c["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    freq = torch.pow(base, -torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    if c["scaling"] == "linear":
        freq = freq / factor
    elif c["scaling"] == "by_parts":
        # pairs that turn more than `high` times within the trained length stay, those below `low` are slowed down
        turns = c["original"] * freq / (2 * math.pi)
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
    angle = torch.arange(c["positions"], dtype=torch.float64, device=DEVICE)[:, None] * freq
    s["out"].copy_(torch.cat([angle.cos(), angle.sin()], 1) * c["magnitude"])
    return s["out"]


def _plain_rotate(s):
    c = s["case"]
    rot = c["rot"]
    pos = s["positions"]
    if pos is None:
        cu = s["cu_seqlens"].long()
        t = torch.arange(s["q"].shape[0], device=cu.device)
        pos = t - cu[torch.searchsorted(cu, t, right=True) - 1]
    cos, sin = s["cos_sin"][pos.long()].chunk(2, 1)
    cos, sin = cos[:, None], -sin[:, None] if c["backward"] else sin[:, None]

    def turn(x):
        x = x.float()
        head, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = head.chunk(2, -1)
            head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([head, rest], -1)

    s["q_out"].copy_(turn(s["q"]))
    s["k_out"].copy_(turn(s["k"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_select(s):
    c = s["case"]
    page, new, top, hkv = c["page"], c["new"], c["top"], c["heads_kv"]
    table, lens = s["block_table"].long(), s["seqlens_k"].long()
    batch, width = table.shape
    # the bounds of the pages that hold new tokens, over the tokens that are there
    span = (new - 1) // page + 2  # pages that `new` tokens can touch
    j = (lens - new)[:, None] // page + torch.arange(span, device=table.device)
    last = (lens[:, None] - 1) // page
    j = torch.minimum(j, last)  # a page named twice is written twice alike
    ids = table.gather(1, j)
    codes = s["k_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()  # [batch, span, heads, page, d]
    there = torch.arange(page, device=table.device) < (lens[:, None] - j * page)[..., None]
    there = there[:, :, None, :, None]
    hi = torch.where(there, codes, torch.full((), -math.inf, device=codes.device)).amax(3)
    lo = torch.where(there, codes, torch.full((), math.inf, device=codes.device)).amin(3)
    s["k_bounds"].view(torch.uint8)[ids] = torch.stack([hi, lo], 3).to(torch.float8_e4m3fn).view(torch.uint8)
    # the sum of the query heads' bounds, in 64 bits: pages next to each other must fall on the right side
    bounds = s["k_bounds"].view(torch.uint8)[table.clamp(min=0)].view(torch.float8_e4m3fn).double()
    bounds *= torch.exp2(s["k_scale"].view(torch.uint8)[table.clamp(min=0)].double() - 127)[..., None, None]
    bounds = bounds.permute(0, 2, 1, 3, 4).flatten(3)  # [batch, heads, width, 2 d]
    q = s["q"].double().view(batch, new, hkv, -1, c["d_qk"])
    q = torch.cat([q.clamp(min=0).sum(3), q.clamp(max=0).sum(3)], -1).transpose(1, 2)  # [batch, heads, new, 2 d]
    scores = torch.matmul(q, bounds.transpose(2, 3))
    # what a token may see
    seen = lens[:, None] - new + torch.arange(1, new + 1, device=table.device)
    pages = (seen + page - 1) // page
    at = torch.arange(width, device=table.device)
    kept = (at < c["first"]) | (at >= (pages - c["last"])[..., None])
    scores = torch.where(kept[:, None], torch.full((), math.inf, device=scores.device, dtype=torch.float64), scores)
    scores = torch.where((at < pages[..., None])[:, None], scores, torch.full_like(scores, -math.inf))
    chosen = scores.sort(dim=-1, descending=True, stable=True)[1][..., :top]
    count = pages.clamp(max=top)
    behind = torch.arange(chosen.shape[-1], device=table.device) >= count[..., None]
    chosen = torch.where(behind[:, None], torch.full((), width, device=table.device), chosen).sort(-1)[0]
    listed_pages = table[:, None, None].expand(-1, hkv, new, -1).gather(3, chosen.clamp(max=width - 1))
    s["lists"].fill_(-1)
    s["lists"][..., :chosen.shape[-1]].copy_(torch.where(behind[:, None], torch.full((), -1, device=table.device),
                                                         listed_pages).transpose(1, 2).flatten(0, 1))
    s["list_lens"].copy_(((count - 1) * page + seen - (pages - 1) * page).flatten())
    return {"lists": s["lists"], "list_lens": s["list_lens"], "k_bounds": s["k_bounds"]}


def _plain_lists(s):
    c = s["case"]
    hkv, page = c["heads_kv"], c["page"]
    lists, lens = s["lists"].long().clamp(min=0), s["list_lens"].long()
    tokens = len(lens)
    heads = torch.arange(hkv, device=lens.device)[None, :, None]

    def dense(cache, scale):  # [tokens, heads, top * page, d]
        x = cache.view(torch.uint8)[lists, heads].view(torch.float8_e4m3fn).float()
        x *= torch.exp2(scale.view(torch.uint8)[lists, heads].float() - 127)[..., None, None]
        return x.flatten(2, 3)

    k, v = dense(s["k_cache"], s["k_scale"]), dense(s["v_cache"], s["v_scale"])
    q = s["q"].float().view(tokens, hkv, -1, c["d_qk"])
    scores = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(c["d_qk"]))
    hidden = torch.arange(k.shape[2], device=lens.device) >= lens[:, None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    best = scores.amax(-1, keepdim=True)
    scores = (scores - best).exp()
    total = scores.sum(-1, keepdim=True)
    s["out"].copy_((torch.matmul(scores, v) / total).view(s["out"].shape))
    s["lse"].copy_((best + total.log()).view(tokens, -1).t())
    return {"o": s["out"], "lse": s["lse"]}


def _plain_fork(s):
    page = s["case"]["page"]
    table, lens, parents = s["block_table"].long(), s["seqlens_k"].long(), s["parents"].long()
    batch, width = table.shape
    rows, cols = torch.arange(batch, device=table.device), torch.arange(width, device=table.device)[None]
    taken = parents >= 0
    source = parents.clamp(min=0)
    # heirs of each old row, the first of them
    heirs = torch.zeros_like(lens).scatter_add_(0, source, taken.long())
    first = torch.full_like(lens, batch).scatter_reduce_(0, source, torch.where(taken, rows, batch), "amin")
    # counts of uses: full pages by heirs, a page that is partly filled stays with one of them
    full, part = lens // page, lens % page
    change = torch.where(cols < full[:, None], heirs[:, None] - 1, torch.zeros_like(cols))
    change = torch.where((cols == full[:, None]) & (part > 0)[:, None], (heirs > 0).long()[:, None] - 1, change)
    refs = s["page_refs"].long().scatter_add(0, table.clamp(min=0).flatten(), change.flatten())
    # new pages: the lowest free ones, row by row
    old = torch.where(taken, lens[source], torch.zeros_like(lens))
    held = (old + page - 1) // page
    copies = taken & (old % page > 0) & (first[source] != rows)
    length = old + s["new_tokens"].long()
    total = (length + page - 1) // page
    need = total - held + copies.long()
    start = torch.cumsum(need, 0) - need
    free = (refs > 0).long().sort(dim=-1, stable=True)[1]
    behind = torch.cumsum(need, 0)[-1]  # a free page that nobody gets
    kept = held - copies.long()  # entries that come from the parent
    fresh = free[(start[:, None] + cols - kept[:, None]).clamp(0, len(refs) - 1)]
    is_fresh = (cols >= kept[:, None]) & (cols < total[:, None])
    out = torch.where(is_fresh, fresh, torch.where(cols < kept[:, None], table[source], torch.full_like(fresh, -1)))
    refs = refs.scatter_add(0, fresh.flatten(), is_fresh.long().flatten())
    s["table_out"].copy_(out)
    s["seqlens_out"].copy_(length)
    s["refs_out"].copy_(refs)
    # the tokens of pages that are partly filled
    src = torch.where(copies, table[source, (held - 1).clamp(min=0)], free[behind])
    dst = torch.where(copies, free[start.clamp(max=len(refs) - 1)], free[behind])
    inside = (torch.arange(page, device=table.device)[None] < (old % page)[:, None])[:, None, :, None]
    k, v = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    k[dst] = torch.where(inside & copies[:, None, None, None], k[src], k[dst])
    v[dst] = torch.where(inside & copies[:, None, None, None], v[src], v[dst])
    k_scale, v_scale, bounds = (s[name].view(torch.uint8) for name in ("k_scale", "v_scale", "k_bounds"))
    k_scale[dst], v_scale[dst], bounds[dst] = k_scale[src], v_scale[src], bounds[src]
    return {"table": s["table_out"], "seqlens": s["seqlens_out"], "refs": s["refs_out"], **_pool(s)}


def _plain_compact(s):
    page = s["case"]["page"]
    refs, table, lens = s["page_refs"].long(), s["block_table"].long(), s["seqlens_k"].long()
    used = refs > 0
    count = used.sum()
    at = torch.arange(len(refs), device=refs.device)
    # pages in use behind the first `count` go to the holes among these, in order
    moves, hole = used & (at >= count), ~used & (at < count)
    holes, movers = (~hole).long().sort(dim=-1, stable=True)[1], (~moves).long().sort(dim=-1, stable=True)[1]
    new = torch.where(moves, holes[(torch.cumsum(moves, 0) - 1).clamp(min=0)], at)
    source = torch.where(hole, movers[(torch.cumsum(hole, 0) - 1).clamp(min=0)], at)
    s["page_map"].copy_(torch.where(used, new, torch.full_like(new, -1)))
    s["refs_out"].copy_(torch.where(at < count, refs[source], torch.zeros_like(refs)))
    s["used"].copy_(count)
    live = torch.arange(table.shape[1], device=refs.device)[None] < ((lens + page - 1) // page)[:, None]
    s["table_out"].copy_(torch.where(live, new[table.clamp(min=0)], torch.full_like(table, -1)))
    k, v, k_scale, v_scale, bounds = (x.view(torch.uint8) for x in _pool(s).values())
    k.copy_(k[source])
    v.copy_(v[source])
    k_scale.copy_(k_scale[source])
    v_scale.copy_(v_scale[source])
    bounds.copy_(bounds[source])
    return {"table": s["table_out"], "refs": s["refs_out"], "page_map": s["page_map"], "used": s["used"], **_pool(s)}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one row after the other
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "rotate": _exact_rotate, "select": _exact_select, "lists": _exact_lists,
            "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)


def _exact_table(s):
    c = s["case"]
    half = c["rot"] // 2
    freq = []
    for i in range(half):
        base = s["base"]
        if c["scaling"] == "base":
            base *= math.pow(c["factor"], c["rot"] / (c["rot"] - 2.0))
        f = math.pow(base, -i / half)
        if c["scaling"] == "linear":
            f /= c["factor"]
        if c["scaling"] == "by_parts":
            keep = (c["original"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])
            keep = min(1.0, max(0.0, keep))
            f = keep * f + (1 - keep) * f / c["factor"]
        freq.append(f)
    at = torch.arange(c["positions"], dtype=torch.float64, device=DEVICE)
    angle = torch.outer(at, torch.tensor(freq, dtype=torch.float64, device=DEVICE))
    return c["magnitude"] * torch.hstack([torch.cos(angle), torch.sin(angle)])


def _exact_rotate(s):
    c = s["case"]
    rot = c["rot"]
    where = [] if s["positions"] is None else s["positions"].tolist()
    if s["positions"] is None:
        for n in _new_tokens(c):
            where += range(n)
    cs = s["cos_sin"].double()[torch.tensor(where, device=DEVICE)][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    first = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
    out = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        a, b = x[..., first].clone(), x[..., second].clone()
        if c["backward"]:
            x[..., first], x[..., second] = a * cos + b * sin, b * cos - a * sin
        else:
            x[..., first], x[..., second] = a * cos - b * sin, b * cos + a * sin
        out[name] = x
    return out


def _exact_select(s):
    c = s["case"]
    page, new, top, hkv = c["page"], c["new"], c["top"], c["heads_kv"]
    table = s["block_table"].tolist()
    codes = s["k_cache"].view(torch.uint8)
    bounds, scale = s["k_bounds"].float().double(), s["k_scale"].float().double()
    lists = torch.full((len(table) * new, hkv, top), -1, dtype=torch.int64)
    lens = torch.zeros(len(table) * new, dtype=torch.int64)
    for b, ctx in enumerate(_contexts(c)):
        for j in range(ctx // page, (ctx + new - 1) // page + 1):
            tokens = codes[table[b][j], :, :min(page, ctx + new - j * page)].view(torch.float8_e4m3fn).float().double()
            bounds[table[b][j], :, 0], bounds[table[b][j], :, 1] = tokens.max(1)[0], tokens.min(1)[0]
        for i in range(new):
            seen = ctx + i + 1
            count = -(-seen // page)
            ids = torch.tensor(table[b][:count], device=DEVICE)
            q = s["q"][b * new + i].double().view(hkv, 1, -1, c["d_qk"])
            hi = (bounds[ids, :, 0] * scale[ids][..., None]).transpose(0, 1)[:, :, None]
            lo = (bounds[ids, :, 1] * scale[ids][..., None]).transpose(0, 1)[:, :, None]
            rate = torch.maximum(q * hi, q * lo).sum((2, 3)).cpu().numpy()  # [heads, pages]
            for h in range(hkv):
                order = sorted(range(count), key=lambda j: (not (j < c["first"] or j >= count - c["last"]), -rate[h][j], j))
                chosen = sorted(order[:top])
                lists[b * new + i, h, :len(chosen)] = torch.tensor([table[b][j] for j in chosen])
            lens[b * new + i] = seen - (count - min(count, top)) * page
    return {"lists": lists, "list_lens": lens, "k_bounds": bounds}


def _exact_lists(s):
    c = s["case"]
    hkv, ratio, page = c["heads_kv"], c["heads_q"] // c["heads_kv"], c["page"]
    q = s["q"].double() / math.sqrt(c["d_qk"])
    o = torch.empty(*q.shape[:2], c["d_v"], dtype=torch.float64, device=DEVICE)
    lse = torch.empty(c["heads_q"], q.shape[0], dtype=torch.float64, device=DEVICE)
    lists = s["lists"].cpu()
    for t, n in enumerate(_list_lengths(c)):
        for h in range(hkv):
            ids = lists[t, h, :-(-n // page)].long().to(DEVICE)
            parts = []
            for name in ("k", "v"):
                x = s[name + "_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).float().double()
                parts.append((x * s[name + "_scale"].float().double()[ids, h][:, None, None]).flatten(0, 1)[:n])
            mine = slice(h * ratio, (h + 1) * ratio)
            scores = q[t, mine] @ parts[0].t()
            l = torch.logsumexp(scores, 1)
            o[t, mine] = torch.exp(scores - l[:, None]) @ parts[1]
            lse[mine, t] = l
    return {"o": o, "lse": lse}


def _values(s):
    return {name: x.float().double() for name, x in _pool(s).items()}


def _exact_fork(s):
    page = s["case"]["page"]
    table, lens, refs = s["block_table"].tolist(), s["seqlens_k"].tolist(), s["page_refs"].tolist()
    parents, grow = s["parents"].tolist(), s["new_tokens"].tolist()
    pool = _values(s)
    out = [[-1] * len(table[0]) for _ in table]
    heirs = [[b for b, p in enumerate(parents) if p == a] for a in range(len(table))]
    for a, row in enumerate(table):  # the old rows go, the new ones come
        for j in range(-(-lens[a] // page)):
            whole = (j + 1) * page <= lens[a]
            refs[row[j]] += len(heirs[a]) - 1 if whole else min(len(heirs[a]), 1) - 1
    free = (p for p, r in enumerate(list(refs)) if r == 0)
    new_lens = []
    for b, (a, g) in enumerate(zip(parents, grow)):
        old = lens[a] if a >= 0 else 0
        for j in range(-(-(old + g) // page)):
            if j < old // page or (j * page < old and heirs[a][0] == b):
                out[b][j] = table[a][j]
                continue
            out[b][j] = p = next(free)
            refs[p] = 1
            if j * page < old:
                for name, x in pool.items():
                    if name in ("k_cache", "v_cache"):
                        x[p, :, :old % page] = x[table[a][j], :, :old % page]
                    else:
                        x[p] = x[table[a][j]]
        new_lens.append(old + g)
    return {"table": torch.tensor(out), "seqlens": torch.tensor(new_lens), "refs": torch.tensor(refs), **pool}


def _exact_compact(s):
    page = s["case"]["page"]
    table, lens, refs = s["block_table"].tolist(), s["seqlens_k"].tolist(), s["page_refs"].tolist()
    pool = _values(s)
    used = sum(r > 0 for r in refs)
    page_map = [p if r > 0 else -1 for p, r in enumerate(refs)]
    holes = iter([p for p in range(used) if refs[p] == 0])
    for p in range(used, len(refs)):
        if refs[p] > 0:
            page_map[p] = to = next(holes)
            refs[to], refs[p] = refs[p], 0
            for x in pool.values():
                x[to] = x[p]
    out = [[page_map[p] if j * page < n else -1 for j, p in enumerate(row)] for row, n in zip(table, lens)]
    return {"table": torch.tensor(out), "refs": torch.tensor(refs), "page_map": torch.tensor(page_map),
            "used": torch.tensor([used]), **pool}
