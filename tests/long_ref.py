"""Plain 64-bit implementations of the operators for long contexts over the paged 8-bit cache: rotary positions, bounds and
selection of pages, attention over lists of pages, and the pages' bookkeeping.

Elementary Python and torch on small CPU tensors; nothing here is shared with the library."""
import math

import torch

import paged_ref as ref


def frequencies(rot, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            w = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def turn(x, cos_sin, interleaved, backward=False):
    """(x rotated in 64 bits, the sum of its terms' sizes); x [tokens, heads, d], cos_sin [tokens, rot]."""
    rot = cos_sin.shape[1]
    x = x.double().cpu()
    cs = cos_sin.double().cpu()[:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:] * (-1 if backward else 1)
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first], size[..., second] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return y, size


def check_turned(got, want, size, what=""):
    """Three fp32 roundings of the terms, then half a step of bf16 (2^-8), or half its smallest."""
    bound = (want.abs() + size * 2.0 ** -22) * 2.0 ** -8 * ref.SLACK + size * 2.0 ** -22 + 2.0 ** -134
    err = (got.double().cpu() - want).abs()
    assert (err <= bound).all(), f"{what}: off by {(err / bound).max().item():.3f} of its bound"


def page_bounds(codes, tokens):
    """[heads, 2, d] of one page's [heads, page, d] codes over its first `tokens`."""
    x = codes.view(torch.uint8).view(torch.float8_e4m3fn).float()[:, :tokens]
    return torch.stack([x.amax(1), x.amin(1)], 1)  # NaN where one is


def all_bounds(cache):
    """k_bounds of a paged_ref.Cache over the tokens that its sequences hold, zeros elsewhere."""
    out = torch.zeros(cache.num_pages, cache.heads, 2, cache.d_qk)
    for b, n in enumerate(cache.lens):
        for j in range(-(-n // cache.page)):
            p = int(cache.table[b, j])
            out[p] = page_bounds(cache.k[p], min(cache.page, n - j * cache.page))
    return out.to(torch.float8_e4m3fn)


def select(q, bounds, scale, table, lens, cu, page, top, causal=True, first=0, last=1):
    """(lists, list_lens) by the definition, -2 in rows of no sequence."""
    total, heads_q, d = q.shape
    heads = bounds.shape[1]
    values, sc = bounds.float().double(), ref.scale_values(scale)
    lists = torch.full((total, heads, top), -2, dtype=torch.int64)
    out_lens = torch.full((total,), -2, dtype=torch.int64)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t = cu[b] + i
            seen = max(length - n + i + 1, 0) if causal else length
            pages = -(-seen // page)
            count = min(pages, top)
            lists[t] = -1
            out_lens[t] = seen - (pages - count) * page
            ids = table[b, :pages].long()
            for h in range(heads):
                g = q[t].double().view(heads, -1, 1, d)[h]                      # [ratio, 1, d]
                hi, lo = (values[ids, h, x] * sc[ids, h][:, None] for x in (0, 1))
                terms = torch.maximum(g * hi, g * lo)
                terms = torch.where(torch.isnan(g * hi) | torch.isnan(g * lo), math.nan, terms)
                score = terms.sum((0, 2)).nan_to_num(nan=math.inf, posinf=math.inf, neginf=-math.inf).tolist()
                order = sorted(range(pages), key=lambda j: (0 if j < first or j >= pages - last else 1, -score[j], j))
                chosen = sorted(order[:count])
                lists[t, h, :count] = torch.tensor([int(ids[j]) for j in chosen], dtype=torch.int64)
    return lists, out_lens


def lists_attention(q, cache, lists, lens, scale=None):
    """What paged_ref.attention returns, each token over its own lists."""
    total, heads_q, d = q.shape
    heads, dv = cache.heads, cache.d_v
    ratio = heads_q // heads
    parts = [torch.zeros(total, heads_q, dv, dtype=torch.float64), torch.full((heads_q, total), -math.inf, dtype=torch.float64),
             torch.zeros(total, heads_q, dv, dtype=torch.float64), torch.zeros(total, heads_q, dtype=torch.float64),
             torch.zeros(total, dtype=torch.float64)]
    q, lists = q.cpu(), lists.cpu()
    for t in range(total):
        for h in range(heads):
            mine = slice(h * ratio, (h + 1) * ratio)
            got = ref.attention(q[t:t + 1, mine], cache.k[:, h:h + 1], cache.v[:, h:h + 1], cache.k_scale[:, h:h + 1],
                                cache.v_scale[:, h:h + 1], lists[t, h][None], [int(lens[t])], [0, 1], cache.page, False, scale)
            parts[0][t, mine], parts[1][mine, t], parts[2][t, mine], parts[3][t, mine] = got[0][0], got[1][:, 0], got[2][0], got[3][0]
            parts[4][t] = got[4][0]
    return tuple(parts)


def fork(table, lens, refs, parents, grow, page, num_pages, width):
    """(rows, lengths, counts, copies (from, to, tokens)): lists of Python numbers; rows that find no page become empty."""
    refs = list(refs)
    heirs = [[] for _ in table]
    for r, a in enumerate(parents):
        if a >= 0:
            heirs[a].append(r)
    for b, row in enumerate(table):
        for j in range(-(-lens[b] // page)):
            refs[row[j]] += len(heirs[b]) - 1 if (j + 1) * page <= lens[b] else min(len(heirs[b]), 1) - 1
    free = [p for p in range(num_pages) if refs[p] <= 0]
    rows, out_lens, copies, undo, at = [], [], [], [], 0
    for r, (a, g) in enumerate(zip(parents, grow)):
        old = lens[a] if a >= 0 else 0
        copy = a >= 0 and old % page != 0 and heirs[a][0] != r
        kept = -(-old // page) - copy
        fresh = -(-(old + g) // page) - kept
        fails = fresh > 0 and at + fresh > len(free)
        mine = free[at:at + fresh]
        at += fresh
        if fails:
            undo += [table[a][j] for j in range(kept) if (j + 1) * page <= old or heirs[a][0] == r]
            rows.append([-1] * width)
            out_lens.append(0)
            continue
        if copy:
            copies.append((table[a][kept], mine[0], old % page))
        for p in mine:
            refs[p] = 1
        rows.append(([table[a][j] for j in range(kept)] + mine + [-1] * width)[:width])
        out_lens.append(old + g)
    for p in undo:
        refs[p] -= 1
    return rows, out_lens, refs, copies


def compact(table, lens, refs, page):
    """(rows, counts, page_map, used, moves)."""
    refs = list(refs)
    used = sum(r > 0 for r in refs)
    page_map = [p if r > 0 else -1 for p, r in enumerate(refs)]
    moves = list(zip([p for p in range(used, len(refs)) if refs[p] > 0], [p for p in range(used) if refs[p] <= 0]))
    for p, to in moves:
        page_map[p] = to
        refs[to], refs[p] = refs[p], 0
    refs = [r if i < used else 0 for i, r in enumerate(refs)]
    rows = [[page_map[p] if j * page < n else -1 for j, p in enumerate(row)] for row, n in zip(table, lens)]
    return rows, refs, page_map, used, moves
