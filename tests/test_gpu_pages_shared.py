"""Forks of rows whose last page, partly filled, has other holders: a second row, a row that goes on behind it, a holder that
only the counts know.  Whoever receives tokens has the page alone afterwards."""
import random

import pytest

torch = pytest.importorskip("torch")
import long_ref as want  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def walk(table, lens, refs, parents, grow, page, num_pages, width):
    """What long_ref.fork returns, from the definition for pages of any number of holders."""
    refs = list(refs)
    heirs = {b: [r for r, a in enumerate(parents) if a == b] for b in range(len(table))}
    ends, keeper = {}, {}
    for b, row in enumerate(table):
        for j in range(lens[b] // page):
            refs[row[j]] += len(heirs[b]) - 1
        if lens[b] % page:
            last = row[lens[b] // page]
            refs[last] -= 1
            ends.setdefault(last, []).extend(heirs[b])
    for last, rows in ends.items():
        if rows and refs[last] <= 0:
            keeper[last] = min(rows)
            refs[last] += 1
    free = [p for p in range(num_pages) if refs[p] <= 0]
    rows, out_lens, copies, undo, at = [], [], [], [], 0
    for r, (a, g) in enumerate(zip(parents, grow)):
        old = lens[a] if a >= 0 else 0
        mine = table[a][:old // page] if a >= 0 else []
        last = table[a][old // page] if old % page else None
        copy = last is not None and keeper.get(last) != r
        if last is not None and not copy:
            mine = mine + [last]
        fresh = -(-(old + g) // page) - len(mine)
        new = free[at:at + fresh]
        at += fresh
        if fresh > 0 and at > len(free):
            undo += mine
            rows.append([-1] * width)
            out_lens.append(0)
            continue
        if copy:
            copies.append((last, new[0], old % page))
        for p in new:
            refs[p] = 1
        rows.append((mine + new + [-1] * width)[:width])
        out_lens.append(old + g)
    for p in undo:
        refs[p] -= 1
    return rows, out_lens, refs, copies


def problem(seed, page=16, batch=None, tight=False, shared=True):
    """(Pool's arguments, outside holders, parents, new tokens): rows of which some end in pages of others."""
    r = random.Random(seed)
    batch = batch or r.choice([2, 3, 9, 40, 200])
    lens = [r.choice([0, 1, page, r.randint(1, 3 * page), r.randint(1, 150)]) for _ in range(batch)]
    share = []
    if shared:
        for b in range(1, batch):
            a = r.randrange(b)
            pages = min(-(-lens[a] // page), -(-lens[b] // page))
            if pages > 0 and r.random() < 0.7:
                share.append((a, b, pages))  # ends in a's page, full or not, or goes on behind it
    rows = r.choice([batch, r.randint(1, 2 * batch)])
    parents = [r.choice([-1, r.randrange(batch), min(i, batch - 1), min(i, batch - 1)]) for i in range(rows)]
    grow = [r.choice([0, 0, 1, 1, r.randint(0, 2 * page)]) for _ in range(rows)]
    kw = dict(lens=lens, page=page, heads=r.choice([1, 3]), spare=r.randint(0, batch) if tight else 12 * batch + 40, width=24,
              share=share, seed=seed)
    return kw, 0.3 if shared else 0.0, parents, grow, r


def make(kw, outside, r):
    from test_gpu_pages import Pool, int32

    pool = Pool(**kw)
    for row in pool.table:  # holders beside the table, of pages of any fill
        for p in row:
            if r.random() < outside:
                pool.refs[p] += r.randint(1, 2)
    pool.page_refs = int32(pool.refs)
    return pool


def check(fa, pool, parents, grow):
    """The call against the walk; returns the copies.  Rows out of pages are reported."""
    from test_gpu_pages import fork

    (table, lens, refs), (code, detail) = fork(fa, pool, parents, grow)
    rows, out_lens, out_refs, copies = walk(pool.table, pool.lens, pool.refs, parents, grow, pool.page, pool.num_pages, pool.width)
    assert table.cpu().tolist() == rows
    assert lens.tolist() == out_lens
    assert refs.tolist() == out_refs
    pool.check_pages(copies)
    lost = [r for r, a in enumerate(parents) if out_lens[r] == 0 and (pool.lens[a] if a >= 0 else 0) + grow[r] > 0]
    assert (code, detail[1:]) == (fa.FA_ERR_INVALID_ARG, (515, lost[0])) if lost else code == 0, (code, detail)
    for r, n in enumerate(out_lens):  # who may receive tokens in a page has it alone
        if n % pool.page:
            assert out_refs[rows[r][n // pool.page]] == 1
    return copies


@pytest.mark.parametrize("seed", range(20))
def test_the_walk_is_the_plain_one_without_other_holders(seed):
    kw, _, parents, grow, r = problem(seed, tight=seed % 2 == 0, shared=False)
    order, table, page = list(range(10000)), [], kw["page"]
    r.shuffle(order)
    for n in kw["lens"]:
        table.append([order.pop() for _ in range(-(-n // page))])
    pages = sorted(p for row in table for p in row)
    name = {p: i for i, p in enumerate(pages)}
    table = [[name[p] for p in row] for row in table]
    num = len(pages) + kw["spare"]
    refs = [1] * len(pages) + [0] * kw["spare"]
    args = (table, kw["lens"], refs, parents, grow, page, num, kw["width"])
    assert walk(*args) == want.fork(*args)


@gpu
def test_two_rows_that_end_in_one_page(fa):
    """Both go on: the first keeps the page, the other copies.  One ends: the other keeps it.  Both end: it is free."""
    kw = dict(lens=[40, 40], page=16, spare=6, width=6, share=[(0, 1, 3)])
    for parents, copied in (([0, 1], 1), ([1, 0], 1), ([1], 0), ([0, -1], 0), ([1, 1, 0], 2), ([-1], 0)):
        pool = make(kw, 0, random.Random(0))
        assert len(check(fa, pool, parents, [1] * len(parents))) == copied


@gpu
def test_rows_of_other_fills_in_one_page(fa):
    """A row's last page is inside another row, which goes on behind it, or is filled further by it."""
    for lens in ([40, 70], [70, 40], [37, 45], [33, 48]):
        for parents in ([0, 1], [1, 0], [0], [1], [0, 0, 1]):
            pool = make(dict(lens=lens, page=16, spare=9, width=8, share=[(0, 1, 3)]), 0, random.Random(0))
            check(fa, pool, parents, [2] * len(parents))


@gpu
def test_a_holder_beside_the_table(fa):
    """The page stays as it is: every heir copies it, once; the copy is the row's own from then on."""
    from test_gpu_pages import Pool, int32

    pool = Pool([40, 21], 16, spare=9, width=6)
    held = pool.table[0][2]
    pool.refs[held] += 1
    pool.page_refs = int32(pool.refs)
    first = check(fa, pool, [0, 0, 1], [1, 0, 1])
    assert [c[0] for c in first] == [held, held]
    pool = Pool([40], 16, spare=9, width=6)
    pool.refs[pool.table[0][2]] += 1
    pool.page_refs = int32(pool.refs)
    args = pool.cache()
    table, lens, refs = fa.kv_fork(int32([0]), *args, pool.block_table, pool.seqlens, pool.page_refs, new_tokens=int32([1]))
    again, lens2, refs2 = fa.kv_fork(int32([0]), *args, table, lens, refs, new_tokens=int32([1]))
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    assert torch.equal(again, table) and torch.equal(refs, refs2) and lens2.tolist() == [42]
    assert refs[pool.table[0][2]] == 1 and table[0, 2] != pool.table[0][2]


@gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("seed", range(16))
def test_shared_last_pages_at_random(fa, seed, page):
    """Trees of rows that end in one another's pages, and holders beside them; too few pages in half of the cases."""
    kw, outside, parents, grow, r = problem(seed, page, tight=seed % 2 == 1)
    check(fa, make(kw, outside, r), parents, grow)


@gpu
@pytest.mark.parametrize("batch", [3000, 16384])
def test_shared_last_pages_of_many_rows(fa, batch):
    """More rows than a block has threads, and than it keeps."""
    kw, outside, parents, grow, r = problem(batch, batch=batch)
    check(fa, make({**kw, "heads": 1, "spare": 4 * batch}, outside, r), parents, grow)


@gpu
def test_appends_leave_other_holders_alone(fa):
    """A prompt that a cache of prompts holds, its last page half full: two requests begin with it and append tokens whose
    scale makes older codes round again; the held pages keep every byte, and both see the prompt."""
    from test_gpu_pages import int32

    g = torch.Generator().manual_seed(0)
    pages, heads, page, d = 12, 2, 16, 64
    k, v = (torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((pages, heads), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2))
    pool = (k, v, ks, vs)
    table, lens, refs = int32([[-1] * 4]), int32([0]), int32([0] * pages)
    table, lens, refs = fa.kv_fork(int32([-1]), *pool, table, lens, refs, new_tokens=int32([24]))
    kn, vn = (torch.randn(24, heads, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    fa.kv_append(kn, vn, *pool, table, lens, int32([0, 24]))
    held = table[0, :2].long()
    refs[held] += 1  # the cache of prompts
    before = [t.view(torch.uint8)[held].clone() for t in pool]
    table, lens, refs = fa.kv_fork(int32([0, 0]), *pool, table, lens, refs, new_tokens=int32([3, 3]))
    kn, vn = (1000 * torch.randn(6, heads, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    fa.kv_append(kn, vn, *pool, table, lens, int32([0, 3, 6]))
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    for t, old in zip(pool, before):
        assert torch.equal(t.view(torch.uint8)[held], old)
    assert table[:, 0].tolist() == [int(held[0])] * 2 and len({int(held[1]), int(table[0, 1]), int(table[1, 1])}) == 3
    assert refs[held].tolist() == [3, 1]
