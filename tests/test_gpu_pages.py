"""Forking, freeing, extending and compacting the paged cache's rows on the GPU: whole numbers and whole pages, equal to a
plain walk over the rows."""
import random

import pytest

torch = pytest.importorskip("torch")
import long_ref as want  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Rows of pages, some shared, in a pool of random bytes."""

    def __init__(self, lens, page, heads=2, d_qk=64, d_v=64, spare=5, width=None, share=(), layout="heads", seed=0):
        r = random.Random(seed)
        counts = [-(-n // page) for n in lens]
        self.width = width or max(counts + [1]) + 3
        self.num_pages = sum(counts) + spare
        order = list(range(self.num_pages))
        r.shuffle(order)
        self.table = [[order.pop() for _ in range(c)] for c in counts]
        for a, b, pages in share:  # row b begins with row a's first pages, full ones
            order += self.table[b][:pages]
            self.table[b][:pages] = self.table[a][:pages]
        self.refs = [0] * self.num_pages
        for row in self.table:
            for p in row:
                self.refs[p] += 1
        self.lens, self.page, self.heads, self.d = list(lens), page, heads, (d_qk, d_v)
        g = torch.Generator().manual_seed(seed)
        self.data = {n: torch.randint(0, 256, (self.num_pages, heads, page, d), generator=g, dtype=torch.uint8)
                     for n, d in zip("kv", self.d)}
        for n in ("ks", "vs"):
            self.data[n] = torch.randint(0, 255, (self.num_pages, heads), generator=g, dtype=torch.uint8)
        self.data["b"] = torch.randint(0, 256, (self.num_pages, heads, 2, d_qk), generator=g, dtype=torch.uint8)
        self.dev = {n: x.cuda() for n, x in self.data.items()}
        if layout == "tokens":
            for n in "kv":
                self.dev[n] = self.dev[n].transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "apart":
            for n in "kv":
                big = torch.zeros(self.num_pages, 2, *self.data[n].shape[1:], dtype=torch.uint8, device="cuda")
                big[:, 1] = self.dev[n]
                self.dev[n] = big[:, 1]
        self.block_table = int32([row + [-7] * (self.width - len(row)) for row in self.table]).view(len(lens), self.width)
        self.seqlens, self.page_refs = int32(self.lens), int32(self.refs)

    def cache(self):
        f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        d = self.dev
        return d["k"].view(f8), d["v"].view(f8), d["ks"].view(e8), d["vs"].view(e8)

    def bounds(self):
        return self.dev["b"].view(torch.float8_e4m3fn)

    def check_pages(self, copies, bounds=True):
        """Copies (from, to, tokens; all of a page if None), everything else as it was."""
        for a, b, tokens in copies:
            n = self.page if tokens is None else tokens
            for name in "kv":
                self.data[name][b, :, :n] = self.data[name][a, :, :n]
            for name in ("ks", "vs") + (("b",) if bounds else ()):
                self.data[name][b] = self.data[name][a]
        for name, x in self.data.items():
            assert torch.equal(self.dev[name].cpu(), x), name


def fork(fa, pool, parents, grow=None, bounds=True, **kw):
    args = (int32(parents), *pool.cache(), pool.block_table, pool.seqlens, pool.page_refs)
    got = fa.kv_fork(*args, new_tokens=None if grow is None else int32(grow), k_bounds=pool.bounds() if bounds else None, **kw)
    torch.cuda.synchronize()
    return got, fa.fa_device_status()


def check_fork(fa, pool, parents, grow=None, bounds=True, **kw):
    """Returns whether all rows found their pages."""
    (table, lens, refs), (code, detail) = fork(fa, pool, parents, grow, bounds, **kw)
    rows, out_lens, out_refs, copies = want.fork(pool.table, pool.lens, pool.refs, parents, grow or [0] * len(parents), pool.page,
                                                 pool.num_pages, pool.width)
    assert table.cpu().tolist() == rows
    assert lens.tolist() == out_lens
    assert refs.tolist() == out_refs
    pool.check_pages(copies, bounds)
    if code == 0:
        return True
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 515, (code, detail)
    missing = [r for r, (a, n) in enumerate(zip(parents, out_lens)) if n == 0 and (pool.lens[a] if a >= 0 else 0) + (grow or [0] * len(parents))[r] > 0]
    assert detail[2] == missing[0]
    return False


DIMS = [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)]


@pytest.mark.parametrize("layout", ["heads", "tokens", "apart"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dims", DIMS)
def test_fork_copies_what_is_partly_filled(fa, dims, page, layout):
    """Every fill of the last page's rows from 1 on; full and empty rows; rows of no heir, of one and of four."""
    lens = [0, 1, page - 1, page, page + 1, 3 * page, 2 * page + 7, 5]
    parents = [1, 2, 2, 2, 3, 3, 4, 6, 6, 6, 6, 0, 0, -1, 5]
    pool = Pool(lens, page, 3, *dims, spare=30, layout=layout)
    assert check_fork(fa, pool, parents)


@pytest.mark.parametrize("bounds", [True, False])
@pytest.mark.parametrize("seed", range(12))
def test_fork_at_random(fa, seed, bounds):
    """Beams, ends, beginnings and growth by nothing, a token or pages, over rows that share their prompts."""
    r = random.Random(seed)
    page = r.choice([16, 32, 64])
    batch = r.choice([1, 2, 7, 40, 130])
    common = r.randint(0, 4)
    lens = [r.choice([0, r.randint(1, 300), common * page + r.randint(0, 200)]) for _ in range(batch)]
    share = [(0, b, common) for b in range(1, batch) if lens[0] >= common * page and lens[b] >= common * page and r.random() < 0.7]
    pool = Pool(lens, page, r.choice([1, 4]), 64, 64, spare=r.choice([400, 3000]), width=60, share=share if common else (), seed=seed)
    rows = r.choice([batch, r.randint(1, 2 * batch)])
    parents = [r.choice([-1, r.randrange(batch), min(i, batch - 1)]) for i in range(rows)]
    grow = None if seed % 3 == 0 else [r.choice([0, 1, 1, r.randint(0, 3 * page)]) for _ in range(rows)]
    assert check_fork(fa, pool, parents, grow, bounds) or pool.num_pages < 2000


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 8])
def test_fork_without_enough_pages(fa, spare):
    """Rows are served in order until one finds too few; that and later ones that need pages become empty and give back
    what they share, a first heir its partly filled page too."""
    lens = [40, 33, 16, 100, 5]
    pool = Pool(lens, 16, spare=spare, share=[(3, 0, 2)], width=12)
    parents = [0, 0, 1, 2, 3, 3, 4, 1, 2]
    grow = [0, 1, 0, 17, 0, 30, 20, 0, 0]
    check_fork(fa, pool, parents, grow)


def test_fork_of_many_rows_and_pages(fa):
    """More rows than a block has threads and more pages than the cluster has; pages freed by the call are used by it."""
    r = random.Random(5)
    lens = [r.randint(0, 60) for _ in range(2500)]
    pool = Pool(lens, 16, 1, 64, 64, spare=20000, width=8)
    parents = [r.choice([-1, r.randrange(2500), r.randrange(2500)]) for _ in range(2500)]
    assert check_fork(fa, pool, parents, [r.randint(0, 40) for _ in range(2500)])
    # 750 rows of 4 pages go: 3000 pages, of which 1500 rows want 4 each, or 750 do
    tight = Pool([16 * 4] * 1500, 16, 1, 64, 64, spare=0, width=8)
    assert not check_fork(fa, tight, [b if b % 2 else -1 for b in range(1500)], [64] * 1500)
    tight = Pool([16 * 4] * 1500, 16, 1, 64, 64, spare=0, width=8)
    assert check_fork(fa, tight, [b if b % 2 else -1 for b in range(1500)], [0 if b % 2 else 64 for b in range(1500)])


@pytest.mark.parametrize("spare", [3000, 9000, 20000])
def test_fork_of_the_largest_tables(fa, spare):
    """As many rows as a call takes, more than a block of the kernel can keep; with too few pages for all of them, and enough:
    the rows want 15323 new pages, and those without an heir free 10502."""
    r = random.Random(9)
    batch = 16384
    pool = Pool([r.randint(0, 30) for _ in range(batch)], 16, 1, 64, 64, spare=spare, width=5)
    parents = [r.choice([-1, r.randrange(batch), r.randrange(batch), b]) for b in range(batch)]
    grow = [r.randint(0, 20) for _ in range(batch)]
    assert check_fork(fa, pool, parents, grow) == (spare >= 15323 - 10502)


def test_fork_wants_more_pages_than_fit_32_bits(fa):
    """Rows that ask for 2^26 pages each, 40 of them: all fail but those before that fit."""
    pool = Pool([40, 20], 16, 1, 64, 64, spare=30, width=12)
    big = 1 << 26
    table = torch.full((2, big), -7, dtype=torch.int32, device="cuda")
    table[:, :12] = pool.block_table
    parents, grow = [0, 1] + [-1] * 40 + [0, 1], [3, 0] + [(big - 8) * 16] * 40 + [0, 5]
    rows = len(parents)
    out = torch.empty(rows, big, dtype=torch.int32, device="cuda")
    got, lens, refs = fa.kv_fork(int32(parents), *pool.cache(), table, pool.seqlens, pool.page_refs, new_tokens=int32(grow),
                                 k_bounds=pool.bounds(), table_out=out)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (515, 2)
    # rows 0 and 1 keep their pages; the 40 find too few, and so do the last two, which want a copy each
    assert lens.tolist() == [43, 20] + [0] * 42
    assert got[0, :3].tolist() == pool.table[0] and got[1, :2].tolist() == pool.table[1]
    assert (got[2:] == -1).all() and (got[:2, 3:] == -1).all()
    assert refs.tolist() == pool.refs
    pool.check_pages([])


def test_fork_into_given_tensors(fa):
    """Counts in place, a wider table's columns, other columns and rows as they were; workspace of any content."""
    pool = Pool([40, 33, 16, 100, 5], 16, spare=20)
    wide = torch.full((4, pool.width + 5), 77, dtype=torch.int32, device="cuda")
    lens = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fa_kv_pages_workspace_size(5, 3, pool.num_pages), dtype=torch.uint8, device="cuda").fill_(255)
    assert check_fork(fa, pool, [3, 0, 0], [1, 1, 1], table_out=wide[:3, 2:2 + pool.width], seqlens_out=lens[:3],
                      refs_out=pool.page_refs, workspace=ws)
    assert (wide[3] == 77).all() and (wide[:, :2] == 77).all() and (wide[:, 2 + pool.width:] == 77).all() and lens[3] == 77


@pytest.mark.parametrize("what,site,index", [("parent", 511, 2), ("parent below", 511, 2), ("grow", 511, 2), ("grow negative", 511, 2),
                                             ("grow most", 511, 2), ("length", 511, 1), ("length negative", 511, 1),
                                             ("page", 512, 1), ("page negative", 512, 1)])
def test_fork_with_numbers_out_of_range(fa, what, site, index):
    """The rows concerned become empty, the others are what they are without them."""
    lens = [40, 33, 16, 100, 5]
    pool = Pool(lens, 16, spare=20)
    parents, grow = [0, 0, 1, 3, 4], [0, 1, 0, 1, 30]
    plain_parents, plain_grow, plain_table = list(parents), list(grow), [list(row) for row in pool.table]
    plain_parents[2], plain_grow[2] = -1, 0
    if what.startswith("parent"):
        parents[2] = 5 if what == "parent" else -2 ** 31
    elif what.startswith("grow"):
        grow[2] = {"grow": pool.width * 16 - 33 + 1, "grow negative": -1, "grow most": 2 ** 31 - 1}[what]
    elif what.startswith("length"):
        pool.seqlens[1] = pool.width * 16 + 1 if what == "length" else -2 ** 31
    else:
        pool.block_table[1, 2] = pool.num_pages if what == "page" else -1
    (table, got, refs), (code, detail) = fork(fa, pool, parents, grow)
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == site, (code, detail)
    assert detail[2] == index or (site == 511 and detail[2] == 2)
    ex_lens = list(lens)
    ex_refs = list(pool.refs)
    if site == 512 or what.startswith("length"):  # the row's pages keep their counts
        for p in plain_table[1]:
            ex_refs[p] += 1
    rows, out_lens, out_refs, copies = want.fork(plain_table, ex_lens, ex_refs, plain_parents, plain_grow, 16, pool.num_pages, pool.width)
    assert table.cpu().tolist() == rows and got.tolist() == out_lens and refs.tolist() == out_refs
    pool.check_pages(copies)


def check_compact(fa, pool, bounds=True, **kw):
    got = fa.kv_compact(*pool.cache(), pool.block_table, pool.seqlens, pool.page_refs, k_bounds=pool.bounds() if bounds else None, **kw)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, (code, detail)
    table, refs, page_map, used = got
    rows, out_refs, out_map, count, moves = want.compact(pool.table, pool.lens, pool.refs, pool.page)
    assert table.cpu().tolist() == [row + [-1] * (pool.width - len(row)) for row in rows]
    assert refs.tolist() == out_refs and page_map.tolist() == out_map and used.tolist() == [count]
    pool.check_pages([(a, b, None) for a, b in moves], bounds)
    return moves


@pytest.mark.parametrize("layout", ["heads", "tokens", "apart"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dims", DIMS)
def test_compact_moves_pages(fa, dims, page, layout):
    pool = Pool([0, 1, page, 3 * page + 1, 40, 2 * page], page, 3, *dims, spare=12, layout=layout, share=[(3, 5, 2)])
    check_compact(fa, pool)


@pytest.mark.parametrize("rows,spare", [(1, 0), (1, 1), (1, 9000), (30, 0), (30, 7), (3000, 17000), (600, 3)])
def test_compact_of_any_fill(fa, rows, spare):
    r = random.Random(rows + spare)
    pool = Pool([r.randint(0, 60) for _ in range(rows)], 16, 1, 64, 64, spare=spare, seed=spare)
    check_compact(fa, pool, bounds=bool(spare))


def test_compact_without_rows_or_pages_in_use(fa):
    """Pages that only the counts know move too; nothing in use at all."""
    pool = Pool([50, 20], 16, spare=9)
    held = [p for p in range(pool.num_pages) if pool.refs[p] == 0][-2:]
    for p in held:
        pool.refs[p] = 3
        pool.page_refs[p] = 3
    check_compact(fa, pool)
    none = Pool([0, 0], 16, spare=20)
    none.page_refs[4] = none.refs[4] = -2  # counts below 0 are free
    moves = check_compact(fa, none)
    assert moves == []


def test_compact_of_pages_in_no_table(fa):
    pool = Pool([50, 20], 16, spare=9)
    held = [p for p in range(pool.num_pages) if pool.refs[p] == 0][1::2]
    for p in held:
        pool.refs[p] = 1
        pool.page_refs[p] = 1
    pool.table, pool.lens = [], []
    pool.block_table, pool.seqlens = pool.block_table[:0], pool.seqlens[:0]
    assert check_compact(fa, pool)


def test_compact_in_place(fa):
    pool = Pool([50, 20, 130], 16, spare=15, seed=3)
    table, refs = pool.block_table, pool.page_refs
    check_compact(fa, pool, table_out=table, refs_out=refs)
    # a second time nothing moves
    pool.table = [row[:-(-n // 16)] for row, n in zip(table.cpu().tolist(), pool.lens)]
    pool.refs = refs.tolist()
    assert check_compact(fa, pool, table_out=table, refs_out=refs) == []


@pytest.mark.parametrize("what,site", [("length", 511), ("length negative", 511), ("page", 512), ("free page", 512)])
def test_compact_with_numbers_out_of_range(fa, what, site):
    pool = Pool([50, 20, 130], 16, spare=15, seed=3)
    if what.startswith("length"):
        pool.seqlens[1] = pool.width * 16 + 1 if what == "length" else -1
    else:
        pool.block_table[1, 0] = -1 if what == "page" else pool.refs.index(0)
    got = fa.kv_compact(*pool.cache(), pool.block_table, pool.seqlens, pool.page_refs, k_bounds=pool.bounds())
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (site, 1)
    rows, refs, page_map, used, moves = want.compact(pool.table, pool.lens, pool.refs, 16)
    rows = [row + [-1] * (pool.width - len(row)) for row in rows]
    if site == 511:
        rows[1] = [-1] * pool.width
    else:
        rows[1][0] = -1
    assert got[0].cpu().tolist() == rows and got[1].tolist() == refs and got[2].tolist() == page_map
    pool.check_pages([(a, b, None) for a, b in moves])


def test_refused_tensors(fa):
    pool = Pool([50, 20, 130], 16, spare=15)
    k, v, ks, vs = pool.cache()
    i32 = dict(dtype=torch.int32, device="cuda")
    good = dict(parents=int32([0, 1]), k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=pool.block_table,
                seqlens_k=pool.seqlens, page_refs=pool.page_refs)
    shared = [dict(k_cache=k.float()), dict(k_cache=k[0]), dict(v_cache=v[1:]), dict(k_scale=ks[1:]), dict(v_scale=vs.float()),
              dict(block_table=pool.block_table.long()), dict(block_table=pool.block_table.t()), dict(block_table=pool.block_table[0]),
              dict(seqlens_k=pool.seqlens[1:]), dict(seqlens_k=pool.seqlens.cpu()), dict(page_refs=pool.page_refs[1:]),
              dict(page_refs=pool.page_refs.float()), dict(k_bounds=pool.bounds()[1:]), dict(k_bounds=pool.bounds().float()),
              dict(refs_out=torch.zeros(3, **i32)), dict(table_out=torch.zeros(2, 3, **i32)),
              dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))]
    for kw in shared + [dict(parents=int32([])), dict(parents=int32([[0]])), dict(parents=torch.zeros(2)), dict(new_tokens=int32([1])),
                        dict(seqlens_out=torch.zeros(3, **i32)), dict(parents=int32([0, 1, 2]), table_out=pool.block_table),
                        dict(parents=int32([0, 1, 2]), seqlens_out=pool.seqlens)]:
        with pytest.raises(fa.FaError):
            fa.kv_fork(**{**good, **kw})
    good.pop("parents")
    for kw in shared + [dict(page_map=pool.page_refs), dict(used=torch.zeros(2, **i32)), dict(page_map=torch.zeros(1, **i32))]:
        with pytest.raises(fa.FaError):
            fa.kv_compact(**{**good, **kw})
    assert fa.fa_device_status()[0] == 0
    pool.check_pages([])
