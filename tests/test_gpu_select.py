"""Bounds of pages and the selection of pages on the GPU: whole numbers, equal to the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
import long_ref as want  # noqa: E402
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status(fa):
    torch.cuda.synchronize()
    return fa.fa_device_status()


def as_values(t):
    return t.float().cpu()


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["heads", "tokens", "apart"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([17, 0, 64], [17, 0, 1]), ([300, 33, 129, 128], [1, 20, 129, 3]),
                                      ([700] * 3, [700, 1, 350])])
def test_bounds_of_touched_pages(fa, lens, new, d, page, layout):
    """Pages with new tokens get the bounds of all their tokens, codes behind them (NaN here) are not looked at; other
    pages keep theirs."""
    cache = ref.Cache(lens, 3, page, d, 64, seed=d + page, layout=layout)
    k, _, _, _, table, seqlens = cache.to_device("cuda")
    got = torch.full((cache.num_pages, 3, 2, d), 0x31, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    expect = got.float().cpu()
    full = want.all_bounds(cache).float()
    for b, (n, m) in enumerate(zip(lens, new)):
        for j in range((n - m) // page, -(-n // page) if m else 0):
            expect[int(cache.table[b, j])] = full[int(cache.table[b, j])]
    fa.kv_bounds(k, got, table, seqlens, int32(offsets(new)), sum(new))
    assert status(fa)[0] == 0
    assert torch.equal(as_values(got), expect)


def test_bounds_show_a_nan_code(fa):
    cache = ref.Cache([40], 2, 32, 64, 64)
    cache.k.view(torch.uint8)[int(cache.table[0, 0]), 1, 5, 9] = 0xFF
    k, _, _, _, table, seqlens = cache.to_device("cuda")
    got = torch.zeros(cache.num_pages, 2, 2, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    fa.kv_bounds(k, got, table, seqlens, int32([0, 40]), 40)
    assert status(fa)[0] == 0
    x = as_values(got)[int(cache.table[0, 0])]
    hit = torch.zeros(2, 2, 64, dtype=torch.bool)
    hit[1, :, 9] = True
    assert torch.isnan(x[hit]).all() and not torch.isnan(x[~hit]).any()


@pytest.mark.parametrize("what", ["length", "page", "offsets"])
def test_bounds_leave_out_what_is_bad(fa, what):
    lens, new = [40, 50, 60], [4, 5, 6]
    cache = ref.Cache(lens, 2, 16, 64, 64)
    k, _, _, _, table, seqlens = cache.to_device("cuda")
    cu, site = int32(offsets(new)), 511
    if what == "length":
        seqlens[1] = 2 ** 30
    elif what == "page":
        table[1, 3], site = cache.num_pages, 512
    else:
        cu[2] = 3
    got = torch.zeros(cache.num_pages, 2, 2, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    fa.kv_bounds(k, got, table, seqlens, cu, 15)
    code, detail = status(fa)
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (site, 1)
    if what != "offsets":
        full = want.all_bounds(cache).float()
        for b in (0, 2):
            p = int(cache.table[b, (lens[b] - 1) // 16])
            assert torch.equal(as_values(got)[p], full[p])


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def check(fa, q, bounds, scale, table, lens, new, page, top, causal=True, first=0, last=1, pad=0, **kw):
    """The call's lists against the definition's; `pad` rows behind the last sequence keep what they hold."""
    total, heads = sum(new) + pad, bounds.shape[1]
    q = torch.cat([q, normal(pad, *q.shape[1:])]) if pad else q
    got = torch.full((total, heads, top), -2, dtype=torch.int32, device="cuda")
    got_lens = torch.full((total,), -2, dtype=torch.int32, device="cuda")
    fa.kv_select(q.cuda(), bounds.cuda(), scale.cuda(), table.cuda(), int32(lens), int32(offsets(new)), max(max(new), 1), page, top,
                 causal=causal, keep_first=first, keep_last=last, lists=got, list_lens=got_lens, **kw)
    code, detail = status(fa)
    assert code == 0, (code, detail)
    lists, list_lens = want.select(q, bounds, scale, table, lens, offsets(new), page, top, causal, first, last)
    assert torch.equal(got_lens.long().cpu(), list_lens)
    assert torch.equal(got.long().cpu(), lists)
    return got, got_lens


@pytest.mark.parametrize("dims", [(1, 1, 64), (8, 2, 128), (6, 3, 192), (32, 1, 128), (40, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,new,top,first,last", [
    ([1], [1], 1, 0, 1), ([0, 5, 900], [0, 1, 1], 4, 0, 1), ([2000, 1500, 40], [1, 1, 1], 9, 2, 3),
    ([900, 3, 2500], [3, 3, 5], 6, 1, 1), ([700], [40], 5, 0, 2), ([3000], [1], 3, 1, 2), ([5, 700], [9, 2], 2, 0, 1)])
def test_selection(fa, lens, new, top, first, last, page, dims):
    """Single tokens, drafts, a chunk; lists longer than the sequence, all places taken by force, rows without a key."""
    hq, hkv, d = dims
    cache = ref.Cache(lens, hkv, page, d, 64, seed=page)
    q = normal(sum(new), hq, d, seed=hq)
    for causal in (True, False):
        check(fa, q, want.all_bounds(cache), cache.k_scale, cache.table, lens, new, page, top, causal, first, last, pad=2)


def wide(pages, heads, d, seed=0, scale=(-3, -1)):
    """Bounds, scales and a table of one sequence of many pages, without the cache behind them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(pages, heads, 2, d, generator=g) * 100
    x = torch.stack([x.amax(2), x.amin(2)], 2).to(torch.float8_e4m3fn)
    s = ref.e8m0(torch.randint(scale[0], scale[1], (pages, heads), generator=g))
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    return x, s, table


@pytest.mark.parametrize("pages,top", [(63, 10), (64, 63), (65, 8), (255, 30), (257, 256), (2000, 64), (4096, 17), (4097, 100),
                                       (9001, 2000)])
@pytest.mark.parametrize("n", [1, 2])
def test_selection_from_many_pages(fa, pages, top, n):
    bounds, scale, table = wide(pages, 2, 64, seed=pages)
    check(fa, normal(n, 6, 64, seed=top), bounds, scale, table, [pages * 16 - 3], [n], 16, top, first=1, last=2)


def test_selection_of_many_sequences(fa):
    """More sequences than a block looks at together, of all lengths, empty ones between them, rows of a wider table."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 400, (700,), generator=g).tolist()
    new = [min(n, 1) if b % 5 else 0 for b, n in enumerate(lens)]
    cache = ref.Cache(lens, 2, 16, 64, 64, width=40)
    table = torch.full((700, 50), 10 ** 9, dtype=torch.int32)
    table[:, :40] = cache.table
    got, _ = check(fa, normal(sum(new), 4, 64), want.all_bounds(cache), cache.k_scale, table[:, :40], lens, new, 16, 5)
    again = fa.kv_select(normal(sum(new), 4, 64).cuda(), want.all_bounds(cache).cuda(), cache.k_scale.cuda(), table.cuda()[:, :40],
                         int32(lens), int32(offsets(new)), 1, 16, 5)[0]
    assert torch.equal(again, got)


@pytest.mark.parametrize("lens,new,dims,page,top", [([3000], [2500], (2, 1, 64), 16, 9), ([900, 40, 700], [700, 40, 1], (4, 2, 128), 32, 5),
                                                    ([1500] * 12, [97] * 12, (3, 1, 192), 64, 3)])
def test_selection_for_prompts(fa, lens, new, dims, page, top):
    """Hundreds and thousands of new tokens: many blocks for the tokens of a tile, small blocks for the choice."""
    hq, hkv, d = dims
    cache = ref.Cache(lens, hkv, page, d, 64, seed=page)
    check(fa, normal(sum(new), hq, d, seed=hq), want.all_bounds(cache), cache.k_scale, cache.table, lens, new, page, top, first=1, pad=1)


def test_equal_scores_take_the_lowest_pages(fa):
    """All pages alike, pages alike in groups, and queries that are 0: only the order decides."""
    for groups in (1, 7, 300):
        bounds, scale, table = wide(300, 2, 64, seed=groups)
        alike = torch.arange(300) % groups
        bounds = bounds.view(torch.uint8)[alike].view(torch.float8_e4m3fn)
        scale = scale.view(torch.uint8)[alike].view(torch.float8_e8m0fnu)
        for q in (normal(1, 4, 64), torch.zeros(1, 4, 64, dtype=torch.bfloat16), -torch.zeros(1, 4, 64, dtype=torch.bfloat16)):
            check(fa, q, bounds, scale, table, [4800], [1], 16, 50)
            check(fa, q, bounds, scale, table, [4799], [1], 16, 50, first=3, last=4)


def test_equal_scores_among_more_pages_than_are_staged(fa):
    bounds, scale, table = wide(5000, 1, 64, seed=2)
    alike = torch.arange(5000) % 40
    bounds = bounds.view(torch.uint8)[alike].view(torch.float8_e4m3fn)
    scale = scale.view(torch.uint8)[alike].view(torch.float8_e8m0fnu)
    check(fa, normal(2, 4, 64), bounds, scale, table, [80000], [2], 16, 333, first=2, last=3)


@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -18, 2.0 ** -24, 2.0 ** -30])
def test_scores_that_fp32_cannot_tell_apart(fa, small):
    """Pages that differ in one channel only, whose query is smaller by 2^12 to 2^30 than the others."""
    bounds, scale, table = wide(500, 1, 128, seed=3)
    bounds = bounds.view(torch.uint8)[:1].repeat(500, 1, 1, 1).view(torch.float8_e4m3fn)
    scale = scale.view(torch.uint8)[:1].repeat(500, 1).view(torch.float8_e8m0fnu)
    values = bounds.float()
    values[:, 0, 0, 77] = torch.randint(1, 100, (500,), generator=torch.Generator().manual_seed(1)).float()
    values[:, 0, 1, 77] = 0
    q = normal(2, 3, 128)
    q[..., 77] = small
    check(fa, q, values.to(torch.float8_e4m3fn), scale, table, [7990], [2], 16, 40)


@pytest.mark.parametrize("spread", [(-63, 60), (-127, 128), (0, 1)])
@pytest.mark.parametrize("q_exp", [-126, 0, 120])
def test_scales_and_queries_at_the_ends_of_their_ranges(fa, spread, q_exp):
    bounds, scale, table = wide(400, 2, 64, seed=8, scale=spread)
    q = (normal(2, 4, 64).double() * 2.0 ** q_exp).to(torch.bfloat16)
    check(fa, q, bounds, scale, table, [6400], [2], 16, 37)


@pytest.mark.parametrize("q_exp", [-133, -120, -95, -90])
def test_queries_that_cannot_be_scaled_all_the_way(fa, q_exp):
    """Largest values down to bf16's smallest numbers, and rows of zeros beside them."""
    bounds, scale, table = wide(300, 2, 64, seed=9)
    q = (normal(3, 4, 64).double() * 2.0 ** q_exp).to(torch.bfloat16)
    q[1] = 0
    q[2, 0] = 0
    check(fa, q, bounds, scale, table, [4800], [3], 16, 21)


@pytest.mark.parametrize("signs", [1, -1])
def test_sums_of_equal_signs(fa, signs):
    """All products of one sign: sums that grow with every term, where products' sums round the most."""
    g = torch.Generator().manual_seed(1)
    x = torch.randint(200, 448, (3000, 1, 2, 192), generator=g).float()
    bounds = (x.sort(2, descending=True)[0] * signs).to(torch.float8_e4m3fn)
    bounds = bounds if signs > 0 else bounds.view(torch.uint8).flip(2).view(torch.float8_e4m3fn)
    scale, table = ref.e8m0(torch.zeros(3000, 1)), torch.randperm(3000, generator=g).to(torch.int32)[None]
    q = normal(4, 8, 192).abs() + 1
    check(fa, q, bounds, scale, table, [48000], [4], 16, 100)


def test_what_is_no_number_is_taken_first(fa):
    """A NaN among a page's bounds or its scale, infinite and NaN queries."""
    bounds, scale, table = wide(300, 2, 64, seed=5)
    bounds.view(torch.uint8)[table[0, [40, 200]].long(), 1, 0, 3] = 0x7F
    scale.view(torch.uint8)[int(table[0, 77]), 0] = 255
    q = normal(1, 4, 64)
    got, _ = check(fa, q, bounds, scale, table, [4800], [1], 16, 12)
    assert table[0, 77] in got[0, 0].tolist() and {int(table[0, 40]), int(table[0, 200])} <= set(got[0, 1].tolist())
    check(fa, torch.zeros_like(q), bounds, scale, table, [4800], [1], 16, 12)
    check(fa, torch.zeros_like(q), bounds, scale, table, [4800], [1], 16, 4, first=1, last=2)
    for value in (math.inf, -math.inf, math.nan):
        q[0, 1, 7] = value
        check(fa, q, bounds, scale, table, [4800], [1], 16, 12)


def test_a_page_outside_the_cache_is_not_followed(fa):
    bounds, scale, table = wide(100, 2, 64)
    for bad in (-1, 100, -2 ** 31, 2 ** 31 - 1):
        broken = table.clone()
        broken[0, 50] = bad
        args = (normal(1, 4, 64).cuda(), bounds.cuda(), scale.cuda(), broken.cuda(), int32([1600]), int32([0, 1]), 1, 16)
        lists, lens = fa.kv_select(*args, 20)
        code, detail = status(fa)
        assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (512, 0)
        assert ((lists >= 0) & (lists < 100)).all() and lens.tolist() == [320]
        lists, lens = fa.kv_select(*args, 100)
        status(fa)
        assert lists[0, 0, 50] == -1 and (lists[0] == -1).sum() == 2


@pytest.mark.parametrize("what", ["length", "negative", "new tokens", "offsets"])
def test_a_bad_sequence_leaves_its_neighbours_right(fa, what):
    lens, new, most = [300, 200, 400], [2, 3, 1], 3
    cache = ref.Cache(lens, 2, 16, 64, 64)
    bounds, q = want.all_bounds(cache), normal(6, 4, 64)
    dev_lens, cu = int32(lens), int32(offsets(new))
    if what == "length":
        dev_lens[1] = cache.width * 16 + 1
    elif what == "negative":
        dev_lens[1] = -2 ** 31
    elif what == "new tokens":
        most = 2
    else:
        cu[3] = 7
    lists = torch.full((6, 2, 7), -2, dtype=torch.int32, device="cuda")
    list_lens = torch.full((6,), -2, dtype=torch.int32, device="cuda")
    fa.kv_select(q.cuda(), bounds.cuda(), cache.k_scale.cuda(), cache.table.cuda(), dev_lens, cu, most, 16, 7, lists=lists,
                 list_lens=list_lens)
    code, detail = status(fa)
    bad = 2 if what == "offsets" else 1
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, bad)
    ex, ex_lens = want.select(q, bounds, cache.k_scale, cache.table, lens, offsets(new), 16, 7)
    for b in range(3):
        rows = slice(offsets(new)[b], offsets(new)[b + 1])
        if b == bad:
            assert (lists[rows] == -2).all() and (list_lens[rows] == -2).all()
        else:
            assert torch.equal(lists[rows].long().cpu(), ex[rows]) and torch.equal(list_lens[rows].long().cpu(), ex_lens[rows])


def test_refused_tensors(fa):
    cache = ref.Cache([100, 50], 2, 16, 64, 64)
    k, _, ks, _, table, lens = cache.to_device("cuda")
    good = dict(q=normal(2, 4, 64).cuda(), k_bounds=want.all_bounds(cache).cuda(), k_scale=ks, block_table=table, seqlens_k=lens,
                cu_seqlens_q=int32([0, 1, 2]), max_seqlen_q=1, page_size=16, top=4)
    fa.kv_select(**good)
    for kw in (dict(q=good["q"].float()), dict(q=good["q"][0]), dict(q=good["q"].transpose(0, 1)), dict(q=normal(2, 3, 64).cuda()),
               dict(k_bounds=good["k_bounds"][1:]), dict(k_bounds=good["k_bounds"].float()), dict(k_scale=ks[0]),
               dict(k_scale=ks.float()), dict(block_table=table.long()), dict(block_table=table[0]), dict(block_table=table.t()),
               dict(seqlens_k=lens[:1]), dict(seqlens_k=lens.cpu()), dict(cu_seqlens_q=int32([0, 1])), dict(top=0), dict(top=-1),
               dict(page_size=20), dict(keep_first=4), dict(keep_last=0), dict(lists=int32([[[0] * 4] * 2])),
               dict(list_lens=int32([0])), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.FaError):
            fa.kv_select(**{**good, **kw})
    more = dict(k_cache=k, k_bounds=good["k_bounds"], block_table=table, seqlens_k=lens, cu_seqlens=int32([0, 1, 2]), total=2)
    for kw in (dict(k_cache=k.float()), dict(k_cache=k[0]), dict(k_bounds=good["k_bounds"][:, :1]), dict(seqlens_k=lens.float()),
               dict(cu_seqlens=int32([0, 1])), dict(total=-1), dict(cu_seqlens=int32([0, 1, 2]).cpu())):
        with pytest.raises(fa.FaError):
            fa.kv_bounds(**{**more, **kw})
    assert status(fa)[0] == 0
