"""Attention over lists of pages on the GPU against 64 bits, with the bounds of the attention over whole sequences."""
import math

import pytest

torch = pytest.importorskip("torch")
import long_ref as want  # noqa: E402
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
EPS_F16 = 2.0 ** -11


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def problem(tokens, heads, page, d_qk, d_v, width, lens, seed=0, layout="heads"):
    """A pool whose pages are full, and random lists of distinct pages for each token and head (-1 behind their ends)."""
    pool = width + 5
    cache = ref.Cache([pool * page], heads, page, d_qk, d_v, seed=seed, spare=0, layout=layout)
    g = torch.Generator().manual_seed(seed + 1)
    lists = torch.stack([torch.randperm(pool, generator=g)[:width] for _ in range(tokens * heads)]).view(tokens, heads, width)
    used = torch.tensor([-(-n // page) for n in lens])
    lists = torch.where(torch.arange(width) < used[:, None, None], lists, -1).to(torch.int32)
    return cache, lists


def attend(fa, q, cache, lists, lens, **kw):
    dev = cache.to_device("cuda")[:4]
    o, lse = fa.attention_forward_lists(q.cuda(), *dev, lists.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), **kw)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, f"device status {code} {detail}"
    return o, lse


@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 1), (9, 1), (16, 1), (32, 1), (17, 1), (48, 2)])
def test_lists(fa, hq, hkv, dims, page, layout):
    """One to 32 query heads a key head, lists of every length from none to all of their pages."""
    width = 7
    lens = [0, 1, page - 1, page, page + 1, 3 * page + 5, width * page]
    cache, lists = problem(len(lens), hkv, page, *dims, width, lens, seed=hq, layout=layout)
    q = normal(len(lens), hq, dims[0], seed=page)
    o, lse = attend(fa, q, cache, lists, lens)
    ref.check_attention(o, lse, want.lists_attention(q, cache, lists, lens), EPS_F16)


@pytest.mark.parametrize("tokens,width,hq,hkv,page", [(1, 150, 8, 2, 64), (3, 300, 2, 1, 16), (300, 3, 2, 2, 16), (40, 40, 4, 1, 32),
                                                     (2, 64, 32, 2, 128)])
def test_lists_that_are_cut(fa, tokens, width, hq, hkv, page):
    """Few long lists, whose pages are split over the GPU and joined, and more tokens than a block looks at together."""
    lens = [width * page - (t * 7) % (2 * page) for t in range(tokens)]
    cache, lists = problem(tokens, hkv, page, 128, 64, width, lens, seed=width)
    q = normal(tokens, hq, 128)
    for scale in (None, 0.02):
        o, lse = attend(fa, q, cache, lists, lens, scale=scale)
        ref.check_attention(o, lse, want.lists_attention(q, cache, lists, lens, scale), EPS_F16)


def test_whole_sequences_as_lists(fa):
    """A list of all of a sequence's pages is the attention over the sequence."""
    lens = [500, 33, 1, 90]
    cache = ref.Cache(lens, 2, 32, 128, 128, width=16)
    q = normal(4, 8, 128)
    dev = cache.to_device("cuda")
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward_paged(q.cuda(), *dev, cu, 1)
    got, got_lse = fa.attention_forward_lists(q.cuda(), *dev[:4], dev[4][:, None].repeat(1, 2, 1).contiguous(), dev[5])
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    # the same products in tiles cut elsewhere: twice what each may be off
    r = want.lists_attention(q, cache, cache.table[:, None].repeat(1, 2, 1), lens)
    ref.check_attention(o, lse, r, EPS_F16)
    ref.check_attention(got, got_lse, r, EPS_F16)


def test_rows_outside_and_results_given(fa):
    cache, lists = problem(3, 2, 16, 64, 64, 4, [20, 64, 7])
    q = normal(3, 4, 64)
    out = torch.full((4, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fa.fa_fwd_lists_workspace_size(4, 2, 64), dtype=torch.uint8, device="cuda").fill_(255)
    o, lse = attend(fa, q, cache, lists, [20, 64, 7], out=out[:3], workspace=ws)
    only = fa.attention_forward_lists(q.cuda(), *cache.to_device("cuda")[:4], lists.cuda(),
                                      torch.tensor([20, 64, 7], dtype=torch.int32, device="cuda"), return_lse=False)
    assert torch.equal(only, o) and (out[3] == 3.0).all()
    ref.check_attention(o, lse, want.lists_attention(q, cache, lists, [20, 64, 7]), EPS_F16)


@pytest.mark.parametrize("bad", [-1, 9, -2 ** 31, 2 ** 31 - 1])
def test_a_page_outside_the_cache_is_not_followed(fa, bad):
    lens = [64, 64, 64]
    cache, lists = problem(3, 2, 16, 64, 64, 4, lens)
    q = normal(3, 4, 64)
    broken = lists.clone()
    broken[1, 1, 2] = bad
    o, lse = fa.attention_forward_lists(q.cuda(), *cache.to_device("cuda")[:4], broken.cuda(),
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (512, 1)
    r = want.lists_attention(q, cache, lists, lens)
    keep = [0, 2]
    ref.check_attention(o[keep], lse[:, keep], (r[0][keep], r[1][:, keep], r[2][keep], r[3][keep], r[4][keep]), EPS_F16)


@pytest.mark.parametrize("bad", [-1, 65, -2 ** 31, 2 ** 31 - 1])
def test_a_length_out_of_range_is_left_out(fa, bad):
    lens = [64, bad, 5]
    cache, lists = problem(3, 2, 16, 64, 64, 4, [64, 64, 5])
    q = normal(3, 4, 64)
    out = torch.full((3, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 3), 3.0, device="cuda")
    fa.attention_forward_lists(q.cuda(), *cache.to_device("cuda")[:4], lists.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out, lse=lse)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 1)
    assert (out[1] == 3.0).all() and (lse[:, 1] == 3.0).all()
    r = want.lists_attention(q, cache, lists, [64, 64, 5])
    keep = [0, 2]
    ref.check_attention(out[keep], lse[:, keep], (r[0][keep], r[1][:, keep], r[2][keep], r[3][keep], r[4][keep]), EPS_F16)


def test_a_nan_reaches_the_rows_that_list_its_page_only(fa):
    lens = [64, 64]
    cache, lists = problem(2, 2, 16, 64, 64, 4, lens)
    bad = int(lists[0, 1, 2])
    clean = attend(fa, normal(2, 4, 64), cache, lists, lens)
    cache.v.view(torch.uint8)[bad, 1, 3, 5] = 0x7F
    o, lse = attend(fa, normal(2, 4, 64), cache, lists, lens)
    hit = torch.zeros(2, 4, dtype=torch.bool)
    for t in range(2):
        if bad in lists[t, 1].tolist():
            hit[t, 2:] = True
    assert hit[0].any()
    assert torch.isnan(o[hit]).all() and torch.isnan(lse.t()[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse.t()[~hit], clean[1].t()[~hit])


def test_the_same_page_twice(fa):
    """Its tokens count twice."""
    cache, lists = problem(1, 1, 16, 64, 64, 4, [64])
    lists[0, 0] = torch.tensor([3, 3, 1, 3])
    q = normal(1, 2, 64)
    o, lse = attend(fa, q, cache, lists, [64])
    ref.check_attention(o, lse, want.lists_attention(q, cache, lists, [64]), EPS_F16)


def test_refused_tensors(fa):
    cache, lists = problem(2, 2, 16, 64, 64, 4, [64, 20])
    k, v, ks, vs = cache.to_device("cuda")[:4]
    lens = torch.tensor([64, 20], dtype=torch.int32, device="cuda")
    good = dict(q=normal(2, 4, 64).cuda(), k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, lists=lists.cuda(), list_lens=lens)
    fa.attention_forward_lists(**good)
    for kw in (dict(q=good["q"].half()), dict(q=good["q"][0]), dict(q=normal(2, 4, 128).cuda()), dict(q=normal(2, 3, 64).cuda()),
               dict(q=normal(3, 4, 64).cuda()), dict(k_cache=k.float()), dict(v_cache=v[:, :1]), dict(k_scale=ks[1:]),
               dict(v_scale=vs.float()), dict(lists=good["lists"].long()), dict(lists=good["lists"][:, :1]), dict(lists=lists),
               dict(lists=good["lists"].transpose(1, 2)), dict(lists=good["lists"][:, :, :0]), dict(list_lens=lens[:1]),
               dict(list_lens=lens.float()), dict(scale=-1.0), dict(scale=math.nan), dict(out=good["q"].float()),
               dict(lse=torch.empty(2, 4, device="cuda")), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.FaError):
            fa.attention_forward_lists(**{**good, **kw})
    none = fa.attention_forward_lists(good["q"][:0], k, v, ks, vs, good["lists"][:0], lens[:0])[0]
    assert none.shape == (0, 4, 64) and fa.fa_device_status()[0] == 0
