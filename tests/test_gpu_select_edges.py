"""Page selection where nothing competes, beside calls that leave their traces in the same shared memory; arguments beyond
the C interface's integers; batches with rows behind the last sequence."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_select import fa, int32, normal, offsets, status, wide  # noqa: E402, F401  (fa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,new", [(100, 300), (1000, 300), (1024, 97), (1000, 5), (4096, 40), (4097, 3)])
@pytest.mark.parametrize("first,last", [(2, 3), (0, 4), (5, 1)])
def test_all_places_forced(fa, pages, new, first, last):  # noqa: F811
    """top == keep_first + keep_last: the first and the last pages, whatever the scores.  Before it, on every SM, selections
    among 60 equal pages, whose blocks settle the choice in the keys that they hold: what they leave behind is no key."""
    heads, page = 4, 16
    bounds, scale, table = wide(pages, heads, 64, seed=pages)
    codes = bounds.view(torch.uint8)
    codes[table[0, 20:80].long()] = torch.tensor([0x7E, 0xFE], dtype=torch.uint8)[None, None, :, None]  # 448, -448
    scale.view(torch.uint8)[table[0, 20:80].long()] = 127
    lens, cu = int32([pages * page]), int32(offsets([new]))
    q = normal(new, 8, 64).cuda()
    args = (q, bounds.cuda(), scale.cuda(), table.cuda(), lens, cu, new, page)
    top = first + last
    expect = torch.full((new, heads, top), -2, dtype=torch.int32)
    expect_lens = torch.zeros(new, dtype=torch.int32)
    for i in range(new):
        seen = pages * page - new + i + 1
        held = -(-seen // page)
        rows = torch.cat([table[0, :first], table[0, held - last:held]])
        expect[i] = rows
        expect_lens[i] = seen - (held - top) * page
    for _ in range(3):
        fa.kv_select(*args, top + 30, keep_first=first, keep_last=last)
        lists = torch.full((new, heads, top), -2, dtype=torch.int32, device="cuda")
        list_lens = torch.full((new,), -2, dtype=torch.int32, device="cuda")
        fa.kv_select(*args, top, keep_first=first, keep_last=last, lists=lists, list_lens=list_lens)
        assert status(fa)[0] == 0
        assert torch.equal(lists.cpu(), expect)
        assert torch.equal(list_lens.cpu(), expect_lens)


def fill_freed(n, value):
    """Leaves `value` in the block of n int32 that the allocator hands out next."""
    blocks = [torch.full((n,), value, dtype=torch.int32, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("side", [False, True])
def test_rows_behind_the_last_sequence_see_no_key(fa, side):  # noqa: F811
    """A padded batch whose list_lens the call allocates: rows of no sequence, and of one that is out of range, have no key
    for the attention, and no error; a graph finds that anew each time, with fewer sequences and with more."""
    import paged_ref as ref

    lens, total = [100, 50, 40, 30], 9
    cache = ref.Cache(lens, 2, 16, 64, 64)
    k, v, ks, vs, table, seqlens = cache.to_device("cuda")
    bounds = torch.zeros(cache.num_pages, 2, 2, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cu_all = int32([0, 100, 150, 190, 220])
    fa.kv_bounds(k, bounds, table, seqlens, cu_all, 220)
    q = normal(total, 4, 64).cuda()
    cu = int32([0, 2, 3, 3, 4])
    args = (q, bounds, ks, table, seqlens, cu, 2, 16, 3)
    whole = fa.kv_select(*args, list_lens=torch.zeros(total, dtype=torch.int32, device="cuda"))
    expect = whole[1].tolist()
    assert expect[4:] == [0] * 5 and min(expect[:4]) > 0
    fill_freed(total, 77)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    lists, list_lens = fa.kv_select(*args, stream=stream)
    torch.cuda.synchronize()
    assert list_lens.tolist() == expect
    o, lse = fa.attention_forward_lists(q, k, v, ks, vs, lists, list_lens)
    assert status(fa)[0] == 0
    assert (o[4:] == 0).all() and torch.isinf(lse[:, 4:]).all() and not torch.isinf(lse[:, :4]).any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lists, list_lens = fa.kv_select(*args)
        o, lse = fa.attention_forward_lists(q, k, v, ks, vs, lists, list_lens)
    for rows, offs in ((9, [0, 2, 4, 7, 9]), (1, [0, 0, 0, 1, 1]), (4, [0, 2, 3, 3, 4])):
        cu.copy_(int32(offs))
        graph.replay()
        code, detail = status(fa)
        if rows == 9:  # three new tokens of one sequence, more than the call allows: that one is left out
            assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 2)
            assert list_lens[4:7].tolist() == [0, 0, 0] and min(list_lens[:4].tolist() + list_lens[7:].tolist()) > 0
            continue
        assert code == 0 and list_lens[rows:].tolist() == [0] * (total - rows) and min(list_lens[:rows].tolist()) > 0
        assert (o[rows:] == 0).all()


BEYOND = [2 ** 32, 2 ** 31, -2 ** 32, 2 ** 64]


def test_numbers_beyond_32_bits_are_refused(fa):  # noqa: F811
    """What the C interface's integers cannot hold is an error, and not its lower 32 bits."""
    import paged_ref as ref

    cache = ref.Cache([100, 50], 2, 16, 64, 64)
    k, _, ks, _, table, lens = cache.to_device("cuda")
    bounds = torch.zeros(cache.num_pages, 2, 2, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cu = int32([0, 1, 2])
    out = torch.full((2, 2, 4), -2, dtype=torch.int32, device="cuda")
    good = dict(q=normal(2, 4, 64).cuda(), k_bounds=bounds, k_scale=ks, block_table=table, seqlens_k=lens, cu_seqlens_q=cu,
                max_seqlen_q=1, page_size=16, top=4, keep_first=0, keep_last=1, lists=out)
    for name in ("max_seqlen_q", "page_size", "top", "keep_first", "keep_last"):
        for more in BEYOND:
            with pytest.raises(fa.FaError):
                fa.kv_select(**{**good, name: good[name] + more})
    for more in BEYOND:
        with pytest.raises(fa.FaError):
            fa.kv_bounds(k, bounds, table, lens, cu, 2 + more)
        with pytest.raises(fa.FaError):
            fa.rotary_table(8 + more, 64)
        with pytest.raises(fa.FaError):
            fa.rotary_table(0, 64 + more)
    assert status(fa)[0] == 0 and (out == -2).all()
