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
