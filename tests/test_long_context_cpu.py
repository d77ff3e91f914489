"""Host-side checks of the operators for long contexts: refusals before any CUDA call, empty calls, workspace sizes."""
import math

import pytest

from test_paged_cpu import BAD_CACHES, FAKE, cache, fa  # noqa: F401  (fa: the fixture)

OTHER = FAKE + 0x1000


def table(fa, **change):
    a = dict(cos_sin=FAKE, positions=8, rot_dim=64, base=10000.0, kind=0, factor=1.0, original=0.0, low=1.0, high=2.0,
             magnitude=1.0)
    a.update(change)
    s = fa.FaRotaryScaling(a["kind"], a["factor"], a["original"], a["low"], a["high"], a["magnitude"])
    return fa.fa_rotary_table(a["cos_sin"], a["positions"], a["rot_dim"], a["base"], s, None)


def rotary(fa, **change):
    a = dict(q=FAKE, k=OTHER, q_out=FAKE, k_out=OTHER, q_stride=512, k_stride=256, q_out_stride=512, k_out_stride=256,
             positions=None, cu=None, batch=0, seqlen=4, total=8, heads_q=4, heads_k=2, d=128, cos_sin=FAKE, max_pos=10,
             rot_dim=64, interleaved=0, backward=0)
    a.update(change)
    return fa.fa_rotary(*a.values(), None)


def bounds(fa, c, **change):
    a = dict(bounds=FAKE, cu=FAKE, batch=2, total=5)
    a.update(change)
    return fa.fa_kv_bounds(c, *a.values(), None)


def select(fa, **change):
    a = dict(q=FAKE, bounds=FAKE, k_scale=FAKE, table=FAKE, table_stride=8, seqlens=FAKE, cu=FAKE, batch=2, total_q=3, max_n=2,
             heads_q=8, heads_kv=2, d_qk=128, num_pages=8, page_size=64, max_pages=8, causal=1, top=4, first=1, last=1,
             lists=FAKE, list_lens=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(change)
    return fa.fa_kv_select(*a.values(), None)


def lists(fa, c, **change):
    a = dict(q=FAKE, cache=c, lists=FAKE, list_lens=FAKE, width=4, o=FAKE, lse=FAKE, total_q=2, heads_q=8, scale=0.0,
             workspace=FAKE, workspace_bytes=1 << 40)
    a.update(change)
    return fa.fa_fwd_lists(*a.values(), None)


def fork(fa, c, **change):
    a = dict(bounds=FAKE, refs=OTHER + 48, batch=2, parents=FAKE, grow=FAKE, rows=3, table_out=OTHER, out_stride=8,
             seqlens_out=OTHER + 16, refs_out=OTHER + 48, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(change)
    return fa.fa_kv_fork(c, *a.values(), None)


def compact(fa, c, **change):
    a = dict(bounds=FAKE, refs=OTHER + 48, batch=2, table_out=FAKE, out_stride=8, refs_out=OTHER + 48, page_map=OTHER,
             used=OTHER + 16, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(change)
    return fa.fa_kv_compact(c, *a.values(), None)


@pytest.mark.parametrize("change", [
    dict(positions=-1), dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=72), dict(rot_dim=208), dict(base=0.5),
    dict(base=math.inf), dict(base=math.nan), dict(kind=-1), dict(kind=4), dict(magnitude=0.0), dict(magnitude=-1.0),
    dict(magnitude=math.nan), dict(magnitude=2.0 ** 65), dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan),
    dict(kind=2, factor=0.0), dict(kind=2, factor=1e200, base=1e200), dict(kind=3, original=0.0),
    dict(kind=3, original=math.inf), dict(kind=3, original=1.0, low=-1.0), dict(kind=3, original=1.0, low=2.0, high=2.0),
    dict(kind=3, original=1.0, high=math.nan), dict(cos_sin=None), dict(cos_sin=FAKE + 8)], ids=str)
def test_rotary_table_refusals(fa, change):
    assert table(fa, **change) == 1


def test_rotary_table_of_no_positions(fa):
    assert table(fa, positions=0, cos_sin=None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(d=96), 2), (dict(d=256), 2), (dict(total=-1), 1), (dict(total=1 << 31), 1), (dict(heads_q=-1), 1), (dict(rot_dim=0), 1),
    (dict(rot_dim=24), 1), (dict(rot_dim=144), 1), (dict(max_pos=0), 1), (dict(interleaved=2), 1), (dict(backward=2), 1),
    (dict(positions=FAKE, cu=FAKE), 1), (dict(cu=FAKE, batch=-1), 1), (dict(cu=FAKE, batch=16385), 1), (dict(seqlen=0), 1),
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(k_out=None), 1), (dict(cos_sin=None), 1),
    (dict(cos_sin=FAKE + 4), 1), (dict(positions=FAKE + 2), 1), (dict(cu=FAKE + 2, batch=1), 1), (dict(q=FAKE + 8), 1),
    (dict(k_out=FAKE + 8), 1), (dict(q_stride=516), 1), (dict(q_stride=504, q_out_stride=504), 1), (dict(k_out_stride=1 << 40), 1),
    (dict(q_out_stride=520), 1), (dict(heads_q=65537, q_stride=1 << 24, q_out_stride=1 << 24), 1),
    (dict(k_out=FAKE), 1), (dict(q_out=OTHER), 1), (dict(q_out=OTHER + 64, k_out=OTHER + 64), 1)], ids=str)
def test_rotary_refusals(fa, change, code):
    assert rotary(fa, **change) == code


@pytest.mark.parametrize("change", [dict(total=0, cos_sin=None), dict(heads_q=0, heads_k=0), dict(cu=FAKE, batch=0),
                                    dict(q=None, q_out=None, k=None, k_out=None)], ids=str)
def test_rotary_of_nothing(fa, change):
    assert rotary(fa, **change) == 0


OF_KEYS = [c for c in BAD_CACHES if "v_stride" not in c[1] and c[0] != "dims v"]


@pytest.mark.parametrize("name,change,code", OF_KEYS, ids=[c[0] for c in OF_KEYS])
def test_bounds_refuse_bad_caches(fa, name, change, code):
    assert bounds(fa, cache(fa, **change)) == code


@pytest.mark.parametrize("name,change,code", BAD_CACHES, ids=[c[0] for c in BAD_CACHES])
def test_page_calls_refuse_bad_caches(fa, name, change, code):
    c = cache(fa, **change)
    assert fork(fa, c, out_stride=1 << 30) == code and compact(fa, c, out_stride=1 << 30) == code
    if name not in ("width", "table stride", "too many tokens"):  # sizes of the table, which lists have in its place
        assert lists(fa, c) == code


@pytest.mark.parametrize("change", [dict(batch=-1), dict(batch=16385), dict(total=-1), dict(total=1 << 31), dict(bounds=None),
                                    dict(bounds=FAKE + 8), dict(cu=None), dict(cu=FAKE + 1)], ids=str)
def test_bounds_refusals(fa, change):
    assert bounds(fa, cache(fa), **change) == 1


def test_bounds_of_nothing_and_without_values(fa):
    assert bounds(fa, cache(fa), batch=0, bounds=None) == 0 and bounds(fa, cache(fa), total=0) == 0
    assert bounds(fa, None) == 1
    assert bounds(fa, cache(fa, v=None, v_scale=None, k_scale=None, d_v=7, v_stride=(0, 0, 0)), total=0) == 0


@pytest.mark.parametrize("change,code", [
    (dict(d_qk=96), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(batch=-1), 1), (dict(batch=16385), 1),
    (dict(total_q=-1), 1), (dict(total_q=1 << 31), 1), (dict(max_n=-1), 1), (dict(max_n=0), 1), (dict(heads_kv=0), 1),
    (dict(heads_q=0), 1), (dict(heads_q=7), 1), (dict(heads_q=65538), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(table_stride=7), 1), (dict(max_pages=1 << 25, table_stride=1 << 25), 1), (dict(first=-1), 1), (dict(last=0), 1),
    (dict(top=0), 1), (dict(top=1), 1), (dict(first=3, last=2), 1), (dict(first=2 ** 31 - 1), 1), (dict(top=(1 << 24) + 1), 1),
    (dict(total_q=1 << 30, heads_kv=2), 1), (dict(workspace_bytes=100), 1)] +
    [({n: v}, 1) for n in ("q", "bounds", "workspace") for v in (None, FAKE + 8)] +
    [({n: v}, 1) for n in ("table", "seqlens", "cu", "lists", "list_lens") for v in (None, FAKE + 2)] + [(dict(k_scale=None), 1)],
    ids=str)
def test_select_refusals(fa, change, code):
    assert select(fa, **change) == code


def test_select_of_nothing(fa):
    assert select(fa, batch=0, q=None) == 0 and select(fa, total_q=0, q=None, max_n=0) == 0


@pytest.mark.parametrize("change", [
    dict(cache=None), dict(width=0), dict(width=1 << 25), dict(total_q=-1), dict(total_q=(1 << 20) + 1), dict(heads_q=0),
    dict(heads_q=7), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(workspace_bytes=100), dict(lists=None),
    dict(lists=FAKE + 2), dict(list_lens=None), dict(list_lens=FAKE + 2), dict(q=None), dict(q=FAKE + 8), dict(o=None),
    dict(o=FAKE + 8), dict(lse=FAKE + 8), dict(workspace=None), dict(workspace=FAKE + 8)], ids=str)
def test_lists_refusals(fa, change):
    assert lists(fa, cache(fa), **change) == 1


def test_lists_of_no_tokens(fa):
    assert lists(fa, cache(fa), total_q=0, q=None, workspace=None) == 0


@pytest.mark.parametrize("change", [
    dict(batch=0), dict(batch=16385), dict(rows=0), dict(rows=16385), dict(out_stride=7), dict(refs=None), dict(refs=FAKE + 2),
    dict(parents=None), dict(parents=FAKE + 2), dict(grow=FAKE + 2), dict(table_out=None), dict(table_out=FAKE),
    dict(table_out=OTHER + 2), dict(seqlens_out=None), dict(seqlens_out=FAKE), dict(seqlens_out=OTHER + 2), dict(refs_out=None),
    dict(refs_out=FAKE + 2), dict(bounds=FAKE + 8), dict(workspace=None), dict(workspace=FAKE + 8), dict(workspace_bytes=100),
    dict(refs_out=FAKE), dict(seqlens_out=OTHER), dict(refs_out=OTHER), dict(seqlens_out=OTHER + 48), dict(table_out=OTHER + 48),
    dict(parents=OTHER + 16), dict(grow=OTHER + 16), dict(grow=OTHER), dict(parents=OTHER + 48)],
    ids=str)
def test_fork_refusals(fa, change):
    assert fork(fa, cache(fa), **change) == 1


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(batch=16385), dict(out_stride=7), dict(out_stride=9), dict(refs=None), dict(refs=FAKE + 2),
    dict(table_out=None), dict(table_out=FAKE + 2), dict(refs_out=None), dict(refs_out=FAKE + 2), dict(page_map=None),
    dict(page_map=FAKE), dict(page_map=FAKE + 2), dict(used=None), dict(used=FAKE + 2), dict(bounds=FAKE + 8),
    dict(workspace=None), dict(workspace=FAKE + 8), dict(workspace_bytes=100), dict(page_map=OTHER + 48), dict(used=OTHER + 48),
    dict(used=FAKE), dict(used=OTHER), dict(table_out=OTHER + 48), dict(refs_out=FAKE)], ids=str)
def test_compact_refusals(fa, change):
    assert compact(fa, cache(fa, seqlens_k=OTHER + 64), **change) == 1


@pytest.mark.parametrize("call", [table, rotary, lambda fa: bounds(fa, cache(fa)), select, lambda fa: lists(fa, cache(fa)),
                                  lambda fa: fork(fa, cache(fa)), lambda fa: compact(fa, cache(fa, seqlens_k=OTHER + 64))])
def test_what_the_refusals_change_is_otherwise_accepted(fa, call):
    """The arguments that the cases above start from pass all checks before the device's: without one the call ends there."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are refused here")
    assert call(fa) == 3


def test_calls_without_a_cache(fa):
    assert fork(fa, None) == 1 and compact(fa, None) == 1 and bounds(fa, None) == 1


def test_workspace_sizes(fa):
    pages = fa.fa_kv_pages_workspace_size
    assert pages(-1, 1, 1) == pages(1, -1, 1) == pages(1, 1, 0) == 0
    assert pages(16, 64, 1000) >= 4 * 1000 + 64 * 20
    sel = fa.fa_kv_select_workspace_size
    assert sel(-1, 1, 1, 1) == sel(1, -1, 1, 1) == sel(1, 1, 0, 1) == sel(1, 1, 1, 0) == 0
    assert sel(4, 1 << 20, 8, 1 << 12) >= 12 << 35  # beyond 32 bits
    size = fa.fa_fwd_lists_workspace_size
    assert size(0, 1, 64) == size(8, 0, 64) == size(7, 2, 64) == size(8, 2, 96) == 0
    assert size(32, 2, 64) > size(8, 2, 64)  # 16 rows a key head
    assert size(64, 2, 64) == size(32, 2, 64)  # 32 rows in two groups
    assert size(34, 2, 64) == size(2, 2, 64)  # 17 rows in 17


def test_binding_refuses_tensors_off_the_gpu(fa):
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    f8 = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: fa.rotary(q, q, torch.zeros(4, 64)), lambda: fa.rotary(None, None, torch.zeros(4, 64)),
                 lambda: fa.rotary_backward(None, q, torch.zeros(4, 64)),
                 lambda: fa.rotary_table(4, 64, out=torch.zeros(4, 64)), lambda: fa.rotary_table(4, 64, device="cpu"),
                 lambda: fa.rotary_table(4, 64, scaling="other"),
                 lambda: fa.kv_bounds(f8, f8, i, i, i, 1),
                 lambda: fa.kv_select(q, f8, i, i, i, i, 1, 16, 2),
                 lambda: fa.attention_forward_lists(q, f8, f8, f8, f8, i, i),
                 lambda: fa.kv_fork(i, f8, f8, f8, f8, i, i, i), lambda: fa.kv_compact(f8, f8, f8, f8, i, i, i)):
        with pytest.raises(fa.FaError):
            call()
