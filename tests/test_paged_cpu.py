"""Host-side checks of the paged 8-bit cache: refusals before any CUDA call, workspace sizes, and the index arithmetic
that maps blocks of work to sequences (restated here and checked by brute force)."""
import ctypes
import itertools
import random

import pytest

FAKE = 0x10000  # aligned, non-null; never dereferenced by these cases


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def cache(fa, **change):
    d_qk, d_v, page, heads = (change.get(n, x) for n, x in (("d_qk", 128), ("d_v", 128), ("page_size", 64), ("heads_kv", 2)))
    c = fa.FaKvCache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, (heads * page * d_qk, page * d_qk, d_qk),
                     (heads * page * d_v, page * d_v, d_v), 8, 16, page, heads, d_qk, d_v, 8)
    for name, value in change.items():
        setattr(c, name, (ctypes.c_int64 * 3)(*value) if name.endswith("_stride") and name != "table_stride" else value)
    return c


def append(fa, c, **change):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=1024, k_stride=256, v_stride=256, q_out=FAKE, cu=FAKE, batch=2, total=5,
             heads_q=8, cos_sin=FAKE, max_positions=100, rot_dim=64, interleaved=0)
    if c is not None and c.d_qk != 128:
        a.update(q_stride=8 * c.d_qk, k_stride=2 * c.d_qk)
    a.update(change)
    return fa.fa_kv_append(c, a["q"], a["k"], a["v"], a["q_stride"], a["k_stride"], a["v_stride"], a["q_out"], a["cu"],
                           a["batch"], a["total"], a["heads_q"], a["cos_sin"], a["max_positions"], a["rot_dim"],
                           a["interleaved"], None)


def attend(fa, c, **change):
    a = dict(q=FAKE, o=FAKE, lse=FAKE, cu=FAKE, batch=2, total_q=2, max_seqlen_q=1, total_k=100, heads_q=8, causal=1,
             scale=0.0, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(change)
    return fa.fa_fwd_paged(a["q"], c, a["o"], a["lse"], a["cu"], a["batch"], a["total_q"], a["max_seqlen_q"], a["total_k"],
                           a["heads_q"], a["causal"], a["scale"], a["workspace"], a["workspace_bytes"], None)


BAD_CACHES = [
    ("heads", dict(heads_kv=0), 1), ("pages", dict(num_pages=0), 1), ("width", dict(max_pages=0), 1),
    ("table stride", dict(table_stride=7), 1), ("dims", dict(d_qk=96), 2), ("dims v", dict(d_qk=64, d_v=128), 2),
    ("page 0", dict(page_size=0), 2), ("page 48", dict(page_size=48), 2), ("page 256", dict(page_size=256), 2),
    ("too many tokens", dict(max_pages=1 << 25, table_stride=1 << 25), 1),
    ("negative stride", dict(k_stride=(-16384, 8192, 128)), 1), ("odd stride", dict(v_stride=(16384, 8192, 136)), 1),
    ("token stride", dict(k_stride=(16384, 8192, 64)), 1), ("head stride 0", dict(k_stride=(16384, 0, 128)), 1),
    ("page stride 0", dict(v_stride=(0, 8192, 128)), 1), ("huge stride", dict(k_stride=(1 << 40, 8192, 128)), 1),
]
BAD_POINTERS = [(n, {n: v}, 1) for n in ("k", "v") for v in (None, FAKE + 8)] + \
               [(n, {n: v}, 1) for n in ("block_table", "seqlens_k") for v in (None, FAKE + 2)] + \
               [(n, {n: None}, 1) for n in ("k_scale", "v_scale")]


@pytest.mark.parametrize("case", BAD_CACHES + BAD_POINTERS, ids=lambda c: c[0])
def test_cache_refusals(fa, case):
    _, change, code = case
    assert append(fa, cache(fa, **change)) == code
    assert attend(fa, cache(fa, **change)) == code


def test_no_cache(fa):
    assert append(fa, None) == 1 and attend(fa, None) == 1


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(batch=16385), dict(total=-1), dict(total=1 << 31), dict(rot_dim=-16), dict(rot_dim=144),
    dict(rot_dim=24), dict(max_positions=0), dict(interleaved=2), dict(q=None), dict(q_out=None), dict(heads_q=0),
    dict(heads_q=3), dict(k=None), dict(v=None), dict(cu=None), dict(cos_sin=None), dict(q=FAKE + 8), dict(q_out=FAKE + 8),
    dict(k=FAKE + 8), dict(v=FAKE + 2), dict(cos_sin=FAKE + 4), dict(cu=FAKE + 2), dict(k_stride=255), dict(k_stride=252),
    dict(v_stride=128), dict(v_stride=-256), dict(q_stride=1020), dict(q_stride=512), dict(k_stride=1 << 41),
    dict(q_stride=2048, q_out=FAKE)], ids=str)
def test_append_refusals(fa, change):
    assert append(fa, cache(fa), **change) == 1


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(batch=16385), dict(total_q=-1), dict(total_q=1 << 31), dict(total_k=-1), dict(max_seqlen_q=-1),
    dict(max_seqlen_q=0), dict(heads_q=0), dict(heads_q=5), dict(scale=-1.0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(q=None), dict(o=None), dict(cu=None), dict(workspace=None), dict(q=FAKE + 8),
    dict(o=FAKE + 8), dict(lse=FAKE + 4), dict(workspace=FAKE + 8), dict(cu=FAKE + 2), dict(workspace_bytes=1000),
    dict(max_seqlen_q=100, total_k=(1 << 31) - 100)], ids=str)
def test_attention_refusals(fa, change):
    assert attend(fa, cache(fa), **change) == 1


def test_nothing_to_do(fa):
    for change in (dict(batch=0), dict(total=0)):
        assert append(fa, cache(fa, k=None, v=None), k=None, v=None, **change) == 0
    for change in (dict(batch=0), dict(total_q=0)):
        assert attend(fa, cache(fa, k=None, v=None), q=None, workspace=None, **change) == 0


def test_workspace_size(fa):
    size = fa.fa_fwd_paged_workspace_size
    assert size(-1, 8, 2, 1, 1, 1, 128, 128) == 0 and size(1, 8, 3, 1, 1, 1, 128, 128) == 0
    assert size(1, 8, 2, 1, 1, 1, 96, 96) == 0
    one = size(1, 8, 2, 1, 1, 1, 128, 128)
    # single tokens: independent of the batch and of the keys
    assert one == size(500, 8, 2, 500, 1, 1 << 30, 128, 128) and 0 < one < 64 << 20
    # 32 tokens x 4 heads are read from the pages, 33 are unpacked: room for the keys and values in bf16
    few, many = size(2, 8, 2, 64, 32, 5000, 128, 128), size(2, 8, 2, 66, 33, 5000, 128, 128)
    assert many >= few + 5000 * 2 * (128 + 128) * 2 + fa.fa_varlen_workspace_size(2, 8, 66)
    assert many == size(2, 8, 2, 66, 1000, 5000, 128, 128)


def test_python_checks_want_cuda_tensors(fa):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FaError):
        fa.kv_append(x, x, *[None] * 7)
    with pytest.raises(fa.FaError):
        fa.attention_forward_paged(x, *[None] * 7, 1)


def warp_search(n, x, key):
    """The 32-lane search of the kernels."""
    lo = 0
    while n > 1:
        step = (n + 31) >> 5
        le = [lane * step < n and key(lo + lane * step) <= x for lane in range(32)]
        sel = (sum(le) - 1) * step if any(le) else 0
        lo += sel
        n = min(n - sel, step)
    return lo


def test_search_finds_the_last_not_above():
    r = random.Random(1)
    for n in [1, 2, 31, 32, 33, 64, 100, 1023, 1024, 1025, 5000]:
        keys = sorted(r.randint(0, 3 * n) for _ in range(n))
        for x in [keys[0], keys[-1], keys[-1] + 5] + [r.randint(keys[0], 3 * n) for _ in range(20)]:
            assert warp_search(n, x, keys.__getitem__) == max(i for i in range(n) if keys[i] <= x)
    garbage = [r.randint(-9, 9) for _ in range(777)]
    for x in range(-12, 12):  # any keys give an index in range
        assert 0 <= warp_search(777, x, garbage.__getitem__) < 777


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_slots_cover_every_touched_page_once(page):
    """Sequence b owns the slots floor(cu[b] / page) + 2 b ..; its j-th is its j-th touched page."""
    r = random.Random(page)
    for _ in range(300):
        batch = r.randint(1, 40)
        new = [r.choice([0, 1, 2, page - 1, page, page + 1, r.randint(0, 5 * page)]) for _ in range(batch)]
        ctx = [r.randint(0, 3 * page) for _ in range(batch)]
        cu = [0] + list(itertools.accumulate(new))
        want = {(b, j) for b in range(batch) if new[b] for j in range(ctx[b] // page, (ctx[b] + new[b] - 1) // page + 1)}
        got = []
        for slot in range(cu[-1] // page + 2 * batch):
            b = warp_search(batch, slot, lambda i: cu[i] // page + 2 * i)
            j = slot - (cu[b] // page + 2 * b)
            if new[b] and ctx[b] // page + j <= (ctx[b] + new[b] - 1) // page:
                got.append((b, ctx[b] // page + j))
        assert len(got) == len(set(got)) and set(got) == want


def test_unpack_slots_cover_every_block_of_16_tokens_once():
    r = random.Random(5)
    for _ in range(300):
        batch = r.randint(1, 40)
        lens = [r.choice([0, 0, 1, 15, 16, 17, r.randint(0, 100)]) for _ in range(batch)]
        cu = [0] + list(itertools.accumulate(lens))
        want = {(b, t) for b in range(batch) for t in range(0, lens[b], 16)}
        got = []
        for slot in range(cu[-1] // 16 + batch):
            b = warp_search(batch, slot, lambda i: cu[i] // 16 + i)
            t = (slot - (cu[b] // 16 + b)) * 16
            if t < lens[b]:
                got.append((b, t))
        assert len(got) == len(set(got)) and set(got) == want
