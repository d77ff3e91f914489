"""fa_fwd_paged on the GPU against a plain attention in 64 bits over the values the cache holds."""
import math

import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

EPS_F16, EPS_BF16 = 2.0 ** -11, 2.0 ** -8
DIMS = [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)]


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def queries(new, heads_q, d, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(sum(new), heads_q, d, generator=g) * size).to(torch.bfloat16)


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def run(fa, cache, new, q, causal=True, scale=None, max_new=None, **kw):
    dev = cache.to_device("cuda")
    cu = torch.tensor(offsets(new), dtype=torch.int32, device="cuda")
    out = fa.attention_forward_paged(q.cuda(), *dev, cu, max(new) if max_new is None else max_new, causal=causal,
                                     scale=scale, **kw)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, f"device status {code} {detail}"
    return out


def check(fa, lens, new, heads_q, heads_kv, dims, page, causal=True, seed=0, scale=None, layout="heads", size=1.0,
          max_new=None, eps=None, **kw):
    cache = ref.Cache(lens, heads_kv, page, *dims, seed=seed, layout=layout)
    q = queries(new, heads_q, dims[0], seed, size)
    o, lse = run(fa, cache, new, q, causal, scale, max_new, **kw)
    want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, lens, offsets(new), page, causal,
                         scale)
    if eps is None:
        rows = (max(new) if max_new is None else max_new) * (heads_q // heads_kv)
        eps = EPS_F16 if rows <= 16 else EPS_BF16  # how the weights are rounded
    return ref.check_attention(o, lse, want, eps, f"{lens} {new} {dims} page {page}")


LENGTHS = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dims", DIMS)
def test_single_tokens(fa, dims, page):
    check(fa, LENGTHS, [1] * len(LENGTHS), 8, 2, dims, page, seed=page)


@pytest.mark.parametrize("ratio", [1, 2, 3, 5, 8, 11, 16, 24, 32, 48, 64])
def test_group_sizes(fa, ratio):
    check(fa, [77, 200, 513], [1, 1, 1], 2 * ratio, 2, (128, 128), 64, seed=ratio)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("rows", [8, 16, 17, 40, 96, 128])
def test_every_build(fa, dims, rows, page):
    check(fa, [100, 33, 1000, 128, 1, 129], [1] * 6, rows, 1, dims, page, seed=rows)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 16, 32])
def test_few_new_tokens(fa, n, causal):
    check(fa, [n, n + 1, 31, 32, 33, 95, 400], [n, n, n, n, n, n, n], 8, 2, (128, 128), 32, causal, seed=n)


@pytest.mark.parametrize("causal", [True, False])
def test_ragged_new_tokens_and_empty_sequences(fa, causal):
    # no new tokens, no keys at all, fewer keys than new tokens (rows without a key)
    check(fa, [40, 0, 3, 100, 17, 0], [1, 2, 6, 0, 4, 0], 6, 3, (64, 64), 16, causal)


@pytest.mark.parametrize("ratio", [4, 16, 24])
@pytest.mark.parametrize("page", [16, 128])
def test_long_and_many_pieces(fa, page, ratio):
    check(fa, [9000], [1], 2 * ratio, 2, (128, 128), page)


@pytest.mark.parametrize("dims", [(64, 64), (192, 128)])
def test_more_units_than_blocks(fa, dims):
    """Pieces that hold several whole (sequence, head)s and parts of others, 20 rows each."""
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(5, 700, (90,), generator=g).tolist()
    check(fa, lens, [5] * 90, 12, 3, dims, 32, seed=2)


@pytest.mark.parametrize("ratio", [2, 20])
def test_many_sequences(fa, ratio):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 150, (700,), generator=g).tolist()
    check(fa, lens, [1] * 700, 2 * ratio, 2, (64, 64), 32)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(fa, dims, causal):
    check(fa, [150, 333, 90], [150, 129, 70], 4, 2, dims, 32, causal)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_prompts_and_tokens_in_one_batch(fa, page):
    # sequences of one token, none, exactly the 128 rows read from the pages, and more
    check(fa, [200, 77, 40, 500, 129, 0, 65], [1, 0, 32, 300, 33, 3, 65], 8, 2, (128, 128), page)


@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (192, 128)])
@pytest.mark.parametrize("ratio", [1, 4, 8, 9])
def test_few_and_many_rows_in_one_batch(fa, dims, ratio):
    # up to 8 rows, and up to 128, next to each other, each kind with units that are cut
    new = [1, 128 // ratio, 8 // ratio or 1, 0, 2, 17, 1, 30 // ratio]
    check(fa, [5000, 3000, 77, 0, 4000, 17, 1, 900], new, 2 * ratio, 2, dims, 64, seed=ratio)


@pytest.mark.parametrize("rows", [24, 56, 120])
def test_cut_where_a_unit_starts(fa, rows):
    """Lengths of one tile more and less, so that pieces begin and end at and near the ends of units."""
    for batch in (3, 29, 37, 61):
        lens = [(128 * (i % 5) + (-1, 0, 1)[i % 3]) or 1 for i in range(batch)]
        check(fa, [max(n, 1) for n in lens], [1] * batch, 4 * rows, 4, (64, 64), 128, seed=batch)


def test_prompt_without_keys(fa):
    check(fa, [0, 0], [100, 1], 4, 4, (64, 64), 16)


@pytest.mark.parametrize("layout", ["tokens", "apart"])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 90]])
def test_other_orders_of_the_cache(fa, layout, new):
    check(fa, [100, 64, 201], new, 8, 4, (128, 64), 32, layout=layout)


def test_scale_and_large_scores(fa):
    check(fa, [500, 300], [1, 2], 8, 2, (128, 128), 64, scale=0.5)
    check(fa, [500, 300], [1, 2], 8, 2, (128, 128), 64, size=30.0)
    check(fa, [500, 300], [1, 5], 16, 2, (128, 128), 64, size=30.0)


def test_queries_of_extreme_size(fa):
    cache = ref.Cache([200, 200, 200], 2, 32, 64, 64, seed=3)
    q = queries([1, 1, 1], 8, 64)
    q[0] = (q[0].double() * 2.0 ** -100).to(torch.bfloat16)  # scores 0 but for rounding
    q[1] *= 0.0
    q[2, :, 0] *= 2.0 ** 10
    o, lse = run(fa, cache, [1, 1, 1], q)
    want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.lens, [0, 1, 2, 3], 32, True)
    ref.check_attention(o, lse, want, EPS_F16)


@pytest.mark.parametrize("new", [1, 20, 80])
def test_scales_far_apart(fa, new):
    """Pages whose scales differ by up to 2^60: none may drown another or overflow."""
    cache = ref.Cache([160], 2, 16, 64, 64, seed=4)
    g = torch.Generator().manual_seed(9)
    cache.v_scale = ref.e8m0(torch.randint(-40, 20, cache.v_scale.shape, generator=g))
    cache.k_scale = ref.e8m0(torch.randint(-30, -5, cache.k_scale.shape, generator=g))
    q = queries([new], 4, 64)
    o, lse = run(fa, cache, [new], q)
    want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, [160], [0, new], 16, True)
    ref.check_attention(o, lse, want, EPS_F16 if new * 2 <= 16 else EPS_BF16)


@pytest.mark.parametrize("n", [6, 30, 80])
@pytest.mark.parametrize("where", ["k", "v", "k_scale", "v_scale"])
def test_nan_reaches_the_rows_that_see_it_only(fa, n, where):
    """Token 97 of 100 holds a NaN (or, for the scales, the last page does): rows before it are untouched."""
    page, lens, new = 16, [100], [n]
    clean = ref.Cache(lens, 2, page, 128, 128, seed=6)
    q = queries(new, 4, 128)
    o0, l0 = run(fa, clean, new, q)
    bad = ref.Cache(lens, 2, page, 128, 128, seed=6)
    p = int(bad.table[0, 97 // page])
    if where in ("k", "v"):
        getattr(bad, where).view(torch.uint8)[p, 1, 97 % page, 5] = 0xFF
        first = 97
    else:
        getattr(bad, where).view(torch.uint8)[p, 1] = 255
        first = 96
    o1, l1 = run(fa, bad, new, q)
    sees = torch.arange(n) + 100 - n >= first
    nan_o, nan_l = torch.isnan(o1).cpu(), torch.isnan(l1).cpu()
    assert nan_o[sees][:, 2:].any(-1).all()          # heads of key head 1
    assert not nan_o[~sees].any() and not nan_o[:, :2].any() and not nan_l[:2].any() and not nan_l[:, ~sees].any()
    assert torch.equal(o1[~sees], o0[~sees]) and torch.equal(o1[:, :2], o0[:, :2])


def test_without_lse_and_given_outputs(fa):
    cache = ref.Cache([70, 300], 2, 64, 128, 128)
    q = queries([1, 1], 8, 128)
    o, lse = run(fa, cache, [1, 1], q)
    alone = run(fa, cache, [1, 1], q, return_lse=False)
    assert torch.equal(alone, o)
    out, l2 = torch.full_like(o, 3.0), torch.full_like(lse, 3.0)
    got = run(fa, cache, [1, 1], q, out=out, lse=l2)
    assert got[0] is out and got[1] is l2 and torch.equal(out, o) and torch.equal(l2, lse)


def test_rows_behind_the_last_sequence_are_left(fa):
    for new in ([1, 2], [1, 90]):
        cache = ref.Cache([70, 300], 2, 64, 128, 128)
        q = queries(new + [5], 8, 128)
        out = torch.full((sum(new) + 5, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((8, sum(new) + 5), 3.0, device="cuda")
        run(fa, cache, new, q, out=out, lse=lse, max_new=max(new))
        assert (out[sum(new):] == 3.0).all() and (lse[:, sum(new):] == 3.0).all()
        assert not (out[:sum(new)] == 3.0).all(-1).any()


@pytest.mark.parametrize("new", [[1] * 9, [1, 9, 2], [1, 3, 100]])
def test_repeats_are_bit_identical_and_the_workspace_needs_no_clearing(fa, new):
    lens = [1000 + 37 * i for i in range(len(new))]
    cache = ref.Cache(lens, 2, 64, 128, 128)
    q = queries(new, 8, 128)
    size = fa.fa_fwd_paged_workspace_size(len(new), 8, 2, sum(new), max(new), sum(lens), 128, 128)
    first = None
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        o, lse = run(fa, cache, new, q, workspace=ws, total_k=sum(lens))
        first = (o, lse) if first is None else first
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_offsets_beyond_32_bits(fa):
    """Pages more than 2^32 bytes into the cache."""
    page, heads, d = 64, 8, 128
    pages = (1 << 32) // (page * heads * d) + 40
    small = ref.Cache([130, 129], heads, page, d, d, seed=8)
    k = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda")
    ks = torch.full((pages, heads), 127, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    first = pages - small.num_pages
    for dst, src in ((k, small.k), (v, small.v), (ks, small.k_scale), (vs, small.v_scale)):
        dst[first:] = src.view(torch.uint8).cuda()
    table = torch.where(small.table >= 0, small.table + first, small.table).to(torch.int32).cuda()
    for new in ([1, 1], [1, 40]):
        q = queries(new, 16, d)
        cu = torch.tensor(offsets(new), dtype=torch.int32, device="cuda")
        o, lse = fa.attention_forward_paged(q.cuda(), k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn),
                                            ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu), table,
                                            small.seqlens.cuda(), cu, max(new))
        torch.cuda.synchronize()
        assert fa.fa_device_status()[0] == 0
        want = ref.attention(q, small.k, small.v, small.k_scale, small.v_scale, small.table, [130, 129], offsets(new), page,
                             True)
        ref.check_attention(o, lse, want, EPS_F16 if max(new) == 1 else EPS_BF16)


def test_side_stream_and_graph_replay(fa):
    """A captured call replayed with other lengths, queries and pages."""
    lens = [500, 40, 900]
    cache = ref.Cache(lens, 2, 32, 128, 128, seed=1)
    dev = cache.to_device("cuda")
    q = queries([1, 1, 1], 8, 128).cuda()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(3, 8, 2, 3, 1, 0, 128, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(8, 3, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda: fa.attention_forward_paged(q, *dev, cu, 1, out=out, lse=lse, workspace=ws)  # noqa: E731
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed, now in ((1, lens), (2, [499, 1, 33]), (3, [500, 40, 0])):
        q.copy_(queries([1, 1, 1], 8, 128, seed).cuda())
        dev[5].copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status()[0] == 0
        want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, now, [0, 1, 2, 3], 32, True)
        ref.check_attention(out, lse, want, EPS_F16, f"replay {now}")
    # outputs allocated for another stream than the current one
    o2, l2 = fa.attention_forward_paged(q, *dev, cu, 1, stream=side)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_replay_with_another_split_of_the_tokens(fa):
    """A captured call of both kernels on pages, replayed with tokens that belong to other sequences, then with fewer."""
    lens, new = [700, 300, 1500], [1, 20, 19]
    cache = ref.Cache(lens, 2, 32, 128, 128, seed=7)
    dev = cache.to_device("cuda")
    q = queries(new, 8, 128).cuda()
    cu = torch.tensor(offsets(new), dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(3, 8, 2, 40, 30, 0, 128, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(40, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(8, 40, device="cuda")
    call = lambda: fa.attention_forward_paged(q, *dev, cu, 30, out=out, lse=lse, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for now in (new, [30, 2, 8], [0, 1, 30], [2, 2, 1]):
        cu.copy_(torch.tensor(offsets(now), dtype=torch.int32))
        out.fill_(-3.0)
        lse.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status()[0] == 0
        used = sum(now)
        want = ref.attention(q[:used], cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, lens, offsets(now),
                             32, True)
        ref.check_attention(out[:used], lse[:, :used], want, EPS_F16, f"replay {now}")
        assert (out[used:] == -3.0).all() and (lse[:, used:] == -3.0).all()


def test_two_calls_at_once(fa):
    """Two streams, each with its own workspace, outputs and batch."""
    batches = [([900, 40, 3000], [1, 1, 1]), ([500, 2500, 60], [6, 1, 20])]
    streams, got, want = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for i, (lens, new) in enumerate(batches):
        cache = ref.Cache(lens, 2, 64, 128, 128, seed=i)
        q = queries(new, 8, 128, i)
        want.append(ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, lens, offsets(new), 64,
                                  True))
        got.append((q.cuda(), cache.to_device("cuda"), torch.tensor(offsets(new), dtype=torch.int32, device="cuda"), max(new)))
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(20):
        for i, (q, dev, cu, most) in enumerate(got):
            with torch.cuda.stream(streams[i]):
                results[i].append(fa.attention_forward_paged(q, *dev, cu, most))
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    for i in range(2):
        ref.check_attention(*results[i][0], want[i], EPS_F16, f"stream {i}")
        for o, lse in results[i][1:]:
            assert torch.equal(o, results[i][0][0]) and torch.equal(lse, results[i][0][1])


@pytest.mark.parametrize("n", [1, 10, 80])
def test_bad_pages_and_lengths_are_reported(fa, n):
    """Found on the device before anything is read: reported, and the other sequences are right."""
    lens, new = [100, 64, 200], [n, n, n]
    cache = ref.Cache(lens, 2, 32, 128, 128, seed=2)
    q = queries(new, 4, 128)
    cu = torch.tensor(offsets(new), dtype=torch.int32, device="cuda")
    want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, lens, offsets(new), 32, True)

    def call(change):
        dev = list(cache.to_device("cuda"))
        c = cu.clone()
        change(dev, c)
        o, lse = fa.attention_forward_paged(q.cuda(), *dev, c, n, total_k=sum(lens))
        torch.cuda.synchronize()
        return o, lse, fa.fa_device_status()

    def others_right(o, lse):
        if n == 80:
            return  # nothing of the long sequences is computed
        keep = [*range(n), *range(2 * n, 3 * n)]
        sub = (want[0][keep], want[1][:, keep], want[2][keep], want[3][keep], want[4][keep])
        ref.check_attention(o[keep], lse[:, keep], sub, EPS_F16 if n == 1 else EPS_BF16)

    for value in (-1, cache.num_pages, 1 << 30):
        def change(dev, c):
            dev[4][1, 1] = value
        o, lse, (code, detail) = call(change)
        assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (512, 1), (code, detail)
        others_right(o, lse)
    for length in (-5, cache.width * 32 + 1, 2 ** 31 - 1):
        def change(dev, c):
            dev[5][1] = length
        o, lse, (code, detail) = call(change)
        assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 1), (code, detail)
        others_right(o, lse)

    def change(dev, c):
        c[2] = c[3] + 1
    _, _, (code, detail) = call(change)
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 511, (code, detail)
    o, lse, (code, detail) = call(lambda dev, c: None)
    assert code == 0, detail


def test_more_keys_than_said_are_reported(fa):
    cache = ref.Cache([100, 64], 2, 32, 128, 128)
    q = queries([70, 1], 4, 128).cuda()
    dev = cache.to_device("cuda")
    cu = torch.tensor([0, 70, 71], dtype=torch.int32, device="cuda")
    fa.attention_forward_paged(q, *dev, cu, 70, total_k=99)  # 140 rows: beyond what is read from the pages
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 513, (code, detail)
    fa.attention_forward_paged(q, *dev, cu, 70, total_k=100)  # the single token's keys are not unpacked
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0


def test_agrees_with_the_dense_forward(fa):
    """The same values as bf16 rows through attention_forward: both are within their bounds of the same sum."""
    page, lens, new = 64, [700, 700], [1, 1]
    cache = ref.Cache(lens, 2, page, 128, 128, seed=7)
    q = queries(new, 8, 128)
    o, lse = run(fa, cache, new, q)
    rows = []
    for name in ("k", "v"):
        codes, scale = getattr(cache, name), getattr(cache, name + "_scale")
        rows.append(torch.stack([ref.dense(codes, scale, cache.table[b], 700, page) for b in range(2)])
                    .transpose(1, 2).to(torch.bfloat16).contiguous().cuda())
    od, ld = fa.attention_forward_splitkv(q.view(2, 1, 8, 128).cuda(), *rows, causal=True)
    want = ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, lens, [0, 1, 2], page, True)
    ref.check_attention(o, lse, want, EPS_F16)
    ref.check_attention(od.view(2, 8, 128), ld.view(2, 8).t().contiguous(), want, EPS_BF16)
