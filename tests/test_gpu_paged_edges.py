"""Edges of the paged 8-bit cache on the GPU: values that no server writes on purpose, and what the two operators promise
about them."""
import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def cuda_offsets(new):
    return torch.tensor(offsets(new), dtype=torch.int32, device="cuda")


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("length", [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 19, -2 ** 31 + 20, -20, -1])
def test_append_leaves_out_lengths_far_below_zero(fa, length):
    """Lengths whose distance to the new tokens does not fit 32 bits: reported, nothing of the sequence stored."""
    lens, new = [40, 20, 33], [3, 20, 1]
    cache = ref.Cache(lens, 2, 16, 64, 64)
    dev = list(cache.to_device("cuda"))
    before = [t.view(torch.uint8).clone() for t in dev[:4]]
    dev[5][1] = length
    k, v = normal(24, 2, 64).cuda(), normal(24, 2, 64, seed=1).cuda()
    q, q_out = normal(24, 4, 64, seed=2).cuda(), torch.full((24, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.kv_append(k, v, *dev, cuda_offsets(new), q=q, cos_sin=ref.cos_sin_table(45, 64).cuda(), q_out=q_out)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 1), (code, detail)
    assert (q_out[3:23] == 3.0).all() and not (q_out[:3] == 3.0).all(-1).any() and not (q_out[23:] == 3.0).all(-1).any()
    mine = cache.table[1, :2].tolist()
    for now, was in zip(dev[:4], before):
        assert torch.equal(now.view(torch.uint8)[mine], was[mine])


EPS_F16, EPS_BF16 = 2.0 ** -11, 2.0 ** -8  # what a weight of the softmax may lose: the kernels on pages, the unpacked keys


def attend(fa, cache, new, q, causal=True, **kw):
    o, lse = fa.attention_forward_paged(q.cuda(), *cache.to_device("cuda"), cuda_offsets(new), max(new), causal=causal, **kw)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, f"device status {code} {detail}"
    return o, lse


def reference(q, cache, new, causal=True):
    return ref.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.lens, offsets(new), cache.page,
                         causal)


@pytest.mark.parametrize("exponent", [17, 20, 24])
@pytest.mark.parametrize("n", [1, 20, 80])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
def test_a_large_query_column_that_meets_no_key(fa, dims, n, exponent):
    """One column of the queries is 2^exponent and all keys are 0 there: the scores are those of the other columns, in all
    their bits (values down to 2^-31 of the row's largest are held exactly; the others here are 2^-6 and more)."""
    cache = ref.Cache([200], 2, 32, *dims, seed=3)
    cache.k.view(torch.uint8)[..., 0] = 0
    q = normal(n, 4, dims[0], seed=n)
    q = torch.where(q.abs() < 2.0 ** -6, torch.full_like(q, 2.0 ** -6), q)
    q[..., 0] = 2.0 ** exponent
    o, lse = attend(fa, cache, [n], q)
    # the reference's bound counts the products that are not 0 only
    ref.check_attention(o, lse, reference(q, cache, [n]), EPS_F16 if 2 * n <= 128 else EPS_BF16)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("q_exp,k_exp", [(-128, 118), (-105, 98), (-95, 88), (-90, 83), (100, -107), (124, -127)])
def test_queries_at_the_ends_of_the_exponents(fa, n, q_exp, k_exp):
    """Queries from bf16's subnormal numbers to its largest, against keys whose scales bring the scores back."""
    cache = ref.Cache([200], 2, 32, 64, 64, seed=5)
    cache.k_scale = ref.e8m0(torch.full(cache.k_scale.shape, k_exp))
    q = (normal(n, 4, 64, seed=n).double() * 2.0 ** q_exp).to(torch.bfloat16)
    assert q.abs().max() > 0 and torch.isfinite(q).all()
    o, lse = attend(fa, cache, [n], q)
    ref.check_attention(o, lse, reference(q, cache, [n]), EPS_F16)


@pytest.mark.parametrize("ratio", [2, 40])
@pytest.mark.parametrize("what", ["length", "negative length", "page", "new tokens", "short one"])
def test_a_bad_sequence_leaves_its_neighbours_right_beside_prompts(fa, what, ratio):
    """Sequences of more rows than are read from the pages, one of which (or a single token between them) is bad."""
    lens, new = [100, 64, 200, 50, 70], [80, 60, 90, 1, 65]
    most, index, site = 90, 1, 511
    cache = ref.Cache(lens, 2, 32, 64, 64, seed=2)
    dev, cu = list(cache.to_device("cuda")), offsets(new)
    q = normal(sum(new), 2 * ratio, 64, seed=4)
    if what == "length":
        dev[5][1] = cache.width * 32 + 1
    elif what == "negative length":
        dev[5][1] = -5
    elif what == "page":
        dev[4][1, 1], site = cache.num_pages, 512
    elif what == "new tokens":
        most, index = 85, 2
    else:
        dev[5][3], index = -1, 3
    o, lse = fa.attention_forward_paged(q.cuda(), *dev, cuda_offsets(new), most, total_k=sum(lens))
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (site, index), (code, detail)
    want = reference(q, cache, new)
    for b in range(5):
        if b != index:
            keep = slice(cu[b], cu[b + 1])
            part = (want[0][keep], want[1][:, keep], want[2][keep], want[3][keep], want[4][keep])
            ref.check_attention(o[keep], lse[:, keep], part, EPS_BF16, f"sequence {b}")


@pytest.mark.parametrize("total_k", [0, 1, None])
def test_prompts_without_keys_leave_rows_behind_the_last_sequence(fa, total_k):
    """No key in any sequence, more rows than are read from the pages: the sequences' rows are written, no others."""
    new = [90, 2]
    cache = ref.Cache([0, 0], 2, 32, 64, 64)
    q = normal(sum(new) + 7, 8, 64)
    out = torch.full((sum(new) + 7, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, sum(new) + 7), 3.0, device="cuda")
    attend(fa, cache, new, q, out=out, lse=lse, total_k=total_k)
    assert (out[:sum(new)] == 0).all() and torch.isneginf(lse[:, :sum(new)]).all()
    assert (out[sum(new):] == 3.0).all() and (lse[:, sum(new):] == 3.0).all()


def test_keys_where_none_were_said(fa):
    """total_k 0 and a prompt that has keys: reported, and nothing of it is written; the single token is computed."""
    lens, new = [100, 64], [90, 1]
    cache = ref.Cache(lens, 2, 32, 64, 64)
    q = normal(sum(new), 8, 64)
    out = torch.full((sum(new), 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, sum(new)), 3.0, device="cuda")
    fa.attention_forward_paged(q.cuda(), *cache.to_device("cuda"), cuda_offsets(new), 90, total_k=0, out=out, lse=lse)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 513, (code, detail)
    assert (out[:90] == 3.0).all() and (lse[:, :90] == 3.0).all()
    o, l, *rest = reference(q, cache, new)
    ref.check_attention(out[90:], lse[:, 90:], (o[90:], l[:, 90:], *(x[90:] for x in rest)), EPS_F16)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("token", [3, 200, 997])
@pytest.mark.parametrize("length,n", [(1000, 1), (1000, 4), (1000, 30), (1000, 60), (1000, 80), (9000, 1), (9000, 20)])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
def test_a_value_that_is_no_number_makes_whole_rows_so(fa, dims, length, n, token, causal):
    """One NaN code among a token's values, wherever the token lies and whichever kernel the rows select: every column and
    the log-sum-exp of the rows that see it are NaN, other rows and heads are what they are without it."""
    page, new = 16, [n]
    clean = ref.Cache([length], 2, page, *dims, seed=6)
    bad = ref.Cache([length], 2, page, *dims, seed=6)
    bad.v.view(torch.uint8)[int(bad.table[0, token // page]), 1, token % page, 5] = 0xFF
    q = normal(n, 4, dims[0], seed=1)
    o0, l0 = attend(fa, clean, new, q, causal)
    o1, l1 = attend(fa, bad, new, q, causal)
    assert torch.isfinite(o0).all() and torch.isfinite(l0).all()
    sees = torch.arange(n) + length - n >= token if causal else torch.ones(n, dtype=torch.bool)
    assert torch.isnan(o1[sees][:, 2:]).all() and torch.isnan(l1[2:][:, sees]).all()
    assert torch.equal(o1[:, :2], o0[:, :2]) and torch.equal(l1[:2], l0[:2])
    assert torch.equal(o1[~sees], o0[~sees]) and torch.equal(l1[:, ~sees], l0[:, ~sees])


@pytest.mark.parametrize("n", [1, 20, 80])
@pytest.mark.parametrize("what", ["key", "query"])
def test_a_key_or_query_that_is_no_number_makes_whole_rows_so(fa, what, n):
    clean, new = ref.Cache([500, 0], 2, 32, 128, 64, seed=6), [n, 1]
    bad = ref.Cache([500, 0], 2, 32, 128, 64, seed=6)
    q = normal(n + 1, 4, 128, seed=1)
    o0, l0 = attend(fa, clean, new, q)
    if what == "key":
        bad.k.view(torch.uint8)[int(bad.table[0, 1]), 1, 3, 7] = 0x7F
        hit = torch.zeros(n + 1, 4, dtype=torch.bool)
        hit[:n, 2:] = True
    else:
        q[n // 2, 1, 9] = float("nan")
        hit = torch.zeros(n + 1, 4, dtype=torch.bool)
        hit[n // 2, 1] = True
    o1, l1 = attend(fa, bad, new, q)
    assert torch.isnan(o1[hit]).all() and torch.isnan(l1.t()[hit]).all()
    assert torch.equal(o1[~hit], o0[~hit]) and torch.equal(l1.t()[~hit], l0.t()[~hit])
    assert (o1[n] == 0).all() and torch.isneginf(l1[:, n]).all()  # without a key


def test_new_tokens_of_any_rank_are_refused(fa):
    cache = ref.Cache([5], 2, 16, 64, 64)
    dev, cu = cache.to_device("cuda"), cuda_offsets([2])
    good = {"k": normal(2, 2, 64).cuda(), "v": normal(2, 2, 64).cuda(), "q": normal(2, 4, 64).cuda()}
    for name in good:
        for change in (lambda t: t[0], lambda t: t[None], lambda t: t[..., 0], lambda t: t.flatten()[0]):
            bad = {**good, name: change(good[name])}
            with pytest.raises(fa.FaError):
                fa.kv_append(bad["k"], bad["v"], *dev, cu, q=bad["q"])
            if name == "q":
                with pytest.raises(fa.FaError):
                    fa.attention_forward_paged(bad["q"], *dev, cu, 2)
    assert fa.fa_device_status()[0] == 0


def test_default_workspace_has_room_for_the_long_sequences_only(fa):
    """64 sequences with room for 32768 tokens each, one of them a prompt that is unpacked: without total_k the call asks
    for what the sequences of that many new tokens could hold, not for the whole block table (8.6 GB here)."""
    new, lens = [33] + [1] * 63, [40] + [1 + i for i in range(63)]
    cache = ref.Cache(lens, 8, 64, 128, 128, width=512)
    q = normal(sum(new), 32, 128)
    dev, cu, qd = cache.to_device("cuda"), cuda_offsets(new), q.cuda()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    o, lse = fa.attention_forward_paged(qd, *dev, cu, 33)
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    assert torch.cuda.max_memory_allocated() - before < 1 << 30
    ref.check_attention(o, lse, reference(q, cache, new), EPS_BF16)


@pytest.mark.parametrize("rows", [17, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)])
def test_weights_keep_eleven_bits_from_the_pages(fa, dims, rows):
    """17 to 128 rows and values' scales close to each other: the weights are f16, not bf16.  Sequences of few keys, where
    many of O's elements are small against their terms, show the difference.

    The bound: half a step of f16 for a weight (2^-11), what the scores' and sums' fp32 leaves (as in paged_ref), and for
    weights in f16's subnormal range 2^-25 of the unit they are kept in, which for a value of the tile's largest scale s
    is an eighth of 1 / s: 2^-28 of 448 s for each key."""
    lens = [2, 3, 4, 5, 6, 8, 11, 300, 1000]
    cache = ref.Cache(lens, 2, 64, *dims, seed=rows)
    new = [1] * len(lens)
    q = normal(len(lens), 2 * rows, dims[0], seed=rows)
    o, lse = attend(fa, cache, new, q)
    want = reference(q, cache, new)
    ow, lw, weight, delta, count = want
    tail = count[:, None, None] * 2.0 ** -28 * 448 * ref.scale_values(cache.v_scale).max()
    rel = EPS_F16 + 2.0 ** -20 + 2 * delta[..., None] + count[:, None, None] * 2.0 ** -24
    bound = (2.0 ** -8 * ow.abs() + (weight * rel + tail) * (1 + 2.0 ** -8)) * ref.SLACK
    worst = ((o.double().cpu() - ow).abs() / bound).max().item()
    assert worst <= 1.0, f"O off by {worst:.3f} of its bound"
    ref.check_attention(o, lse, want, EPS_BF16)


@pytest.mark.parametrize("n,eps,tail", [(1, EPS_F16, 2.0 ** -32), (8, EPS_F16, 2.0 ** -32), (20, EPS_BF16, 2.0 ** -22),
                                        (80, EPS_BF16, 0.0)])
def test_small_weights_of_large_values(fa, n, eps, tail):
    """Scores that differ by 2^60 and values' scales that differ as much: what a weight may lose is what the header says.

    Up to 16 rows the larger of 2^-11 of the weight and 2^-32 of the largest one, whatever its values; up to 128 rows 2^-8
    of it where the scales are far apart, or 2^-11 and 2^-28 S / s, at most 2^-22, where they are not; above 2^-8."""
    cache = ref.Cache([160], 2, 16, 64, 64, seed=4)
    g = torch.Generator().manual_seed(9)
    cache.v_scale = ref.e8m0(torch.randint(-40, 20, cache.v_scale.shape, generator=g))
    cache.k_scale = ref.e8m0(torch.randint(-4, -1, cache.k_scale.shape, generator=g))
    q = normal(n, 4, 64, seed=n)
    o, lse = attend(fa, cache, [n], q)
    ow, lw, weight, delta, count = reference(q, cache, [n])
    size = ref.dense(cache.v, cache.v_scale, cache.table[0], 160, 16).abs().sum(1).repeat_interleave(2, 0)  # [heads_q, d_v]
    rel = eps + 2.0 ** -20 + 2 * delta[..., None] + count[:, None, None] * 2.0 ** -24
    bound = (2.0 ** -8 * ow.abs() + (weight * rel + tail * size) * (1 + 2.0 ** -8)) * ref.SLACK
    worst = ((o.double().cpu() - ow).abs() / bound).max().item()
    assert worst <= 1.0, f"O off by {worst:.3f} of its bound"


@pytest.mark.parametrize("small", [-63, 55])
@pytest.mark.parametrize("n", [1, 20, 80])
def test_values_up_to_two_to_the_sixty_fourth(fa, n, small):
    """Values' scales of 2^55 throughout, and next to pages of the smallest scale that the append writes."""
    cache = ref.Cache([300], 2, 32, 128, 128, seed=4)
    exps = torch.full(cache.v_scale.shape, 55)
    exps[cache.table[0, :5].long()] = small  # the first tile's pages and one more
    cache.v_scale = ref.e8m0(exps)
    q = normal(n, 4, 128, seed=n)
    o, lse = attend(fa, cache, [n], q)
    wide = small != 55 and n == 20  # bf16 weights from the second tile on
    ref.check_attention(o, lse, reference(q, cache, [n]), EPS_F16 if n * 2 <= 128 and not wide else EPS_BF16)
