"""fa_kv_append on the GPU: codes and scales against the operator's definition, and the two operators run together."""
import math

import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 64), (128, 128), (192, 64), (192, 128)]


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def u8(t):
    return t.view(torch.uint8)


def expected(cache, x, name, new, dtype, cos_sin, rot, interleaved):
    """(codes, exponents) after the append of x [total, heads, d], by the definition, token by token, in `dtype`."""
    codes, scale = u8(getattr(cache, name)).clone(), u8(getattr(cache, name + "_scale")).clone()
    page = cache.page
    done = 0
    for b, (n, length) in enumerate(zip(new, cache.lens)):
        start = length - n
        part = x[done:done + n].to(dtype)
        if rot and n:
            part = ref.rotate(part, cos_sin[start:length], rot, interleaved)
        done += n
        j = start // page
        while j * page < length and n:
            lo, hi = max(start, j * page), min(length, (j + 1) * page)
            p = int(cache.table[b, j])
            for h in range(cache.heads):
                vals = part[lo - start:hi - start, h]
                finite = vals[torch.isfinite(vals)]
                amax = finite.abs().max().item() if finite.numel() else 0.0
                e = ref.needed_scale(amax) + 127
                old = lo - j * page
                if old:
                    e = max(e, int(scale[p, h]))
                    was = codes[p, h, :old].view(torch.float8_e4m3fn).to(dtype) * 2.0 ** (int(scale[p, h]) - e)
                    codes[p, h, :old] = u8(was.float().to(torch.float8_e4m3fn))
                now = torch.where(torch.isfinite(vals), vals, torch.full_like(vals, math.nan)) * 2.0 ** (127 - e)
                codes[p, h, old:old + hi - lo] = u8(now.float().to(torch.float8_e4m3fn))
                scale[p, h] = e
            j += 1
    return codes, scale


def same_codes(got, want):
    """Equal bytes, any NaN code counting as any other."""
    g, w = got.clone(), want.clone()
    g[(g & 0x7F) == 0x7F] = 0x7F
    w[(w & 0x7F) == 0x7F] = 0x7F
    return torch.equal(g, w)


def tokens(new, heads_q, heads_kv, d_qk, d_v, seed=0, size=1.0):
    """q, k, v as views of one projection's output."""
    g = torch.Generator().manual_seed(seed + 7)
    width = [heads_q * d_qk, heads_kv * d_qk, heads_kv * d_v]
    qkv = (torch.randn(sum(new), sum(width), generator=g) * size).to(torch.bfloat16).cuda()
    q, k, v = qkv.split(width, 1)
    return q.unflatten(1, (heads_q, d_qk)), k.unflatten(1, (heads_kv, d_qk)), v.unflatten(1, (heads_kv, d_v))


def append(fa, dev, new, k, v, **kw):
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    out = fa.kv_append(k, v, *dev, cu, **kw)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, f"device status {code} {detail}"
    return out


def check(fa, lens, new, heads_q, heads_kv, dims, page, rot, interleaved=False, layout="heads", seed=0, size=1.0):
    cache = ref.Cache(lens, heads_kv, page, *dims, seed=seed, layout=layout)
    # bytes behind a sequence's last token are any bytes; tokens to come are overwritten
    dev = cache.to_device("cuda")
    q, k, v = tokens(new, heads_q, heads_kv, *dims, seed=seed, size=size)
    cs = ref.cos_sin_table(max(lens) + 1, rot) if rot else None
    qr = append(fa, dev, new, k, v, q=q, cos_sin=cs.cuda() if rot else None, interleaved=interleaved)
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        r = rot if name == "k" else 0
        codes, scale = expected(cache, x.cpu(), name, new, torch.float32, cs, r, interleaved)
        assert torch.equal(u8(dev[2 + i]).cpu(), scale), f"{name}: scales"
        assert same_codes(u8(dev[i]).cpu(), codes), f"{name}: codes"
        # and against 64 bits: half a step of e4m3, half its smallest step, three fp32 roundings of the rotation
        got = ref.code_values(dev[i].cpu()) * ref.scale_values(dev[2 + i].cpu())[..., None, None]
        done = 0
        for b, n in enumerate(new):
            start = lens[b] - n
            exact = x[done:done + n].double().cpu()
            biggest = exact.abs().amax().item() if n else 0.0
            if r and n:
                exact = ref.rotate(exact, cs[start:lens[b]].double(), r, interleaved)
            for t in range(n):
                p, slot = int(cache.table[b, (start + t) // page]), (start + t) % page
                s = ref.scale_values(dev[2 + i].cpu())[p][:, None]
                bound = 2.0 ** -4 * exact[t].abs() + 0.5 * ref.E4M3_TINY * s + 3 * 2.0 ** -24 * 2 * biggest
                assert ((got[p, :, slot] - exact[t]).abs() <= bound).all(), f"{name}: sequence {b} token {t}"
            done += n
    # queries: the rotation in fp32, one rounding
    where = torch.cat([torch.arange(length - n, length) for n, length in zip(new, lens)])
    if rot:
        want = ref.rotate(q.float().cpu(), cs[where], rot, interleaved).to(torch.bfloat16)
    else:
        want = q.cpu()
    assert torch.equal(qr.cpu(), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dims", DIMS)
def test_ragged_batch(fa, dims, page, interleaved):
    # fresh and begun pages, one token, none, a whole prompt, several pages
    lens = [1, 17, 40, 130, 131, 64, 200]
    new = [1, 1, 40, 3, 131, 0, 137]
    check(fa, lens, new, 6, 2, dims, page, min(dims[0], 64), interleaved, seed=page)


@pytest.mark.parametrize("rot", [0, 16, 48, 96, 192])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_columns(fa, rot, interleaved):
    check(fa, [30, 5], [4, 5], 4, 4, (192, 128), 32, rot, interleaved)


@pytest.mark.parametrize("layout", ["tokens", "apart"])
def test_other_orders_of_the_cache(fa, layout):
    check(fa, [70, 33], [35, 1], 4, 2, (128, 64), 32, 128, layout=layout)


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -60, 2.0 ** -8, 1e4, 1e37])
def test_sizes_of_values(fa, size):
    check(fa, [90, 20], [35, 20], 4, 2, (64, 64), 32, 64, size=size)


def test_many_sequences(fa):
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(1, 90, (600,), generator=g).tolist()
    new = [min(n, int(k)) for n, k in zip(lens, torch.randint(0, 4, (600,), generator=g))]
    check(fa, lens, new, 2, 1, (64, 64), 16, 64)


def test_no_page_but_the_new_tokens_and_older_codes_changes(fa):
    lens, new, page = [50, 100], [2, 40], 32
    cache = ref.Cache(lens, 2, page, 64, 64, tail=0x33)
    dev = cache.to_device("cuda")
    _, k, v = tokens(new, 2, 2, 64, 64)
    append(fa, dev, new, k, v)
    written = torch.zeros(cache.num_pages, page, dtype=torch.bool)
    for b, n in enumerate(new):
        for t in range(lens[b] - n, lens[b]):
            written[int(cache.table[b, t // page]), t % page] = True
    touched = written.any(1)
    for i, name in enumerate(("k", "v")):
        before, after = u8(getattr(cache, name)), u8(dev[i]).cpu()
        assert torch.equal(before[~touched], after[~touched])
        held = torch.zeros_like(written)
        for b, length in enumerate(lens):
            for t in range(length):
                held[int(cache.table[b, t // page]), t % page] = True
        behind = ~held
        assert torch.equal(before.transpose(1, 2)[behind], after.transpose(1, 2)[behind])
        s0, s1 = u8(getattr(cache, name + "_scale")), u8(dev[2 + i]).cpu()
        assert torch.equal(s0[~touched], s1[~touched])


def test_scale_grows_and_older_codes_follow(fa):
    """Tokens appended one by one, each larger than the last: the older values stay within half a step of themselves."""
    page, heads, d = 32, 2, 64
    cache = ref.Cache([20], heads, page, d, d, spare=0)
    dev = list(cache.to_device("cuda"))
    p = int(cache.table[0, 0])
    g = torch.Generator().manual_seed(3)
    stored = []
    for t in range(20):
        x = (torch.randn(1, heads, d, generator=g) * 1.5 ** t).to(torch.bfloat16)
        dev[5].fill_(t + 1)
        append(fa, dev, [1], x.cuda(), x.cuda())
        stored.append(x[0])
        got = ref.code_values(dev[0].cpu()) * ref.scale_values(dev[2].cpu())[..., None, None]
        s = ref.scale_values(dev[2].cpu())[p][:, None]
        for i, y in enumerate(stored):
            # one rounding to e4m3 in all but the subnormal codes, where every growth may add half a step
            bound = 2.0 ** -4 * y.double().abs() + ref.E4M3_TINY * s
            assert ((got[p, :, i] - y.double()).abs() <= bound).all()
    at_once = ref.Cache([20], heads, page, d, d, spare=0)
    dev2 = at_once.to_device("cuda")
    every = torch.stack(stored).cuda()
    append(fa, dev2, [20], every, every)
    assert torch.equal(u8(dev2[2]), u8(dev[2]))  # the same scales


def test_a_begun_page_of_a_fresh_sequence_ignores_the_old_scale(fa):
    cache = ref.Cache([5], 1, 16, 64, 64)
    u8(cache.k_scale).fill_(200)
    u8(cache.v_scale).fill_(200)
    dev = cache.to_device("cuda")
    _, k, v = tokens([5], 1, 1, 64, 64)
    append(fa, dev, [5], k, v)
    p = int(cache.table[0, 0])
    assert int(u8(dev[2])[p, 0]) < 127 and int(u8(dev[3])[p, 0]) < 127


def test_values_that_are_no_numbers(fa):
    cache = ref.Cache([40], 2, 32, 64, 64)
    dev = cache.to_device("cuda")
    _, k, v = tokens([3], 2, 2, 64, 64)
    k, v = k.clone(), v.clone()
    k[1, 0, 3] = math.inf
    v[1, 1, 4] = -math.inf
    v[2, 0, 5] = math.nan
    k[0] = math.nan
    v[0, 0] = math.inf
    append(fa, dev, [3], k, v)
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        codes, scale = expected(cache, x.cpu(), name, [3], torch.float32, None, 0, False)
        assert torch.equal(u8(dev[2 + i]).cpu(), scale) and same_codes(u8(dev[i]).cpu(), codes)
    p = int(cache.table[0, 1])
    assert torch.isnan(dev[0].float()[p, 0, 37 % 32]).all()


def test_queries_in_place_and_without_queries(fa):
    lens, new = [30, 9], [2, 9]
    cs = ref.cos_sin_table(40, 64).cuda()
    got = []
    for case in ("apart", "in place", "none"):
        cache = ref.Cache(lens, 2, 16, 64, 64)
        dev = cache.to_device("cuda")
        q, k, v = tokens(new, 4, 2, 64, 64)
        if case == "apart":
            first = append(fa, dev, new, k, v, q=q, cos_sin=cs)
        elif case == "in place":
            q = q.contiguous()
            assert append(fa, dev, new, k, v, q=q, cos_sin=cs, q_out=q) is q
            assert torch.equal(q, first)
        else:
            assert append(fa, dev, new, k, v, cos_sin=cs) is None
        got.append((u8(dev[0]).clone(), u8(dev[1]).clone(), u8(dev[2]).clone(), u8(dev[3]).clone()))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_full_pages_may_be_shared(fa):
    """Two sequences behind one cached prefix of whole pages."""
    cache = ref.Cache([64, 40], 2, 32, 64, 64)
    cache.table = torch.tensor([[0, 1, 2], [0, 3, -1]], dtype=torch.int32)
    cache.lens, cache.seqlens = [66, 40], torch.tensor([66, 40], dtype=torch.int32)
    dev = cache.to_device("cuda")
    _, k, v = tokens([2, 8], 2, 2, 64, 64)
    append(fa, dev, [2, 8], k, v)
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        codes, scale = expected(cache, x.cpu(), name, [2, 8], torch.float32, None, 0, False)
        assert torch.equal(u8(dev[2 + i]).cpu(), scale) and same_codes(u8(dev[i]).cpu(), codes)


def test_offsets_beyond_32_bits(fa):
    page, heads, d = 64, 8, 128
    pages = (1 << 32) // (page * heads * d) + 4
    k = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((pages, heads), 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    dev = (k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks.view(torch.float8_e8m0fnu),
           vs.view(torch.float8_e8m0fnu), torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda"),
           torch.tensor([70], dtype=torch.int32, device="cuda"))
    _, kn, vn = tokens([70], 8, heads, d, d)
    append(fa, dev, [70], kn, vn)
    for i, x in enumerate((kn, vn)):
        for j, p in enumerate((pages - 1, pages - 2)):
            part = x[j * page:(j + 1) * page].float().cpu()
            got = dev[i][p].float().cpu() * ref.scale_values(dev[2 + i].cpu())[p].float()[:, None, None]
            err = (got[:, :part.shape[0]].transpose(0, 1) - part).abs()
            assert (err <= 2.0 ** -4 * part.abs() + 2.0 ** -10).all()
        assert not u8(dev[i])[:pages - 2].any()


def test_bad_pages_lengths_and_positions_are_reported(fa):
    lens, new = [40, 20, 33], [3, 20, 1]
    _, k, v = tokens(new, 2, 2, 64, 64)
    cu = torch.tensor([0, 3, 23, 24], dtype=torch.int32, device="cuda")
    cs = ref.cos_sin_table(45, 64).cuda()

    def call(change, table=cs):
        cache = ref.Cache(lens, 2, 16, 64, 64)
        dev, c = list(cache.to_device("cuda")), cu.clone()
        change(dev, c)
        fa.kv_append(k, v, *dev, c, cos_sin=table)
        torch.cuda.synchronize()
        return cache, dev, fa.fa_device_status()

    def others_right(cache, dev):
        for b in (0, 2):
            j = (lens[b] - 1) // 16
            p = int(cache.table[b, j])
            lo, hi = max(lens[b] - new[b] - 16 * j, 0), lens[b] - 16 * j
            x = v[int(cu[b + 1]) - (hi - lo):int(cu[b + 1])].float().cpu()
            got = dev[1][p].float().cpu() * ref.scale_values(dev[3].cpu())[p].float()[:, None, None]
            err = (got[:, lo:hi].transpose(0, 1) - x).abs()
            bound = 2.0 ** -4 * x.abs() + 2.0 ** -10 * ref.scale_values(dev[3].cpu())[p].float()[None, :, None]
            assert (err <= bound).all()

    for value in (-1, 1000, -2 ** 31):
        cache, dev, (code, detail) = call(lambda d, c: d[4][1].fill_(value))
        assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (512, 1), (code, detail)
        others_right(cache, dev)
    for length in (19, -1, 16 * 3 + 1, 2 ** 31 - 1):
        cache, dev, (code, detail) = call(lambda d, c: d[5][1:2].fill_(length))
        assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 1), (code, detail)
        others_right(cache, dev)
    cache, dev, (code, detail) = call(lambda d, c: None, cs[:35].contiguous())  # sequence 0 is at position 39
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (511, 0), (code, detail)
    for value in (30, -7):
        _, _, (code, detail) = call(lambda d, c: c[2:3].fill_(value))
        assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 511, (code, detail)
    _, _, (code, detail) = call(lambda d, c: None)
    assert code == 0, detail


@pytest.mark.parametrize("graph", [False, True])
def test_prompt_then_tokens(fa, graph):
    """A prompt appended and attended to, then tokens one by one (eagerly, or one captured step replayed): at every step
    the attention is that over the values the cache holds, and the cache holds the rotated keys."""
    heads_q, heads_kv, d, page, prompt, steps = 8, 2, 128, 16, [45, 70], 20
    end = [n + steps for n in prompt]
    cache = ref.Cache(end, heads_kv, page, d, d, tail=0x00)
    dev = list(cache.to_device("cuda"))
    cs = ref.cos_sin_table(max(end), d).cuda()
    q, k, v = tokens(prompt, heads_q, heads_kv, d, d)
    dev[5].copy_(torch.tensor(prompt, dtype=torch.int32))
    cu = torch.tensor([0, 45, 115], dtype=torch.int32, device="cuda")
    kept = [[k[:45].cpu()], [k[45:].cpu()]]
    qr = fa.kv_append(k, v, *dev, cu, q=q, cos_sin=cs)
    o, lse = fa.attention_forward_paged(qr, *dev, cu, 70)
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    want = ref.attention(qr, dev[0].cpu(), dev[1].cpu(), dev[2], dev[3], cache.table, prompt, [0, 45, 115], page, True)
    ref.check_attention(o, lse, want, 2.0 ** -8)

    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    qs, ks, vs = (torch.empty(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (heads_q, heads_kv, heads_kv))
    q1, o1 = torch.empty_like(qs), torch.empty_like(qs)
    l1 = torch.empty(heads_q, 2, device="cuda")
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(2, heads_q, heads_kv, 2, 1, 0, d, d), dtype=torch.uint8, device="cuda")

    def step():
        dev[5].add_(1)
        fa.kv_append(ks, vs, *dev, one, q=qs, cos_sin=cs, q_out=q1)
        fa.attention_forward_paged(q1, *dev, one, 1, out=o1, lse=l1, workspace=ws)

    g = None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for t in range(steps):
        a, b, c = tokens([1, 1], heads_q, heads_kv, d, d, seed=50 + t, size=1.0 + t % 5)
        qs.copy_(a), ks.copy_(b), vs.copy_(c)
        for i in range(2):
            kept[i].append(b[i:i + 1].cpu())
        g.replay() if graph else step()
        torch.cuda.synchronize()
        assert fa.fa_device_status()[0] == 0
        lens = [n + t + 1 for n in prompt]
        assert dev[5].tolist() == lens
        want = ref.attention(q1, dev[0].cpu(), dev[1].cpu(), dev[2], dev[3], cache.table, lens, [0, 1, 2], page, True)
        ref.check_attention(o1, l1, want, 2.0 ** -11, f"step {t}")
    for b in range(2):
        x = ref.rotate(torch.cat(kept[b]).double(), cs.cpu()[:end[b]].double(), d, False)
        got = ref.dense(dev[0].cpu(), dev[2], cache.table[b], end[b], page).transpose(0, 1)
        # e4m3: half a step, and up to a whole smallest step under the page's scale (448 of it hold the largest value)
        big = x.abs().amax().item()
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + ref.E4M3_TINY * 2 * big / 448).all()
