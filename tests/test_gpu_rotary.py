"""Rotary positions on the GPU: the table and the rotation against 64 bits, strides, positions, gradients, refusals."""
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


def ok(fa):
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == 0, f"device status {code} {detail}"


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="by_parts", factor=32.0, original=4096.0, low=1.0, high=4.0),
            dict(scaling="by_parts", factor=10.5, original=100.0, low=0.0, high=32.0)]


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k.get("scaling", "none"))
@pytest.mark.parametrize("rot", [16, 32, 48, 64, 128, 176, 192])
@pytest.mark.parametrize("positions,base,magnitude", [(1, 10000.0, 1.0), (7, 1.0, 0.5), (1000, 500000.0, 1.25), (70001, 10000.0, 1.0)])
def test_table(fa, positions, base, magnitude, rot, kw):
    """The turns' fraction is off by 2^-64 a position and by the frequency's double rounding; the reduced angle, at most an
    eighth of a turn, is rounded to fp32 (2^-24 of itself), sincospif is off by 2 units of the last place, the product
    with the magnitude rounds once more."""
    out = torch.full((positions + 1, rot), 7.0, device="cuda")
    fa.rotary_table(positions, rot, base=base, magnitude=magnitude, out=out[:positions], **kw)
    ok(fa)
    assert (out[positions] == 7.0).all()
    pos = torch.arange(positions, dtype=torch.float64)[:, None]
    angle = pos * want.frequencies(rot, base, **kw)
    exact = torch.cat([angle.cos(), angle.sin()], 1) * magnitude
    slack = angle.repeat(1, 2) * 2.0 ** -50 + pos * 2.0 ** -60  # frequencies in double, fractions of 2^64
    bound = magnitude * (exact.abs() / magnitude * 3 * 2.0 ** -23 + math.pi / 4 * 2.0 ** -24 + slack)
    assert ((out[:positions].double().cpu() - exact).abs() <= bound).all()


def test_table_of_far_positions(fa):
    """A million positions: the angle's fraction is still exact where fp32 would keep 4 bits of it."""
    n = 1 << 20
    got = fa.rotary_table(n, 16, base=10000.0)
    ok(fa)
    pos = torch.arange(n - 5000, n, dtype=torch.float64)[:, None]
    angle = pos * want.frequencies(16, 10000.0)
    exact = torch.cat([angle.cos(), angle.sin()], 1)
    assert ((got[-5000:].double().cpu() - exact).abs() <= 2.0 ** -22 + angle.repeat(1, 2) * 2.0 ** -50).all()


CASES = [(1, 1, 64, 64), (4, 2, 64, 16), (3, 3, 128, 128), (8, 1, 128, 48), (32, 8, 128, 128), (5, 5, 192, 64), (16, 16, 192, 192),
         (1, 1, 192, 16), (9, 3, 192, 176)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [1, 3, 200, 5000])
@pytest.mark.parametrize("hq,hk,d,rot", CASES)
def test_rotation(fa, hq, hk, d, rot, tokens, interleaved, backward):
    """Any positions of the table; queries as views of a projection, keys by themselves, into a strided result."""
    if tokens * hq * d > 2e6 and hq != 16:
        tokens = 700
    both = normal(tokens, hq * d + 24, seed=tokens)
    q, k = both[:, 16:16 + hq * d].view(tokens, hq, d), normal(tokens, hk, d, seed=1)
    cs = ref.cos_sin_table(300, rot)
    pos = torch.randint(0, 300, (tokens,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    dev = both.cuda()
    k_wide = torch.full((tokens, hk + 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
    call = fa.rotary_backward if backward else fa.rotary
    qo, ko = call(dev[:, 16:16 + hq * d].view(tokens, hq, d), k.cuda(), cs.cuda(), positions=pos.cuda(), interleaved=interleaved,
                  k_out=k_wide[:, 1:1 + hk])
    ok(fa)
    want.check_turned(qo, *want.turn(q, cs[pos.long()], interleaved, backward), "q")
    want.check_turned(ko, *want.turn(k, cs[pos.long()], interleaved, backward), "k")
    assert torch.equal(qo[..., rot:].cpu(), q[..., rot:])
    assert (k_wide[:, 0] == 3.0).all() and (k_wide[:, -1] == 3.0).all()


@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128), (192, 64)])
@pytest.mark.parametrize("new", [[5], [0, 0, 3, 0], [1] * 40, [300, 0, 1, 77], [1, 2, 3] * 30 + [900]])
def test_positions_of_packed_sequences(fa, new, d, rot):
    """Each sequence counts from 0; rows before, between and behind the sequences keep what they hold."""
    cu = [2]
    for n in new:
        cu.append(cu[-1] + n)
    total = cu[-1] + 3
    q, k = normal(total, 4, d), normal(total, 2, d, seed=1)
    cs = ref.cos_sin_table(max(max(new), 1), rot)
    q_out = torch.full((total, 4, d), 3.0, dtype=torch.bfloat16, device="cuda")
    k_dev = k.cuda()
    fa.rotary(q.cuda(), k_dev, cs.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), q_out=q_out, k_out=k_dev)
    ok(fa)
    pos = torch.tensor([i for n in new for i in range(n)], dtype=torch.long)
    keep = slice(cu[0], cu[-1])
    want.check_turned(q_out[keep], *want.turn(q[keep], cs[pos], False))
    want.check_turned(k_dev[keep], *want.turn(k[keep], cs[pos], False))
    assert (q_out[:2] == 3.0).all() and (q_out[cu[-1]:] == 3.0).all()
    assert torch.equal(k_dev[:2].cpu(), k[:2]) and torch.equal(k_dev[cu[-1]:].cpu(), k[cu[-1]:])


def test_dense_batches_and_one_sequence(fa):
    cs = ref.cos_sin_table(50, 64)
    wide = normal(3, 50, 4 + 2 + 2, 128)
    dev = wide.cuda()
    q, k = fa.rotary(dev[:, :, :4], dev[:, :, 4:6], cs.cuda())
    ok(fa)
    for got, x in ((q, wide[:, :, :4]), (k, wide[:, :, 4:6])):
        w, size = want.turn(x.reshape(150, -1, 128), cs.repeat(3, 1), False)
        want.check_turned(got.reshape(150, -1, 128), w, size)
    flat = wide[0, :, :4]
    got, none = fa.rotary(flat.cuda(), None, cs.cuda())
    ok(fa)
    assert none is None and torch.equal(got, q[0])
    pos = torch.randint(0, 50, (3, 50), dtype=torch.int32)
    none, got = fa.rotary(None, dev[:, :, 4:6], cs.cuda(), positions=pos.cuda(), interleaved=True)
    ok(fa)
    want.check_turned(got.reshape(150, 2, 128), *want.turn(wide[:, :, 4:6].reshape(150, 2, 128), cs[pos.flatten().long()], True))
    empty = fa.rotary(torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda"), None, cs.cuda())[0]
    assert empty.shape == (0, 4, 128)


def test_in_place_over_a_projection(fa):
    both = normal(33, 6 * 64).cuda()
    before = both.cpu().clone()
    cs = ref.cos_sin_table(33, 64)
    q = both[:, :256].view(33, 4, 64)
    fa.rotary(q, None, cs.cuda(), q_out=q)
    ok(fa)
    want.check_turned(q, *want.turn(before[:, :256].view(33, 4, 64), cs, False))
    assert torch.equal(both[:, 256:].cpu(), before[:, 256:])


def test_infinities_and_nan_stay_in_their_pairs(fa):
    x = normal(4, 2, 64)
    x[1, 0, 3], x[2, 1, 40] = math.inf, math.nan
    cs = ref.cos_sin_table(4, 64)
    got = fa.rotary(x.cuda(), None, cs.cuda())[0].cpu()
    ok(fa)
    hit = torch.zeros(4, 2, 64, dtype=torch.bool)
    hit[1, 0, [3, 35]] = hit[2, 1, [8, 40]] = True
    assert not torch.isfinite(got[hit]).any() and torch.isfinite(got[~hit]).all()


@pytest.mark.parametrize("bad", [-1, 50, -2 ** 31, 2 ** 31 - 1])
def test_positions_outside_the_table_are_reported(fa, bad):
    x = normal(9, 2, 64)
    pos = torch.arange(9, dtype=torch.int32)
    pos[4] = bad
    cs = ref.cos_sin_table(50, 64)
    out = torch.full((9, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.rotary(x.cuda(), None, cs.cuda(), positions=pos.cuda(), q_out=out)
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1:] == (514, 4)
    keep = [i for i in range(9) if i != 4]
    assert (out[4] == 3.0).all()
    want.check_turned(out[keep], *want.turn(x[keep], cs[pos[keep].long()], False))


@pytest.mark.parametrize("cu,index", [([0, 5, 3, 9], 1), ([-1, 2, 4, 9], 0), ([0, 2, 4, 10], 2), ([0, 2 ** 31 - 1, 4, 9], 0)])
def test_bad_offsets_are_reported(fa, cu, index):
    x = normal(9, 2, 64).cuda()
    fa.rotary(x, None, ref.cos_sin_table(50, 64).cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    code, detail = fa.fa_device_status()
    assert code == fa.FA_ERR_INVALID_ARG and detail[1] == 511


def test_refused_tensors(fa):
    x, cs = normal(6, 2, 64).cuda(), ref.cos_sin_table(50, 64).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(q=x.float()), dict(q=x[0]), dict(q=x.transpose(0, 1)), dict(q=x[..., ::2]), dict(cos_sin=cs.double()),
               dict(cos_sin=cs[:, :40]), dict(cos_sin=cs.cpu()), dict(cos_sin=cs[0]), dict(positions=torch.zeros(5, **i32)),
               dict(positions=torch.zeros(6, device="cuda")), dict(positions=torch.zeros(6, dtype=torch.int32)),
               dict(positions=torch.zeros(6, **i32), cu_seqlens=torch.zeros(2, **i32)), dict(cu_seqlens=torch.zeros(0, **i32)),
               dict(q_out=x.float()), dict(q_out=x[:5]), dict(k_out=x), dict(k=normal(6, 2, 128).cuda()),
               dict(k=normal(5, 2, 64).cuda()), dict(q=normal(2, 3, 4, 2, 64).cuda())):
        args = {"q": x, "k": None, "cos_sin": cs, **kw}
        with pytest.raises(fa.FaError):
            fa.rotary(**args)
    assert fa.fa_device_status()[0] == 0


def test_same_rotation_as_the_append(fa):
    """kv_append's rotated queries, bit by bit."""
    cache = ref.Cache([40, 7], 2, 16, 128, 64)
    q, k, v = normal(12, 4, 128).cuda(), normal(12, 2, 128, seed=1).cuda(), normal(12, 2, 64, seed=2).cuda()
    cs = fa.rotary_table(40, 96, scaling="by_parts", factor=4.0, original=20.0, high=4.0)
    cu = torch.tensor([0, 9, 12], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        got = fa.kv_append(k, v, *cache.to_device("cuda"), cu, q=q, cos_sin=cs, interleaved=interleaved)
        pos = torch.tensor([*range(31, 40), 4, 5, 6], dtype=torch.int32, device="cuda")
        assert torch.equal(got, fa.rotary(q, None, cs, positions=pos, interleaved=interleaved)[0])
    ok(fa)


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_gradient(fa, interleaved):
    """Against differences of the forward pass along a random direction h: g . (R(x + h) - R(x - h)) / 2 = (R^T g) . h up to
    each side's rounding to bf16 (2^-8 of every value)."""
    cs = fa.rotary_table(64, 64, magnitude=1.25)
    x, h, g = (normal(64, 3, 128, seed=s).cuda() for s in range(3))
    up, down = ((x.float() + s * h.float()).to(torch.bfloat16) for s in (1, -1))
    step = (up.double() - down.double()) / 2
    f = [fa.rotary(t, None, cs, interleaved=interleaved)[0].double() for t in (up, down)]
    back = fa.rotary_backward(g, None, cs, interleaved=interleaved)[0].double()
    ok(fa)
    left, right = (g.double() * (f[0] - f[1]) / 2).sum(), (back * step).sum()
    bound = ((g.double().abs() * (f[0].abs() + f[1].abs()) / 2).sum() + (back.abs() * step.abs()).sum()) * 2.0 ** -8 * 1.01
    assert abs(left - right) <= bound and abs(right) > 0
    # and the two maps are each other's transpose times the square of the magnitude
    turned = fa.rotary_backward(f[0].to(torch.bfloat16), None, cs, interleaved=interleaved)[0].double()
    exact = up.double().clone()
    exact[..., :64] *= 1.25 ** 2
    assert ((turned - exact).abs() <= (exact.abs() + 2 * f[0].abs().amax()) * 3 * 2.0 ** -8).all()


def test_training_step_through_attention(fa):
    """Rotation, attention, its backward pass and the rotation's: gradients of the unrotated q and k against fp64 autograd.

    The bound is the attention backward's own (2e-2 of the largest gradient) and two roundings to bf16 beside it."""
    B, S, Hq, Hk, d = 2, 130, 4, 2, 64
    q, k, v, g = (normal(B, S, h, d, seed=i) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    cs = fa.rotary_table(S, 32, scaling="linear", factor=2.0)
    qr, kr = fa.rotary(q.cuda(), k.cuda(), cs, interleaved=True)
    o, lse = fa.attention_forward(qr, kr, v.cuda(), causal=True)
    dq, dk, dv = fa.attention_backward(qr, kr, v.cuda(), o, lse, g.cuda(), causal=True)
    dq, dk = fa.rotary_backward(dq, dk, cs, interleaved=True, q_out=dq, k_out=dk)
    ok(fa)
    ql, kl, vl = (t.double().requires_grad_() for t in (q, k, v))

    def turned(x):
        c = cs.double().cpu()[None, :, None]
        cos, sin = c[..., :16], c[..., 16:]
        a, b = x[..., 0:32:2], x[..., 1:32:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., 32:]], -1)

    scores = torch.einsum("bihd,bjhd->bhij", turned(ql), turned(kl).repeat_interleave(2, 2)) / 8
    scores = scores.masked_fill(torch.ones(S, S).triu(1).bool(), -math.inf)
    out = torch.einsum("bhij,bjhd->bihd", scores.softmax(-1), vl.repeat_interleave(2, 2))
    out.backward(g.double())
    for got, x in ((dq, ql), (dk, kl), (dv, vl)):
        assert (got.double().cpu() - x.grad).abs().max() <= (2e-2 + 2 * 2.0 ** -8) * x.grad.abs().max()


def test_another_stream_and_a_graph(fa):
    x, cs = normal(500, 8, 128).cuda(), ref.cos_sin_table(500, 128).cuda()
    want_q = fa.rotary(x, None, cs)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rotary(x, None, cs, stream=side)[0]
    table = fa.rotary_table(500, 128, stream=side)
    side.synchronize()
    assert torch.equal(got, want_q)
    assert torch.equal(table, fa.rotary_table(500, 128))
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.rotary(x, None, cs, q_out=out)
    x.copy_(x.flip(1))
    graph.replay()
    ok(fa)
    assert torch.equal(out, want_q.flip(1))
