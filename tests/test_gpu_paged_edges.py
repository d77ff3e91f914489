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
