"""Attention over lists for prompts and for as many tokens as a call takes, against 64 bits on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
import paged_ref as ref  # noqa: E402
from test_gpu_lists import EPS_F16, fa  # noqa: E402, F401  (fa: the fixture)

pytestmark = pytest.mark.gpu


def attention(q, k, v, lists, lens):
    """paged_ref.attention's five results for tokens over lists; k, v [pages, heads, page, d] in 64 bits."""
    total, heads_q, d = q.shape
    heads = k.shape[1]
    at = torch.arange(heads, device=q.device)[None, :, None]
    k, v = (x[lists.long(), at].flatten(2, 3) for x in (k, v))
    q = q.double().view(total, heads, -1, d)
    s = 1.0 / math.sqrt(d)
    hidden = (torch.arange(k.shape[2], device=q.device) >= lens[:, None])[:, None, None]
    scores = (q @ k.transpose(2, 3) * s).masked_fill(hidden, -math.inf)
    lse = scores.logsumexp(-1)
    p = (scores - lse[..., None].nan_to_num(neginf=0.0)).exp()
    size = (q.abs() @ k.abs().transpose(2, 3) * s).masked_fill(hidden, 0.0).amax(-1)
    out = (p @ v).flatten(1, 2), lse.flatten(1, 2).t(), (p @ v.abs()).flatten(1, 2), size.flatten(1, 2) * (d + 8) * 2.0 ** -24
    return (*(x.cpu() for x in out), lens.double().cpu())


@pytest.mark.parametrize("total,width,hq,hkv,page,chunk", [(2500, 40, 8, 2, 16, 64), (3001, 9, 17, 1, 64, 64), (1 << 20, 1, 1, 1, 16, 1 << 15)])
def test_many_tokens(fa, total, width, hq, hkv, page, chunk):  # noqa: F811
    d, pages = 64, 500
    g = torch.Generator(device="cuda").manual_seed(total)
    codes = [(torch.randn(pages, hkv, page, d, generator=g, device="cuda").clamp(-4, 4) * 60).to(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.randint(-8, -4, (pages, hkv), generator=g, device="cuda") for _ in range(2)]
    scales = [(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu) for e in exps]
    values = [c.double() * (2.0 ** e.double())[..., None, None] for c, e in zip(codes, exps)]
    lists = torch.randint(0, pages, (total, hkv, width), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, width * page + 1, (total,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(total, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fa.attention_forward_lists(q, *codes, *scales, lists, lens)
    torch.cuda.synchronize()
    assert fa.fa_device_status()[0] == 0
    for t in range(0, total, chunk):
        rows = slice(t, min(t + chunk, total))
        ref.check_attention(o[rows], lse[:, rows], attention(q[rows], *values, lists[rows], lens[rows]), EPS_F16, f"tokens from {t}")
