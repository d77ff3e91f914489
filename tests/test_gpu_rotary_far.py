"""The rotary table's values to the bound that the header gives, relative to each value, against frequencies of 60 digits:
far positions, and among all positions those whose cosine or sine is the smallest."""
import math
from decimal import Decimal, getcontext

import pytest

torch = pytest.importorskip("torch")
from test_gpu_rotary import fa, ok  # noqa: E402, F401  (fa: the fixture)

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
BITS = 160


def exact_turns(rot, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    """(scaled, plain) frequencies in turns as integers of 2^-160, of the doubles that the call gets."""
    getcontext().prec = 60
    base, factor, original, low, high = (Decimal(x) for x in (base, factor, original, low, high))
    if scaling == "base":
        base *= (factor.ln() * rot / (rot - 2)).exp()
    out = []
    for i in range(rot // 2):
        plain = f = (-2 * base.ln() * i / rot).exp() / (2 * PI)
        if scaling == "linear":
            f = f / factor
        if scaling == "by_parts":
            w = min(Decimal(1), max(Decimal(0), (original * f - low) / (high - low)))
            f = w * f + (1 - w) * f / factor
        out.append((int(f * 2 ** BITS), float(plain)))
    return out, float(base.ln())


def cos_sin(turns):
    """(cos, sin) of an angle in 2^-160 turns, relative to 2^-50 of each."""
    quarter, rest = divmod(turns + (1 << (BITS - 3)), 1 << (BITS - 2))
    x = (rest - (1 << (BITS - 3))) / 2 ** BITS * (2 * math.pi)  # at most an eighth of a turn; the quotient of integers rounds once
    c, s = math.cos(x), math.sin(x)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quarter % 4]


@pytest.mark.parametrize("positions,rot,base,magnitude,kw", [
    (1 << 22, 16, 10000.0, 1.0, dict()), (1 << 20, 64, 500000.0, 1.25, dict(scaling="linear", factor=3.0)),
    (1 << 20, 48, 10000.0, 0.7, dict(scaling="base", factor=10.5)),
    (1 << 20, 64, 10000.0, 1.2772588722239782, dict(scaling="by_parts", factor=16.0, original=8192.0, low=1.0, high=32.0)),
    (1 << 20, 64, 1e7, 1.0, dict(scaling="by_parts", factor=10.5, original=5000.0, low=3.9, high=4.1)),
    (300, 192, 1e300, 1.0, dict()), (1 << 24, 16, 1.0, 1.0, dict())], ids=lambda x: str(x) if not isinstance(x, dict) else x.get("scaling", "none"))
def test_values_to_the_stated_bound(fa, positions, rot, base, magnitude, kw):  # noqa: F811
    """A frequency in double: (2 ln base + 8) 2^-53 of itself, by parts (ln base + 10) (1 + high / (high - low)) 2^-53 of the
    unscaled one; half of 2^-64 turns for its fraction.  The value: the angle's two parts are rounded to fp32 with their
    factors and summed, 2.5 steps of 2^-24 of it and 2^-51 where they cancel; the series 1.6 steps; the magnitude's rounding
    and its product two."""
    got = fa.rotary_table(positions, rot, base=base, magnitude=magnitude, **kw)
    ok(fa)
    turns, ln_base = exact_turns(rot, base, **kw)
    g = torch.Generator().manual_seed(0)
    half, worst = rot // 2, 0.0
    spread = 1 + kw["high"] / (kw["high"] - kw["low"]) if kw.get("scaling") == "by_parts" else None
    for i in sorted({0, 1, 2, half // 3, half // 2, half - 1}):
        rel = (2 * ln_base + 8 if spread is None else (ln_base + 10) * spread) * 2.0 ** -53
        pick = [torch.randint(0, positions, (200,), generator=g), torch.arange(max(0, positions - 100), positions),
                torch.arange(min(positions, 100))]
        for column in (i, half + i):
            pick.append(got[:, column].abs().topk(min(200, positions), largest=False).indices.cpu())
        pick = torch.unique(torch.cat(pick))
        values = got[pick.cuda()][:, [i, half + i]].double().cpu().tolist()
        for p, pair in zip(pick.tolist(), values):
            f = turns[i][0] / 2 ** BITS if spread is None else turns[i][1]
            angle = p * (f * rel + 2.0 ** -65) * 2 * math.pi
            for have, want in zip(pair, cos_sin(p * turns[i][0])):
                bound = abs(magnitude) * (angle + abs(want) * 6.1 * 2.0 ** -24 + 2.0 ** -51) * (1 + 2.0 ** -20)
                worst = max(worst, abs(have - want * magnitude) / bound)
    assert worst <= 1, f"off by {worst:.3f} of the bound"
    print(f"off by {worst:.3f} of the bound")
