"""Edges of the paged 8-bit cache that need no GPU: the range checks of the kernels, compiled for the host, and the
checks and defaults of the Python binding."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_forward_08_gb300", "csrc")

RANGE_PROGRAM = r"""
#include <cstdio>
#include "fa_paged_range.h"
int main() {
  int kind, c0, c1, len, max_new;
  long long total, most;
  while (std::scanf("%d %d %d %d %lld %d %lld", &kind, &c0, &c1, &len, &total, &max_new, &most) == 7) {
    int start = 0, n = 0;
    const bool ok = kind == 0 ? fa::paged_append_range(c0, c1, len, total, most, start, n)
                              : fa::paged_attend_range(c0, c1, len, total, max_new, most, n);
    std::printf("%d %d %d\n", ok ? 1 : 0, start, n);
  }
}
"""


def test_range_checks_hold_for_any_offsets_and_lengths(tmp_path):
    """Offsets and lengths are device memory and may hold anything: the checks agree with unbounded integers and no step of
    them overflows (a signed overflow stops the program)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    source, program = tmp_path / "range.cpp", tmp_path / "range"
    source.write_text(RANGE_PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I",
                    CSRC, str(source), "-o", str(program)], check=True)
    low, high = -2 ** 31, 2 ** 31 - 1
    offsets = [low, low + 1, -7, -1, 0, 1, 20, 24, 25, high - 1, high]
    lengths = [low, low + 1, low + 20, -21, -20, -1, 0, 1, 19, 20, 21, 44, 45, 46, 1 << 30, high - 20, high]
    cases = [(kind, c0, c1, length, total, max_new, most) for kind in (0, 1) for c0 in offsets for c1 in offsets
             for length in lengths for total in (24, high) for max_new in (1, 24) for most in (45, 1 << 30)]
    run = subprocess.run([str(program)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, capture_output=True)
    assert run.returncode == 0, "an overflow"
    got = [tuple(map(int, line.split())) for line in run.stdout.splitlines()]
    assert len(got) == len(cases)
    for (kind, c0, c1, length, total, max_new, most), (ok, start, n) in zip(cases, got):
        new, rows = c1 - c0, 0 <= c0 <= c1 <= total
        if kind == 0:
            want = rows and new <= length <= most
        else:
            want = rows and new <= max_new and 0 <= length <= most
        assert ok == want, (kind, c0, c1, length, total, max_new, most)
        if ok:
            assert n == new and (kind == 1 or start == length - new)


def paged_tensors(pages=3, heads=2, page=16, d_qk=64, d_v=64, batch=2):
    """The cache's tensors as the binding takes them, on the CPU."""
    torch = pytest.importorskip("torch")
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    u8 = dict(dtype=torch.uint8)
    return dict(k_cache=torch.zeros(pages, heads, page, d_qk, **u8).view(f8),
                v_cache=torch.zeros(pages, heads, page, d_v, **u8).view(f8),
                k_scale=torch.zeros(pages, heads, **u8).view(e8), v_scale=torch.zeros(pages, heads, **u8).view(e8),
                block_table=torch.zeros(batch, 4, dtype=torch.int32), seqlens_k=torch.zeros(batch, dtype=torch.int32),
                cu_seqlens=torch.zeros(batch + 1, dtype=torch.int32))


def test_tensors_of_any_rank_are_refused_by_name():
    """A dimension too few or too many in any of the cache's tensors is an FaError that names it, nothing else."""
    import exact_attention_forward_08_gb300 as fa
    good = paged_tensors()
    assert fa._paged_cache(*good.values(), -1)[1:] == (2, 64, 64, 2, 64)
    for name in good:
        for change in (lambda t: t[0], lambda t: t[None], lambda t: t[..., 0], lambda t: t[..., None], lambda t: t.flatten()[0]):
            bad = dict(good)
            bad[name] = change(good[name])
            with pytest.raises(fa.FaError, match=name):
                fa._paged_cache(*bad.values(), -1)


def test_default_limit_of_keys_covers_every_batch():
    """What attention_forward_paged takes for total_k when none is given: never below the keys that the sequences of more
    than 128 rows can have, whatever the lengths (checked over all splits of the new tokens), and no more than that."""
    import exact_attention_forward_08_gb300 as fa

    def longest(batch, total, least, at=0):  # most sequences of `least` tokens or more among all splits of `total`
        if at == batch:
            return 0
        return max((n >= least) + longest(batch, total - n, least, at + 1) for n in range(total + 1))

    for ratio, most in ((128, 7), (64, 8), (43, 9), (129, 6), (40, 9)):  # 2, 3, 3, 1 and 4 tokens are more than 128 rows
        least = 128 // ratio + 1
        assert (least - 1) * ratio <= 128 < least * ratio
        for batch in (1, 2, 3):
            for total in range(most):
                assert fa._paged_total_k(batch, 1000, total, ratio) == 1000 * longest(batch, total, least)
    assert fa._paged_total_k(64, 32768, 96, 4) == 2 * 32768  # one prompt of 33 tokens and 63 single ones
    # the row limit is the library's: one row more than it asks for room for unpacked keys
    size = fa.fa_fwd_paged_workspace_size
    rows = fa._PAGED_ROWS
    assert size(1, 1, 1, rows, rows, 1 << 20, 64, 64) < 1 << 28 <= size(1, 1, 1, rows + 1, rows + 1, 1 << 20, 64, 64)
