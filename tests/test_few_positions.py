"""Masked and shared decodes that see a few positions, where nothing averages the roundings of small weights.

A tile's operands below 2^-6 have steps of 2^-9 (64 rows), and an offset of up to half a step is added before they are rounded: a
step in all.  A row that meets its first tile puts its largest operand, weight x scale mantissa (below 2), at 2^3.75 or above.  The
oracle's floor counts weight x 2^floor(log2 scale), so an operand is off by at most 2^-9 / 2^3.75 x 2 = 2^-11.75 of it where
masked_util has 2^-13.75 (half a step, no offset, no mantissa).  Results below 2^-126 may be flushed to zero."""
import pytest
import torch

import test_masked_decode as masked
import test_shared_decode as shared
from cache_util import bits, make_dense
from masked_util import check_decode
from oracle import masked_oracle

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _check(out, lse, want):
    want = list(want)
    want[3] = 4 * want[3] + 2.0 ** (13.75 - 126)
    check_decode(out, lse, want)


@pytest.mark.parametrize("H", [16, 17, 64, 128])
@pytest.mark.parametrize("q_scale", [0.1, 1.0, 6.0])
@pytest.mark.parametrize("form", ["plain", "cap", "slopes", "window"])
def test_masked(H, q_scale, form):
    lens = [1, 2, 3, 5, 14, 27, 44, 0, 121]
    q, cache, bt, ln = make_dense(lens, H, seed=H, q_scale=q_scale)
    cap = 30.0 if form == "cap" else 0.0
    slopes = torch.tensor(masked._alibi(H)) if form == "slopes" else None
    starts = [max(0, n - 3) for n in lens] if form == "window" else None
    want = masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(), SCALE, cap,
                                       None if slopes is None else slopes.numpy(), starts, None)
    for wide in masked._row_groups(q, cache, bt):
        out, lse, err = masked._run(q, cache, wide, ln, cap, slopes, masked._i32(starts))
        assert err == 0
        _check(out, lse, want)


@pytest.mark.parametrize("H,s_q", [(16, 3), (64, 1), (100, 2)])
@pytest.mark.parametrize("q_scale", [0.1, 1.0, 6.0, 30.0])
@pytest.mark.parametrize("n", [0, 1, 3, 40])
def test_shared(H, s_q, q_scale, n):
    case = shared.make([n], [max(0, x - (s_q - 1 - j)) for x in (0, 1, 2, 7, 3) for j in range(s_q)], H, s_q, seed=H + n,
                       q_scale=q_scale)
    for c in (case, shared._widened(case)):
        out, lse, err = shared._run(c)
        assert err == 0
        _check(out, lse, shared._want(c))
