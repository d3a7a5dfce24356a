"""Prefix kernel: records of one size beside records without values, which have no size."""
import pytest
import torch

import test_shared_decode as shared
from masked_util import check_decode

pytestmark = pytest.mark.gpu


def _empty(cache, page):
    """Records as the appends write them for zeros: codes 0, scales 1, rope 0."""
    cache[page] = 0
    cache[page, :, 512:528] = torch.ones((64, 4)).view(torch.uint8)


def _scaled(cache, power):
    cache[:, :, 512:528] = (cache[:, :, 512:528].contiguous().view(torch.float32) * 2.0 ** power).view(torch.uint8)
    rope = cache[:, :, 528:].contiguous().view(torch.bfloat16)
    cache[:, :, 528:] = (rope.float() * 2.0 ** power).to(torch.bfloat16).view(torch.uint8)


@pytest.mark.parametrize("power", [-44, -30, -20, -10, 0, 10, 20, 40])
@pytest.mark.parametrize("first", [0, 2])
def test_records_without_values_take_no_bits_from_the_others(power, first):
    """Values of 2^power, with scores of the usual size, and pages of zeros in every third tile of 128 positions (whole tiles, which
    the oracle's bound counts with their own values).  16 blocks of rows x 21 tiles: a pair takes five at a time, so that
    references pass from tiles without values to others."""
    q, cache, pt, pl, bt, ln = shared.make([2600], [(i * 37) % 90 for i in range(32)], 64, seed=7, q_scale=2.0 ** -power)
    _scaled(cache, power)
    for i in range(first, 40, 6):
        _empty(cache, int(pt[0, i]))
        _empty(cache, int(pt[0, i + 1]))
    case = (q, cache, pt, pl, bt, ln)
    out, lse, err = shared._run(case)
    assert err == 0
    check_decode(out, lse, shared._want(case))


def test_no_values_at_all():
    q, cache, pt, pl, bt, ln = shared.make([2500], [64, 3], 64, seed=8)
    for pg in range(cache.shape[0]):
        _empty(cache, pg)
    case = (q, cache, pt, pl, bt, ln)
    out, lse, err = shared._run(case)
    assert err == 0 and torch.all(out == 0)
    check_decode(out, lse, shared._want(case))
