"""Items of the prefix kernel that follow one another quickly: segments of one or two tiles whose rows differ by powers of two from
item to item."""
import pytest
import torch

import test_shared_decode as shared
from masked_util import check_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [1, 100, 128, 200])
@pytest.mark.parametrize("G,own", [(160, 0), (160, 70), (90, 5)])
def test_rows_of_an_item_keep_their_factors(length, G, own):
    """(A row's factor is a power of two that follows its largest element; each item's are other ones than the next's.)"""
    q, *rest = shared.make([length] * G, [own if i % 3 else 0 for i in range(2 * G)], 64, seed=length + G)
    power = (torch.arange(2 * G) // 2 * 5 + torch.arange(2 * G)) % 9 - 7          # 2^-7 .. 2^1
    q = (q.float() * torch.exp2(power.float())[:, None, None]).to(torch.bfloat16)
    case = shared._widened((q, *rest))
    out, lse, err = shared._run(case)
    assert err == 0
    check_decode(out, lse, shared._want(case))
    for _ in range(3):
        again = shared._run(case)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
