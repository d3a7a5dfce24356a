"""The dense decode's oracle and error bounds on the CPU: results known in closed form, and wrong results refused."""
import numpy as np
import pytest
import torch

from cache_util import bits, check_dense, make_dense
from oracle import dense_oracle


def _oracle(q, cache, bt, lens, scale):
    return dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens.numpy(), scale)


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.05])
def test_the_score_bound_does_not_depend_on_the_sign_of_the_scale(scale):
    q, cache, bt, lens = make_dense([321, 50], 4, seed=12)
    up, down = _oracle(q, cache, bt, lens, scale)[4], _oracle(q, cache, bt, lens, -scale)[4]
    assert np.array_equal(up, down) and np.all(up >= 0) and (scale == 0.0 or np.all(up > 0))


@pytest.mark.parametrize("scale", [-0.05, 0.05])
def test_a_wrong_lse_is_refused(scale):
    q, cache, bt, lens = make_dense([321, 50], 4, seed=12)
    out, lse = (torch.from_numpy(x).float() for x in _oracle(q, cache, bt, lens, scale)[:2])
    check_dense(out.to(torch.bfloat16), lse, q, cache, bt, lens, scale)
    with pytest.raises(AssertionError):
        check_dense(out.to(torch.bfloat16), torch.full_like(lse, 123.0), q, cache, bt, lens, scale)
    with pytest.raises(AssertionError):
        check_dense(out.to(torch.bfloat16), lse + 0.01, q, cache, bt, lens, scale)
