"""The dense decode's oracle and error bounds on the CPU: results known in closed form, and wrong results refused."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import bits, check_dense, make_dense
from dense_util import check_weights
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


def _sink(n=3000, H=4):
    """One position, whose own value is zero, outweighs every other by about e^14."""
    q, cache, bt, lens = make_dense([n], H, seed=10)
    q[:] = 0
    q[:, :, 512] = 1.0
    cache[..., 528:530] = torch.tensor([0.0], dtype=torch.bfloat16).view(torch.uint8)
    cache[int(bt[0, 3]), 17, 528:530] = torch.tensor([14.0], dtype=torch.bfloat16).view(torch.uint8)
    cache[int(bt[0, 3]), 17, :512] = 0
    return q, cache, bt, lens


def _as_results(out, lse):
    return torch.from_numpy(out).to(torch.bfloat16), torch.from_numpy(lse).float()


@pytest.mark.parametrize("rows", [16, 64])
def test_a_sink_without_value_leaves_the_rest_to_be_checked(rows):
    case = _sink()
    out, lse = _oracle(*case, 1.0)[:2]
    check_weights(*_as_results(out, lse), *case, 1.0, rows)
    for wrong in (0 * out, -out, out * 0.98, np.roll(out, 1, axis=-1)):
        with pytest.raises(AssertionError):
            check_weights(*_as_results(wrong, lse), *case, 1.0, rows)


@pytest.mark.parametrize("n", [256, 1000, 4097])
def test_a_position_left_out_is_found(n):
    q, cache, bt, lens = make_dense([n], 2, seed=n)
    out, lse = _oracle(q, cache, bt, lens, 576 ** -0.5)[:2]
    check_weights(*_as_results(out, lse), q, cache, bt, lens, 576 ** -0.5, 16)
    rows, _ = dense_oracle.positions_rows(bt[0].numpy(), n, cache.shape[0])
    k = oracle.dequantize_record(cache.numpy().reshape(-1, 656)[rows])
    p = np.exp(576 ** -0.5 * (oracle.as_f64_q(bits(q)).reshape(q.shape)[0] @ k.T) - lse[0][:, None])
    # A position of weight p changes a block by p |v| in the root mean square.  The bound is 1.5 times 2^-8 of the result
    # and of the root of sum (p v)^2, which is about as large: 1.5 * 2^-7.5 |v| sqrt(sum p^2).  Scores of deviation s have
    # sum p^2 = exp(s^2) / n; with s = 1.3 at most 0.02 |v| / sqrt(n): below 3 |v| / n up to n = 22000.  Such a position is
    # left out of the sum of values, but not of lse.
    found = np.flatnonzero((p > 3 / n).any(axis=0))
    assert len(found) > 5
    for t in found[::max(1, n // 200)]:
        with pytest.raises(AssertionError):
            check_weights(*_as_results(out - p[None, :, t, None] * k[None, None, t, :512], lse), q, cache, bt, lens,
                          576 ** -0.5, 16)


def test_a_block_of_small_scale_is_checked_against_itself():
    q, cache, bt, lens = make_dense([200], 3, seed=3, poison=False)
    sc = cache[..., 512:528].contiguous().view(torch.float32)
    sc[..., 2] *= 2.0 ** -12
    cache[..., 512:528] = sc.view(torch.uint8)
    out, lse = _oracle(q, cache, bt, lens, 0.04)[:2]
    check_weights(*_as_results(out, lse), q, cache, bt, lens, 0.04, 64)
    out[..., 256:384] *= 1.03
    with pytest.raises(AssertionError):
        check_weights(*_as_results(out, lse), q, cache, bt, lens, 0.04, 64)
