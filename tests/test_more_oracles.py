"""The oracles of the masked and shared decode, the weights and the eviction on closed forms."""
import numpy as np

import oracle  # noqa: F401
from oracle import cache_weights_oracle as cw, dense_oracle, masked_oracle as mo
from cache_util import bits, make_dense

SCALE = 576 ** -0.5


def _case(lens, H=3, s_q=1, seed=0):
    q, cache, bt, ln = make_dense(lens, H, s_q, seed=seed)
    return bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy()


def test_nothing_given_is_the_dense_decode():
    case = _case([130, 0, 7])
    for a, b in zip(mo.masked_decode(*case, SCALE), dense_oracle.dense_decode(*case, SCALE)):
        assert np.allclose(a, b, rtol=1e-12, atol=0)


def test_a_window_is_the_dense_decode_of_what_it_shows():
    """A start at a page's border: the same as a table without the pages before it."""
    q, cache, bt, ln = _case([200])
    a = mo.masked_decode(q, cache, bt, ln, SCALE, starts=[64])
    b = dense_oracle.dense_decode(q, cache, bt[:, 1:], ln - 64, SCALE)
    assert np.allclose(a[0], b[0], rtol=1e-12) and np.allclose(a[1], b[1], rtol=1e-12)


def test_caps_and_slopes_on_one_position():
    q, cache, bt, ln = _case([1])
    s = dense_oracle.dense_decode(q, cache, bt, ln, SCALE)[1]
    assert np.allclose(mo.masked_decode(q, cache, bt, ln, SCALE, softcap=0.5)[1], 0.5 * np.tanh(s / 0.5))
    # the query's own position has no bias
    assert np.allclose(mo.masked_decode(q, cache, bt, ln, SCALE, slopes=[3.0, -2.0, 0.5])[1], s)
    q, cache, bt, ln = _case([2], seed=1)
    first, both = [dense_oracle.dense_decode(q, cache, bt, [n], SCALE)[1] for n in (1, 2)]
    last = np.log(np.exp(both) - np.exp(first))
    slopes = np.array([3.0, -2.0, 0.5])
    assert np.allclose(mo.masked_decode(q, cache, bt, ln, SCALE, slopes=slopes)[1], np.logaddexp(first - slopes, last))


def test_a_prefix_and_own_positions_are_one_context():
    q, cache, bt, ln = _case([200])
    one = dense_oracle.dense_decode(q, cache, bt, ln, SCALE)
    two = mo.shared_decode(q, cache, bt[:, :2], [128], bt[:, 2:], [72], SCALE)
    assert np.allclose(one[0], two[0], rtol=1e-12) and np.allclose(one[1], two[1], rtol=1e-12)


def test_weights_of_a_decode_sum_to_one_per_row():
    q, cache, bt, ln = _case([100, 64], H=5)
    lse = dense_oracle.dense_decode(q, cache, bt, ln, SCALE)[1]
    w, err = cw.attention_weights(q, cache, bt, ln, lse, SCALE, np.full((2, 120), 2.0), 0.5)
    for r, n in enumerate(ln):
        assert np.isclose((w[r, :n] - 1.0).sum(), 5.0, rtol=1e-9) and np.all(w[r, n:] == 2.0)
    assert np.all(err >= 0)


def test_eviction_by_hand():
    w = np.array([[5, 1, 1, 9, 1, 0, 3, 2]], dtype=np.float32)
    pos = np.array([[0, 1, 2, 3, 4, 5, 6, 7]], dtype=np.int32)
    cache = np.arange(64 * 656, dtype=np.uint32).astype(np.uint8).reshape(1, 64, 656).copy()
    cache[0, :, 0] = np.arange(64)
    # held: position 0 and the last one; then weights 9, 3 and the first of the ones: slots 0, 1, 3, 6, 7
    nw, npos, nc, new = cw.evict(w, pos, [8], [8], 5, cache, np.array([[0]]), 1, 1)
    assert new[0] == 5
    assert npos[0, :5].tolist() == [0, 1, 6, 3, 7] and nw[0].tolist() == [5, 1, 3, 9, 2, 0, 0, 0]
    assert nc[0, :5, 0].tolist() == [0, 1, 6, 3, 7] and np.array_equal(nc[0, 5:], cache[0, 5:])


def test_order_of_special_values():
    x = np.array([np.nan, np.inf, 1, 1e-45, 0.0, -0.0, -1, -np.inf, -np.nan], dtype=np.float32)
    x[8] = np.array([0xFFC00000], dtype=np.uint32).view(np.float32)[0]
    k = cw.order_key(x)
    assert np.all(np.diff(k) < 0)
