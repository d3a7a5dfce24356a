"""Attention weights accumulated per cached position against the float64 oracle: lengths from none to several thousand, head
counts, several queries per request, positions that no query sees, bad pages, strides, streams, graphs."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, make_dense
from oracle import cache_weights_oracle as ref
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _lse(q, cache, bt, lens):
    """Near the true lse, and fp32: any will do."""
    from oracle import dense_oracle
    return torch.from_numpy(dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens.numpy(),
                                                      SCALE)[1].astype(np.float32))


def _check(lens, H, s_q=1, decay=1.0, seed=0, extra=5, stride=0, flags=0, change=None, cols=None):
    q, cache, bt, ln = make_dense(lens, H, s_q, seed=seed)
    lse = _lse(q, cache, bt, ln)
    if change:
        change(bt, ln)
    n = cols if cols is not None else max(0, max(lens)) + extra
    g = torch.Generator().manual_seed(seed + 1)
    w = torch.rand((bt.shape[0], n + stride), generator=g)[:, :n]
    dw = torch.full((bt.shape[0], n + stride), -7.0, device=DEV)
    view = dw[:, :n]
    view.copy_(w)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = api.sparse_mla_attention_weights(q.to(DEV), cache.to(DEV), bt.to(DEV), ln.to(DEV), lse.to(DEV), SCALE, view,
                                           decay=decay, err_word=err)
    torch.cuda.synchronize()
    assert got is view and int(err) == flags
    assert torch.all(dw[:, n:] == -7.0)
    want, tol = ref.attention_weights(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(), lse.numpy(), SCALE,
                                      w.numpy(), decay)
    off = np.abs(got.cpu().double().numpy() - want)
    assert np.all(off <= tol), f"error {(off / np.maximum(tol, 1e-300)).max():.2f} of its bound"
    return got


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 127, 128, 129, 256, 1000, 4097])
def test_lengths(n):
    _check([n], 16, seed=n)


@pytest.mark.parametrize("H", [1, 5, 8, 16, 17, 24, 32, 33, 64, 65, 100, 128])
def test_head_counts(H):
    _check([300, 77], H, seed=H)


@pytest.mark.parametrize("H,s_q", [(16, 2), (24, 3), (128, 2), (64, 5), (5, 13), (128, 3)])
def test_queries_of_a_request_have_their_own_lengths(H, s_q):
    _check([max(0, n - (s_q - 1 - j)) for n in (1500, 64, 130) for j in range(s_q)], H, s_q, seed=H + s_q)


def test_lengths_of_one_request_in_any_order():
    _check([5, 700, 0, 129, 1, 300], 40, 3, seed=8)


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, 3.0])
def test_decay(decay):
    _check([300, 0, 129], 16, decay=decay, seed=4)


def test_decay_of_zero_reads_nothing():
    q, cache, bt, ln = make_dense([200], 16, seed=3)
    lse = _lse(q, cache, bt, ln)
    w = torch.full((1, 260), float("nan"), device=DEV)
    api.sparse_mla_attention_weights(q.to(DEV), cache.to(DEV), bt.to(DEV), ln.to(DEV), lse.to(DEV), SCALE, w, decay=0.0)
    torch.cuda.synchronize()
    assert torch.isfinite(w[:, :200]).all() and torch.isnan(w[:, 200:]).all()
    # every row's weights sum to 1 (2^-18: lse and the terms are off by less than 2^-19 each)
    assert abs(float(w[0, :200].double().sum()) - 16) <= 16 * 2.0 ** -18


def test_many_requests_of_mixed_lengths():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 400, (700,), generator=g).tolist()
    _check(lens, 8, seed=5)


def test_strided_rows():
    _check([130, 64, 1], 16, seed=6, stride=11)


def test_fewer_columns_than_positions():
    _check([300, 77], 16, seed=7, cols=150, flags=_native.DEVERR_LEN_RANGE)


def test_bad_pages_add_nothing():
    def change(bt, ln):
        bt[0, 1], bt[0, 3], bt[1, 0] = -1, 10 ** 6, -5
    _check([300, 77, 200], 32, seed=9, change=change, flags=_native.DEVERR_PAGE_RANGE)


def test_lengths_beyond_the_table_are_clamped():
    def change(bt, ln):
        ln[0] = 64 * bt.shape[1] + 9
        ln[1] = -3
    _check([320, 77], 16, seed=10, change=change, extra=100, flags=_native.DEVERR_LEN_RANGE)


def test_runs_are_equal_and_captured_calls_follow_the_lengths():
    q, cache, bt, ln = make_dense([3000, 500], 64, seed=11)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    lse = _lse(q, cache, bt, ln).to(DEV)
    out = []
    for _ in range(3):
        w = torch.zeros((2, 3000), device=DEV)
        api.sparse_mla_attention_weights(*d, lse, SCALE, w)
        out.append(w)
    w = torch.zeros((2, 3000), device=DEV)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        api.sparse_mla_attention_weights(*d, lse, SCALE, w, decay=0.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[0], x) for x in (*out[1:], w))
    d[3].copy_(torch.tensor([100, 0], dtype=torch.int32))
    w.fill_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w[0, :100], out[0][0, :100]) and torch.all(w[0, 100:] == -1) and torch.all(w[1] == -1)


def test_on_another_stream():
    q, cache, bt, ln = make_dense([900], 16, seed=12)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    lse = _lse(q, cache, bt, ln).to(DEV)
    a, b = torch.zeros((1, 900), device=DEV), torch.zeros((1, 900), device=DEV)
    api.sparse_mla_attention_weights(*d, lse, SCALE, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.sparse_mla_attention_weights(*d, lse, SCALE, b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_a_wait_that_runs_out_is_reported():
    q, cache, bt, ln = make_dense([900], 16, seed=13)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    lse = _lse(q, cache, bt, ln).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.zeros((1, 900), device=DEV)
    try:
        api.debug_set_wait_limit(1)
        api.sparse_mla_attention_weights(*d, lse, SCALE, w, err_word=err)
        torch.cuda.synchronize()
    finally:
        api.debug_set_wait_limit(0)
    assert int(err) & _native.DEVERR_TIMEOUT and torch.all(w == 0)


def test_a_nan_reaches_its_position_alone():
    q, cache, bt, ln = make_dense([200], 16, seed=14)
    lse = _lse(q, cache, bt, ln)
    cache[int(bt[0, 1]), 3, 7] = 0x7F
    w = torch.zeros((1, 200), device=DEV)
    api.sparse_mla_attention_weights(q.to(DEV), cache.to(DEV), bt.to(DEV), ln.to(DEV), lse.to(DEV), SCALE, w)
    torch.cuda.synchronize()
    assert torch.isnan(w[0]).nonzero().flatten().tolist() == [67]
