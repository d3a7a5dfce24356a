"""Decode with capped, biased and masked scores against the float64 oracle: caps and slopes small and large, windows, documents
and prefixes at every place in a tile, queries of one request with sights of their own, unseen pages, graphs, streams."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, make_dense
from masked_util import check_decode
from oracle import masked_oracle
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32)


def _run(q, cache, bt, lens, softcap=0.0, slopes=None, starts=None, prefix=None, ctas=0, scale=SCALE):
    d = [t.to(DEV) for t in (q, cache, bt, lens)]
    opt = [None if t is None else t.to(DEV) for t in (slopes, starts, prefix)]
    ws = api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2], ctas), DEV)
    out = torch.full((q.shape[0], q.shape[1], 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    api.sparse_mla_masked_decode(*d, scale, softcap=softcap, slopes=opt[0], starts=opt[1], prefix_lens=opt[2], out=out,
                                 lse=lse, workspace=ws, ctas=ctas)
    torch.cuda.synchronize()
    return out, lse, api.read_errors(ws)


def _row_groups(q, cache, bt):
    """The table as it is and widened, so that CTAs take 16, 32 and 64 rows at once."""
    seen, pages = {}, bt.shape[1]
    while pages < 1 << 20:
        wide = torch.full((bt.shape[0], pages), -1, dtype=torch.int32)
        wide[:, :bt.shape[1]] = bt
        rows = api.dense_plan(api.dense_dims_of(q, cache, wide), 0).rows_per_cta
        seen.setdefault(rows, wide)
        if rows >= min(64, q.shape[0] // bt.shape[0] * q.shape[1]):
            break
        pages *= 2
    return seen.values()


def _check(lens, H, s_q=1, seed=0, softcap=0.0, slopes=None, starts=None, prefix=None, q_scale=1.0, ctas=0, flags=0,
           change=None):
    q, cache, bt, ln = make_dense(lens, H, s_q, seed=seed, q_scale=q_scale)
    if change:
        change(bt)
    slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32)
    st, pr = _i32(starts), _i32(prefix)
    want = masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(), SCALE, softcap,
                                       None if slopes is None else slopes.numpy(), starts, prefix)
    for wide in _row_groups(q, cache, bt):
        out, lse, err = _run(q, cache, wide, ln, softcap, slopes, st, pr, ctas)
        assert err == flags
        check_decode(out, lse, want)


def _alibi(H):
    return [2.0 ** (-8 * (h + 1) / H) for h in range(H)]


@pytest.mark.parametrize("cap,q_scale", [(30.0, 1.0), (30.0, 8.0), (2.0, 8.0), (0.01, 1.0), (1000.0, 4.0), (2.0 ** 20, 1.0),
                                         (2.0 ** -20, 1.0), (5.0, 300.0)])
def test_caps(cap, q_scale):
    _check([300, 1, 0, 130], 64, seed=1, softcap=cap, q_scale=q_scale)


@pytest.mark.parametrize("H", [1, 5, 16, 24, 64, 128])
def test_slopes(H):
    _check([700, 64, 3], H, seed=H, slopes=_alibi(H))


@pytest.mark.parametrize("slope", [0.0, -0.25, 8.0, -1e-3])
def test_slopes_of_any_sign(slope):
    _check([900], 16, seed=2, slopes=[slope] * 16)


def test_cap_and_slopes_together():
    _check([900, 33], 64, s_q=1, seed=3, softcap=20.0, slopes=_alibi(64), q_scale=6.0)


@pytest.mark.parametrize("start", [0, 1, 63, 64, 65, 127, 128, 129, 300, 511, 512, 899, 900, 901, -5, 10 ** 9])
@pytest.mark.parametrize("prefix", [None, 0, 1, 64, 130, 400, 2000, -1])
def test_starts_and_prefixes(start, prefix):
    _check([900], 16, seed=4, starts=[start], prefix=None if prefix is None else [prefix])


@pytest.mark.parametrize("H", [16, 40, 64, 128])
def test_windows_of_a_batch(H):
    lens = [3000, 0, 1, 640, 641, 2000, 100]
    _check(lens, H, seed=5, starts=[max(0, n - 300) for n in lens], prefix=[4] * len(lens))


@pytest.mark.parametrize("H,s_q", [(16, 2), (64, 2), (5, 13), (128, 2), (24, 3)])
def test_queries_of_a_request_have_their_own_sight(H, s_q):
    lens = [max(0, n - (s_q - 1 - j)) for n in (1500, 64, 700) for j in range(s_q)]
    starts = [(37 * i * 41) % max(1, n) for i, n in enumerate(lens)]
    _check(lens, H, s_q, seed=6, starts=starts, prefix=[(i * 53) % 200 for i in range(len(lens))], slopes=_alibi(H))


def test_rows_whose_mask_leaves_nothing():
    _check([500, 300, 0, 64], 64, seed=7, starts=[500, 299, 0, 70], prefix=[0, 0, 9, 0])


def test_everything_at_once_with_any_number_of_ctas():
    for ctas in (1, 3, 31, 200):
        _check([2000, 17, 900, 4000], 64, seed=8, starts=[1500, 0, 900, 2100], prefix=[130, 5, 700, 300], softcap=15.0,
               slopes=_alibi(64), ctas=ctas)


def test_pages_that_no_query_sees_may_be_gone():
    def gone(bt):
        bt[0, 3:12] = -1
        bt[1, :5] = 10 ** 6
    _check([1500, 700], 64, seed=9, starts=[12 * 64, 330], prefix=[3 * 64, 0], change=gone)


def test_a_missing_page_that_is_seen_is_reported():
    def gone(bt):
        bt[0, 14] = -1
    _check([1500], 64, seed=10, starts=[12 * 64 + 5], prefix=[64], change=gone, flags=_native.DEVERR_PAGE_RANGE)


def test_without_anything_given_it_is_the_dense_decode():
    q, cache, bt, ln = make_dense([700, 64, 0], 64, seed=11)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    a, b = api.sparse_mla_masked_decode(*d, SCALE), api.sparse_mla_dense_decode(*d, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_mask_that_hides_nothing_is_the_dense_decode():
    q, cache, bt, ln = make_dense([700, 64, 0], 64, seed=12)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    z = torch.zeros(3, dtype=torch.int32, device=DEV)
    a, b = api.sparse_mla_masked_decode(*d, SCALE, starts=z), api.sparse_mla_dense_decode(*d, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(a[1], b[1]) or float((a[1] - b[1]).nan_to_num(0).abs().max()) < 2.0 ** -19


def test_a_hidden_nan_or_infinity_does_no_harm():
    q, cache, bt, ln = make_dense([700], 64, seed=13)
    bad = cache.clone()
    for t in range(200, 500):
        bad[int(bt[0, t // 64]), t % 64] = torch.full((656,), 0x7F, dtype=torch.uint8)
    st, pr = _i32([500]), _i32([200])
    a, b = _run(q, cache, bt, ln, starts=st, prefix=pr), _run(q, bad, bt, ln, starts=st, prefix=pr)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[1]).all()


def test_a_captured_call_follows_lengths_and_starts():
    q, cache, bt, ln = make_dense([2000, 900], 64, seed=14)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    ws = api.alloc_dense_workspace(api.dense_dims_of(*d[:3]), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.sparse_mla_masked_decode(*d, SCALE, softcap=10.0, starts=st, workspace=ws)
    for lens, starts in (([2000, 900], [1000, 10]), ([130, 900], [0, 899]), ([2000, 1], [1999, 0])):
        d[3].copy_(_i32(lens))
        st.copy_(_i32(starts))
        graph.replay()
        torch.cuda.synchronize()
        check_decode(out, lse, masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens, SCALE,
                                                           10.0, None, starts, None))


def test_on_another_stream():
    q, cache, bt, ln = make_dense([2000], 64, seed=15)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    st = _i32([700]).to(DEV)
    a = api.sparse_mla_masked_decode(*d, SCALE, starts=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = api.sparse_mla_masked_decode(*d, SCALE, starts=st, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
