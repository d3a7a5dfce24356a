"""Decode behind shared prefixes against the float64 oracle: prefix and own lengths from none to several thousand, groups,
heads, queries of one request, bad pages, graphs, streams, and the dense decode of the same positions."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits
from masked_util import check_decode
from oracle import masked_oracle
from sparse_mla_decode_paged_gb300 import _native, api
from sparse_mla_decode_paged_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _tables(lens, cache, perm, at, poison):
    """Block table of rows of these lengths over perm[at:]; records behind a row's length are poisoned."""
    pages = [(max(0, n) + 63) // 64 for n in lens]
    bt = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32)
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
        if lens[r] % 64 and n:
            cache[int(bt[r, n - 1]), lens[r] % 64:] = poison
    return bt, at


def make(prefixes, lens, H, s_q=1, seed=0, q_scale=1.0):
    """CPU inputs: lens[b] per query of R = len(lens) / s_q requests in len(prefixes) groups."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens) // s_q
    own = [max(lens[r * s_q:(r + 1) * s_q]) for r in range(R)]
    total = sum((max(0, n) + 63) // 64 for n in [*prefixes, *own]) + 2
    cache = wl.fill_kv_cache(total, g, "cpu", outlier_channels=5)
    poison = torch.full((656,), 0x7F, dtype=torch.uint8)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    pt, at = _tables(prefixes, cache, perm, 0, poison)
    bt, at = _tables(own, cache, perm, at, poison)
    for pg in perm[at:].tolist():
        cache[pg] = poison
    q = (torch.randn((len(lens), H, 576), generator=g) * q_scale).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return q, cache, pt, i32(prefixes), bt, i32(lens)


def _run(case, ws=None, **kw):
    d = [t.to(DEV) for t in case]
    if ws is None:
        ws = api.alloc_shared_workspace(d[0], d[1], d[2], d[4])
    out = torch.full((*d[0].shape[:2], 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(d[0].shape[:2], float("nan"), device=DEV)
    api.sparse_mla_shared_decode(*d, SCALE, out=out, lse=lse, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, lse, api.read_errors(ws)


# Prefixes of so many rows and pages are taken by pairs of CTAs, with keys rounded to fp16.
PAIR_ROWS, PAIR_PAGES = 128, 16


def _want(case):
    q, cache, pt, pl, bt, ln = case
    pairs = q.shape[0] * q.shape[1] // pt.shape[0] >= PAIR_ROWS and pt.shape[1] >= PAIR_PAGES
    return masked_oracle.shared_decode(bits(q).reshape(q.shape), cache.numpy(), pt.numpy(), pl.numpy(), bt.numpy(),
                                       ln.numpy(), SCALE, half_keys=pairs)


def _widened(case):
    """The same prefixes in a table of as many pages as pairs of CTAs take."""
    pt = torch.full((case[2].shape[0], max(PAIR_PAGES, case[2].shape[1])), -1, dtype=torch.int32)
    pt[:, :case[2].shape[1]] = case[2]
    return (*case[:2], pt, *case[3:])


def _check(*args, flags=0, wide=False, **kw):
    case = make(*args, **kw)
    if wide:
        case = _widened(case)
    out, lse, err = _run(case)
    assert err == flags
    check_decode(out, lse, _want(case))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 300, 1000, 1024, 2500])
def test_pairs_of_ctas_lengths(n):
    _check([n], [100, 0], 64, seed=n, wide=True)


@pytest.mark.parametrize("H,R", [(64, 3), (128, 1), (128, 2), (100, 2), (16, 9), (5, 40), (1, 130)])
def test_pairs_of_ctas_rows(H, R):
    _check([1100], [(i * 37) % 90 for i in range(R)], H, seed=H, wide=True)


@pytest.mark.parametrize("G,each", [(2, 2), (3, 2), (9, 2), (200, 2)])
def test_pairs_of_ctas_groups(G, each):
    """More blocks than pairs, empty prefixes among them."""
    _check([0 if i % 4 == 1 else (i * 331 + 500) % 1300 for i in range(G)], [(i * 97) % 70 for i in range(G * each)], 64 if G < 20 else 66,
           seed=G, wide=True)


def test_pairs_of_ctas_nothing_to_see():
    _check([0, 0], [0, 3, 0, 0], 64, seed=1, wide=True)


@pytest.mark.parametrize("q_scale", [0.01, 8.0, 60.0])
def test_pairs_of_ctas_scores_far_apart(q_scale):
    _check([2000], [100, 5], 64, seed=2, q_scale=q_scale, wide=True)


def test_pairs_of_ctas_long():
    _check([20000], [10, 300], 64, seed=3, wide=True)


def test_pairs_of_ctas_bad_pages():
    case = _widened(make([1500], [300, 200], 64, seed=3))
    case[2][0, 2], case[2][0, 7], case[4][1, 0] = -1, 10 ** 6, 10 ** 6
    out, lse, err = _run(case)
    assert err == _native.DEVERR_PAGE_RANGE
    check_decode(out, lse, _want(case))


def test_pairs_of_ctas_scales_far_apart():
    """Tiles whose scales differ by powers of two, rising and falling: the references and the sums follow."""
    q, cache, pt, pl, bt, ln = make([1500], [64, 64], 64, seed=9)
    for i, pg in enumerate(pt[0].tolist()):
        sc = cache[pg, :, 512:528].contiguous().view(torch.float32) * 2.0 ** ((i * 7) % 23 - 16)
        cache[pg, :, 512:528] = sc.view(torch.uint8)
    case = _widened((q, cache, pt, pl, bt, ln))
    out, lse, err = _run(case)
    check_decode(out, lse, _want(case))


def test_pairs_of_ctas_runs_are_equal():
    case = _widened(make([9000], [100, 200, 3], 64, seed=10))
    a = _run(case)
    for _ in range(5):
        b = _run(case)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pairs_of_ctas_a_nan_that_one_query_sees():
    """The last query of a request sees a position that is no number, the one before does not; nor do other requests."""
    case = _widened(make([1200], [39, 40, 64, 64], 64, s_q=2, seed=12))
    case[1][int(case[4][0, 0]), 39, 7] = 0x7F
    out, lse, err = _run(case)
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()
    keep = [0, 2, 3]
    case[1][int(case[4][0, 0]), 39] = 0
    want = _want(case)
    check_decode(out[keep], lse[keep], tuple(x[keep] for x in want))


@pytest.mark.parametrize("own", [1, 64, 200, 700, 2000])
def test_pairs_of_ctas_own_positions(own):
    """Few own positions go with the prefixes, many to the dense kernel."""
    _check([1100, 900], [own, 0, 3, own // 2], 64, seed=own, wide=True)
    _check([1100], [max(0, own - 2), own - 1, own, 0, 1, 2], 64, s_q=3, seed=own + 1, wide=True)


def test_pairs_of_ctas_nan():
    case = _widened(make([1200], [10, 20], 64, seed=11))
    case[1][int(case[2][0, 3]), 5, 100] = 0x7F
    out, lse, err = _run(case)
    assert torch.isnan(lse).all() and torch.isnan(out).all()


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 128, 129, 500, 1000, 3000])
@pytest.mark.parametrize("own", [0, 1, 64, 200])
def test_lengths(n, own):
    _check([n], [own, 3], 16, seed=n + own)


@pytest.mark.parametrize("H", [1, 5, 16, 24, 40, 64, 100, 128])
def test_head_counts(H):
    _check([700], [10, 0, 129], H, seed=H)


@pytest.mark.parametrize("G,each", [(1, 1), (1, 9), (2, 3), (5, 2), (7, 1)])
def test_groups(G, each):
    _check([(i * 331 + 5) % 900 for i in range(G)], [(i * 97) % 300 for i in range(G * each)], 16, seed=G)


@pytest.mark.parametrize("H,s_q", [(16, 2), (64, 2), (5, 13), (24, 3)])
def test_queries_of_a_request_have_their_own_lengths(H, s_q):
    _check([900, 130], [max(0, n - (s_q - 1 - j)) for n in (70, 0, 1, 200) for j in range(s_q)], H, s_q, seed=H)


def test_nothing_to_see():
    _check([0, 0, 5], [0, 3, 0], 16, seed=1)


def test_scores_far_apart():
    _check([600], [100, 5], 64, seed=2, q_scale=20.0)


def test_bad_pages_are_skipped_and_reported():
    case = make([600], [300, 200], 16, seed=3)
    case[2][0, 2], case[4][1, 0] = -1, 10 ** 6
    out, lse, err = _run(case)
    assert err == _native.DEVERR_PAGE_RANGE
    check_decode(out, lse, _want(case))


def test_lengths_beyond_the_tables_are_reported():
    case = make([128], [64], 16, seed=4)
    want = _want(case)
    case[3][0], case[5][0] = 500, 70
    out, lse, err = _run(case)
    assert err == _native.DEVERR_PAGE_RANGE
    check_decode(out, lse, want)
    case[3][0], case[5][0] = -5, 64
    out, lse, err = _run(case)
    check_decode(out, lse, _want((*case[:3], torch.zeros(1, dtype=torch.int32), *case[4:])))


def test_the_same_pages_as_prefix_and_own():
    """A page may be in the prefix and in rows of the block table: nothing is written."""
    case = list(make([256], [64, 64], 16, seed=5))
    case[4] = case[2][:, :1].repeat(2, 1).contiguous()
    out, lse, err = _run(case)
    assert err == 0
    check_decode(out, lse, _want(case))


def test_a_captured_call_follows_the_lengths_and_two_calls_have_their_own_workspace():
    case = make([1500], [100, 200, 0], 64, seed=6)
    d = [t.to(DEV) for t in case]
    ws = api.alloc_shared_workspace(d[0], d[1], d[2], d[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.sparse_mla_shared_decode(*d, SCALE, workspace=ws)
    for pl, ln in ((1500, [100, 200, 0]), (77, [1, 0, 0]), (0, [0, 130, 0])):
        d[3].fill_(pl)
        d[5].copy_(torch.tensor(ln, dtype=torch.int32))
        graph.replay()
        other = _run(case)
        torch.cuda.synchronize()
        check_decode(out, lse, _want((*case[:3], torch.tensor([pl], dtype=torch.int32), case[4], torch.tensor(ln))))
        check_decode(*other[:2], _want(case))


def test_on_another_stream():
    case = make([900], [64] * 4, 16, seed=7)
    d = [t.to(DEV) for t in case]
    a = api.sparse_mla_shared_decode(*d, SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = api.sparse_mla_shared_decode(*d, SCALE, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_wait_that_runs_out_is_reported():
    case = make([900], [64], 16, seed=8)
    d = [t.to(DEV) for t in case]
    ws = api.alloc_shared_workspace(d[0], d[1], d[2], d[4])
    try:
        api.debug_set_wait_limit(1)
        api.sparse_mla_shared_decode(*d, SCALE, workspace=ws)
        torch.cuda.synchronize()
    finally:
        api.debug_set_wait_limit(0)
    assert api.read_errors(ws) & _native.DEVERR_TIMEOUT
    api.clear_errors(ws)
    out, lse, err = _run(case, ws=ws)
    assert err == 0
    check_decode(out, lse, _want(case))
