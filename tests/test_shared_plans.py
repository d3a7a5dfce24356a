"""The three ways of a decode behind shared prefixes, told apart by their workspaces: everything with the dense kernel, prefixes
and own positions with the prefix kernel, prefixes with the prefix kernel and own positions with the dense one.  The last,
which wide tables of the requests' own take, against the oracle."""
import ctypes as C

import pytest
import torch

import test_shared_decode as shared
from cache_util import DEV
from masked_util import check_decode
from sparse_mla_decode_paged_gb300 import _native, api
from sparse_mla_decode_paged_gb300._native import SmlaSharedDims

SCALE = 576 ** -0.5
TILE_BYTES = 128 * 576 * 2                                  # a tile of 128 positions in fp16


def planned(lib, sms, B, H, s_q, G, prefix_pages, own_pages):
    """(the prefix kernel takes the prefixes, it takes the requests' own positions, too).  Workspaces grow with the expanded
    tables, by that many bytes per tile; what else is in them changes at two widths of a table at most, with the rows per
    CTA of the dense kernel."""
    def size(more_prefix, more_own):
        d = SmlaSharedDims(B, H, 64, own_pages + more_own, 512, 64, 1 << 20, s_q, G, prefix_pages + more_prefix)
        n = C.c_size_t(0)
        assert lib.sparse_mla_shared_workspace_size(d, sms, C.byref(n)) == 0
        return n.value
    p = [size(i, 0) for i in (0, 2)]
    o = [size(0, i) for i in (0, 2, 4, 6)]
    grows = lambda v, by: [by <= b - a < 1.1 * by for a, b in zip(v, v[1:])]
    return all(grows(p, G * TILE_BYTES)), sum(grows(o, B // s_q * TILE_BYTES)) >= 2


def _case_plan(lib, case, s_q=1):
    q, _, pt, _, bt, _ = case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return planned(lib, sms, q.shape[0], q.shape[1], s_q, pt.shape[0], pt.shape[1], bt.shape[1])


@pytest.mark.parametrize("shape,plan", [
    ((64, 16, 1, 1, 15, 16), (False, False)),               # few pages of prefix
    ((4, 16, 1, 1, 16, 16), (False, False)),                # few rows
    ((64, 16, 1, 1, 512, 1), (True, True)),
    ((32, 64, 1, 1, 512, 2), (True, True)),
    ((64, 16, 1, 1, 16, 16), (True, False)),
    ((32, 64, 1, 1, 512, 512), (True, False)),
    ((2, 64, 1, 1, 18, 188), (True, False)),
    ((200, 16, 1, 1, 16, 2), (True, False))])
def test_plans(lib, shape, plan):
    assert planned(lib, 152, *shape) == plan


def _wider(case, own_pages):
    bt = torch.full((case[4].shape[0], max(own_pages, case[4].shape[1])), -1, dtype=torch.int32)
    bt[:, :case[4].shape[1]] = case[4]
    return (*case[:4], bt, case[5])


def _mixed(lib, prefixes, lens, H, s_q=1, own_pages=0, seed=0, **kw):
    case = _wider(shared._widened(shared.make(prefixes, lens, H, s_q, seed=seed, **kw)), own_pages)
    assert _case_plan(lib, case, s_q) == (True, False)
    return case


def _check(lib, *args, flags=0, **kw):
    case = _mixed(lib, *args, **kw)
    out, lse, err = shared._run(case)
    assert err == flags
    check_decode(out, lse, shared._want(case))
    return case, out, lse


RAGGED = [(i * 53) % 900 if i % 5 else 0 for i in range(64)]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [0, 1, 129, 1024, 2500])
def test_requests_of_mixed_lengths(lib, n):
    _check(lib, [n], RAGGED, 16, own_pages=16, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("H,R,own_pages", [(128, 20, 40), (100, 8, 100), (5, 70, 30), (1, 200, 20), (64, 4, 512)])
def test_head_counts_and_wide_tables(lib, H, R, own_pages):
    _check(lib, [1100], [(i * 37 + 60) % 300 for i in range(R)], H, own_pages=own_pages, seed=H)


@pytest.mark.gpu
@pytest.mark.parametrize("G,R,H", [(2, 40, 32), (5, 40, 16), (7, 21, 64), (20, 160, 16)])
def test_groups(lib, G, R, H):
    _check(lib, [0 if i % 3 == 2 else (i * 331 + 500) % 1500 for i in range(G)], [(i * 97) % 500 for i in range(R)], H,
           own_pages=40, seed=G)


@pytest.mark.gpu
@pytest.mark.parametrize("H,s_q,R", [(32, 2, 20), (16, 3, 24), (64, 2, 12)])
def test_queries_of_a_request_have_their_own_lengths(lib, H, s_q, R):
    _check(lib, [1300, 700], [max(0, (i * 61) % 700 - (s_q - 1 - j)) for i in range(R) for j in range(s_q)], H, s_q,
           own_pages=40, seed=H + s_q)


@pytest.mark.gpu
def test_own_positions_that_cross_runs(lib):
    _check(lib, [1100], [12000, 9001], 64, seed=3)
    _check(lib, [1100], [0, 20000], 64, seed=4)
    _check(lib, [3000, 0], [7000, 0, 1, 6999], 64, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("own_pages", [1, 2])
def test_tables_of_one_tile(lib, own_pages):
    _check(lib, [1000], [(i * 7) % (64 * own_pages + 1) for i in range(200)], 16, own_pages=own_pages, seed=own_pages)


@pytest.mark.gpu
def test_nothing_to_see(lib):
    _check(lib, [0], [0] * 64, 16, own_pages=16, seed=1)
    _check(lib, [0, 0], [0, 70] * 32, 16, own_pages=16, seed=2)


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_reported(lib):
    case = _mixed(lib, [1500], RAGGED, 16, own_pages=16, seed=6)
    case[2][0, 2], case[4][3, 0], case[4][4, 1] = -1, 10 ** 6, -1
    out, lse, err = shared._run(case)
    assert err == _native.DEVERR_PAGE_RANGE
    check_decode(out, lse, shared._want(case))
    case = _mixed(lib, [1500], RAGGED, 16, own_pages=16, seed=6)
    want = shared._want(case)
    case[5][0] = -3                                         # (its length is 0)
    out, lse, err = shared._run(case)
    assert err == 0
    check_decode(out, lse, want)
    case[5][1] = 16 * 64 + 1
    out, lse, err = shared._run(case)
    assert err == _native.DEVERR_PAGE_RANGE
    keep = [0, *range(2, 64)]
    check_decode(out[keep], lse[keep], tuple(x[keep] for x in want))


@pytest.mark.gpu
def test_positions_that_are_no_numbers(lib):
    """One of the request's own reaches that request alone, one of the prefix everybody."""
    case = _mixed(lib, [1200], RAGGED, 16, own_pages=16, seed=7)
    want = shared._want(case)
    case[1][int(case[4][2, 0]), 5, 100] = 0x7F
    out, lse, err = shared._run(case)
    assert err == 0 and torch.isnan(lse[2]).all() and torch.isnan(out[2]).all()
    keep = [0, 1, *range(3, 64)]
    check_decode(out[keep], lse[keep], tuple(x[keep] for x in want))
    case[1][int(case[2][0, 3]), 5, 100] = 0x7F
    out, lse, err = shared._run(case)
    assert torch.isnan(lse).all() and torch.isnan(out).all()


@pytest.mark.gpu
def test_a_captured_call_follows_the_lengths(lib):
    case = _mixed(lib, [2000], RAGGED, 16, own_pages=16, seed=8)
    d = [t.to(DEV) for t in case]
    ws = api.alloc_shared_workspace(d[0], d[1], d[2], d[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.sparse_mla_shared_decode(*d, SCALE, workspace=ws)
    none = torch.zeros(64, dtype=torch.int32)
    some = torch.where(torch.arange(64) % 3 == 0, case[5], none)
    for pl, ln in ((2000, case[5]), (77, some), (0, none), (0, case[5]), (2000, none), (1, some)):
        d[3].fill_(pl)
        d[5].copy_(ln)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert api.read_errors(ws) == 0
        check_decode(out, lse, shared._want((*case[:3], torch.tensor([pl], dtype=torch.int32), case[4], ln)))


@pytest.mark.gpu
def test_two_calls_at_once_are_equal_to_calls_alone(lib):
    cases = [_mixed(lib, [1700 + 100 * i], RAGGED, 16, own_pages=16, seed=9 + i) for i in range(2)]
    alone = [shared._run(c) for c in cases]
    dev = [[t.to(DEV) for t in c] for c in cases]
    ws = [api.alloc_shared_workspace(d[0], d[1], d[2], d[4]) for d in dev]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [api.sparse_mla_shared_decode(*d, SCALE, workspace=w, stream=st) for d, w, st in zip(dev, ws, side)]
    torch.cuda.synchronize()
    for c, a, g in zip(cases, alone, got):
        assert torch.equal(a[0], g[0]) and torch.equal(a[1], g[1])
        check_decode(*g, shared._want(c))


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported(lib):
    case = _mixed(lib, [1300], RAGGED, 16, own_pages=16, seed=11)
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
    out, lse, err = shared._run(case, ws=ws)
    assert err == 0
    check_decode(out, lse, shared._want(case))
