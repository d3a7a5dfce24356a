"""Calls at once, captured calls whose lengths change, and slopes at the ends of their range, of the masked and the shared decode
and the eviction."""
import numpy as np
import pytest
import torch

import test_kv_evict as evict
import test_masked_decode as masked
import test_shared_decode as shared
from cache_util import DEV, bits, make_dense
from masked_util import check_decode
from oracle import masked_oracle
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _pairs_case(prefixes, lens, H, seed):
    return shared._widened(shared.make(prefixes, lens, H, seed=seed))


def test_pairs_of_ctas_two_calls_at_once():
    cases = [_pairs_case([1700 + 100 * i], [60, 0, 130], 64, 30 + i) for i in range(2)]
    dev = [[t.to(DEV) for t in c] for c in cases]
    ws = [api.alloc_shared_workspace(d[0], d[1], d[2], d[4]) for d in dev]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = [api.sparse_mla_shared_decode(*d, SCALE, workspace=w, stream=st) for d, w, st in zip(dev, ws, side)]
    torch.cuda.synchronize()
    for c, w, (out, lse) in zip(cases, ws, got):
        assert api.read_errors(w) == 0
        check_decode(out, lse, shared._want(c))


def test_pairs_of_ctas_captured_follow_the_lengths():
    case = _pairs_case([1500], [100, 200, 0], 64, 33)
    d = [t.to(DEV) for t in case]
    ws = api.alloc_shared_workspace(d[0], d[1], d[2], d[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.sparse_mla_shared_decode(*d, SCALE, workspace=ws)
    for pl, ln in ((0, [0, 0, 0]), (1500, [100, 200, 0]), (77, [1, 0, 0]), (0, [0, 130, 0]), (0, [0, 0, 0]), (1, [0, 0, 0])):
        d[3].fill_(pl)
        d[5].copy_(torch.tensor(ln, dtype=torch.int32))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert api.read_errors(ws) == 0
        check_decode(out, lse, shared._want((*case[:3], torch.tensor([pl], dtype=torch.int32), case[4], torch.tensor(ln))))


def test_pairs_of_ctas_a_wait_that_runs_out_is_reported():
    case = _pairs_case([1300], [64, 10], 64, 34)
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


def test_two_masked_calls_at_once():
    cases = [make_dense([900, 1300], 64, 1, seed=40 + i) for i in range(2)]
    starts = torch.tensor([700, 5], dtype=torch.int32)
    dev = [[t.to(DEV) for t in c] for c in cases]
    st = starts.to(DEV)
    ws = [api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2], 0), DEV) for d in dev]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [api.sparse_mla_masked_decode(*d, SCALE, softcap=20.0, starts=st, workspace=w, stream=s)
               for d, w, s in zip(dev, ws, side)]
    torch.cuda.synchronize()
    for (q, cache, bt, ln), (out, lse) in zip(cases, got):
        check_decode(out, lse, masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(),
                                                           SCALE, 20.0, None, starts.tolist(), None))


@pytest.mark.parametrize("H", [16, 64])
def test_a_slope_that_leaves_the_last_position_alone(H):
    """A bias of -1e30 per position: the query's own position has all of the weight."""
    masked._check([300, 1, 900], H, seed=41, slopes=[1e30] * H)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_slope_that_is_no_number_reaches_its_head_alone(H, bad):
    """(An infinite slope times the distance 0 of the last position is no number either.)"""
    q, cache, bt, ln = make_dense([300, 700], H, 1, seed=42)
    slopes = torch.full((H,), 0.01)
    want = masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(), SCALE, 0.0,
                                       slopes.numpy(), None, None)
    slopes[3] = bad
    rest = [h for h in range(H) if h != 3]
    out, lse, err = masked._run(q, cache, bt, ln, slopes=slopes)
    assert err == 0
    assert torch.isnan(lse[:, 3]).all() and torch.isnan(out[:, 3]).all()
    check_decode(out[:, rest], lse[:, rest], tuple(x[:, rest] for x in want))


def test_a_captured_eviction_over_a_large_cluster():
    cols = 340000
    w, pos, nxt, lens, cache, bt = evict._inputs([cols], seed=43)
    d = [t.to(DEV) for t in (w, pos, nxt, lens, cache, bt)]
    ws = api.alloc_evict_workspace(d[0])
    new = torch.zeros(1, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sparse_mla_kv_evict(*d[:4], 200000, *d[4:], sinks=4, new_lens=new, workspace=ws)
    for n in (cols, 260000, 100):
        for t, v in zip(d, (w, pos, nxt, torch.tensor([n], dtype=torch.int32), cache, bt)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = evict.ref.evict(w.numpy(), pos.numpy(), nxt.numpy(), [n], 200000, cache.numpy(), bt.numpy(), 4, 0)
        for t, v in zip((d[0], d[1], d[4], new), want):
            assert np.array_equal(t.cpu().numpy(), v)
