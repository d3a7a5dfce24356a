"""Eviction from the paged cache against the oracle, exactly: lengths, budgets, held positions, ties, special values, strides,
bad pages, graphs, lengths in place."""
import numpy as np
import pytest
import torch

from cache_util import DEV
from oracle import cache_weights_oracle as ref
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu


def _inputs(lens, seed=0, cols=None, values="heavy", spare=2):
    g = torch.Generator().manual_seed(seed)
    R, need = len(lens), [max(0, n) for n in lens]
    pages = [(n + 63) // 64 for n in need]
    total = sum(pages) + spare
    cache = torch.randint(0, 256, (total, 64, 656), generator=g, dtype=torch.uint8)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    bt = torch.full((R, max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
    cols = cols or max(1, max(need))
    w = torch.randn((R, cols), generator=g)
    if values == "heavy":
        w = torch.exp(3 * w)
    elif values == "ties":
        w = torch.randint(0, 3, (R, cols), generator=g).float()
    elif values == "one":
        w = torch.ones((R, cols))
    elif values == "special":
        pick = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), -float("nan"), 1e-45, -1e-45, 1.0, -1.0])
        w = pick[torch.randint(0, 10, (R, cols), generator=g)]
    pos = torch.stack([torch.randperm(cols, generator=g) for _ in range(R)]).to(torch.int32) * 2
    nxt = torch.tensor([2 * cols] * R, dtype=torch.int32)
    return w, pos, nxt, torch.tensor(lens, dtype=torch.int32), cache, bt


def _check(w, pos, nxt, lens, cache, bt, keep, sinks=0, recent=0, flags=0, in_place=False):
    k = keep.numpy() if isinstance(keep, torch.Tensor) else keep
    want = ref.evict(w.numpy(), pos.numpy(), nxt.numpy(), lens.numpy(), k, cache.numpy(), bt.numpy(), sinks, recent)
    dw, dp, dn, dl, dc, db = [t.to(DEV) for t in (w, pos, nxt, lens, cache, bt)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = api.sparse_mla_kv_evict(dw, dp, dn, dl, keep.to(DEV) if isinstance(keep, torch.Tensor) else keep, dc, db,
                                  sinks=sinks, recent=recent, new_lens=dl if in_place else None, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == flags
    assert np.array_equal(new.cpu().numpy(), want[3])
    assert np.array_equal(dw.cpu().numpy().view(np.int32), want[0].view(np.int32))
    assert np.array_equal(dp.cpu().numpy(), want[1])
    assert np.array_equal(dc.cpu().numpy(), want[2])
    return new


@pytest.mark.parametrize("n", [0, 1, 2, 31, 32, 33, 64, 65, 1000, 1023, 1024, 1025, 5000])
@pytest.mark.parametrize("part", [0.0, 0.5, 0.97, 1.0])
def test_lengths(n, part):
    _check(*_inputs([n], seed=n), keep=int(n * part))


@pytest.mark.parametrize("values", ["ties", "one", "special"])
def test_ties_and_special_values(values):
    _check(*_inputs([777, 64, 3], seed=3, values=values), keep=300)
    _check(*_inputs([777, 64, 3], seed=4, values=values), keep=10, sinks=9, recent=30)


@pytest.mark.parametrize("sinks,recent", [(5, 0), (0, 40), (7, 33), (10 ** 6, 0), (0, 2 ** 31 - 1)])
def test_held_positions_stay(sinks, recent):
    _check(*_inputs([700, 20, 129], seed=5), keep=60, sinks=sinks, recent=recent)


def test_more_held_than_the_budget():
    new = _check(*_inputs([700], seed=6), keep=10, recent=200)
    assert int(new[0]) == 100                              # positions are even: 100 of them among the last 200


def test_a_budget_per_request_and_lengths_in_place():
    keep = torch.tensor([0, 5, 100, -3, 10 ** 9, 64], dtype=torch.int32)
    _check(*_inputs([300, 300, 77, 40, 129, 0], seed=7), keep=keep, in_place=True)


@pytest.mark.parametrize("cols,lens", [(9000, [9000]), (20000, [20000, 7000]), (70000, [70000]), (340000, [340000, 1]),
                                       (400001, [400001])])
def test_long_requests_over_several_ctas(cols, lens):
    for values in ("heavy", "ties"):
        _check(*_inputs(lens, seed=cols, values=values), keep=lens[0] // 2, sinks=4, recent=64)


def test_many_requests():
    g = torch.Generator().manual_seed(8)
    _check(*_inputs(torch.randint(0, 500, (300,), generator=g).tolist(), seed=8), keep=120, sinks=2, recent=20)


def test_strided_rows():
    w, pos, nxt, lens, cache, bt = _inputs([200, 100], seed=9)
    want = ref.evict(w.numpy(), pos.numpy(), nxt.numpy(), lens.numpy(), 60, cache.numpy(), bt.numpy(), 0, 0)
    dw = torch.full((2, 333), 5.0, device=DEV)
    dp = torch.full((2, 250), 6, dtype=torch.int32, device=DEV)
    dw[:, 3:203], dp[:, :200] = w.to(DEV), pos.to(DEV)
    api.sparse_mla_kv_evict(dw[:, 3:203], dp[:, :200], nxt.to(DEV), lens.to(DEV), 60, cache.to(DEV), bt.to(DEV))
    torch.cuda.synchronize()
    assert np.array_equal(dw[:, 3:203].cpu().numpy(), want[0]) and np.array_equal(dp[:, :200].cpu().numpy(), want[1])
    assert torch.all(dw[:, :3] == 5) and torch.all(dw[:, 203:] == 5) and torch.all(dp[:, 200:] == 6)


def test_bad_pages_leave_the_record():
    w, pos, nxt, lens, cache, bt = _inputs([400], seed=10)
    bt[0, 1], bt[0, 5] = -1, 10 ** 6
    _check(w, pos, nxt, lens, cache, bt, keep=200, flags=_native.DEVERR_PAGE_RANGE)


def test_lengths_beyond_the_columns_are_clamped():
    w, pos, nxt, lens, cache, bt = _inputs([300, 200], seed=11, cols=250)
    _check(w, pos, nxt, lens, cache, bt, keep=100, flags=_native.DEVERR_LEN_RANGE)
    lens[1] = -7
    _check(w, pos, nxt, lens, cache, bt, keep=100, flags=_native.DEVERR_LEN_RANGE)


def test_a_captured_call_follows_the_lengths():
    w, pos, nxt, lens, cache, bt = _inputs([500, 300], seed=12)
    d = [t.to(DEV) for t in (w, pos, nxt, lens, cache, bt)]
    ws = api.alloc_evict_workspace(d[0])
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sparse_mla_kv_evict(*d[:4], 100, *d[4:], sinks=3, new_lens=new, workspace=ws)
    for ln in ([500, 300], [130, 99], [0, 300]):
        for t, v in zip(d, (w, pos, nxt, torch.tensor(ln, dtype=torch.int32), cache, bt)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.evict(w.numpy(), pos.numpy(), nxt.numpy(), ln, 100, cache.numpy(), bt.numpy(), 3, 0)
        for t, v in zip((d[0], d[1], d[4], new), want):
            assert np.array_equal(t.cpu().numpy(), v)


def test_two_evictions_at_once():
    cases = [_inputs([900], seed=20 + i) for i in range(2)]
    dev = [[t.to(DEV) for t in c] for c in cases]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for d, st in zip(dev, side):
        api.sparse_mla_kv_evict(*d[:4], 400, *d[4:], stream=st)
    torch.cuda.synchronize()
    for c, d in zip(cases, dev):
        want = ref.evict(*[t.numpy() for t in c[:4]], 400, c[4].numpy(), c[5].numpy(), 0, 0)
        assert np.array_equal(d[0].cpu().numpy(), want[0]) and np.array_equal(d[4].cpu().numpy(), want[2])
