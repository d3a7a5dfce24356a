"""Evictions whose keys do not fit into the shared memory of the CTAs that a request gets: every pass reads them anew."""
import numpy as np
import pytest
import torch

import test_kv_evict as evict
from cache_util import DEV
from sparse_mla_decode_paged_gb300 import api

pytestmark = pytest.mark.gpu
FIT = 40960                                                 # slots of a CTA whose keys fit


def _lens(requests, long):
    """A CTA per request, the others short."""
    return [long[i // 20] if i % 20 == 0 and i // 20 < len(long) else (i * 37) % 200 for i in range(requests)]


@pytest.mark.parametrize("requests", [80, 130])
@pytest.mark.parametrize("values", ["heavy", "ties", "one", "special"])
def test_a_cta_per_request(requests, values):
    """(Lengths on either side of what fits.)"""
    lens = _lens(requests, [FIT, FIT + 1, 41100, 50000])
    case = evict._inputs(lens, seed=requests, cols=50000, values=values)
    evict._check(*case, keep=20000, sinks=4, recent=64)


def test_budgets_from_none_to_all():
    lens = _lens(100, [41100, 41000, 45000, 41100, 41100])
    keep = torch.tensor([0, 0, 0, 0, 0] * 20, dtype=torch.int32)
    keep[0], keep[20], keep[40], keep[60], keep[80] = 0, 1, 44999, 41100, 30000
    evict._check(*evict._inputs(lens, seed=5, cols=45000, values="ties"), keep=keep, in_place=True)
    evict._check(*evict._inputs(lens, seed=6, cols=45000), keep=keep, sinks=30000)


def test_one_request_of_more_than_the_largest_cluster_holds():
    evict._check(*evict._inputs([700000], seed=7, values="ties"), keep=350000, sinks=4, recent=640)


def test_captured():
    lens = _lens(80, [41100, 50000])
    w, pos, nxt, ln, cache, bt = evict._inputs(lens, seed=8, cols=50000)
    d = [t.to(DEV) for t in (w, pos, nxt, ln, cache, bt)]
    ws = api.alloc_evict_workspace(d[0])
    new = torch.zeros(80, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sparse_mla_kv_evict(*d[:4], 15000, *d[4:], sinks=4, new_lens=new, workspace=ws)
    for step in range(3):
        n = ln.clone()
        if step == 1:
            n[0], n[20] = 300, 40961
        elif step == 2:
            n[:] = 0
            n[20] = 50000
        for t, v in zip(d, (w, pos, nxt, n, cache, bt)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = evict.ref.evict(w.numpy(), pos.numpy(), nxt.numpy(), n.tolist(), 15000, cache.numpy(), bt.numpy(), 4, 0)
        for t, v in zip((d[0], d[1], d[4], new), want):
            got = t.cpu().numpy()
            assert np.array_equal(got.view(np.int32) if got.dtype == np.float32 else got,
                                  v.view(np.int32) if v.dtype == np.float32 else v)
