"""Dense decode: the merge reads what its own call wrote, whatever an earlier call left in the workspace."""
import pytest
import torch

from cache_util import DEV, make_dense
from sparse_mla_decode_paged_gb300 import api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


@pytest.mark.parametrize("lens", [[40000], [3000] * 6 + [7, 0]], ids=["many_parts", "few_parts"])
def test_calls_one_after_the_other_in_one_workspace(lens):
    q, cache, bt, n = [t.to(DEV) for t in make_dense(lens, 64, seed=50, poison=False)]
    qs = [(q.float() * f).to(torch.bfloat16) for f in (1.0, -0.5, 3.0, 0.0)]
    want = [api.sparse_mla_dense_decode(x, cache, bt, n, SCALE) for x in qs]         # a workspace each
    ws = api.alloc_dense_workspace(api.dense_dims_of(q, cache, bt), DEV)
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    for _ in range(3):
        for x, (o, l) in zip(qs, outs):
            api.sparse_mla_dense_decode(x, cache, bt, n, SCALE, out=o, lse=l, workspace=ws)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    # and replayed: the graph's kernels keep the launch that overlaps the decode with its merge
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, (o, l) in zip(qs, outs):
            api.sparse_mla_dense_decode(x, cache, bt, n, SCALE, out=o, lse=l, workspace=ws)
    for o, l in outs:
        o.zero_()
        l.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
