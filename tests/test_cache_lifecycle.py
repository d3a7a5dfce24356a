"""The operators on one cache as a server runs them: append, decode, accumulate the weights, evict, append again, decode with a
mask and behind a shared prefix; step by step against the oracles, and a whole step captured."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, check_dense
from masked_util import check_decode
from oracle import cache_weights_oracle, masked_oracle
from sparse_mla_decode_paged_gb300 import api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
R, H, CTX, PAGES = 3, 16, 300, 6


class Server:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.cache = torch.zeros((R * PAGES + 2, 64, 656), dtype=torch.uint8, device=DEV)
        perm = torch.randperm(R * PAGES, generator=self.g).to(torch.int32)
        self.bt = perm.view(R, PAGES).to(DEV)
        self.table = api.rope_table(4096, device=DEV)
        self.norm = torch.ones(512, device=DEV)
        self.lens = torch.zeros(R, dtype=torch.int32, device=DEV)
        self.next = torch.zeros(R, dtype=torch.int32, device=DEV)
        self.weights = torch.zeros((R, PAGES * 64), device=DEV)
        self.positions = torch.zeros((R, PAGES * 64), dtype=torch.int32, device=DEV)
        self.ws = api.alloc_evict_workspace(self.weights)

    def append(self, kv):
        """One token per request at its next position, into its next slot.  (The rotation's angle follows the position, the
        slot follows the length.)"""
        rope = api.sparse_mla_norm_rope(kv[:, None, 512:], self.next, self.table, norm=False)[:, 0]
        latent = api.sparse_mla_norm_rope(kv[:, None, :512].contiguous(), weight=self.norm)[:, 0]
        api.sparse_mla_kv_append(latent.contiguous(), rope.contiguous(), self.bt, self.lens, self.cache)
        self.positions.scatter_(1, self.lens.long()[:, None], self.next[:, None])
        self.lens += 1
        self.next += 1

    def decode(self, q):
        q = api.sparse_mla_norm_rope(q, self.next - 1, self.table, norm=False, rope_offset=512)
        out, lse = api.sparse_mla_dense_decode(q, self.cache, self.bt, self.lens, SCALE)
        api.sparse_mla_attention_weights(q, self.cache, self.bt, self.lens, lse, SCALE, self.weights, decay=0.95)
        return q, out, lse

    def token(self):
        return (torch.randn((R, 576), generator=self.g).to(torch.bfloat16).to(DEV),
                torch.randn((R, H, 576), generator=self.g).to(torch.bfloat16).to(DEV))


def _filled(seed):
    s = Server(seed)
    for _ in range(CTX):
        s.append(s.token()[0])
    return s


def _host(*ts):
    return [t.cpu().numpy() for t in ts]


def test_decode_weights_evict_and_go_on():
    s = _filled(1)
    for step in range(6):
        kv, q = s.token()
        s.append(kv)
        old = s.weights.cpu().numpy()
        q, out, lse = s.decode(q)
        check_dense(out, lse, q.cpu(), s.cache.cpu(), s.bt.cpu(), s.lens.cpu(), SCALE)
        w, tol = cache_weights_oracle.attention_weights(bits(q).reshape(q.shape), *_host(s.cache, s.bt, s.lens, lse), SCALE, old,
                                                        0.95)
        assert np.all(np.abs(s.weights.cpu().double().numpy() - w) <= tol)
        if step % 2 == 1:
            before = _host(s.weights, s.positions, s.next, s.lens, s.cache, s.bt)
            new = api.sparse_mla_kv_evict(s.weights, s.positions, s.next, s.lens, 200 - 20 * step, s.cache, s.bt, sinks=4,
                                          recent=32, new_lens=s.lens, workspace=s.ws)
            want = cache_weights_oracle.evict(before[0], before[1], before[2], before[3], 200 - 20 * step, before[4],
                                              before[5], 4, 32)
            assert new is s.lens and np.array_equal(new.cpu().numpy(), want[3])
            for got, x in zip((s.weights, s.positions, s.cache), want):
                assert np.array_equal(got.cpu().numpy(), x)
            held = set(range(4)) | set(range(int(s.next[0]) - 32, int(s.next[0])))
            assert held <= set(s.positions[0, :int(s.lens[0])].tolist())


def test_masked_and_shared_decode_of_the_same_cache():
    s = _filled(2)
    _, q = s.token()
    starts = torch.tensor([100, 0, 299], dtype=torch.int32, device=DEV)
    prefix = torch.tensor([7, 0, 64], dtype=torch.int32, device=DEV)
    slopes = torch.exp2(-torch.arange(1, H + 1, device=DEV) / 2)
    out, lse = api.sparse_mla_masked_decode(q, s.cache, s.bt, s.lens, SCALE, softcap=5.0, slopes=slopes, starts=starts,
                                            prefix_lens=prefix)
    check_decode(out, lse, masked_oracle.masked_decode(bits(q).reshape(q.shape), *_host(s.cache, s.bt, s.lens), SCALE, 5.0,
                                                       *_host(slopes, starts, prefix)))
    # request 0's positions as a prefix of the other two
    pl = s.lens[:1].contiguous()
    out, lse = api.sparse_mla_shared_decode(q[1:], s.cache, s.bt[:1], pl, s.bt[1:], s.lens[1:], SCALE)
    check_decode(out, lse, masked_oracle.shared_decode(bits(q[1:]).reshape(2, H, 576),
                                                       *_host(s.cache, s.bt[:1], pl, s.bt[1:], s.lens[1:]), SCALE))


def test_a_captured_step():
    """append, decode, weights and eviction in one graph, replayed with the lengths that each replay leaves."""
    a, b = _filled(3), _filled(3)
    kv, q = a.token()
    torch.cuda.synchronize()

    def step(s, kv, q, out):
        s.append(kv)
        _, o, l = s.decode(q)
        out[0].copy_(o)
        out[1].copy_(l)
        api.sparse_mla_kv_evict(s.weights, s.positions, s.next, s.lens, 250, s.cache, s.bt, sinks=2, recent=16, new_lens=s.lens,
                                workspace=s.ws)

    outs = [(torch.zeros((R, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((R, H), device=DEV)) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(a, kv, q, outs[0])
    for _ in range(4):
        nkv, nq = b.token()
        kv.copy_(nkv)
        q.copy_(nq)
        graph.replay()
        step(b, nkv, nq, outs[1])
        torch.cuda.synchronize()
        for x, y in ((outs[0][0], outs[1][0]), (outs[0][1], outs[1][1]), (a.weights, b.weights), (a.positions, b.positions),
                     (a.lens, b.lens), (a.cache, b.cache)):
            assert torch.equal(x, y)
