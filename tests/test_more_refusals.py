"""Refusals of the masked and the shared decode, the attention weights and the eviction: through the C ABI (nothing launches) and
of the Python entry points."""
import ctypes as C

import pytest
import torch

from sparse_mla_decode_paged_gb300 import _native, api

P = C.c_void_p(1 << 20)      # aligned non-null stand-in; never dereferenced by these calls
ODD = C.c_void_p((1 << 20) + 2)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F = C.c_float


def _masked(lib, cap=0.0, slopes=None, starts=None, prefix=None, q=P, ws=P, n=1 << 40, **k):
    d = api.make_dense_dims(**{**dict(B=4, H=64, max_pages_per_seq=16, num_pages=100), **k})
    return lib.sparse_mla_masked_decode(C.byref(d), q, P, P, P, F(0.04), F(cap), slopes, starts, prefix, P, P, ws,
                                        C.c_size_t(n), None)


@pytest.mark.parametrize("cap", [-1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21, -0.5])
def test_masked_refuses_caps(lib, cap):
    assert _masked(lib, cap=cap) == INVALID


def test_masked_refusals(lib):
    assert _masked(lib, prefix=P) == INVALID                     # a prefix without starts
    assert _masked(lib, slopes=ODD) == INVALID
    assert _masked(lib, starts=ODD) == INVALID
    assert _masked(lib, starts=P, prefix=ODD) == INVALID
    assert _masked(lib, q=None) == INVALID
    assert _masked(lib, ws=None) == WORKSPACE
    assert _masked(lib, n=100) == WORKSPACE
    assert _masked(lib, H=129) == UNSUPPORTED
    assert _masked(lib, B=0) == INVALID


def _shared_dims(**k):
    v = dict(batch=8, num_heads=64, page_size=64, max_pages_per_seq=4, d_latent=512, d_rope=64, num_pages=100,
             queries_per_request=1, num_prefixes=2, prefix_pages=16)
    return _native.SmlaSharedDims(**{**v, **k})


def _shared(lib, q=P, table=P, ws=P, n=1 << 40, out=P, **k):
    return lib.sparse_mla_shared_decode(C.byref(_shared_dims(**k)), q, P, table, P, P, P, F(0.04), out, P, ws,
                                        C.c_size_t(n), None)


def test_shared_refusals(lib):
    assert _shared(lib, q=None) == INVALID
    assert _shared(lib, table=None) == INVALID
    assert _shared(lib, table=ODD) == INVALID
    assert _shared(lib, out=C.c_void_p((1 << 20) + 8)) == INVALID
    assert _shared(lib, ws=None) == WORKSPACE
    assert _shared(lib, ws=C.c_void_p((1 << 20) + 16)) == WORKSPACE
    assert _shared(lib, n=255) == WORKSPACE
    for bad in (dict(batch=0), dict(num_heads=0), dict(num_prefixes=0), dict(num_prefixes=3), dict(prefix_pages=0),
                dict(max_pages_per_seq=0), dict(num_pages=0), dict(queries_per_request=-1), dict(queries_per_request=3)):
        assert _shared(lib, **bad) == INVALID, bad
    for bad in (dict(page_size=32), dict(d_latent=256), dict(d_rope=32), dict(num_heads=129), dict(batch=65536),
                dict(num_pages=1 << 31)):
        assert _shared(lib, **bad) == UNSUPPORTED, bad
    assert lib.sparse_mla_shared_decode(None, P, P, P, P, P, P, F(1), P, P, P, C.c_size_t(1), None) == INVALID


def test_shared_workspace(lib):
    n = C.c_size_t(0)
    size = lambda sms=152, **k: (lib.sparse_mla_shared_workspace_size(C.byref(_shared_dims(**k)), sms, C.byref(n)), n.value)
    assert size(sms=0)[0] == INVALID and size(num_prefixes=3)[0] == INVALID
    assert lib.sparse_mla_shared_workspace_size(C.byref(_shared_dims()), 152, None) == INVALID
    assert lib.sparse_mla_shared_workspace_size(None, 152, C.byref(n)) == INVALID
    # results of 8 x 64 rows, twice, in any case; expanded records for many rows and long tables alone
    results = 2 * 8 * 64 * 513 * 4
    ok, few = size(prefix_pages=15)
    assert ok == 0 and results < few < results + (64 << 20)
    ok, many = size(prefix_pages=1000)
    assert ok == 0 and many > 2 * 1000 * 64 * 1152
    # not more than 4 GiB of them: wider tables stay with the dense kernel
    ok, wide = size(prefix_pages=40000)
    assert ok == 0 and wide < results + (64 << 20)
    # one SM has no pair
    assert size(sms=1, prefix_pages=1000)[0] == 0


def _weights(lib, decay=1.0, lse=P, w=P, err=None, **k):
    v = dict(batch=4, num_heads=64, page_size=64, max_pages_per_seq=16, d_latent=512, d_rope=64, num_pages=100,
             queries_per_request=1, num_cols=1000, weights_stride=1000)
    d = _native.SmlaWeightsDims(**{**v, **k})
    return lib.sparse_mla_attention_weights(C.byref(d), P, P, P, P, lse, F(0.04), F(decay), w, err, None)


def test_weights_refusals(lib):
    for decay in (-1.0, float("nan"), float("inf")):
        assert _weights(lib, decay=decay) == INVALID
    assert _weights(lib, lse=None) == INVALID
    assert _weights(lib, w=ODD) == INVALID
    assert _weights(lib, err=ODD) == INVALID
    for bad in (dict(batch=-1), dict(num_heads=0), dict(max_pages_per_seq=0), dict(num_pages=0), dict(num_cols=-1),
                dict(weights_stride=999), dict(queries_per_request=3)):
        assert _weights(lib, **bad) == INVALID, bad
    for bad in (dict(page_size=32), dict(num_heads=129), dict(batch=65536), dict(num_pages=1 << 31),
                dict(num_cols=(1 << 30) + 1, weights_stride=1 << 31)):
        assert _weights(lib, **bad) == UNSUPPORTED, bad
    # nothing to do is no error, whatever the pointers
    assert _weights(lib, batch=0, lse=None) == 0 and _weights(lib, num_cols=0, w=None) == 0


def _evict_dims(**k):
    v = dict(num_requests=4, num_cols=1000, page_size=64, max_pages_per_seq=16, d_latent=512, d_rope=64, num_pages=100,
             weights_stride=1000, positions_stride=1000, keep=10, sinks=0, recent=0)
    return _native.SmlaEvictDims(**{**v, **k})


def _evict(lib, w=P, keep=None, new=P, ws=P, n=1 << 40, **k):
    return lib.sparse_mla_kv_evict(C.byref(_evict_dims(**k)), w, P, P, P, keep, P, P, new, ws, C.c_size_t(n), None, None)


def test_evict_refusals(lib):
    assert _evict(lib, w=None) == INVALID
    assert _evict(lib, w=ODD) == INVALID
    assert _evict(lib, new=None) == INVALID
    assert _evict(lib, keep=ODD) == INVALID
    assert _evict(lib, ws=None) == WORKSPACE
    assert _evict(lib, n=lib.sparse_mla_kv_evict_workspace_size(C.byref(_evict_dims())) - 1) == WORKSPACE
    for bad in (dict(num_requests=-1), dict(num_cols=0), dict(max_pages_per_seq=0), dict(num_pages=0), dict(keep=-1),
                dict(sinks=-1), dict(recent=-1), dict(weights_stride=999), dict(positions_stride=999)):
        assert _evict(lib, **bad) == INVALID, bad
    for bad in (dict(page_size=32), dict(d_rope=32), dict(num_requests=65536), dict(num_pages=1 << 31),
                dict(num_cols=(1 << 30) + 1, weights_stride=1 << 31, positions_stride=1 << 31)):
        assert _evict(lib, **bad) == UNSUPPORTED, bad
    assert _evict(lib, num_requests=0, w=None, ws=None) == 0


def test_evict_workspace(lib):
    # half of a request's slots can move at most: two lists of them, and the counts
    assert lib.sparse_mla_kv_evict_workspace_size(C.byref(_evict_dims())) == 256 + 4 * 2 * 501 * 4
    assert lib.sparse_mla_kv_evict_workspace_size(None) == 0


# ------------------------------------------------------------------ Python

@pytest.fixture
def on_cpu(monkeypatch):
    """Checks that look at the device are answered as if the tensors were on the GPU."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _decode_args(B=4, H=8, R=4, pages=3):
    return [torch.zeros((B, H, 576), dtype=torch.bfloat16), torch.zeros((9, 64, 656), dtype=torch.uint8), _i32(R, pages),
            _i32(B)]


def test_masked_arguments(on_cpu):
    a = _decode_args()
    run = lambda slopes=None, starts=None, prefix=None, out=None, lse=None, args=a: api._masked_dims(
        *args, slopes, starts, prefix, out, lse, None, 0)
    assert run(torch.zeros(8), _i32(4), _i32(4)).batch == 4
    with pytest.raises(ValueError, match="slopes"):
        run(slopes=torch.zeros(7))
    with pytest.raises(TypeError, match="slopes"):
        run(slopes=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="starts"):
        run(starts=_i32(3))
    with pytest.raises(TypeError, match="starts"):
        run(starts=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="prefix_lens without starts"):
        run(prefix=_i32(4))
    with pytest.raises(ValueError, match="out"):
        run(out=torch.zeros((4, 8, 511), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="lse"):
        run(lse=torch.zeros((8, 4)))
    with pytest.raises(TypeError, match="q must be"):
        run(args=[None, *a[1:]])
    with pytest.raises(ValueError, match="divisor"):
        run(args=_decode_args(R=3))


def test_shared_arguments(on_cpu):
    q, kv, bt, ln = _decode_args()
    run = lambda pt=_i32(2, 5), pl=_i32(2), bt=bt, ln=ln: api._shared_dims(q, kv, pt, pl, bt, ln, None, None, None)
    d = run()
    assert (d.num_prefixes, d.prefix_pages, d.queries_per_request, d.max_pages_per_seq) == (2, 5, 1, 3)
    with pytest.raises(ValueError, match="group"):
        run(pt=_i32(3, 5), pl=_i32(3))
    with pytest.raises(ValueError, match="group"):
        run(pl=_i32(3))
    with pytest.raises(TypeError, match="prefix_lens"):
        run(pl=[1, 2])
    with pytest.raises(TypeError, match="prefix_table"):
        run(pt=torch.zeros((2, 5), dtype=torch.int64))


def test_weights_arguments(on_cpu):
    q, kv, bt, ln = _decode_args()
    run = lambda lse=torch.zeros((4, 8)), w=torch.zeros((4, 100)): api._weights_dims(q, kv, bt, ln, lse, w, None)
    assert run(w=torch.zeros((4, 300))[:, :100]).weights_stride == 300
    with pytest.raises(ValueError, match="lse"):
        run(lse=torch.zeros((4, 7)))
    with pytest.raises(TypeError, match="weights"):
        run(w=torch.zeros((4, 100), dtype=torch.float64))
    with pytest.raises(ValueError, match="weights"):
        run(w=torch.zeros((5, 100)))
    with pytest.raises(ValueError, match="weights"):
        run(w=torch.zeros((4, 200))[:, ::2])
    with pytest.raises(ValueError, match="weights"):
        run(w=torch.zeros((1, 100)).expand(4, 100))
    with pytest.raises(TypeError, match="weights must be a torch.Tensor"):
        run(w=None)


def test_evict_arguments(on_cpu):
    def run(w=torch.zeros((2, 100)), pos=_i32(2, 100), nxt=_i32(2), lens=_i32(2), keep=5, sinks=0, recent=0, new=None):
        return api._evict_dims(w, pos, nxt, lens, keep, torch.zeros((9, 64, 656), dtype=torch.uint8), _i32(2, 3), sinks, recent,
                               new, None)
    assert run().keep == 5 and run(keep=_i32(2)).keep == 0
    for bad in (dict(keep=-1), dict(sinks=-1), dict(recent=1 << 31), dict(keep=_i32(3)), dict(nxt=_i32(1)),
                dict(lens=_i32(2, 1)), dict(new=_i32(3)), dict(pos=_i32(2, 99)), dict(w=torch.zeros((2, 0)), pos=_i32(2, 0))):
        with pytest.raises(ValueError):
            run(**bad)
    for bad in (dict(keep=1.5), dict(keep=True), dict(sinks=None), dict(keep=torch.zeros(2)), dict(pos=torch.zeros((2, 100)))):
        with pytest.raises(TypeError):
            run(**bad)
