"""Host-side checks of the operators around the paged cache through the C ABI (no GPU needed: nothing launches), and
their oracles on closed forms."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from oracle import dense_oracle, norm_rope_oracle as nr
from sparse_mla_decode_paged_gb300 import _native, api

P = C.c_void_p(1 << 20)      # aligned non-null stand-in; never dereferenced by these calls
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _dense(lib, dims, q=P, out=P, ws=P, ws_bytes=1 << 40):
    return lib.sparse_mla_dense_decode(C.byref(dims), q, P, P, P, C.c_float(0.04), out, P, ws, C.c_size_t(ws_bytes), None)


def test_dense_refusals(lib):
    ok = lambda **k: api.make_dense_dims(**{**dict(B=4, H=64, max_pages_per_seq=16, num_pages=100, queries_per_request=1), **k})
    assert _dense(lib, ok(), q=None) == INVALID
    assert _dense(lib, ok(), q=C.c_void_p((1 << 20) + 8)) == INVALID
    assert _dense(lib, ok(), out=C.c_void_p((1 << 20) + 4)) == INVALID
    assert _dense(lib, ok(), ws=None) == WORKSPACE
    assert _dense(lib, ok(), ws=C.c_void_p((1 << 20) + 16)) == WORKSPACE
    assert _dense(lib, ok(), ws_bytes=255) == WORKSPACE
    assert _dense(lib, ok(B=0)) == INVALID
    assert _dense(lib, ok(H=0)) == INVALID
    assert _dense(lib, ok(B=5, queries_per_request=2)) == INVALID
    assert _dense(lib, ok(ctas=-1)) == INVALID
    assert _dense(lib, ok(H=129)) == UNSUPPORTED
    assert _dense(lib, ok(B=65536)) == UNSUPPORTED
    assert _dense(lib, ok(ctas=1025)) == UNSUPPORTED
    assert _dense(lib, ok(num_pages=1 << 31)) == UNSUPPORTED
    bad = ok()
    bad.page_size = 32
    assert _dense(lib, bad) == UNSUPPORTED
    assert lib.sparse_mla_dense_decode(None, P, P, P, P, C.c_float(1.0), P, P, P, C.c_size_t(1 << 40), None) == INVALID


def test_dense_plan(lib):
    for H, sq, rows, groups in ((1, 1, 16, 1), (16, 1, 16, 1), (17, 1, 32, 1), (16, 2, 32, 1), (64, 1, 64, 1),
                                (128, 1, 64, 2), (128, 3, 64, 6), (5, 13, 64, 2)):
        p = api.dense_plan_for(api.make_dense_dims(sq * 3, H, 65536, 100, sq), 152)
        assert (p.rows_per_cta, p.row_groups) == (rows, groups)
        assert p.ctas == 152 and p.workspace_bytes >= 256
    # short tables: smaller row groups while a CTA has at most 4 (16 rows) or 24 (32 rows) tiles
    for pages, sq, rows, groups in ((128, 1, 16, 4), (304, 1, 16, 4), (306, 1, 32, 2), (3648, 1, 32, 2), (3650, 1, 64, 1),
                                    (304, 2, 32, 4), (1, 9, 16, 36)):
        p = api.dense_plan_for(api.make_dense_dims(sq, 64, pages, 100, sq), 152)
        assert (p.rows_per_cta, p.row_groups) == (rows, groups)
    # very wide tables: a CTA counts its tiles in 32 bits
    assert api.dense_plan_for(api.make_dense_dims(65535, 128, 1 << 17, 100), 152).row_groups == 2
    assert lib.sparse_mla_dense_plan_for(C.byref(api.make_dense_dims(65535, 128, 1 << 24, 100)), 152,
                                         C.byref(p)) == UNSUPPORTED
    p = api.dense_plan_for(api.make_dense_dims(3, 64, 8, 100, ctas=40), 152)
    assert p.ctas == 40
    assert lib.sparse_mla_dense_plan_for(None, 152, C.byref(p)) == INVALID
    assert lib.sparse_mla_dense_plan_for(C.byref(api.make_dense_dims(3, 64, 8, 100)), 0, C.byref(p)) == INVALID


def _na(**k):
    d = dict(tokens=4, num_requests=2, page_size=64, max_pages_per_seq=8, d_latent=512, d_rope=64, num_pages=100,
             latent_stride=576, rope_stride=576, dtype=0, weight_dtype=0, max_positions=100, interleaved=1)
    return _native.SmlaNormAppendDims(**{**d, **k})


def test_norm_append_refusals(lib):
    def call(d, lat=P, rope=P, w=P, eps=1e-6, cs=P, pos=P, kv=P):
        return lib.sparse_mla_kv_norm_append(C.byref(d), lat, rope, w, C.c_float(eps), cs, P, None, pos, kv, None, None)
    odd = C.c_void_p((1 << 20) + 1)
    for kw in (dict(lat=None), dict(rope=None), dict(w=None), dict(cs=None), dict(pos=None), dict(kv=None), dict(lat=odd),
               dict(kv=C.c_void_p((1 << 20) + 8)), dict(cs=C.c_void_p((1 << 20) + 4)), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(_na(), **kw) == INVALID, kw
    for kw in (dict(tokens=-1), dict(num_requests=0), dict(latent_stride=511), dict(rope_stride=63), dict(dtype=3),
               dict(dtype=0, weight_dtype=1), dict(max_positions=0), dict(interleaved=2), dict(num_pages=0)):
        assert call(_na(**kw)) == INVALID, kw
    for kw in (dict(page_size=32), dict(d_latent=256), dict(d_rope=32)):
        assert call(_na(**kw)) == UNSUPPORTED, kw


def _nr(**k):
    d = dict(tokens=4, num_heads=2, head_dim=128, rope_dim=64, rope_offset=64, dtype=0, weight_dtype=0, norm=1,
             interleaved=1, max_positions=10, x_token_stride=256, x_head_stride=128, out_token_stride=256,
             out_head_stride=128)
    return _native.SmlaNormRopeDims(**{**d, **k})


def test_norm_rope_refusals(lib):
    def call(d, x=P, w=P, eps=1e-6, cs=P, pos=P, out=P):
        return lib.sparse_mla_norm_rope(C.byref(d), x, w, C.c_float(eps), cs, pos, out, None, None)
    for kw in (dict(x=None), dict(out=None), dict(cs=None), dict(pos=None), dict(eps=-1e-6),
               dict(x=C.c_void_p((1 << 20) + 1)), dict(cs=C.c_void_p((1 << 20) + 2))):
        assert call(_nr(), **kw) == INVALID, kw
    for kw in (dict(tokens=-1), dict(num_heads=0), dict(head_dim=0), dict(rope_dim=63), dict(rope_dim=-2),
               dict(rope_offset=65), dict(rope_offset=-1), dict(dtype=7), dict(norm=2), dict(max_positions=0),
               dict(x_head_stride=-1), dict(out_head_stride=127), dict(out_token_stride=255),
               dict(out_token_stride=0), dict(rope_offset=2147483647), dict(out_token_stride=128, out_head_stride=256)):
        assert call(_nr(**kw)) == INVALID, kw
    assert call(_nr(head_dim=1025, rope_offset=0, x_head_stride=2000, out_head_stride=2000, out_token_stride=4000)) == \
        UNSUPPORTED


def test_read_refusals(lib):
    def call(d, kv=P, out=P, dt=0):
        return lib.sparse_mla_kv_read(C.byref(d), kv, P, None, P, out, dt, None, None)
    D = _native.SmlaAppendDims
    assert call(D(4, 2, 64, 8, 512, 64, 100), kv=None) == INVALID
    assert call(D(4, 2, 64, 8, 512, 64, 100), out=C.c_void_p((1 << 20) + 8)) == INVALID
    assert call(D(4, 2, 64, 8, 512, 64, 100), dt=3) == INVALID
    assert call(D(-1, 2, 64, 8, 512, 64, 100)) == INVALID
    assert call(D(4, 2, 32, 8, 512, 64, 100)) == UNSUPPORTED


# --------------------------------------------------------------------------- the oracles

def test_dense_oracle_equals_the_sparse_oracle_over_every_position():
    from cache_util import bits, make_dense
    q, cache, bt, lens = make_dense([70, 3, 0, 130], 3, 2, seed=1)
    tk = np.tile(np.arange(192), (4, 1))
    a = dense_oracle.dense_decode(bits(q), cache.numpy(), bt.numpy(), lens.numpy(), 0.05)
    b = oracle.sparse_mla_decode(bits(q), cache.numpy(), bt.numpy(), tk, lens.numpy(), 0.05)
    assert np.allclose(a[0], b[0], rtol=1e-12, atol=1e-14) and np.allclose(a[1], b[1], rtol=1e-12)
    assert np.all(a[2] >= np.abs(a[0]) - 1e-12) and np.all(a[3] >= 0) and np.all(a[4] >= 0)


def test_rotation_oracle_turns_by_the_angle():
    tab = api.rope_table(7, 4, device="cpu").numpy().astype(np.float64)
    x = np.array([1.0, 0.0, 0.0, 1.0])
    y, _ = nr.rotate(x, tab[3], True)
    assert np.allclose(y, [np.cos(3), np.sin(3), -np.sin(0.03), np.cos(0.03)], atol=1e-6)
    y, _ = nr.rotate(np.array([1.0, 0.0, 0.0, 1.0]), tab[3], False)      # pairs (0, 2), (1, 3)
    assert np.allclose(y, [np.cos(3), -np.sin(0.03), np.sin(3), np.cos(0.03)], atol=1e-6)
    z = np.random.default_rng(0).standard_normal((5, 4))
    assert np.allclose(np.linalg.norm(nr.rotate(z, tab[:5], True)[0], axis=1), np.linalg.norm(z, axis=1), rtol=1e-6)
    n = nr.rms_norm(z, None, 0.0)
    assert np.allclose((n * n).mean(-1), 1.0)
    with pytest.raises(ValueError):
        api.rope_table(5, 3, device="cpu")
    assert api.rope_table(5, device="cpu").shape == (5, 64) and api.rope_table(5, device="cpu").dtype == torch.float32
