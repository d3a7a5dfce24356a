"""Norm + rotation (per head, and fused with the FP8 append) and reading records back, against float64 oracles."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import DEV, bits, check_dense
from oracle import dense_oracle, kv_append_oracle as ka, norm_rope_oracle as nr
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
# float32 norm: 21 roundings in the sum of squares (halved by the root), the reciprocal root within 2 ulp, two
# products: below 2^-19 in all; a rotation adds three more
NORM_ERR = 2.0 ** -19


def _table(n, dim=64):
    return api.rope_table(n, dim, device="cpu")


def _f64(t):
    return t.double().cpu().numpy()


# --------------------------------------------------------------------------- per head

def _norm_rope_case(T, H, D, off, rdim, dtype, interleaved=True, norm=True, weight="x", seed=0, maxpos=5000):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    x = (torch.randn((T, H, D), generator=g) * 2).to(dt)
    w = None if weight is None else (1 + 0.3 * torch.randn(D, generator=g)).to(torch.float32 if weight == "fp32" else dt)
    tab = _table(maxpos, rdim) if rdim else None
    pos = torch.randint(0, maxpos, (T,), generator=g).to(torch.int32)
    return x, w, tab, pos


def _check_norm_rope(got, x, w, tab, pos, dtype, norm, off, interleaved, eps=1e-6):
    ref, mag = nr.norm_rope(_f64(x), pos.numpy(), None if tab is None else tab.numpy(),
                            None if w is None else _f64(w), eps, norm, off, interleaved)
    # fp16 results below 2^-14 have steps of 2^-24
    tol = HALF_STEP[dtype] * np.abs(ref) + 2 * NORM_ERR * mag + (2.0 ** -25 if dtype == "fp16" else 0.0)
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,D,off,rdim", [(1, 1, 64, 0, 64), (1, 64, 192, 128, 64), (7, 5, 128, 0, 64),
                                           (33, 3, 576, 512, 64), (5, 2, 1024, 0, 128), (4, 3, 512, 0, 0),
                                           (3, 7, 100, 36, 64), (6, 2, 96, 8, 30), (2, 3, 2, 0, 2), (3, 1, 1, 0, 0),
                                           (2, 2, 257, 1, 256), (11, 4, 80, 16, 64)])
def test_norm_rope(T, H, D, off, rdim, dtype):
    for interleaved in (True, False):
        x, w, tab, pos = _norm_rope_case(T, H, D, off, rdim, dtype, seed=D + T)
        got = api.sparse_mla_norm_rope(x.to(DEV), pos.to(DEV) if rdim else None, tab.to(DEV) if rdim else None,
                                       weight=w.to(DEV), rope_offset=off, interleaved=interleaved)
        _check_norm_rope(got, x, w, tab, pos, dtype, True, off, interleaved)


@pytest.mark.parametrize("norm,weight", [(True, None), (True, "fp32"), (False, None)])
def test_norm_rope_without_weight_or_norm(norm, weight):
    for D, off in ((192, 128), (70, 3)):
        x, w, tab, pos = _norm_rope_case(9, 4, D, off, 64, "bf16", weight=weight, seed=3)
        got = api.sparse_mla_norm_rope(x.to(DEV), pos.to(DEV), tab.to(DEV), weight=None if w is None else w.to(DEV),
                                       norm=norm, rope_offset=off)
        _check_norm_rope(got, x, w, tab, pos, "bf16", norm, off, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_strides_and_in_place(interleaved, dtype):
    g = torch.Generator().manual_seed(4)
    dt = TYPES[dtype]
    for shift in (0, 1, 8):                                     # element offsets: wide and element-wise accesses
        base = torch.randn((13, 6, 200 + 16), generator=g).to(dt)
        x = base[:, 1:5, shift:shift + 192]
        w = (1 + 0.1 * torch.randn(192, generator=g)).to(dt)
        tab, pos = _table(300), torch.randint(0, 300, (13,), generator=g).to(torch.int32)
        dbase = base.to(DEV)
        dx = dbase[:, 1:5, shift:shift + 192]
        # heads outermost
        out = torch.empty((4, 13, 192), dtype=dt, device=DEV).transpose(0, 1)
        api.sparse_mla_norm_rope(dx, pos.to(DEV), tab.to(DEV), weight=w.to(DEV), rope_offset=128,
                                 interleaved=interleaved, out=out)
        _check_norm_rope(out, x, w, tab, pos, dtype, True, 128, interleaved)
        assert torch.equal(dbase.cpu(), base)
        api.sparse_mla_norm_rope(dx, pos.to(DEV), tab.to(DEV), weight=w.to(DEV), rope_offset=128,
                                 interleaved=interleaved, out=dx)
        assert torch.equal(dx, out)
        keep = torch.ones_like(base, dtype=torch.bool)
        keep[:, 1:5, shift:shift + 192] = False
        assert torch.equal(dbase.cpu()[keep], base[keep])


def test_norm_rope_writes_into_another_layout():
    # the rotated part of 192-dim heads into the last 64 dims of 576-dim query rows
    x, _, tab, pos = _norm_rope_case(5, 16, 192, 0, 64, "bf16", seed=6)
    q = torch.full((5, 16, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    api.sparse_mla_norm_rope(x.to(DEV)[..., 128:], pos.to(DEV), tab.to(DEV), norm=False, out=q[..., 512:])
    _check_norm_rope(q[..., 512:], x[..., 128:], None, tab, pos, "bf16", False, 0, True)
    assert torch.all(q[..., :512] == 3.0)


def test_norm_rope_positions_out_of_range():
    for D in (64, 70):
        x, w, tab, pos = _norm_rope_case(6, 3, D, 0, 64, "bf16", seed=7, maxpos=50)
        pos[1], pos[4] = 50, -1
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = api.sparse_mla_norm_rope(x.to(DEV), pos.to(DEV), tab.to(DEV), weight=w.to(DEV), err_word=err)
        _check_norm_rope(got, x, w, tab, pos, "bf16", True, 0, True)
        assert int(err) == _native.DEVERR_LEN_RANGE
        assert not got[1].any() and not got[4].any()


def test_norm_rope_special_values():
    x, w, tab, pos = _norm_rope_case(4, 2, 128, 64, 64, "bf16", seed=8)
    x[0, 0] = 0                                                # all zero: eps alone under the root
    x[1, 1, 5] = float("nan")
    x[2, 0] = 1e-20
    got = api.sparse_mla_norm_rope(x.to(DEV), pos.to(DEV), tab.to(DEV), weight=w.to(DEV), rope_offset=64).cpu()
    assert not got[0, 0].any() and torch.isnan(got[1, 1]).all()
    rest = torch.ones((4, 2), dtype=torch.bool)
    rest[1, 1] = False
    ref, mag = nr.norm_rope(_f64(x), pos.numpy(), tab.numpy(), _f64(w), 1e-6, True, 64, True)
    tol = 2.0 ** -8 * np.abs(ref) + 2 * NORM_ERR * mag
    assert np.all((np.abs(_f64(got) - ref) <= tol)[rest.numpy()])


def test_norm_rope_empty_and_refused():
    x, w, tab, pos = [t.to(DEV) for t in _norm_rope_case(4, 2, 128, 0, 64, "bf16")]
    assert api.sparse_mla_norm_rope(x[:0], pos[:0], tab, weight=w).shape == (0, 2, 128)
    with pytest.raises(TypeError):
        api.sparse_mla_norm_rope(x.double(), pos, tab)
    with pytest.raises(TypeError):
        api.sparse_mla_norm_rope(x, pos.long(), tab)
    with pytest.raises(TypeError):
        api.sparse_mla_norm_rope(x, pos, tab, weight=w.half())
    with pytest.raises(ValueError):
        api.sparse_mla_norm_rope(x, pos[:2], tab)
    with pytest.raises(ValueError):
        api.sparse_mla_norm_rope(x, pos, tab, weight=w, norm=False)
    with pytest.raises(ValueError):
        api.sparse_mla_norm_rope(x.transpose(1, 2), pos, tab)
    with pytest.raises(ValueError):
        api.sparse_mla_norm_rope(x[:3], pos[:3], tab, out=x[1:])          # overlapping, shifted by a token
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_norm_rope(x, pos, tab, rope_offset=65)
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_norm_rope(x, pos, tab, eps=-1.0)
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_norm_rope(torch.zeros((1, 1, 1032), device=DEV))
    with pytest.raises(_native.SmlaError):                                # rows of out on top of one another
        api.sparse_mla_norm_rope(x, pos, tab, out=torch.empty((4, 1, 128), dtype=x.dtype, device=DEV).expand(4, 2, 128))


# --------------------------------------------------------------------------- fused append

def _append_case(T, dtype, seed, strided=True, pages=60, R=5, P=10, weight="x"):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    kv = torch.randn((T, 600), generator=g)
    kv[:, :512] *= torch.exp(torch.randn(T, 512, generator=g))
    if T > 3:
        kv[2, 128:256] = 0                                     # an all-zero block
        kv[3, :512] = 0                                        # an all-zero latent
    kv = kv.to(dt)
    lat, rope = kv[:, :512], kv[:, 512:576]
    if not strided:
        lat, rope = lat.contiguous(), rope.contiguous()
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.float32 if weight == "fp32" else dt)
    cache = torch.randint(0, 256, (pages, 64, 656), generator=g, dtype=torch.uint8)
    bt = torch.randperm(pages, generator=g)[:R * P].reshape(R, P).to(torch.int32)
    flat = torch.randperm(R * P * 64, generator=g)[:T]
    return lat, rope, w, cache, bt, (flat // (P * 64)).to(torch.int32), (flat % (P * 64)).to(torch.int32)


def _check_append(new, old, lat, rope, w, tab, bt, req, pos, interleaved, eps, skipped=()):
    new, old = new.cpu().numpy(), old.numpy()
    n = nr.rms_norm(_f64(lat), _f64(w), eps)
    touched = np.zeros(old.shape[:2], dtype=bool)
    for i in range(lat.shape[0]):
        if i in skipped:
            continue
        page, slot = int(bt[int(req[i]), int(pos[i]) // 64]), int(pos[i]) % 64
        touched[page, slot] = True
        codes, scales, y = oracle.decode_record(new[page, slot])
        blk = n[i].reshape(4, 128)
        amax = np.abs(blk).max(-1)
        ref_scale = np.where(amax > 0, amax / 448.0, 1.0)
        assert np.all(np.abs(scales - ref_scale) <= 2 * NORM_ERR * ref_scale)
        # a code is that of a value within the float32 error of n / scale: between the codes of its two ends
        quot = blk / ref_scale[:, None]
        lo, hi = (oracle.e4m3_to_f64(ka.e4m3_encode(quot - s * 4 * NORM_ERR * np.abs(quot))) for s in (1, -1))
        got = codes.reshape(4, 128)
        assert np.all((got >= lo) & (got <= hi))
        yr, mag = nr.rotate(_f64(rope[i]), tab[int(pos[i])].numpy(), interleaved)
        assert np.all(np.abs(y - yr) <= 2.0 ** -8 * np.abs(yr) + 2.0 ** -21 * mag)
    assert np.array_equal(new[~touched], old[~touched])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,strided", [(1, True), (5, False), (130, True), (131, False)])
def test_norm_append(T, strided, dtype):
    for interleaved in (True, False):
        lat, rope, w, cache, bt, req, pos = _append_case(T, dtype, seed=T, strided=strided)
        tab = _table(640)
        dc = cache.to(DEV)
        kv = torch.cat([lat, rope, torch.zeros((T, 24), dtype=lat.dtype)], 1).to(DEV)
        dl, dr = (kv[:, :512], kv[:, 512:576]) if strided else (lat.to(DEV), rope.to(DEV))
        api.sparse_mla_kv_norm_append(dl, dr, w.to(DEV), 1e-5, tab.to(DEV), bt.to(DEV), pos.to(DEV), dc,
                                      requests=req.to(DEV), interleaved=interleaved)
        torch.cuda.synchronize()
        _check_append(dc, cache, lat, rope, w, tab, bt, req, pos, interleaved, 1e-5)


def test_norm_append_odd_strides_fp32_weight_and_no_requests():
    lat, rope, w, cache, bt, _, _ = _append_case(5, "bf16", seed=31, weight="fp32")
    pos = torch.tensor([0, 63, 64, 639, 200], dtype=torch.int32)
    kv = torch.zeros((5, 577), dtype=lat.dtype)                # rows 1154 bytes apart: element-wise loads
    kv[:, 1:513], kv[:, 513:] = lat, rope
    dc, tab, dkv = cache.to(DEV), _table(640), kv.to(DEV)
    api.sparse_mla_kv_norm_append(dkv[:, 1:513], dkv[:, 513:], w.to(DEV), 1e-6, tab.to(DEV), bt.to(DEV), pos.to(DEV), dc)
    torch.cuda.synchronize()
    _check_append(dc, cache, lat, rope, w, tab, bt, torch.arange(5), pos, True, 1e-6)


def test_norm_append_with_unit_norm_matches_the_plain_append():
    # latents of power-of-two scaled unit rows: the norm multiplies by an exact power of two, so the
    # records equal those of the append of the normed latents
    g = torch.Generator().manual_seed(32)
    sign = torch.where(torch.rand((9, 512), generator=g) < 0.5, -1.0, 1.0)
    lat = (sign * 2.0 ** torch.arange(-4, 5)[:, None]).to(torch.bfloat16)
    rope = torch.randn((9, 64), generator=g).to(torch.bfloat16)
    bt, pos = torch.arange(9, dtype=torch.int32)[:, None], torch.zeros(9, dtype=torch.int32)
    a, b = (torch.zeros((9, 64, 656), dtype=torch.uint8, device=DEV) for _ in range(2))
    tab = _table(1).to(DEV)                                    # position 0: no turn
    api.sparse_mla_kv_norm_append(lat.to(DEV), rope.to(DEV), torch.ones(512, device=DEV), 0.0, tab, bt.to(DEV),
                                  pos.to(DEV), a)
    api.sparse_mla_kv_append(sign.to(torch.bfloat16).to(DEV), rope.to(DEV), bt.to(DEV), pos.to(DEV), b)
    codes = a[:, 0, :512].cpu().numpy()
    assert np.array_equal(codes, b[:, 0, :512].cpu().numpy())
    assert torch.equal(a[..., 528:], b[..., 528:])


def test_norm_append_skips_and_flags():
    lat, rope, w, cache, bt, _, _ = _append_case(7, "bf16", seed=33)
    bt[2, 1] = 99
    req = torch.tensor([0, 1, 2, 9, 0, 2, 3], dtype=torch.int32)
    pos = torch.tensor([3, 640, 100, 0, -1, 63, 500], dtype=torch.int32)
    tab = _table(500)                                          # position 500 is past the table
    dc, err = cache.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    api.sparse_mla_kv_norm_append(lat.to(DEV), rope.to(DEV), w.to(DEV), 1e-6, tab.to(DEV), bt.to(DEV), pos.to(DEV), dc,
                                  requests=req.to(DEV), err_word=err)
    torch.cuda.synchronize()
    assert int(err) == _native.DEVERR_PAGE_RANGE
    _check_append(dc, cache, lat, rope, w, tab, bt, req, pos, True, 1e-6, skipped=(1, 2, 3, 4, 6))


def test_norm_append_nan_latent_writes_nan_codes():
    lat, rope, w, cache, bt, req, pos = _append_case(2, "bf16", seed=34, strided=False)
    lat[1, 77] = float("nan")
    dc = cache.to(DEV)
    api.sparse_mla_kv_norm_append(lat.to(DEV), rope.to(DEV), w.to(DEV), 1e-6, _table(640).to(DEV), bt.to(DEV),
                                  pos.to(DEV), dc, requests=req.to(DEV))
    rec = dc[int(bt[int(req[1]), int(pos[1]) // 64]), int(pos[1]) % 64, :512].cpu()
    assert torch.all((rec & 0x7F) == 0x7F)


def test_norm_append_blocks_of_tiny_values():
    # block maxima down to where amax / 448, or its reciprocal, is no normal float: no code may become NaN
    g = torch.Generator().manual_seed(36)
    lat, rope = torch.randn((6, 512), generator=g), torch.zeros((6, 64))
    lat *= torch.tensor([1e-30, 1e-35, 1e-36, 1e-38, 1e-41, 1e-44])[:, None]
    lat[:, ::7] = 0
    bt, pos = torch.arange(6, dtype=torch.int32)[:, None], torch.zeros(6, dtype=torch.int32)
    cache = torch.full((6, 64, 656), 0x7F, dtype=torch.uint8, device=DEV)
    api.sparse_mla_kv_norm_append(lat.to(DEV), rope.to(DEV), torch.ones(512, device=DEV), 1.0, _table(1).to(DEV),
                                  bt.to(DEV), pos.to(DEV), cache)
    rec = cache.cpu().numpy()
    for i in range(6):
        codes, scales, _ = oracle.decode_record(rec[i, 0])
        n = lat[i].double().numpy().reshape(4, 128)            # (the mean square is 0 beside eps)
        got = codes.reshape(4, 128) * np.asarray(scales, dtype=np.float64)[:, None]
        # half a step of a code (2^-4 of it, 2^-10 scales at least), and the scale's own rounding in steps of 2^-149
        tol = 2.0 ** -4 * np.abs(n) * 1.001 + 2.0 ** -10 * scales[:, None] + 448 * 2.0 ** -150
        if i == 5:
            tol = np.abs(n)                                    # a scale of 1: codes of 0
        assert np.all(np.abs(got - n) <= tol)
        assert np.all(got[n == 0] == 0)


def test_norm_append_refused():
    lat, rope, w, cache, bt, req, pos = [t.to(DEV) for t in _append_case(4, "bf16", seed=35)]
    tab = _table(640).to(DEV)
    ok = dict(requests=req)
    with pytest.raises(TypeError):
        api.sparse_mla_kv_norm_append(lat.double(), rope.double(), w, 1e-6, tab, bt, pos, cache, **ok)
    with pytest.raises(ValueError):
        api.sparse_mla_kv_norm_append(lat, rope.float(), w, 1e-6, tab, bt, pos, cache, **ok)
    with pytest.raises(TypeError):
        api.sparse_mla_kv_norm_append(lat, rope, w.half(), 1e-6, tab, bt, pos, cache, **ok)
    with pytest.raises(ValueError):
        api.sparse_mla_kv_norm_append(lat[:1].expand(4, 512), rope, w, 1e-6, tab, bt, pos, cache, **ok)
    with pytest.raises(ValueError):
        api.sparse_mla_kv_norm_append(lat, rope, w, 1e-6, tab, bt, pos[:3], cache, **ok)
    with pytest.raises(ValueError):
        api.sparse_mla_kv_norm_append(lat, rope, w, 1e-6, tab, bt, pos, cache[..., :640], **ok)
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_kv_norm_append(lat, rope, w, float("nan"), tab, bt, pos, cache, **ok)
    api.sparse_mla_kv_norm_append(lat[:0], rope[:0], w, 1e-6, tab, bt, pos[:0], cache, requests=req[:0])


# --------------------------------------------------------------------------- read back

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 8, 9, 300])
def test_read_is_exact(T, dtype):
    _, _, _, cache, bt, req, pos = _append_case(T, "bf16", seed=40 + T)
    from sparse_mla_decode_paged_gb300 import workloads as wl
    cache = wl.fill_kv_cache(cache.shape[0], torch.Generator().manual_seed(41), "cpu")
    got = api.sparse_mla_kv_read(cache.to(DEV), bt.to(DEV), pos.to(DEV), requests=req.to(DEV), dtype=TYPES[dtype]).cpu()
    ref = dense_oracle.read_records(cache.numpy(), bt.numpy(), pos.numpy(), req.numpy())
    # a code times a scale has 28 bits: one rounding to float32, one to the output type
    assert torch.equal(got, torch.from_numpy(ref.astype(np.float32)).to(TYPES[dtype]))


def test_read_out_of_range_and_rows_behind():
    from sparse_mla_decode_paged_gb300 import workloads as wl
    _, _, _, cache, bt, _, _ = _append_case(7, "bf16", seed=42)
    cache = wl.fill_kv_cache(cache.shape[0], torch.Generator().manual_seed(43), "cpu")
    bt[2, 1] = 99
    req = torch.tensor([0, 1, 2, 9, 0, 2], dtype=torch.int32)
    pos = torch.tensor([3, 640, 100, 0, -1, 63], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    whole = torch.full((9, 576), 5.0, dtype=torch.bfloat16, device=DEV)
    api.sparse_mla_kv_read(cache.to(DEV), bt.to(DEV), pos.to(DEV), requests=req.to(DEV), out=whole[:6], err_word=err)
    ref = dense_oracle.read_records(cache.numpy(), bt.numpy(), pos.numpy(), req.numpy())
    assert torch.equal(whole[:6].cpu(), torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16))
    assert torch.all(whole[6:] == 5.0) and int(err) == _native.DEVERR_PAGE_RANGE


def test_read_special_records():
    cache = torch.zeros((1, 64, 656), dtype=torch.uint8)
    cache[0, 0, 0] = 0x7F                                      # NaN code
    cache[0, 0, 512:516] = torch.tensor([2.0]).view(torch.uint8)
    cache[0, 1, 0] = 0x7E                                      # 448 * 1e6: infinite in fp16 alone
    cache[0, 1, 512:516] = torch.tensor([1e6]).view(torch.uint8)
    bt, pos, req = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([[0]], [0, 1], [0, 0]))
    h = api.sparse_mla_kv_read(cache.to(DEV), bt, pos, requests=req, dtype=torch.float16)
    assert torch.isnan(h[0, 0]) and torch.isinf(h[1, 0]) and torch.isfinite(h[:, 1:]).all()
    assert float(api.sparse_mla_kv_read(cache.to(DEV), bt, pos, requests=req, dtype=torch.float32)[1, 0]) == 448e6


def test_read_refused():
    _, _, _, cache, bt, req, pos = [t.to(DEV) for t in _append_case(4, "bf16", seed=44)]
    with pytest.raises(TypeError):
        api.sparse_mla_kv_read(cache, bt, pos, requests=req, dtype=torch.float64)
    with pytest.raises(ValueError):
        api.sparse_mla_kv_read(cache, bt, pos, requests=req, out=torch.empty((5, 576), device=DEV))
    with pytest.raises(TypeError):
        api.sparse_mla_kv_read(cache, bt, pos.long(), requests=req)
    assert api.sparse_mla_kv_read(cache, bt, pos[:0], requests=req[:0]).shape == (0, 576)


# --------------------------------------------------------------------------- together

def test_a_captured_step_replayed_over_new_tokens():
    """Append, query rotation and dense decode captured on a stream of their own and replayed with the positions moved
    on: each step attends over what the steps before it wrote."""
    g = torch.Generator().manual_seed(51)
    R, H, start = 2, 16, torch.tensor([62, 0], dtype=torch.int32)
    tab, w = _table(128).to(DEV), torch.ones(512, device=DEV)
    bt = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32)
    from sparse_mla_decode_paged_gb300 import workloads as wl
    cache = wl.fill_kv_cache(4, torch.Generator().manual_seed(52), "cpu").to(DEV)
    kv, raw = torch.zeros((R, 576), device=DEV), torch.zeros((R, H, 576), dtype=torch.bfloat16, device=DEV)
    pos, dbt, q, seq = start.to(DEV), bt.to(DEV), torch.empty_like(raw), torch.zeros(R, dtype=torch.int32, device=DEV)
    ws = api.alloc_dense_workspace(api.dense_dims_of(raw, cache, dbt), DEV)
    out, lse = torch.empty((R, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((R, H), device=DEV)
    stream = torch.cuda.Stream()

    def step():
        api.sparse_mla_kv_norm_append(kv[:, :512], kv[:, 512:], w, 1e-6, tab, dbt, pos, cache)
        api.sparse_mla_norm_rope(raw, pos, tab, rope_offset=512, out=q)
        torch.add(pos, 1, out=seq)
        api.sparse_mla_dense_decode(q, cache, dbt, seq, 576 ** -0.5, out=out, lse=lse, workspace=ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(4):
        kv.copy_(torch.randn((R, 576), generator=g))
        raw.copy_(torch.randn((R, H, 576), generator=g))
        pos.copy_(start + i)
        before = cache.cpu()
        graph.replay()
        torch.cuda.synchronize()
        _check_append(cache, before, kv[:, :512].cpu(), kv[:, 512:].cpu(), w.cpu(), tab.cpu(), bt, torch.arange(R),
                      start + i, True, 1e-6)
        check_dense(out, lse, q.cpu(), cache.cpu(), bt, start + i + 1, 576 ** -0.5)
    assert api.read_errors(ws) == 0


def test_calls_on_a_stream_of_their_own():
    lat, rope, w, cache, bt, req, pos = _append_case(40, "bf16", seed=53)
    tab, dc = _table(640).to(DEV), cache.to(DEV)
    d = [t.to(DEV) for t in (lat, rope, w, bt, req, pos)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.sparse_mla_kv_norm_append(d[0], d[1], d[2], 1e-5, tab, d[3], d[5], dc, requests=d[4], stream=s)
    rows = api.sparse_mla_kv_read(dc, d[3], d[5], requests=d[4], dtype=torch.float32, stream=s)
    x = api.sparse_mla_norm_rope(rows.view(40, 1, 576), d[5], tab, norm=False, rope_offset=512, stream=s)
    s.synchronize()
    _check_append(dc, cache, lat, rope, w, tab.cpu(), bt, req, pos, True, 1e-5)
    ref = dense_oracle.read_records(dc.cpu().numpy(), bt.numpy(), pos.numpy(), req.numpy()).astype(np.float32)
    assert np.array_equal(rows.cpu().numpy(), ref)
    _check_norm_rope(x, rows.view(40, 1, 576).cpu(), None, tab.cpu(), pos, "fp32", False, 512, True)
    with pytest.raises((TypeError, AttributeError)):
        api.sparse_mla_kv_read(dc, d[3], d[5], requests=d[4], stream=0)


def test_a_decode_step_from_projections_to_output():
    """Prompt and new token written by the fused append, queries normed and rotated in place, the dense decode over
    the cache, and the context read back: each stage against the float64 oracle on what the stage before it wrote."""
    g = torch.Generator().manual_seed(50)
    R, H, prompt = 3, 16, [150, 64, 1]
    tab = _table(256).to(DEV)
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16).to(DEV)
    P = 4
    bt = torch.randperm(R * P, generator=g).view(R, P).to(torch.int32).to(DEV)
    cache = torch.full((R * P, 64, 656), 0x7F, dtype=torch.uint8, device=DEV)      # unwritten records are NaN
    for lens, start in ((prompt, [0] * R), ([1] * R, prompt)):
        req = torch.cat([torch.full((n,), r) for r, n in enumerate(lens)]).to(torch.int32)
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(start, lens)]).to(torch.int32)
        kv = torch.randn((len(req), 576), generator=g).to(torch.bfloat16)
        before = cache.cpu()
        dkv = kv.to(DEV)
        api.sparse_mla_kv_norm_append(dkv[:, :512], dkv[:, 512:], w, 1e-6, tab, bt, pos.to(DEV), cache,
                                      requests=req.to(DEV))
        _check_append(cache, before, kv[:, :512], kv[:, 512:], w.cpu(), tab.cpu(), bt.cpu(), req, pos, True, 1e-6)
    seq = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    q = torch.randn((R, H, 576), generator=g).to(torch.bfloat16).to(DEV)
    raw = q.clone()
    api.sparse_mla_norm_rope(q, seq, tab, rope_offset=512, out=q)
    _check_norm_rope(q, raw.cpu(), None, tab.cpu(), seq.cpu(), "bf16", True, 512, True)
    out, lse = api.sparse_mla_dense_decode(q, cache, bt, seq + 1, 576 ** -0.5)
    check_dense(out, lse, q.cpu(), cache.cpu(), bt.cpu(), (seq + 1).cpu(), 576 ** -0.5)
    rows = api.sparse_mla_kv_read(cache, bt, torch.arange(151, dtype=torch.int32, device=DEV),
                                  requests=torch.zeros(151, dtype=torch.int32, device=DEV), dtype=torch.float32)
    k = rows.double()
    s = (q[0].double() @ k.T) * 576 ** -0.5
    assert torch.allclose(torch.logsumexp(s, -1), lse[0].double(), atol=2e-5)
    assert bits(out).shape == (R, H, 512)
