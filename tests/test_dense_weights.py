"""Dense decode: the bits that a position's weight keeps in each 128-dim block, beside positions that dominate a tile, blocks
of small scale and blocks without values, in every row group; errors element by element and by blocks."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, make_dense
from dense_util import block_errors, check_weights
from oracle import dense_oracle
from sparse_mla_decode_paged_gb300 import api
from test_dense_decode import SCALE, _every_row_group, _run

pytestmark = pytest.mark.gpu


def _check(q, cache, bt, lens, scale=SCALE, worst_block=None):
    for rows, wide in _every_row_group(q, cache, bt).items():
        out, lse, err = _run(q, cache, wide, lens, scale)
        assert err == 0
        check_weights(out, lse, q, cache, bt, lens, scale, rows)
        if worst_block is not None:
            ref = dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens.numpy(), scale)[0]
            got = block_errors(out.float().cpu().double().numpy(), ref)
            assert np.nanmax(got) <= worst_block, (rows, np.nanmax(got))


def _scales(cache):
    return cache[..., 512:528].contiguous().view(torch.float32)


def _put_scales(cache, sc):
    cache[..., 512:528] = sc.contiguous().view(torch.uint8)


def _rope_scores(q, cache, bt, lead):
    """Scores are the first rope value alone: those of request 0's positions."""
    q[:] = 0
    q[:, :, 512] = 1.0
    flat = torch.zeros(bt.shape[1] * 64)
    flat[:len(lead)] = torch.as_tensor(lead, dtype=torch.float32)
    for i in range(bt.shape[1]):
        if bt[0, i] >= 0:
            cache[int(bt[0, i]), :, 528:530] = flat[64 * i:64 * i + 64, None].to(torch.bfloat16).view(torch.uint8)


def _record(latent):
    """An appended record's latent part and scales, as the append writes them."""
    cache = torch.zeros((1, 64, 656), dtype=torch.uint8, device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    rope = torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)
    api.sparse_mla_kv_append(latent.to(torch.bfloat16).view(1, 512).to(DEV), rope, one.view(1, 1), one, cache)
    return cache[0, 0, :528].cpu()


@pytest.mark.parametrize("n", [1, 2, 3, 65, 127, 128, 129, 300, 1000, 4097])
def test_lengths(n):
    _check(*make_dense([n], 64, seed=n))


@pytest.mark.parametrize("H,s_q", [(1, 1), (5, 13), (16, 3), (33, 1), (64, 2), (128, 1)])
def test_heads_and_queries(H, s_q):
    lens = [max(0, n - (s_q - 1 - j)) for n in (700, 130) for j in range(s_q)]
    _check(*make_dense(lens, H, s_q, seed=H))


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.3])
def test_score_scales(scale):
    _check(*make_dense([321, 50], 64, seed=12), scale=scale)


@pytest.mark.parametrize("n", [128, 3000])
@pytest.mark.parametrize("lead", [0, 2, 4, 6, 8, 10, 12, 16, 25])
def test_a_zero_latent_that_dominates(lead, n):
    # as the append writes it: codes of 0 with scales of 1; the others' results are lead nats down, and keep their bits
    q, cache, bt, lens = make_dense([n], 64, seed=lead)
    _rope_scores(q, cache, bt, [lead if t == 57 else 0.02 * (t % 50) for t in range(n)])
    rec = _record(torch.zeros(512))
    assert not rec[:512].any() and torch.equal(rec[512:].view(torch.float32), torch.ones(4))
    cache[int(bt[0, 0]), 57, :528] = rec
    _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -6)


@pytest.mark.parametrize("lead", [0, 5, 10])
def test_a_zero_latent_with_any_scale(lead):
    q, cache, bt, lens = make_dense([200], 64, seed=lead)
    _rope_scores(q, cache, bt, [lead if t == 57 else 0.0 for t in range(200)])
    cache[int(bt[0, 0]), 57, :512] = torch.tensor([0x00, 0x80], dtype=torch.uint8).repeat(256)      # zeros of both signs
    sc = _scales(cache)
    sc[int(bt[0, 0]), 57] = torch.tensor([1e-3, 1e9, 0.0, 1e30])
    _put_scales(cache, sc)
    _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -6)


@pytest.mark.parametrize("lead", [0, 4, 8])
def test_zero_blocks_in_an_ordinary_record(lead):
    # the append writes a zero block's scale as 1: far above the other blocks'
    q, cache, bt, lens = make_dense([300], 64, seed=lead)
    _rope_scores(q, cache, bt, [lead if t == 200 else 0.0 for t in range(300)])
    g = torch.Generator().manual_seed(1)
    for t, empty in ((200, (1,)), (130, (0, 2, 3)), (10, (3,))):
        x = torch.randn(512, generator=g)
        for b in empty:
            x[128 * b:128 * b + 128] = 0
        cache[int(bt[0, t // 64]), t % 64, :528] = _record(x)
    _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -6)


@pytest.mark.parametrize("power", [5, 9, 11, 13, 16])
def test_blocks_of_small_scale(power):
    # block 1 of every record, and blocks 0 and 3 of every other record
    q, cache, bt, lens = make_dense([500, 90], 64, seed=power, poison=False)
    sc = _scales(cache)
    sc[..., 1] *= 2.0 ** -power
    sc[:, ::2, 0] *= 2.0 ** -power
    sc[:, 1::2, 3] *= 2.0 ** -power
    _put_scales(cache, sc)
    _check(q, cache, bt, lens, worst_block=2.0 ** -5)


@pytest.mark.parametrize("power", [5, 7, 9])
def test_a_dominating_position_of_small_scale_in_one_block(power):
    # its block 2 adds nothing to speak of, so that block is the others'
    q, cache, bt, lens = make_dense([128], 64, seed=power, poison=False)
    _rope_scores(q, cache, bt, [6.0 if t == 31 else 0.0 for t in range(128)])
    sc = _scales(cache)
    sc[int(bt[0, 0]), 31, 2] *= 2.0 ** -power
    _put_scales(cache, sc)
    _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -6)


@pytest.mark.parametrize("lead", [4, 8, 10])
def test_a_sink_of_small_value(lead):
    # 1/32 of the others' values, with the scales that come with it; its tile and 45 tiles behind it
    for n in (128, 6000):
        q, cache, bt, lens = make_dense([n], 64, seed=lead, poison=False)
        _rope_scores(q, cache, bt, [lead if t == 0 else 0.0 for t in range(n)])
        sc = _scales(cache)
        sc[int(bt[0, 0]), 0] /= 32
        _put_scales(cache, sc)
        _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -6)


@pytest.mark.parametrize("step", [-0.7, -0.2, 0.2, 0.7])
def test_scores_that_drift(step):
    # by less than a reference's window per tile, over 40 tiles
    n = 5000
    q, cache, bt, lens = make_dense([n], 64, seed=5, poison=False)
    g = torch.Generator().manual_seed(2)
    _rope_scores(q, cache, bt, (torch.randn(n, generator=g) * 2 + step * (torch.arange(n) // 128)).tolist())
    _check(q, cache, bt, lens, 1.0, worst_block=2.0 ** -5)


def test_agrees_with_the_sparse_decode_beside_a_sink():
    n = 400
    q, cache, bt, lens = make_dense([n], 64, seed=7)
    _rope_scores(q, cache, bt, [8.0 if t == 3 else 0.01 * (t % 100) for t in range(n)])
    cache[int(bt[0, 0]), 3, :512] = 0
    d = [t.to(DEV) for t in (q, cache, bt, lens)]
    so, _ = api.sparse_mla_decode(d[0], d[1], d[2], torch.arange(512, dtype=torch.int32, device=DEV)[None], d[3], 1.0)
    for wide in _every_row_group(q, cache, bt).values():
        do, _, _ = _run(q, cache, wide, lens, 1.0)
        assert block_errors(do.float().cpu().double().numpy(), so.float().cpu().double().numpy()).max() <= 2.0 ** -6


@pytest.mark.parametrize("power", [-50, 60, 100])
def test_scales_of_every_magnitude(power):
    q, cache, bt, lens = make_dense([200], 64, seed=14, poison=False)
    _put_scales(cache, _scales(cache) * 2.0 ** power)
    q[..., :512] *= 2.0 ** -max(power, 0)
    ref = dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens.numpy(), SCALE)[0]
    for rows, wide in _every_row_group(q, cache, bt).items():
        out, lse, err = _run(q, cache, wide, lens)
        assert err == 0 and block_errors(out.float().cpu().double().numpy(), ref).max() <= 2.0 ** -6


def test_negative_scales():
    q, cache, bt, lens = make_dense([300], 64, seed=15, poison=False)
    sc = _scales(cache)
    sc[:, ::3, 1:3] *= -1
    _put_scales(cache, sc)
    _check(q, cache, bt, lens)


@pytest.mark.parametrize("n", [1, 2, 90])
@pytest.mark.parametrize("power", [18, 20, 22])
def test_blocks_of_very_small_scale(power, n):
    # beyond what a factor between two blocks' references can hold: fewer bits, but the right size.  (Off by at most
    # 2^-23.5 of the row's largest operand; scales of ordinary records differ by less than 2^4 among themselves.)
    q, cache, bt, lens = make_dense([n], 64, seed=power, poison=False)
    sc = _scales(cache)
    sc[..., 1] *= 2.0 ** -power
    sc[..., 2] *= 2.0 ** (6 - power)
    _put_scales(cache, sc)
    _check(q, cache, bt, lens, worst_block=2.0 ** (power - 19.5) if power < 19 else None)


def test_block_scales_that_spread_over_time():
    # block 0 grows by 2^26 over the tiles while the others stay: their references have to follow its weights
    n = 128 * 14
    q, cache, bt, lens = make_dense([n], 64, seed=3, poison=False)
    _rope_scores(q, cache, bt, [0.0] * n)
    sc = _scales(cache)
    for i in range(bt.shape[1]):
        sc[int(bt[0, i]), :, 0] *= 2.0 ** (i - 10)
    _put_scales(cache, sc)
    for rows, wide in _every_row_group(q, cache, bt).items():
        out, lse, err = _run(q, cache, wide, lens, 1.0)
        check_weights(out, lse, q, cache, bt, lens, 1.0, rows)


def test_a_context_of_zero_latents_alone():
    q, cache, bt, lens = make_dense([200, 3], 64, seed=4, poison=False)
    cache[..., :512] = 0
    _put_scales(cache, torch.ones_like(_scales(cache)))
    ref = dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), lens.numpy(), SCALE)
    for wide in _every_row_group(q, cache, bt).values():
        out, lse, err = _run(q, cache, wide, lens)
        # (such positions' scores are rounded beside an exponent of 60: 2^-19 in units of log2)
        assert err == 0 and not out.any() and np.abs(lse.cpu().numpy() - ref[1]).max() <= ref[4].max() + 2.0 ** -18
