"""Dense decode (every cached position) against the float64 oracle: lengths from none to several thousand, head
counts, several queries per request, CTA counts, positions that must not be read, bad pages, streams, graphs."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, check_dense, make_dense
from sparse_mla_decode_paged_gb300 import _native, api
from sparse_mla_decode_paged_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def _run(q, cache, bt, lens, scale=SCALE, ctas=0, ws=None):
    d = [t.to(DEV) for t in (q, cache, bt, lens)]
    if ws is None:
        ws = api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2], ctas), DEV)
    out = torch.full((q.shape[0], q.shape[1], 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    api.sparse_mla_dense_decode(*d, scale, out=out, lse=lse, workspace=ws, ctas=ctas)
    torch.cuda.synchronize()
    return out, lse, api.read_errors(ws)


def _every_row_group(q, cache, bt, ctas=0):
    """The block table as it is and widened, so that a CTA handles 16, 32 and 64 rows at once as far as the query has
    them (long tables make for large groups)."""
    seen = {}
    pages = bt.shape[1]
    while pages < 1 << 20:
        wide = torch.full((bt.shape[0], pages), -1, dtype=torch.int32)
        wide[:, :bt.shape[1]] = bt
        rows = api.dense_plan(api.dense_dims_of(q, cache, wide, ctas), 0).rows_per_cta
        seen.setdefault(rows, wide)
        if rows >= min(64, q.shape[0] // bt.shape[0] * q.shape[1]):
            break
        pages *= 2
    return seen


def _check(q, cache, bt, lens, scale=SCALE, ctas=0, flags=0):
    for rows, wide in _every_row_group(q, cache, bt, ctas).items():
        out, lse, err = _run(q, cache, wide, lens, scale, ctas)
        assert err == flags
        check_dense(out, lse, q, cache, bt, lens, scale)


@pytest.mark.parametrize("H,groups", [(16, [16]), (32, [16, 32]), (64, [16, 32, 64]), (128, [16, 32, 64])])
def test_the_checks_below_reach_every_row_group(H, groups):
    q, cache, bt, _ = make_dense([300], H, seed=1)
    assert sorted(_every_row_group(q, cache, bt)) == groups


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 256, 1000, 4097])
def test_lengths(n):
    _check(*make_dense([n], 16, seed=n))


@pytest.mark.parametrize("H", [1, 5, 8, 16, 17, 24, 32, 33, 40, 64, 65, 100, 128])
def test_head_counts(H):
    _check(*make_dense([300, 77], H, seed=H))


@pytest.mark.parametrize("H,s_q", [(16, 2), (16, 3), (64, 2), (128, 2), (8, 5), (24, 3), (5, 13), (64, 1)])
def test_queries_of_a_request_have_their_own_lengths(H, s_q):
    base = [500, 64, 130]
    lens = [max(0, n - (s_q - 1 - j)) for n in base for j in range(s_q)]
    _check(*make_dense(lens, H, s_q, seed=H + s_q))


def test_lengths_of_one_request_in_any_order():
    _check(*make_dense([5, 700, 0, 129, 1, 300], 40, 3, seed=8))


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 31, 200, 1024])
def test_any_number_of_ctas(ctas):
    _check(*make_dense([0, 900, 1, 64, 2000, 0, 128, 257], 64, seed=ctas), ctas=ctas)


def test_ragged_batch_with_empty_requests():
    g = np.random.default_rng(5)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(1500), 60))] + [0, 0, 0]
    _check(*make_dense(lens, 16, seed=6))


@pytest.mark.parametrize("R", [31, 32, 33, 127, 128, 129, 200])
def test_request_counts(R):
    g = np.random.default_rng(R)
    lens = [0 if i % 9 == 4 else int(x) for i, x in enumerate(np.exp(g.uniform(0, np.log(700), R)))]
    _check(*make_dense(lens, 16, seed=R))


def test_largest_batch():
    # 65535 queries of one position each: the output is that position's value, lse its score
    B, g = 65535, torch.Generator().manual_seed(40)
    cache = wl.fill_kv_cache(64, g, "cpu").to(DEV)
    bt = torch.randint(0, 64, (B, 1), generator=g).to(torch.int32).to(DEV)
    q = torch.randn((B, 1, 576), generator=g).to(torch.bfloat16).to(DEV)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    ws = api.alloc_dense_workspace(api.dense_dims_of(q, cache, bt), DEV)
    out, lse = api.sparse_mla_dense_decode(q, cache, bt, lens, SCALE, workspace=ws)
    k = api.sparse_mla_kv_read(cache, bt, torch.zeros(B, dtype=torch.int32, device=DEV), dtype=torch.float32).double()
    score = SCALE * (q[:, 0].double() * k).sum(-1)
    size = SCALE * (q[:, 0].double() * k).abs().sum(-1)
    # q's terms are exact but for 2^-17 of the largest element, the rest are float32 sums
    err = 2.0 ** -17 * SCALE * q[:, 0].abs().amax(-1).double() * k.abs().sum(-1) + 2.0 ** -18 * size + 2.0 ** -20
    assert bool(((lse[:, 0].double() - score).abs() <= err).all())
    # a weight's two terms: 2^-8 of the value with its own rounding, and one of the output
    assert bool(((out[:, 0].double() - k[:, :512]).abs() <= 2.0 ** -7 * k[:, :512].abs() + 1e-30).all())
    assert api.read_errors(ws) == 0


def test_many_short_requests():
    lens = [i % 4 for i in range(3000)]
    _check(*make_dense(lens, 2, seed=7))


def test_result_does_not_depend_on_timing_or_earlier_calls():
    q, cache, bt, lens = make_dense([1500, 3, 800, 640], 64, seed=9)
    d = [t.to(DEV) for t in (q, cache, bt, lens)]
    ws = api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2]), DEV)
    first = [t.clone() for t in api.sparse_mla_dense_decode(*d, SCALE, workspace=ws)]
    for _ in range(5):
        again = api.sparse_mla_dense_decode(*d, SCALE, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_an_attention_sink_keeps_the_rest():
    # one position outweighs every other by about e^14 while 3000 others share what is left
    q, cache, bt, lens = make_dense([3000], 16, seed=10)
    q[:] = 0
    q[:, :, 512] = 1.0                                         # scores: the first rope value
    rope = cache[..., 528:530]
    rope[:] = torch.tensor([0.0], dtype=torch.bfloat16).view(torch.uint8)
    cache[int(bt[0, 3]), 17, 528:530] = torch.tensor([14.0], dtype=torch.bfloat16).view(torch.uint8)
    cache[int(bt[0, 3]), 17, :512] = 0                         # the sink's own value is zero
    _check(q, cache, bt, lens, 1.0)


def test_rising_scores_move_the_reference():
    # scores grow by 4 per page: the running reference of every row has to move again and again
    q, cache, bt, lens = make_dense([1400], 24, seed=11)
    q[:] = 0
    q[:, :, 512] = torch.linspace(0.5, 2.0, 24).to(torch.bfloat16)[None]
    for i in range(bt.shape[1]):
        v = torch.tensor([4.0 * i - 30], dtype=torch.bfloat16).view(torch.uint8)
        cache[int(bt[0, i]), :, 528:530] = v
    _check(q, cache, bt, lens, 1.0)


@pytest.mark.parametrize("steps", ["rise", "fall", "both"])
def test_scores_that_jump_from_page_to_page(steps):
    # whole pages 50 (in units of e) above or below the one before, in rows of every magnitude: accumulators in
    # registers and in TMEM are scaled back by far more than a tile's own range, or keep what a later tile adds to
    q, cache, bt, lens = make_dense([1300, 257], 64, seed=30)
    q[:] = 0
    q[:, :, 512] = torch.linspace(0.02, 1.0, 64).to(torch.bfloat16)[None]
    for r in range(bt.shape[0]):
        for i in range(bt.shape[1]):
            if bt[r, i] < 0:
                continue
            h = 50.0 * {"rise": i, "fall": -i, "both": (i * 7) % 5 - 2}[steps]
            cache[int(bt[r, i]), :, 528:530] = torch.tensor([h], dtype=torch.bfloat16).view(torch.uint8)
    _check(q, cache, bt, lens, 1.0)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_score_scales(scale):
    _check(*make_dense([321, 50], 16, seed=12), scale=scale)


def test_query_magnitudes():
    q, cache, bt, lens = make_dense([400], 16, seed=13)
    gain = torch.logspace(-12, 1, 16).view(1, 16, 1)
    q = (q.float() * gain).to(torch.bfloat16)
    q[0, 3] = 0
    q[0, 5, 7] = 90.0                                          # outliers in a block
    q[0, 6, 300] = -2000.0 * 2 ** -9
    _check(q, cache, bt, lens)


@pytest.mark.parametrize("mag", [1e-4, 1e-2, 60.0])
def test_latent_magnitudes(mag):
    # scales from far below fp16's normal range up
    q, cache, bt, lens = make_dense([200], 16, seed=14, poison=False)
    sc = cache[..., 512:528].contiguous().view(torch.float32) * mag
    cache[..., 512:528] = sc.view(torch.uint8)
    q = (q.float() / max(mag, 1.0)).to(torch.bfloat16)
    _check(q, cache, bt, lens)


def test_nan_query_and_nan_position_stay_in_their_rows():
    q, cache, bt, lens = make_dense([200, 150], 16, seed=15)
    q[0, 3, 40] = float("nan")
    q[0, 4, 530] = float("nan")
    q[0, 5, 100] = float("inf")
    out, lse, _ = _run(q, cache, bt, lens)
    bad = torch.zeros(2, 16, dtype=torch.bool)
    bad[0, 3:6] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), bad) and torch.equal(torch.isnan(out).any(-1).cpu(), bad)
    # a NaN code inside request 1's context reaches that request's rows and no others
    q, cache, bt, lens = make_dense([200, 150], 16, seed=15)
    cache[int(bt[1, 0]), 9, 100] = 0x7F
    out, lse, _ = _run(q, cache, bt, lens)
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()
    assert torch.isfinite(lse[0]).all() and torch.isfinite(out[0].float()).all()


def test_a_later_query_sees_a_nan_that_an_earlier_one_does_not():
    q, cache, bt, lens = make_dense([140, 141], 16, 2, seed=16)
    cache[int(bt[0, 2]), 140 - 128, 5] = 0x7F                   # position 140: query 1 alone reads it
    out, lse, _ = _run(q, cache, bt, lens)
    assert torch.isfinite(lse[0]).all() and torch.isfinite(out[0].float()).all()
    assert torch.isnan(lse[1]).all()


def test_nan_positions_in_every_row_group():
    q, cache, bt, lens = make_dense([260, 259, 130, 127], 64, 2, seed=31)
    cache[int(bt[0, 4]), 3, 300] = 0x7F                         # position 259: query 0 alone reads it
    cache[int(bt[1, 1]), 64 - 1, 512 + 4:512 + 8] = torch.tensor([float("nan")]).view(torch.uint8)   # 127: query 2 alone
    for wide in _every_row_group(q, cache, bt).values():
        out, lse, err = _run(q, cache, wide, lens)
        assert err == 0
        bad = torch.tensor([True, False, True, False])
        assert torch.equal(torch.isnan(lse).all(1).cpu(), bad) and torch.equal(torch.isnan(lse).any(1).cpu(), bad)
        assert torch.equal(torch.isnan(out.float()).all(2).all(1).cpu(), bad)
        assert torch.equal(torch.isnan(out.float()).any(2).any(1).cpu(), bad)


def test_a_wait_that_runs_out_is_reported_and_recoverable():
    q, cache, bt, lens = make_dense([1300, 257, 5], 64, seed=32)
    for wide in _every_row_group(q, cache, bt).values():
        d = [t.to(DEV) for t in (q, cache, wide, lens)]
        ws = api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2]), DEV)
        out = torch.full((3, 64, 512), 3.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((3, 64), 3.0, device=DEV)
        try:
            api.debug_set_wait_limit(1)                        # no wait of this call is issued anything to wait for
            api.sparse_mla_dense_decode(*d, SCALE, out=out, lse=lse, workspace=ws)
            torch.cuda.synchronize()
        finally:
            api.debug_set_wait_limit(0)
        assert api.read_errors(ws) & _native.DEVERR_TIMEOUT
        assert torch.all(out[2] == 3.0) and torch.all(lse[2] == 3.0)      # a request of one tile: unwritten
        api.clear_errors(ws)
        api.sparse_mla_dense_decode(*d, SCALE, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert api.read_errors(ws) == 0
        check_dense(out, lse, q, cache, bt, lens, SCALE)


def test_bad_pages_are_skipped_and_flagged():
    q, cache, bt, lens = make_dense([500, 300], 16, seed=17)
    bt[0, 2] = cache.shape[0] + 5
    bt[1, 1] = -7
    _check(q, cache, bt, lens, flags=_native.DEVERR_PAGE_RANGE)
    q, cache, bt, lens = make_dense([500, 300], 16, seed=17)
    bt[:] = -1                                                  # no page at all: empty rows
    _check(q, cache, bt, lens, flags=_native.DEVERR_PAGE_RANGE)


def test_lengths_outside_the_table():
    q, cache, bt, lens = make_dense([256, 100], 16, seed=18, poison=False)
    lens[0] = 256 + 200                                         # past the table's four pages: skipped and flagged
    lens[1] = -5                                                # counts as 0
    _check(q, cache, bt, lens, flags=_native.DEVERR_PAGE_RANGE)


def test_latents_beyond_fp16():
    # one position far beyond fp16's range beside ordinary ones, and scales that differ by 2^40 within one
    q, cache, bt, lens = make_dense([100], 16, seed=19, poison=False)
    cache[int(bt[0, 0]), 3, 512:516] = torch.tensor([1000.0]).view(torch.uint8)        # up to 448 * 1000
    cache[int(bt[0, 0]), 5, 512:528] = torch.tensor([1e-9, 1e3, 1e-3, 0.0]).view(torch.uint8)
    _check(torch.zeros_like(q), cache, bt, lens)
    q[:] = 0
    q[:, :, 560] = 2.0
    _check(q, cache, bt, lens)


def test_cache_beyond_4_gib():
    # pages past the 32-bit byte offsets; only the pages in use are filled
    total = 110000                                              # 4.6 GB
    q, cache, bt, lens = make_dense([700, 200], 64, seed=20, spare_pages=0)
    big = torch.empty((total, 64, 656), dtype=torch.uint8, device=DEV)
    where = torch.randperm(40000, generator=torch.Generator().manual_seed(1))[:cache.shape[0]] + total - 40000
    big[where.to(DEV)] = cache.to(DEV)
    btb = torch.where(bt >= 0, where[bt.clamp_min(0).long()].to(torch.int32), bt)
    for wide in _every_row_group(q, cache, btb).values():
        out, lse = api.sparse_mla_dense_decode(q.to(DEV), big, wide.to(DEV), lens.to(DEV), SCALE)
        torch.cuda.synchronize()
        check_dense(out, lse, q, cache, bt, lens, SCALE)


@pytest.mark.parametrize("H,rows", [(32, 16), (32, 32), (64, 32), (64, 64)])
def test_captured_call_follows_new_lengths(H, rows):
    q, cache, bt, lens = make_dense([900, 500, 64], H, seed=21, poison=False)
    d = [t.to(DEV) for t in (q, cache, _every_row_group(q, cache, bt)[rows], lens)]
    ws = api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2]), DEV)
    out, lse = api.sparse_mla_dense_decode(*d, SCALE, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.sparse_mla_dense_decode(*d, SCALE, out=out, lse=lse, workspace=ws)
    for new in ([900, 500, 64], [3, 0, 60], [128, 129, 1], [870, 499, 33]):
        lens = torch.tensor(new, dtype=torch.int32)
        d[3].copy_(lens)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_dense(out, lse, q, cache, bt, lens, SCALE)


def test_two_streams_with_a_workspace_each():
    a = make_dense([1200, 700], 64, seed=22)
    b = make_dense([100, 2000, 50], 16, seed=23)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [[t.to(DEV) for t in x] for x in (a, b)]
    ws = [api.alloc_dense_workspace(api.dense_dims_of(d[0], d[1], d[2]), DEV) for d in dev]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for d, w, s in zip(dev, ws, streams):
            got.append(api.sparse_mla_dense_decode(*d, SCALE, workspace=w, stream=s))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        x = (a, b)[i % 2]
        if i >= 6:
            check_dense(out, lse, *x, SCALE)
        else:
            assert torch.equal(out, got[6 + i % 2][0]) and torch.equal(lse, got[6 + i % 2][1])


def test_agrees_with_the_sparse_decode_over_every_position():
    w = wl.make_custom(B=3, H=64, topk=512, ctx_lens=[512, 200, 64], seed=24, device=DEV)
    w.topk_idx = torch.arange(512, dtype=torch.int32, device=DEV).repeat(3, 1)
    so, sl = api.sparse_mla_decode(w.q, w.kv_cache, w.block_table, w.topk_idx, w.seq_lens, w.sm_scale)
    do, dl = api.sparse_mla_dense_decode(w.q, w.kv_cache, w.block_table, w.seq_lens, w.sm_scale)
    torch.cuda.synchronize()
    check_dense(do, dl, w.q.cpu(), w.kv_cache.cpu(), w.block_table.cpu(), w.seq_lens.cpu(), w.sm_scale)
    assert (sl - dl).abs().max() < 1e-3                         # the sparse decode's own tolerance


def test_python_refusals():
    q, cache, bt, lens = [t.to(DEV) for t in make_dense([70, 10], 16, seed=25)]
    with pytest.raises(TypeError):
        api.sparse_mla_dense_decode(q.float(), cache, bt, lens, SCALE)
    with pytest.raises(ValueError):
        api.sparse_mla_dense_decode(q.transpose(0, 1), cache, bt, lens, SCALE)
    with pytest.raises(ValueError):
        api.sparse_mla_dense_decode(q, cache, bt, lens[:1], SCALE)
    with pytest.raises(ValueError):
        api.sparse_mla_dense_decode(q, cache.cpu(), bt, lens, SCALE)
    with pytest.raises(ValueError):
        api.sparse_mla_dense_decode(q, cache, bt, lens, SCALE, out=torch.empty((2, 16, 576), dtype=q.dtype, device=DEV))
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_dense_decode(q, cache, bt, lens, SCALE, workspace=torch.zeros(128, dtype=torch.uint8, device=DEV))
    with pytest.raises(_native.SmlaError):
        api.sparse_mla_dense_decode(torch.zeros((2, 129, 576), dtype=q.dtype, device=DEV), cache, bt, lens, SCALE)
