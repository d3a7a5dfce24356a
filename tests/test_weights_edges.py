"""Attention weights from an lse of no positions, and of lengths that no column holds."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bits, make_dense
from oracle import cache_weights_oracle as ref
from sparse_mla_decode_paged_gb300 import _native, api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


@pytest.mark.parametrize("H", [16, 32, 64, 128, 100])
@pytest.mark.parametrize("decay", [0.0, 0.9])
def test_a_row_that_saw_nothing_adds_nothing(H, decay):
    """A window that leaves the last query of a request nothing: its lse is -inf."""
    q, cache, bt, ln = make_dense([300, 301, 500, 500], H, 2, seed=H)
    d = [t.to(DEV) for t in (q, cache, bt, ln)]
    starts = torch.tensor([0, 301, 500, 0], dtype=torch.int32, device=DEV)
    _, lse = api.sparse_mla_masked_decode(*d, SCALE, starts=starts)
    gone = torch.isneginf(lse).all(1).cpu()
    assert gone.tolist() == [False, True, True, False]
    w = torch.rand((2, 510), generator=torch.Generator().manual_seed(H))
    got = api.sparse_mla_attention_weights(*d, lse, SCALE, w.to(DEV), decay=decay)
    # what the rows that saw something add; the decay reaches as far as the longest length of all
    host = lse.cpu()
    host[gone] = 0.0
    want, tol = ref.attention_weights(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), torch.where(gone, 0, ln).numpy(),
                                      host.numpy(), SCALE, w.numpy(), decay)
    assert int(ln[1]) == 301
    if decay != 0:
        want[0, 300], tol[0, 300] = decay * np.float64(w[0, 300]), 2.0 ** -23 * w[0, 300]
    else:
        want[0, 300] = tol[0, 300] = 0
    off = np.abs(got.cpu().double().numpy() - want)
    assert np.all(off <= tol), f"error {(off / np.maximum(tol, 1e-300)).max():.2f} of its bound"


@pytest.mark.parametrize("lens,flags", [([5, 0], _native.DEVERR_LEN_RANGE), ([0, 1], _native.DEVERR_LEN_RANGE), ([0, -3], 0)])
def test_no_columns(lens, flags):
    q, cache, bt, ln = make_dense([64, 64], 16, seed=1)
    ln = torch.tensor(lens, dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.zeros((2, 0), device=DEV)
    api.sparse_mla_attention_weights(q.to(DEV), cache.to(DEV), bt.to(DEV), ln.to(DEV), torch.zeros((2, 16), device=DEV), SCALE, w,
                                     err_word=err)
    torch.cuda.synchronize()
    assert int(err) == flags


def test_no_columns_of_many_requests():
    lens = [0] * 3000
    lens[2999] = 7
    q, cache, bt, ln = make_dense([1] * 3000, 1, seed=2)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.sparse_mla_attention_weights(q.to(DEV), cache.to(DEV), bt.to(DEV), ln, torch.zeros((3000, 1), device=DEV), SCALE,
                                     torch.zeros((3000, 0), device=DEV), err_word=err)
    torch.cuda.synchronize()
    assert int(err) == _native.DEVERR_LEN_RANGE
