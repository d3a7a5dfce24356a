"""A mask that hides nothing: outputs as well as lse, against the oracle and the dense decode."""
import pytest
import torch

import test_masked_decode as masked
from cache_util import DEV, bits, make_dense
from masked_util import check_decode
from oracle import masked_oracle
from sparse_mla_decode_paged_gb300 import api

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


@pytest.mark.parametrize("H", [16, 40, 64, 128])
@pytest.mark.parametrize("starts,prefix", [([0, 0, 0], None), ([700, 64, 0], [700, 64, 0]), ([-3, -3, -3], [5, 5, 5])])
def test_outputs(H, starts, prefix):
    q, cache, bt, ln = make_dense([700, 64, 0], H, seed=H)
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32)
    out, lse, err = masked._run(q, cache, bt, ln, starts=i32(starts), prefix=i32(prefix))
    assert err == 0
    want = masked_oracle.masked_decode(bits(q).reshape(q.shape), cache.numpy(), bt.numpy(), ln.numpy(), SCALE)
    check_decode(out, lse, want)
    check_decode(*api.sparse_mla_dense_decode(*[t.to(DEV) for t in (q, cache, bt, ln)], SCALE), want)
