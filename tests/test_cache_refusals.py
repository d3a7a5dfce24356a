"""Refusals of the Python entry points that need no GPU: arguments of the wrong kind are named, views of equal layout are
accepted in place."""
import pytest
import torch

from sparse_mla_decode_paged_gb300 import api


@pytest.fixture
def on_cpu(monkeypatch):
    """Checks that look at the device are answered as if the tensors were on the GPU."""
    monkeypatch.setattr(api, "_need_rows", lambda t, name, cols: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))


@pytest.mark.parametrize("weight", [None, [1.0] * 512, 1.0])
def test_a_norm_weight_that_is_no_tensor_is_named(on_cpu, weight):
    bf = torch.zeros((2, 576), dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="norm_weight"):
        api._norm_append_dims(bf[:, :512], bf[:, 512:], weight, torch.zeros((4, 64)), torch.zeros((2, 1), dtype=torch.int32),
                              i32, torch.zeros((2, 64, 656), dtype=torch.uint8), None, True, None)


def test_a_head_weight_that_is_no_tensor_is_named(on_cpu):
    with pytest.raises(TypeError, match="weight"):
        api._norm_rope_dims(torch.zeros((2, 3, 64)), None, None, [1.0] * 64, True, 0, True, None, None)


def _apart(x, out):
    return api._apart(x, out, api._span_bytes(x), api._span_bytes(out))


def test_strides_of_dims_of_size_one_do_not_tell_layouts_apart():
    x = torch.zeros((6, 1, 64))[:5]
    assert _apart(x, x.as_strided((5, 1, 64), (64, 7, 1)))                  # one head: x itself
    assert _apart(x[:1], x.as_strided((1, 1, 64), (999, 7, 1)))             # one row
    y = torch.zeros((4, 1, 200))
    assert _apart(y[..., :64], y.as_strided((4, 1, 64), (200, 3, 1), 64))   # other columns of the rows
    assert not _apart(y[..., :64], y.as_strided((4, 1, 64), (200, 3, 1), 63))
    assert not _apart(x, x.as_strided((5, 1, 64), (65, 64, 1))) and not _apart(x[:1], x.as_strided((1, 1, 64), (64, 64, 1), 1))


def test_overlapping_layouts_stay_refused():
    x = torch.zeros((4, 3, 128))
    assert _apart(x, x) and _apart(x[..., :64], x[..., 64:]) and _apart(x[:2], x[2:])
    assert not _apart(x[..., :64], x[..., 32:96]) and not _apart(x[:3], x[1:])
    assert not _apart(x, x.as_strided((4, 3, 128), (128, 512, 1)))          # its heads outermost
