"""The compiled part of the language-model operators' binding, without a GPU:
what is not a plain call is left to Python, and nothing is done."""
import pytest
import torch

import recurrent_nn_amd as ra
from recurrent_nn_amd import _lib, lm


@pytest.fixture(scope="module")
def compiled():
    return lm._bind()


def test_other_tensors_are_left_to_python(compiled):
    x, f = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    none = [None] * 12
    for bad in (x, None, 5, "x"):
        assert compiled.conv(bad, f, None, False, *none[:4], 0, 0) is None
        assert compiled.scan(bad, bad, f, x, x, *none[:3], False, *none[:4], 0, 0) is None
        assert compiled.quantize(bad, 0, 0) is None
        assert compiled.project(bad, f, f, *none[:4], 0, 0) is None
        assert compiled.scores(bad, None, 3, 0, 0) is None


def test_wrong_arguments_are_errors(compiled):
    with pytest.raises(TypeError):
        compiled.conv(None)
    with pytest.raises(TypeError):
        compiled.quantize(None, "device", 0)
    with pytest.raises(TypeError):
        compiled.bind(1, 2)


def test_every_entry_point_is_bound():
    assert set(lm._ENTRIES) == set(_lib.EXPORTED[-8:])


def test_rows_too_long_are_refused():
    run = _lib.load().rnn_quantize_rows
    assert run(0, 1, 1 << 31, 0, 1 << 20, 1 << 31, 1 << 21, 1 << 31, 1 << 20) == ra.RNN_ERR_UNSUPPORTED


def test_a_flag_without_a_truth_value_raises_what_it_says(compiled):
    from torch._subclasses.fake_tensor import FakeTensorMode

    class Neither:
        def __bool__(self):
            raise ArithmeticError("neither")

    with FakeTensorMode():
        def new(*shape):
            return torch.empty(*shape, device="cuda")
        x, B = new(2, 3, 8), new(2, 3, 4)
        with pytest.raises(ArithmeticError, match="neither"):
            compiled.conv(x, new(8, 4), None, Neither(), None, None, new(2, 3, 8), new(2, 3, 8), 0, 0)
        with pytest.raises(ArithmeticError, match="neither"):
            compiled.scan(x, x, new(8, 4), B, B, None, None, None, Neither(), None, None, new(2, 3, 8),
                          new(2, 8, 4), 0, 0)
    f = torch.zeros(2, 3, 8)
    with pytest.raises(ArithmeticError, match="neither"):
        ra.causal_conv(f, torch.zeros(8, 4), silu=Neither())
