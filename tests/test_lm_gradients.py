"""The language-model operators go forward only: while gradients are recorded
a tensor that requires one is refused, so that none is lost without a word."""
import pytest
import torch

import recurrent_nn_amd as ra
from recurrent_nn_amd import lm


def every_input(device):
    """(call, its float inputs by name) of each operator."""
    def new(*shape):
        return torch.full(shape, 0.25, device=device)
    lens = torch.tensor([3, 2], dtype=torch.int32, device=device)
    w = torch.ones(4, 16, dtype=torch.int8, device=device)
    return {
        "conv": (lambda **t: ra.causal_conv(sequence_lens=lens, **t),
                 dict(x=new(2, 3, 8), weight=new(8, 4), bias=new(8), state=new(2, 3, 8))),
        "scan": (lambda **t: ra.selective_scan(sequence_lens=lens, **t),
                 dict(x=new(2, 3, 8), dt=new(2, 3, 8), A=-new(8, 4), B=new(2, 3, 4), C=new(2, 3, 4),
                      D=new(8), z=new(2, 3, 8), dt_bias=new(8), state=new(2, 8, 4))),
        "quantize": (ra.quantize_rows, dict(x=new(3, 16))),
        "project": (lambda **t: ra.quant_project(w=w, **t), dict(x=new(3, 16), w_scale=new(4), bias=new(4))),
        "scores": (lambda **t: ra.token_scores(top=2, **t), dict(logits=new(3, 16))),
    }


CASES = [(op, name) for op, (_, tensors) in every_input("cpu").items() for name in tensors]


@pytest.mark.parametrize("op,name", CASES)
def test_an_input_that_requires_a_gradient_is_refused(op, name):
    call, tensors = every_input("cpu")[op]
    tensors[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        call(**tensors)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):        # its place is the next thing
        call(**tensors)


def test_the_compiled_calls_leave_it_to_python():
    from torch._subclasses.fake_tensor import FakeTensorMode
    compiled = lm._bind()
    with FakeTensorMode():
        x = torch.empty(3, 16, device="cuda", requires_grad=True)
        assert compiled.quantize(x, 0, 0) is None
        assert compiled.scores(x, None, 2, 0, 0) is None


@pytest.mark.gpu
@pytest.mark.parametrize("op,name", CASES)
def test_on_the_device(op, name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    call, tensors = every_input("cuda")[op]
    want = call(**tensors)
    tensors[name].requires_grad_()
    for stream in (None, torch.cuda.current_stream()):      # the compiled call, and the other way
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call(**tensors, stream=stream)
        with torch.no_grad():
            got = call(**tensors, stream=stream)
        for a, b in zip(got, want):
            assert (a is None and b is None) or (torch.equal(a, b) and not a.requires_grad)
