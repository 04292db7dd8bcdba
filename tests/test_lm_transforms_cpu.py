"""The language-model operators under torch's transforms, without a GPU (fake
device tensors): a wrapper has no memory of its own, which is an error to the
caller.  In a process of its own, so that a crash is a failed test."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, warnings
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from recurrent_nn_amd import lm

warnings.simplefilter("ignore")
op, kind = sys.argv[1:]
compiled = lm._bind()
lm._device, lm._raw_stream = (lambda: 0), (lambda index: 0)
none = [None] * 8
with FakeTensorMode(allow_non_fake_inputs=True):
    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    calls = {
        "conv": (new(5, 2, 3, 8), lambda x: (x, new(8, 4), None, False, None, None, new(2, 3, 8),
                                             new(2, 3, 8)), lm.causal_conv),
        "scan": (new(5, 2, 3, 8), lambda x: (x, x, new(8, 4), new(2, 3, 4), new(2, 3, 4), None, None,
                                             None, False, None, None, new(2, 3, 8), new(2, 8, 4)),
                 lm.selective_scan),
        "quantize": (new(5, 3, 16), lambda x: (x,), lm.quantize_rows),
        "project": (new(5, 3, 16), lambda x: (x, new(4, 16, dtype=torch.int8), new(4), None, None, None,
                                              new(3, 4)), lm.quant_project),
        "scores": (new(5, 3, 16), lambda x: (x, new(3, dtype=torch.int64), 2), lm.token_scores),
    }
    x, args, public = calls[op]
    seen = []

    def under(v):
        # the compiled call leaves it to Python, which says what is wrong
        seen.append(getattr(compiled, op)(*args(v), 0, 0))
        try:
            public(*args(v))
        except (RuntimeError, ValueError) as e:
            seen.append(e)
        return v

    if kind == "vmap":
        torch.vmap(under)(x)
    elif kind == "vjp":
        torch.func.vjp(under, x[0])
    else:
        torch.func.jvp(under, (x[0],), (x[0],))
assert seen[0] is None and isinstance(seen[1], (RuntimeError, ValueError)), seen
print("said:", seen[1])
"""


@pytest.mark.parametrize("kind", ["vmap", "vjp", "jvp"])
@pytest.mark.parametrize("op", ["conv", "scan", "quantize", "project", "scores"])
def test_a_transform_is_an_error_and_no_crash(op, kind):
    r = subprocess.run([sys.executable, "-c", PROGRAM, op, kind], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0 and "said:" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])
