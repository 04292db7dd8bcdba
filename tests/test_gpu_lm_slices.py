"""Projections of 8-bit rows and weights that are column slices of wider
matrices, whose other columns hold anything: against exact integer sums."""
import pytest
import torch

import recurrent_nn_amd as ra
from tests.test_gpu_lm import Draw, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# every kernel form: few rows, few rows beside 64 MiB of weights, columns among the
# waves, and the tiles from 64 x 64 to 256 x 256
FORMS = [(1, 40), (3, 500), (16, 130), (17, 70), (130, 200), (900, 1500), (500, 3970), (1700, 1900),
         (1700, 3900), (3500, 3600)]


def sums(q, w):
    """q w^T, exact: in 64 bits."""
    return (q.double() @ w.double().t().contiguous()).float()


@pytest.mark.parametrize("cols", [1, 15, 17, 60, 63, 100, 127, 249, 255, 500])
@pytest.mark.parametrize("rows,outs", FORMS)
def test_columns_past_the_last_do_not_count(rows, outs, cols):
    r = Draw(rows + 3 * outs + 7 * cols)
    x, w = (torch.randint(-128, 128, (n, 512), generator=r.g, dtype=torch.int8).cuda()
            for n in (rows, outs))
    x[:, cols:] |= 1                        # nothing past the slice is zero
    w[:, cols:] |= 1
    one = torch.ones(max(rows, outs)).cuda()
    got = ra.quant_project(x[:, :cols], w[:, :cols], one[:outs], x_scale=one[:rows])
    assert torch.equal(got, sums(x[:, :cols], w[:, :cols]))


def test_columns_past_the_last_of_few_rows_and_many_weights():
    r = Draw(5)
    x, w = (torch.randint(-128, 128, (n, 4112), generator=r.g, dtype=torch.int8).cuda() | 1
            for n in (3, 16400))
    one = torch.ones(16400).cuda()
    for cols in (4099, 4111, 4095):
        got = ra.quant_project(x[:, :cols], w[:, :cols], one, x_scale=one[:3])
        assert torch.equal(got, sums(x[:, :cols], w[:, :cols]))


@pytest.mark.parametrize("lo,hi", [(1024, 2048), (0, 1024), (1936, 2048), (2032, 2041), (16, 1999)])
@pytest.mark.parametrize("rows", [2, 40])
def test_column_slices_of_weights_are_taken(rows, lo, hi):
    r = Draw(rows + lo)
    x = r.normal(rows, hi - lo).cuda()
    w = torch.randint(-128, 128, (64, 2048), generator=r.g, dtype=torch.int8).cuda()
    ws = r.uniform(64, lo=0.5, hi=1.5).cuda()
    dense = torch.zeros(64, 2048, dtype=torch.int8, device="cuda")[:, :hi - lo]
    dense.copy_(w[:, lo:hi])
    want = ra.quant_project(x, dense, ws)
    q = ra.quantize_rows(x)
    wide = torch.ones(rows, 2048, dtype=torch.int8, device="cuda")
    wide[:, lo:hi] = q.q
    for stream in (None, torch.cuda.current_stream()):      # the compiled call, and the other way
        assert torch.equal(ra.quant_project(x, w[:, lo:hi], ws, stream=stream), want)
        assert torch.equal(ra.quant_project(wide[:, lo:hi], w[:, lo:hi], ws, x_scale=q.scale,
                                            stream=stream), want)


def test_rows_that_end_inside_a_piece_of_16_bytes_are_refused():
    x, ws = torch.zeros(2, 8).cuda(), torch.ones(4).cuda()
    w = torch.zeros(4 * 16 - 8, dtype=torch.int8).cuda().as_strided((4, 8), (16, 1))
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(ValueError, match="w: its last row"):
            ra.quant_project(x, w, ws, stream=stream)
