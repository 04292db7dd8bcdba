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
