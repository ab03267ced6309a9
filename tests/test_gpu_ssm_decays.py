"""GPU: the state space scan's forward and gradient at decays that vanish within
a token, hold everything, or lie between, against the literal fp64 recurrence
(tolerances in ssm_checks.py): without a decay everything cancels against what
the chunks carry on, at steep ones all but the diagonal is zero."""
import pytest
import torch

from ssm_checks import check_backward, check_forward
from test_gpu_ssm_scan import BF, F, backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [330, 1100])   # walked whole, and in spans
@pytest.mark.parametrize("A", [0.0, -1e-4, -50.0, -3000.0])
def test_decays(A, T, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(81, 1, T, 2, 1, 64, 64, dtype, F)
    for t in (d, c):
        t["A"].fill_(A)
    c["A"] = d["A"].cpu().double()
    check_forward(forward(gdr, d), c, None, dtype)
    check_backward(backward(gdr, d), c, None, dtype, F)


@pytest.mark.parametrize("dtype", [BF, F])
def test_steps_that_write_nothing(dtype):
    """Tokens whose raw step is the lowest value of fp32, or -inf, pass the state on as it is."""
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(82, 1, 200, 2, 1, 64, 64, dtype, F, [0, 40, 200])
    for at, v in ((slice(0, 40), torch.finfo(F).min), (slice(70, 140), -float("inf"))):
        for t in (d, c):
            t["dt"][:, at] = v
    check_forward(forward(gdr, d), c, [0, 40, 200], dtype)
    got = backward(gdr, d)
    low = c["dt"] < -1e30
    c["dt"][low] = -1e4   # as good as -inf: a step of zero; the reference's own derivative there would be 0 times inf
    check_backward(got, c, [0, 40, 200], dtype, F)
    assert (got[1][low.cuda()] == 0).all()
