"""GPU: outputs of the state space scan in bf16 carry their own rounding and no
other (tolerances in ssm_checks.py; short sequences, where a term's own rounding
is not lost in the sum of the others)."""
import pytest
import torch

from ssm_checks import check_backward, check_forward
from test_gpu_ssm_scan import BF, F, backward, forward, make

pytestmark = pytest.mark.gpu

CASES = [
    # B, T, H, G, n, p, gate, cu, state
    (2, 1, 2, 1, 64, 64, BF, None, True),
    (1, 5, 4, 2, 128, 64, F, [0, 2, 2, 5], True),
    (3, 3, 2, 1, 64, 128, BF, None, False),
    (1, 20, 4, 1, 128, 128, F, [0, 7, 20], True),
    (1, 130, 2, 2, 128, 128, BF, None, True),
    (1, 1100, 2, 1, 128, 64, F, [0, 1000, 1000, 1100], True),   # in spans
]


@pytest.mark.parametrize("B,T,H,G,n,p,gate,cu,state", CASES)
def test_one_rounding(B, T, H, G, n, p, gate, cu, state):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(31, B, T, H, G, n, p, BF, gate, cu, state)
    check_forward(forward(gdr, d), c, cu, BF)
    check_backward(backward(gdr, d), c, cu, BF, gate)
