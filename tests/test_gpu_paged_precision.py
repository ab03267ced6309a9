"""GPU: one token over the bf16 cache keeps its probabilities to 2^-15 and rounds
its output alone.

Tolerance: that of fp32 (attn_ref.py), 2^-15 of sum p |v| for the probabilities,
which stand in two bf16 parts (the first is cut, which leaves 2^-7 of p at most,
the second holds what is left, rounded by 2^-8 of itself), and half a step, 2^-8,
of the output."""
import pytest
import torch

import attn_ref as ref
from mixer_ref import check
from test_gpu_paged import BF, F, ints, pages_of, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,page,hq,hk,d,window", [
    ([1, 2, 3, 40], 16, 2, 1, 64, 0),
    ([700, 129, 64], 24, 8, 2, 128, 0),
    ([900, 33], 16, 33, 1, 128, 100),
    ([9000], 100, 4, 1, 64, 0),                 # chunks that are joined
])
def test_probabilities_are_not_rounded_to_bf16(lens, page, hq, hk, d, window):
    import chunked_gated_delta_fwd_amd as gdr
    kp, vp, table = pages_of(lens, page, hk, d, BF)
    q = queries(len(lens), hq, d, BF)
    o = gdr.attn_paged_step(q.cuda(), kp.cuda(), vp.cuda(), ints(table), ints(lens), window=window)
    args = table, lens, window
    want, tol = ref.paged(q.double(), kp.double(), vp.double(), *args, dtype=torch.float32)
    size, _ = ref.paged(q.double(), kp.double(), vp.double().abs(), *args, dtype=torch.float32)
    check("o", o, want, tol + 2.0 ** -15 * size + 2.0 ** -8 * want.abs())


@pytest.mark.parametrize("lens", [[1, 2], [40, 300], [9000, 5]])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_value_stays_one(lens, dtype, value):
    """Where its probability is above zero (a single key's is 1): the second part of a probability is none of 0 times it."""
    import chunked_gated_delta_fwd_amd as gdr
    kp, vp, table = pages_of(lens, 16, 2, 64, dtype)
    q = queries(2, 4, 64, dtype)
    want = gdr.attn_paged_step(q.cuda(), kp.cuda(), vp.cuda(), ints(table), ints(lens))
    vp[table[0][0], 0, 1, 9] = value               # key 0 of sequence 0, head 1
    q[0] /= 16                                     # every probability above e^-20
    few = gdr.attn_paged_step(q.cuda(), kp.cuda(), vp.cuda(), ints(table), ints(lens))
    assert (few[0, 2:, 9] == value).all()
    few[0, 2:, 9] = 0
    assert torch.isfinite(few).all() and torch.equal(few[1], want[1])
