"""GPU: the state space scan where it is cut into spans of several chunks, at
every n and p, in both types, packed and as rows, with ragged last spans and
chunks, against the literal fp64 recurrence (tolerances in ssm_checks.py; the
reference runs on the GPU in fp64, elementwise); and states that are stored past
the caches."""
import pytest
import torch

from mixer_ref import U
from ssm_checks import NAMES, check_backward, check_forward
from test_gpu_ssm_scan import BF, F, backward, forward, make

pytestmark = pytest.mark.gpu


def span_len(T, B, heads, cu, dtype, bwd):
    """Tokens of a span as the launch rule has it, 0 where sequences are walked whole: 512 walks forward, 256
    backward, twice as many packed; whole when none is longer than some (of packed ones, whose lengths the host does
    not know, the longest is taken for four times the average, and a third of the tokens at least)."""
    total = B * T
    length = max(64, (total * heads // ((256 if bwd else 512) * (2 if cu else 1)) + 63) // 64 * 64)
    longest = T if cu is None else max(min(total, 4 * total // (len(cu) - 1)), total // 3)
    few = (768 if dtype == BF else 448) if bwd else (512 if dtype == BF else 192)
    whole = (4 if cu and not bwd else 2) * length
    known = T if cu is None else max(b - a for a, b in zip(cu, cu[1:]))
    return 0 if longest <= few or (total if cu else longest) <= whole or known <= whole else length


# packed: one long sequence that ends inside a chunk, one in one span, single tokens and empty ones
def packed(T):
    return [0, 0, 1, T - 700, T - 700, T - 637, T - 636, T]


FORWARD = [
    # B, T, H, G, packed
    (1, 1133, 32, 4, False),
    (2, 1029, 24, 24, False),
    (1, 2309, 32, 2, True),
]
BACKWARD = [
    (1, 1133, 16, 4, False),
    (2, 1029, 12, 1, False),
    (1, 1501, 32, 2, True),
]
SHAPES = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,p", SHAPES)
@pytest.mark.parametrize("B,T,H,G,pack", FORWARD)
def test_forward(B, T, H, G, pack, n, p, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    cu = packed(T) if pack else None
    assert span_len(T, B, H, cu, dtype, False) >= 128
    d, c = make(61, B, T, H, G, n, p, dtype, F, cu, wide=pack)
    check_forward(forward(gdr, d), c, cu, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,p", SHAPES)
@pytest.mark.parametrize("B,T,H,G,pack", BACKWARD)
def test_backward(B, T, H, G, pack, n, p, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    cu = packed(T) if pack else None
    assert span_len(T, B, H, cu, dtype, True) >= 128
    d, c = make(62, B, T, H, G, n, p, dtype, dtype, cu, wide=pack)
    got = backward(gdr, d)
    check_backward(got, c, cu, dtype, dtype)
    again = backward(gdr, d)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [BF, F])
def test_large_states(dtype):
    """A gradient whose chunk states go past the caches, against calls on a quarter of the heads each, whose states
    do not.  Spans may be cut elsewhere: twice the 512 U of the terms' sizes, which are some 15 times the largest
    result, and for bf16 outputs a half step on either side."""
    import chunked_gated_delta_fwd_amd as gdr
    T, H = 4160, 32
    cu = [0, 3000, T]
    d, _ = make(63, 1, T, H, H, 128, 128, dtype, F, cu)
    assert (T // 64) * H * 128 * 128 * 4 >= 1 << 27
    whole = dict(zip(NAMES, backward(gdr, d)))
    for q in range(4):
        s = slice(8 * q, 8 * q + 8)
        assert (T // 64 + 2) * 8 * 128 * 128 * 4 < 1 << 27
        one = dict(d)
        for k in ("x", "b", "c", "dy"):
            one[k] = d[k][:, :, s].contiguous()
        one["dt"] = d["dt"][..., s].contiguous()
        for k in ("A", "D", "dt_bias"):
            one[k] = d[k][s]
        for k in ("h0", "dht"):
            one[k] = d[k][:, s].contiguous()
        part = dict(zip(NAMES, backward(gdr, one)))
        for name in NAMES:
            w = whole[name]
            w = w[:, :, s] if name in ("dx", "db", "dc") else w[..., s] if name == "ddt" else w[:, s] if name == "dh0" else w[s]
            w, g = w.double(), part[name].double()
            half = 2 * 2.0 ** -8 if dtype == BF and name in ("dx", "db", "dc") else 0
            room = 512 * U * 30 * g.abs().max() + half * torch.maximum(w.abs(), g.abs())
            assert bool(((w - g).abs() <= room).all()), (name, q)
