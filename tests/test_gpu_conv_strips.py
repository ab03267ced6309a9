"""GPU: the convolution's gradient at sizes where a thread walks strips of 16, 32
and 64 tokens (small calls, as in test_gpu_conv.py, take strips of 8), against
the plain fp64 evaluation on the GPU (elementwise).  Tolerances as there: 32 U
(1 + mag) |dy| for each dz, 128 U for the sums over tokens (64 additions in a
strip, 4 strips of a block, an eighth of the blocks' rows and 3)."""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step
from test_gpu_conv import BF, F

pytestmark = pytest.mark.gpu


def strip_of(T, ch, dtype, vec):
    """Tokens of a strip as the launch rule has it: 64, halved while there are fewer than 1024 blocks."""
    pieces = ch // 4 if vec else ch
    lanes = 1
    while lanes < 64 and lanes < pieces:
        lanes *= 2
    strip = 64
    while strip > 8 and -(-T // (256 // lanes * strip)) * -(-pieces // lanes) < 1024:
        strip //= 2
    return strip


@pytest.mark.parametrize("strip,T,ch,W,dtype,bias,silu,vec", [
    (16, 4100, 4096, 4, BF, True, True, True),
    (32, 8197, 4096, 3, BF, False, True, True),
    (64, 8261, 8192, 4, BF, True, True, True),
    (64, 8261, 2051, 4, BF, True, True, False),      # single channels
    (16, 4100, 4096, 2, F, True, True, True),
    (64, 16390, 4096, 4, F, False, False, True),
    (32, 8197, 1027, 4, F, True, True, False),
])
def test_gradient(strip, T, ch, W, dtype, bias, silu, vec):
    import chunked_gated_delta_fwd_amd as gdr
    assert strip_of(T, ch, dtype, vec) == strip
    cu = [0, 1, 1, 3, 130, T // 2 + 5, T - 2, T]
    N = len(cu) - 1
    g = torch.Generator(device="cuda").manual_seed(71)

    def r(*s, k=1.0):
        return (k * torch.randn(s, generator=g, device="cuda")).to(dtype)

    x, w, b, s0 = r(1, T, ch), r(ch, W, k=0.4), r(ch) if bias else None, r(N, W - 1, ch)
    dy, dst = r(1, T, ch), r(N, W - 1, ch)
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = gdr.short_conv_bwd(x, w, dy, b, offsets, s0, dst, activation="silu" if silu else None)

    def grads(leaves, gy, gst, act):
        leaves = [t.requires_grad_() for t in leaves]
        y, st = ref.conv(leaves[0], leaves[1], leaves[3] if bias else None, cu, leaves[2], act)
        return torch.autograd.grad([y, st], leaves, [gy, gst])

    leaves = [t.double() for t in (x, w, s0)] + ([b.double()] if bias else [])
    rx, rw, rs, *rb = grads([t.clone() for t in leaves], dy.double(), dst.double(), silu)
    a = [t.abs() for t in leaves]
    with torch.no_grad():
        mag = ref.conv(a[0], a[1], a[3] if bias else None, cu, a[2], False)[0]
    mx, mw, ms, *mb = grads(a, dy.double().abs() * 1.1 * (1 + mag), dst.double().abs(), False)
    half = half_step(dtype) if dtype == BF else 0
    check("dx", got[0], rx.cpu(), (32 * U * mx + half * rx.abs()).cpu())
    check("dw", got[1], rw.cpu(), ((32 + 128) * U * mw).cpu())
    if bias:
        check("db", got[2], rb[0].cpu(), ((32 + 128) * U * mb[0]).cpu())
    check("ds0", got[3], rs.cpu(), (32 * U * ms + half * rs.abs()).cpu())
