"""GPU: one token of the state space scan against the fp64 recurrence.

Tolerances, per element: the decay is off by (4 + |dt A|) U of itself, the
write by 8 U, so the state by 16 U (1 + |dt A|) (|a S| + |dt b x|); y is a sum
of n such terms, (n + 32) U of sum |c| (those) + |D x|, plus half a step of bf16.
"""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(B, H, G, n, p, dtype, gate, extras=True, seed=1):
    g = torch.Generator().manual_seed(seed)

    def r(*s, dt=dtype, k=1.0):
        return (k * torch.randn(s, generator=g)).to(dt)

    c = dict(x=r(B, 3, H, p), dt=r(B, 3, H, dt=gate), A=-torch.rand(H, generator=g) * 8, b=r(B, 3, G, n), c=r(B, 3, G, n),
             h=r(B, H, n, p, dt=F, k=0.5), D=r(H, dt=F) if extras else None, dt_bias=r(H, dt=F) - 2 if extras else None)
    return {k: None if v is None else v.cuda() for k, v in c.items()}, {k: None if v is None else v.double() for k, v in c.items()}


@pytest.mark.parametrize("B,H,G,n,p,dtype,gate,extras", [
    (1, 1, 1, 64, 64, F, F, True), (3, 6, 2, 128, 64, BF, F, True), (2, 4, 1, 64, 128, BF, BF, False),
    (5, 8, 8, 128, 128, F, BF, True), (33, 2, 1, 128, 128, BF, BF, True)])
def test_three_tokens(B, H, G, n, p, dtype, gate, extras):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(B, H, G, n, p, dtype, gate, extras)
    h = d["h"].clone()
    ys = [gdr.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["b"][:, t], d["c"][:, t], h, d["D"], d["dt_bias"])
          for t in range(3)]
    torch.cuda.synchronize()
    y, ht, step = ref.ssm(c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], None, c["h"])
    ab = {k: None if v is None else v.abs() for k, v in c.items()}
    my, mh, _ = ref.ssm(ab["x"], c["dt"], c["A"], ab["b"], ab["c"], ab["D"], c["dt_bias"], None, ab["h"])
    worst = 3 * (1 + (step * c["A"].abs()).max().item())   # three tokens' roundings
    check("state", h, ht, 16 * U * worst * mh)
    check("y", torch.stack(ys, 1), y, (n + 32 + 16 * worst) * U * my + (half_step(dtype) * y.abs() if dtype == BF else 0))


@pytest.mark.parametrize("dtype,n,p", [(BF, 128, 128), (F, 64, 128)])
def test_large_states(dtype, n, p):
    """States that go past the caches have the bits of each sequence alone, over three tokens."""
    import chunked_gated_delta_fwd_amd as gdr
    B, H = 5 * 128 // n, 65
    d, _ = make(B, H, 5, n, p, dtype, dtype, seed=2)
    h = d["h"].clone()
    assert h.numel() * 4 >= 1 << 24
    ys = [gdr.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["b"][:, t], d["c"][:, t], h, d["D"], d["dt_bias"]) for t in range(3)]
    for i in range(B):
        s = slice(i, i + 1)
        one = d["h"][s].clone()
        for t in range(3):
            y = gdr.ssm_step(d["x"][s, t], d["dt"][s, t], d["A"], d["b"][s, t], d["c"][s, t], one, d["D"], d["dt_bias"])
            assert torch.equal(y[0], ys[t][i])
        assert torch.equal(one[0], h[i])
