"""GPU: attention, its paged cache and the recurrent layer run together as
examples/hybrid_stack.py runs them.

Tolerances, on the relative 2-norm of whole tensors, by the count of
test_gpu_token_mixer.py: a layer rounds some six tensors to bf16 between its
input and its output, three layers 18, two evaluations of the same formulas 36
roundings of 2^-8, independent (sqrt(36) 2^-8 = 0.024 together); products of q
and k cancel to a tenth of their terms before the norm brings them back to 1,
which makes 5 of it: 0.12, and twice that for a gradient, which passes the same
tensors once more on the way back.  fp32: seven sums of 512 terms follow each
other, cancellation costs a factor of 10 at most: 7 * 512 * 10 * 2^-24 = 2.2e-3.
"""
import os
import sys

import pytest
import torch

import attn_ref
import mixer_ref as ref
from test_gpu_token_mixer import plain_delta

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain_attention(layer, x, cu):
    """AttentionLayer.forward in fp64."""
    P = {k: v.detach().double().cpu().requires_grad_() for k, v in layer.named_parameters()}
    q, k, v = (x @ P["proj"]).unflatten(-1, (layer.hq + 2 * layer.hk, layer.d)).split([layer.hq, layer.hk, layer.hk], -2)
    pos = torch.cat([torch.arange(e - s) for s, e in zip(cu[:-1], cu[1:])])[None]
    cos, sin = (t.double().cpu() for t in layer.tables)
    q, k = (ref.norm_rope(t, None, cos, sin, pos, False, 1e-6, False) for t in (q, k))
    o = attn_ref.attention(q * layer.d ** 0.5, k, v, cu, window=layer.window)[0]
    return o.flatten(-2) @ P["out"], P


def test_tokens_after_a_prompt_match_the_whole_pass():
    import hybrid_stack as hs
    for dtype, tol in ((torch.float32, 2.2e-3), (torch.bfloat16, 0.12)):
        torch.manual_seed(1)
        model = hs.Stack(width=256, window=40).cuda().to(dtype)
        far, _ = hs.decode_and_compare(model, [1, 70, 200], 5, dtype)
        print(dtype, "relative distance %.3g" % far, flush=True)
        assert far <= tol


def test_forward_and_gradients_match_the_formulas():
    import hybrid_stack as hs
    import token_mixer as tm
    torch.manual_seed(2)
    model = hs.Stack(width=256, window=20).cuda().bfloat16()
    lengths, cu = [3, 66, 1], [0, 3, 69, 70]
    x, dy = (torch.randn(1, 70, 256).bfloat16() for _ in range(2))
    xg = x.cuda().requires_grad_()
    y = model(xg, tm.packed(lengths, "cuda"))
    y.backward(dy.cuda())
    xr = x.double().requires_grad_()
    want, params = xr, []
    for layer, plain in zip(model.layers, (plain_delta, plain_attention, plain_attention)):
        step, P = plain(layer, want, cu)
        want = want + step
        params.append(P)
    want.backward(dy.double())

    def far(what, got, r, tol):
        d = ((got.detach().double().cpu() - r).norm() / r.norm()).item()
        print("%s: relative distance %.3g" % (what, d), flush=True)
        assert d <= tol, what

    far("y", y, want.detach(), 0.12)
    far("dx", xg.grad, xr.grad, 0.24)
    for layer, P in zip(model.layers, params):
        for name in P:
            if name in ("proj", "out"):
                far(type(layer).__name__ + " d" + name, dict(layer.named_parameters())[name].grad, P[name].grad, 0.24)


def test_it_trains_and_prints():
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "hybrid_stack.py"), "--tokens", "200", "--new", "3",
                        "--steps", "2"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "single tokens" in r.stdout and "training" in r.stdout
