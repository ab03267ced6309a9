"""GPU: the operators run together as examples/token_mixer.py runs them.

Tolerances, on the relative 2-norm of whole tensors.  bf16: some 12 tensors are
rounded to bf16 between input and output of the stack (projections, convolution,
norm, recurrence and output of two layers, two sums), each by at most 2^-8 of
its value, so two evaluations of the same formulas differ by 24 roundings.
Those are independent (sqrt(24) 2^-8 = 0.019 together) and the products of q
and k, which cancel to a tenth of their terms before the norm brings the result
back to 1, make 5 of it; a gradient passes the same tensors once more on the
way back.  Tolerances: 0.1 and 0.2.  fp32: the longest sum has 512
terms, five of them follow each other, and cancellation costs a factor of 10 at
most: 5 * 512 * 10 * 2^-24 = 1.5e-3.
"""
import os
import sys

import pytest
import torch

import mixer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain_delta(layer, x, cu):
    """DeltaLayer.forward in fp64, the recurrence one token at a time."""
    P = {k: v.detach().double().cpu().requires_grad_() for k, v in layer.named_parameters()}
    mixed, gate, beta = (x @ P["proj"]).split([layer.qk + layer.vd, layer.hv, layer.hv], -1)
    g, beta = torch.nn.functional.logsigmoid(gate + 2), torch.sigmoid(beta)
    m, _ = ref.conv(mixed, P["conv_w"], P["conv_b"], cu, None, True)
    q, k, v = layer.heads(m[..., :layer.qk], m[..., layer.qk:])
    pos = torch.cat([torch.arange(e - s) for s, e in zip(cu[:-1], cu[1:])])[None]
    cos, sin = (t.double().cpu() for t in layer.tables)
    q, k = (ref.norm_rope(t, None, cos, sin, pos, False, 1e-6, False)[0].repeat_interleave(layer.hv // layer.hk, 1)
            for t in (q, k))
    out = []
    for s, e in zip(cu[:-1], cu[1:]):
        H = x.new_zeros(layer.hv, layer.d, layer.d)
        for t in range(s, e):
            H = g[0, t].exp()[:, None, None] * H
            d = beta[0, t][:, None] * (v[0, t] - (k[t][:, :, None] * H).sum(1))
            H = H + k[t][:, :, None] * d[:, None]
            out.append(layer.d ** -0.5 * (q[t][:, :, None] * H).sum(1))
    o = torch.stack(out)[None]
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6)
    return o.flatten(-2) @ P["out"], P


def plain_ssm(layer, x, cu):
    P = {k: v.detach().double().cpu().requires_grad_() for k, v in layer.named_parameters()}
    mixed, dt = (x @ P["proj"]).split([sum(layer.sizes), layer.h], -1)
    m, _ = ref.conv(mixed, P["conv_w"], P["conv_b"], cu, None, True)
    u, b, c = layer.split(m)
    y, _, _ = ref.ssm(u, dt, P["A"], b, c, P["D"], P["dt_bias"], cu, None)
    return y.flatten(-2) @ P["out"], P


def test_tokens_after_a_prompt_match_the_whole_pass():
    import token_mixer as tm
    for dtype, tol in ((torch.float32, 1.5e-3), (torch.bfloat16, 0.1)):
        torch.manual_seed(1)
        model = tm.Stack(width=256).cuda().to(dtype)
        far, _ = tm.decode_and_compare(model, [1, 70, 200], 5, dtype)
        print(dtype, "relative distance %.3g" % far, flush=True)
        assert far <= tol


def test_forward_and_gradients_match_the_formulas():
    import token_mixer as tm
    torch.manual_seed(2)
    model = tm.Stack(width=256).cuda().bfloat16()
    lengths = [3, 66, 1]
    cu = [0, 3, 69, 70]
    x = torch.randn(1, 70, 256).bfloat16()
    dy = torch.randn(1, 70, 256).bfloat16()
    xg = x.cuda().requires_grad_()
    y = model(xg, tm.packed(lengths, "cuda"))
    y.backward(dy.cuda())
    xr = x.double().requires_grad_()
    y1, p_ssm = plain_ssm(model.layers[0], xr, cu)
    x1 = xr + y1
    y2, p_delta = plain_delta(model.layers[1], x1, cu)
    want = x1 + y2
    want.backward(dy.double())

    def far(what, got, ref, tol):
        d = ((got.detach().double().cpu() - ref).norm() / ref.norm()).item()
        print("%s: relative distance %.3g" % (what, d), flush=True)
        assert d <= tol, what

    far("y", y, want.detach(), 0.1)
    far("dx", xg.grad, xr.grad, 0.2)
    for layer, P in zip(model.layers, (p_ssm, p_delta)):
        for name in ("proj", "conv_w", "conv_b", "out"):
            far(type(layer).__name__ + " d" + name, dict(layer.named_parameters())[name].grad, P[name].grad, 0.2)


def test_training_lowers_the_loss():
    import token_mixer as tm
    torch.manual_seed(3)
    model = tm.Stack(width=256).cuda().bfloat16()
    losses = tm.train(model, tm.packed([40, 100], "cuda"), 10)
    print(losses, flush=True)
    assert losses[-1] < losses[0]
