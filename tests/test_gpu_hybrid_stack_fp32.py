"""GPU: forward and gradients of examples/hybrid_stack.py in fp32 against the
formulas in 64 bits.  Tolerance on the relative 2-norm: 2.2e-3 as counted in
test_gpu_hybrid_stack.py for a pass, twice that for a gradient, which passes the
same tensors once more on the way back.  The delta rule's own gradient rounds the
operands of its products to bf16, whatever its inputs are: what comes through it
(of x and of that layer's projection) is held to that file's 0.24."""
import pytest
import torch

from test_gpu_hybrid_stack import plain_attention
from test_gpu_token_mixer import plain_delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,window", [([3, 66, 1], 20), ([130], 128)])
def test_forward_and_gradients(lengths, window):
    import hybrid_stack as hs
    import token_mixer as tm
    torch.manual_seed(4)
    model = hs.Stack(width=256, window=window).cuda()
    T, cu = sum(lengths), [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    x, dy = torch.randn(1, T, 256), torch.randn(1, T, 256)
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

    far("y", y, want.detach(), 2.2e-3)
    far("dx", xg.grad, xr.grad, 0.24)
    for layer, P in zip(model.layers, params):
        for name in P:
            if name in ("proj", "out"):
                tol = 0.24 if layer is model.layers[0] and name == "proj" else 4.4e-3
                far(type(layer).__name__ + " d" + name, dict(layer.named_parameters())[name].grad, P[name].grad, tol)
