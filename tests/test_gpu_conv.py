"""GPU: the short causal convolution (forward, gradient, one token) against the
plain fp64 evaluation of its definition.

Tolerances.  z is W products and a bias in fp32: an error of at most
(W + 1) U mag, mag = |bias| + sum |w x|.  |silu'| < 1.1 and the sigmoid's own
error (exp, add, reciprocal: a few units of U) is at most 8 U |y|, so 16 U mag
covers y in fp32 and bf16 adds half a step.  |silu''| < 0.5 likewise gives
32 U (1 + mag) |dy| for dz, and sums of k terms k U more of the terms' sizes.
"""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(seed, B, T, ch, W, dtype, bias=True, cu=None, state=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1

    def r(*s):
        return torch.randn(s, generator=g).to(dtype)

    c = dict(x=r(B, T, ch), w=(r(ch, W).float() * 0.4).to(dtype), bias=r(ch) if bias else None,
             s0=r(N, W - 1, ch) if state else None, dy=r(B, T, ch), dst=r(N, W - 1, ch) if state else None)
    c["cu"] = cu
    dev = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in c.items()}
    if wide:   # x and dy as columns of a wider projection
        for k in ("x", "dy"):
            big = torch.zeros(B, T, ch + wide, dtype=dtype, device="cuda")
            big[..., wide // 2:wide // 2 + ch] = dev[k]
            dev[k] = big[..., wide // 2:wide // 2 + ch]
    dev["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    dbl = {k: (v.double() if torch.is_tensor(v) else v) for k, v in c.items()}
    return dev, dbl


CASES = [
    # B, T, ch, W, dtype, bias, silu, cu, state, wide
    (1, 1, 64, 4, BF, True, True, None, True, 0),
    (1, 1, 7, 2, F, False, False, None, True, 0),
    (2, 2, 24, 4, BF, True, True, None, True, 0),            # shorter than the state
    (3, 65, 72, 3, BF, False, True, None, False, 0),
    (2, 130, 40, 4, F, True, True, None, True, 16),          # rows of a wider projection
    (2, 37, 40, 4, BF, True, True, None, True, 6),           # such rows off 16 bytes
    (1, 200, 136, 4, BF, True, True, [0, 0, 1, 3, 3, 64, 131, 200, 200], True, 0),
    (1, 97, 131, 3, F, True, False, [0, 2, 2, 96, 97], True, 0),
    (1, 97, 129, 2, BF, False, True, [0, 33, 97], False, 0),
    (1, 700, 520, 4, BF, True, True, [0, 1, 2, 300, 629, 700], True, 24),
]


@pytest.mark.parametrize("B,T,ch,W,dtype,bias,silu,cu,state,wide", CASES)
def test_conv_forward(B, T, ch, W, dtype, bias, silu, cu, state, wide):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(1, B, T, ch, W, dtype, bias, cu, state, wide)
    y, st = gdr.short_conv_fwd(d["x"], d["w"], d["bias"], d["cu"], d["s0"], activation="silu" if silu else None)
    torch.cuda.synchronize()
    ry, rst = ref.conv(c["x"], c["w"], c["bias"], cu, c["s0"], silu)
    mag = ref.conv(c["x"].abs(), c["w"].abs(), None if c["bias"] is None else c["bias"].abs(), cu,
                   None if c["s0"] is None else c["s0"].abs(), False)[0]
    check("y", y, ry, 16 * U * mag + (half_step(dtype) * ry.abs() if dtype == BF else 0))
    assert torch.equal(st.double().cpu(), rst)


@pytest.mark.parametrize("B,T,ch,W,dtype,bias,silu,cu,state,wide", CASES)
def test_conv_backward(B, T, ch, W, dtype, bias, silu, cu, state, wide):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(2, B, T, ch, W, dtype, bias, cu, state, wide)
    got = gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"], d["s0"], d["dst"],
                             activation="silu" if silu else None)
    torch.cuda.synchronize()
    s0 = torch.zeros(len(ref.bounds(cu, B, T)), W - 1, ch, dtype=torch.double) if c["s0"] is None else c["s0"]
    leaves = [t.clone().requires_grad_() for t in (c["x"], c["w"], s0)] + ([c["bias"].clone().requires_grad_()] if bias else [])
    y, st = ref.conv(leaves[0], leaves[1], leaves[3] if bias else None, cu, leaves[2], silu)
    loss = (y * c["dy"]).sum() + ((st * c["dst"]).sum() if state else 0 * leaves[2].sum())
    rx, rw, rs, *rb = torch.autograd.grad(loss, leaves)
    # the same gradients of the magnitudes: sum |w| |dz| with |dz| <= 1.1 |dy|, each dz off by 32 U (1 + mag) |dy|
    a = [t.detach().abs() for t in leaves]
    mag = ref.conv(a[0], a[1], a[3] if bias else None, cu, a[2], False)[0]
    size = (c["dy"].abs() * 1.1 * (1 + mag)).requires_grad_(False)
    m = [t.clone().requires_grad_() for t in a]
    ym, sm = ref.conv(m[0], m[1], m[3] if bias else None, cu, m[2], False)
    mx, mw, ms, *mb = torch.autograd.grad((ym * size).sum() + ((sm * c["dst"].abs()).sum() if state else 0), m)
    half = half_step(dtype) if dtype == BF else 0
    check("dx", got[0], rx, 32 * U * mx + half * rx.abs())
    check("dw", got[1], rw, (32 + 128) * U * mw)
    if bias:
        check("db", got[2], rb[0], (32 + 128) * U * mb[0])
    else:
        assert got[2] is None
    check("ds0", got[3], rs, 32 * U * ms + half * rs.abs())


def test_conv_backward_differences():
    """Directional differences of the fp64 forward against the kernel's gradients."""
    import chunked_gated_delta_fwd_amd as gdr
    cu = [0, 3, 3, 40, 90]
    d, c = make(3, 1, 90, 24, 4, F, True, cu)
    dx, dw, db, ds0 = (t.double().cpu() for t in gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"], d["s0"], d["dst"]))

    def loss(x, w, b, s):
        y, st = ref.conv(x, w, b, cu, s, True)
        return ((y * c["dy"]).sum() + (st * c["dst"]).sum()).item()

    base = [c["x"], c["w"], c["bias"], c["s0"]]
    for i, grad in enumerate((dx, dw, db, ds0)):
        v = torch.randn(base[i].shape, dtype=torch.double, generator=torch.Generator().manual_seed(i))
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + 1e-5 * v, base[i] - 1e-5 * v
        diff = (loss(*up) - loss(*dn)) / 2e-5
        terms = (grad * v).abs().sum().item()
        # fp32 gradients: 200 U of the terms; the differences: third derivatives x 1e-10 and fp64 noise / 1e-5
        assert abs(diff - (grad * v).sum().item()) <= (200 * U + 1e-6) * terms, i


@pytest.mark.parametrize("B,ch,W,dtype", [(1, 8, 4, BF), (5, 70, 3, BF), (3, 33, 2, F), (65, 264, 4, F)])
def test_conv_step_continues_the_forward(B, ch, W, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(4, B, 6, ch, W, dtype)
    y, st = gdr.short_conv_fwd(d["x"], d["w"], d["bias"], None, d["s0"])
    state = d["s0"].clone()
    ys = [gdr.short_conv_step(d["x"][:, t], state, d["w"], d["bias"]) for t in range(6)]   # strided rows
    torch.cuda.synchronize()
    ry, _ = ref.conv(c["x"], c["w"], c["bias"], None, c["s0"], True)
    mag = ref.conv(c["x"].abs(), c["w"].abs(), c["bias"].abs(), None, c["s0"].abs(), False)[0]
    check("y", torch.stack(ys, 1), ry, 16 * U * mag + (half_step(dtype) * ry.abs() if dtype == BF else 0))
    assert torch.equal(state, st)


def test_conv_repeats_and_splits_bit_identically():
    """Two calls over a split sequence give one call's bits; repeats too."""
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(5, 1, 300, 96, 4, BF)
    y, st = gdr.short_conv_fwd(d["x"], d["w"], d["bias"], None, d["s0"])
    a, s1 = gdr.short_conv_fwd(d["x"][:, :131], d["w"], d["bias"], None, d["s0"])
    b, s2 = gdr.short_conv_fwd(d["x"][:, 131:], d["w"], d["bias"], None, s1)
    assert torch.equal(torch.cat([a, b], 1), y) and torch.equal(s2, st)
    first = gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], None, d["s0"], d["dst"])
    for _ in range(3):
        again = gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], None, d["s0"], d["dst"])
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_conv_special_values():
    """Infinities and NaN stay in the rows that read them, and large |z| does not overflow the sigmoid."""
    import chunked_gated_delta_fwd_amd as gdr
    x = torch.randn(1, 20, 16, device="cuda")
    x[0, 5, 3], x[0, 9, 4] = float("nan"), float("inf")
    x[0, 15, 5], x[0, 15, 6] = 1e30, -1e30
    w = torch.full((16, 4), 0.5, device="cuda")
    y, _ = gdr.short_conv_fwd(x, w)
    bad = ~torch.isfinite(y[0])
    want = torch.zeros_like(bad)
    want[5:9, 3] = True
    want[9:13, 4] = True
    assert torch.equal(bad, want)
    assert torch.equal(y[0, 15:19, 6], torch.zeros(4, device="cuda")) or (y[0, 15:19, 6].abs() < 1e-20).all()
    assert (y[0, 15, 5] - 5e29).abs() < 1e24


def test_conv_backward_in_a_graph():
    """Captured with a workspace of its own; replays with eager work between them."""
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(6, 2, 150, 64, 4, BF)
    args = (d["x"], d["w"], d["dy"], d["bias"], None, d["s0"], d["dst"])
    eager = gdr.short_conv_bwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = gdr.short_conv_bwd(*args)
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        gdr.short_conv_bwd(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager, out))


def test_large_outputs():
    """An output that is stored past the caches has the bits of its rows computed alone."""
    import chunked_gated_delta_fwd_amd as gdr
    g = torch.Generator(device="cuda").manual_seed(21)
    for dtype, ch in ((BF, 4096), (F, 2048)):
        x = torch.randn(2, 8192, ch, generator=g, device="cuda").to(dtype)
        w = torch.randn(ch, 4, generator=g, device="cuda").to(dtype)
        s0 = torch.randn(2, 3, ch, generator=g, device="cuda").to(dtype)
        y, st = gdr.short_conv_fwd(x, w, s0=s0)
        assert y.numel() * y.element_size() >= 1 << 27
        for i in range(2):
            one, s1 = gdr.short_conv_fwd(x[i:i + 1], w, s0=s0[i:i + 1])
            assert torch.equal(one[0], y[i]) and torch.equal(s1[0], st[i])
