"""GPU: the selective state space scan (prompt and gradient) against the literal
fp64 recurrence and its derivative.

Tolerances, per element, from sums of the terms' sizes (the recurrence and its
gradient on absolute values).  Every decay e^-|G| is off by at most 8 U (1 + |G|)
of itself, and |G| e^-|G| <= e^(-|G|/2), so sizes taken with half the decay
exponents bound the decays' errors too:

* fp32 results: 8 U for the decay and step, 3 U for the products, and one U for
  each addition on a term's way (at most 3 x 64 in a chunk, 64 chunks, n or p
  in a dot product): 512 U of the sizes at the test's lengths;
* bf16 results add one rounding of an operand (half a step of each term) and
  the result's own half step.

The gradient of a decay's logarithm is a sum over the rest of the chunk, so its
error is that of the sum of the terms' sizes there.
"""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(seed, B, T, H, G, n, p, dtype, gate, cu=None, state=True, extras=True, wide=False):
    g = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1

    def r(*s, dt=dtype, k=1.0):
        return (k * torch.randn(s, generator=g)).to(dt)

    c = dict(x=r(B, T, H, p), dt=r(B, T, H, dt=gate, k=0.7), A=-torch.exp(2 * torch.rand(H, generator=g)), b=r(B, T, G, n),
             c=r(B, T, G, n), D=r(H, dt=F) if extras else None, dt_bias=r(H, dt=F) - 3 if extras else None,
             h0=r(N, H, n, p, dt=F, k=0.4) if state else None, dy=r(B, T, H, p),
             dht=r(N, H, n, p, dt=F, k=0.4) if state else None)
    dev = {k: None if v is None else v.cuda() for k, v in c.items()}
    if wide:   # x, b and c as columns of one projection, dt of another
        w = torch.cat([dev["x"].flatten(2), dev["b"].flatten(2), dev["c"].flatten(2)], 2)
        dev["x"] = w[..., :H * p].unflatten(-1, (H, p))
        dev["b"] = w[..., H * p:H * p + G * n].unflatten(-1, (G, n))
        dev["c"] = w[..., H * p + G * n:].unflatten(-1, (G, n))
        dev["dt"] = torch.cat([dev["dt"], dev["dt"]], 2)[..., H:]
    dev["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return dev, {k: None if v is None else v.double() for k, v in c.items()}


CASES = [
    # B, T, H, G, n, p, dtype, gate, cu, state, extras, wide
    (1, 1, 1, 1, 64, 64, BF, BF, None, True, True, False),
    (1, 64, 2, 1, 128, 64, BF, F, None, False, True, False),
    (2, 65, 4, 2, 64, 128, BF, BF, None, True, False, True),
    (1, 200, 4, 1, 128, 128, BF, F, None, True, True, False),
    (1, 321, 6, 2, 128, 64, BF, F, [0, 0, 1, 65, 65, 130, 321, 321], True, True, True),
    (1, 150, 3, 3, 64, 64, BF, BF, [0, 3, 3, 150], False, True, False),
    (2, 127, 2, 1, 64, 64, F, F, None, True, True, False),
    (1, 190, 4, 2, 128, 64, F, BF, [0, 64, 64, 190], True, True, True),
    (1, 70, 2, 2, 128, 128, F, F, None, True, False, False),
    (1, 66, 1, 1, 64, 128, F, F, [0, 0, 66], False, True, False),
    # walked in spans, in both directions; rows; and packed sequences that are all short
    (1, 1100, 2, 1, 64, 64, BF, F, [0, 1000, 1000, 1100], True, True, False),
    (2, 900, 2, 2, 64, 64, BF, BF, None, True, True, False),
    (1, 700, 2, 1, 64, 64, F, F, [0, 30, 700], True, True, False),
    (1, 900, 4, 2, 64, 64, BF, F, list(range(0, 901, 100)), True, True, False),
]
IDS = ["%dx%d H%d/%d n%d p%d %s%s" % (c[0], c[1], c[2], c[3], c[4], c[5], "bf16" if c[6] == BF else "f32",
                                      " packed" if c[8] else "") for c in CASES]


def forward(gdr, d):
    return gdr.ssm_scan_fwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["D"], d["dt_bias"], d["cu"], d["h0"])


def backward(gdr, d):
    return gdr.ssm_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["dy"], d["D"], d["dt_bias"], d["cu"], d["h0"], d["dht"])


def sizes(c):
    """Absolute values, the steps, and the decays with half their exponents."""
    step = ref.softplus(c["dt"] if c["dt_bias"] is None else c["dt"] + c["dt_bias"])
    a = {k: None if v is None else v.abs() for k, v in c.items()}
    return a, step, torch.exp(step * c["A"] / 2)


@pytest.mark.parametrize("B,T,H,G,n,p,dtype,gate,cu,state,extras,wide", CASES, ids=IDS)
def test_forward(B, T, H, G, n, p, dtype, gate, cu, state, extras, wide):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(1, B, T, H, G, n, p, dtype, gate, cu, state, extras, wide)
    y, ht = forward(gdr, d)
    torch.cuda.synchronize()
    ry, rh, _ = ref.ssm(c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], cu, c["h0"])
    a, step, dec = sizes(c)
    my, mh = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], cu, a["h0"])
    half = half_step(dtype) if dtype == BF else 0
    check("y", y, ry, 512 * U * my + half * (my + ry.abs()))
    check("ht", ht, rh, 512 * U * mh)


@pytest.mark.parametrize("B,T,H,G,n,p,dtype,gate,cu,state,extras,wide", CASES, ids=IDS)
def test_backward(B, T, H, G, n, p, dtype, gate, cu, state, extras, wide):
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(2, B, T, H, G, n, p, dtype, gate, cu, state, extras, wide)
    got = dict(zip(("dx", "ddt", "dA", "db", "dc", "dD", "dbias", "dh0"), backward(gdr, d)))
    torch.cuda.synchronize()
    N = len(ref.bounds(cu, B, T))
    zero = torch.zeros(N, H, n, p, dtype=torch.double)
    names = ["x", "dt", "A", "b", "c", "h0"] + (["D", "dt_bias"] if extras else [])
    leaf = {k: (zero if c[k] is None else c[k]).clone().requires_grad_() for k in names}
    y, ht, _ = ref.ssm(leaf["x"], leaf["dt"], leaf["A"], leaf["b"], leaf["c"], leaf.get("D"), leaf.get("dt_bias"), cu, leaf["h0"])
    dht = zero if c["dht"] is None else c["dht"]
    r = dict(zip(names, torch.autograd.grad((y * c["dy"]).sum() + (ht * dht).sum(), list(leaf.values()))))

    # the same on absolute values, with the steps and decays as leaves of their own
    a, step, dec = sizes(c)
    m = dict(x=a["x"], st=step, dec=dec, b=a["b"], c=a["c"], h0=zero if a["h0"] is None else a["h0"])
    m = {k: v.clone().requires_grad_() for k, v in m.items()}
    ym, hm = ref.ssm_walk(m["x"], m["st"], m["dec"], m["b"], m["c"], a["D"], cu, m["h0"])
    s = dict(zip(m, torch.autograd.grad((ym * a["dy"]).sum() + (hm * dht.abs()).sum(), list(m.values()))))
    half = half_step(dtype) if dtype == BF else 0
    k = 512 * U
    for name, key in (("dx", "x"), ("db", "b"), ("dc", "c")):
        check(name, got[name], r[key], k * s[key] + half * (s[key] + r[key].abs()))
    check("dh0", got["dh0"], r["h0"], k * s["h0"])
    # l_t: the rest of the chunk's c . dc and dt v, and <E, S> at its end
    per = (a["c"] * s["c"]).sum(-1).repeat_interleave(H // G, 2) + step * s["st"]
    end = dec * s["dec"]
    size = torch.zeros_like(per).reshape(-1, H)
    P_, E_ = per.reshape(-1, H), end.reshape(-1, H)
    tail = (dht.abs() * hm.detach()).sum((2, 3))
    for i, (b0, e0) in enumerate(ref.bounds(cu, B, T)):
        for t0 in range(b0, e0, 64):
            t1 = min(t0 + 64, e0)
            at_end = E_[t1] if t1 < e0 else tail[i]
            size[t0:t1] = P_[t0:t1].flip(0).cumsum(0).flip(0) + at_end
    size = size.reshape(per.shape)
    tol = k * (s["st"] + c["A"].abs() * size)   # sigmoid <= 1
    gh = half_step(gate) if gate == BF else 0
    check("ddt", got["ddt"], r["dt"], tol + gh * r["dt"].abs())
    check("dA", got["dA"], r["A"], k * (step * size).sum((0, 1)))
    if extras:
        check("dD", got["dD"], r["D"], k * (a["x"] * a["dy"]).sum((0, 1, 3)))
        check("dbias", got["dbias"], r["dt_bias"], tol.sum((0, 1)) + k * r["dt"].abs().sum((0, 1)))
    else:
        assert got["dD"] is None and got["dbias"] is None


def test_backward_differences():
    """Directional differences of the fp64 forward against the kernel's gradients."""
    import chunked_gated_delta_fwd_amd as gdr
    cu = [0, 5, 5, 75, 90]
    d, c = make(3, 1, 90, 2, 1, 64, 64, F, F, cu)
    dx, ddt, dA, db, dc, dD, dbias, dh0 = (t.double().cpu() for t in backward(gdr, d))
    base = [c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], c["h0"]]

    def loss(*t):
        y, ht, _ = ref.ssm(t[0], t[1], t[2], t[3], t[4], t[5], t[6], cu, t[7])
        return ((y * c["dy"]).sum() + (ht * c["dht"]).sum()).item()

    for i, grad in enumerate((dx, ddt, dA, db, dc, dD, dbias, dh0)):
        v = torch.randn(base[i].shape, dtype=torch.double, generator=torch.Generator().manual_seed(i))
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + 1e-5 * v, base[i] - 1e-5 * v
        diff = (loss(*up) - loss(*dn)) / 2e-5
        terms = (grad * v).abs().sum().item()
        # fp32 gradients of up to 512 U of terms that are some ten times the result; differences: 1e-10 of
        # third derivatives and the fp64 noise of the loss over the step
        assert abs(diff - (grad * v).sum().item()) <= (5120 * U + 1e-5) * terms, i


@pytest.mark.parametrize("dtype", [BF, F])
def test_many_spans(dtype):
    """A sequence of many spans, and one token at a time from the state it left."""
    import chunked_gated_delta_fwd_amd as gdr
    cu = [0, 1500, 1500, 1733]
    d, c = make(4, 1, 1733, 2, 1, 64, 64, dtype, F, cu)
    y, ht = forward(gdr, d)
    ry, rh, _ = ref.ssm(c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], cu, c["h0"])
    a, step, dec = sizes(c)
    my, mh = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], cu, a["h0"])
    half = half_step(dtype) if dtype == BF else 0
    check("y", y, ry, 512 * U * my + half * (my + ry.abs()))
    check("ht", ht, rh, 512 * U * mh)
    h = d["h0"].clone()
    steps = []
    for t in range(1500, 1507):   # the third sequence's first tokens
        steps.append(gdr.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["b"][:, t], d["c"][:, t], h[2:3], d["D"], d["dt_bias"]))
    check("steps", torch.stack(steps, 1), ry[:, 1500:1507], 512 * U * my[:, 1500:1507] + half * (my + ry.abs())[:, 1500:1507])


def test_segments_do_not_meet():
    """Packed sequences give the bits of separate calls on the same spans; repeats and ghosts change nothing."""
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(5, 1, 60, 2, 1, 64, 64, BF, F, [0, 25, 60])
    y, ht = forward(gdr, d)
    for lo, hi, i in ((0, 25, 0), (25, 60, 1)):
        one, h1 = gdr.ssm_scan_fwd(d["x"][:, lo:hi], d["dt"][:, lo:hi], d["A"], d["b"][:, lo:hi], d["c"][:, lo:hi], d["D"],
                                   d["dt_bias"], None, d["h0"][i:i + 1].contiguous())
        assert torch.equal(one, y[:, lo:hi]) and torch.equal(h1[0], ht[i])
    g, _ = make(5, 1, 60, 2, 1, 64, 64, BF, F, [0, 25, 60])
    g["cu"] = torch.tensor([0, 0, 25, 25, 60, 60], dtype=torch.int32, device="cuda")
    z = torch.randn_like(d["h0"][:1])
    g["h0"] = torch.cat([z, d["h0"][:1], z, d["h0"][1:], z])
    y2, h2 = forward(gdr, g)
    assert torch.equal(y2, y) and torch.equal(h2[1], ht[0]) and torch.equal(h2[3], ht[1])
    assert all(torch.equal(h2[i], z[0]) for i in (0, 2, 4))
    first = backward(gdr, d)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, backward(gdr, d)))


def test_non_finite_values_stay_in_their_sequence():
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(6, 1, 150, 2, 1, 64, 64, BF, F, [0, 70, 150])
    want = forward(gdr, d)
    d["x"][0, 69, 0, 0] = float("inf")
    d["b"][0, 68, 0, 3] = float("nan")
    y, ht = forward(gdr, d)
    assert torch.equal(y[:, 70:], want[0][:, 70:]) and torch.equal(ht[1], want[1][1])
    assert torch.equal(y[:, :64], want[0][:, :64])   # earlier chunks


def test_steep_and_flat_decays():
    """Decays that vanish within a token, and none at all."""
    import chunked_gated_delta_fwd_amd as gdr
    for A in (-3000.0, 0.0):
        d, c = make(7, 1, 130, 2, 1, 64, 64, F, F, None)
        d["A"].fill_(A)
        c["A"].fill_(A)
        y, ht = forward(gdr, d)
        ry, rh, step = ref.ssm(c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], None, c["h0"])
        a, step, dec = sizes(c)
        my, mh = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], None, a["h0"])
        check("y", y, ry, 512 * U * my)
        check("ht", ht, rh, 512 * U * mh)
        assert all(torch.isfinite(t).all() for t in backward(gdr, d))


@pytest.mark.parametrize("T,cu", [(0, None), (0, [0, 0, 0])])
def test_no_tokens(T, cu):
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(8, 1, T, 2, 1, 64, 64, BF, F, cu)
    y, ht = forward(gdr, d)
    assert y.numel() == 0 and torch.equal(ht, d["h0"])
    dx, ddt, dA, db, dc, dD, dbias, dh0 = backward(gdr, d)
    assert torch.equal(dh0, d["dht"]) and all((t == 0).all() for t in (dA, dD, dbias))


@pytest.mark.parametrize("T", [700, 1000])
def test_in_a_graph(T):
    """Forward with spans and backward (with spans where T is 1000), captured with workspaces of their own, replayed with eager work between."""
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(9, 1, T, 2, 1, 64, 64, BF, F, [0, 300, T])
    eager = list(forward(gdr, d)) + list(backward(gdr, d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = list(forward(gdr, d)) + list(backward(gdr, d))
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        backward(gdr, d)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager, out))


@pytest.mark.parametrize("cu", [None, [0, 0, 1010, 2500]])
@pytest.mark.parametrize("T,H,G", [(2500, 12, 4), (2500, 8, 1)])
def test_groups_alone_and_together(T, H, G, cu):
    """Gradients of a call whose blocks take several heads, across groups, against calls on one group and one
    head each (which the tests above hold to fp64): twice the 512 U of the terms' sizes at most, which are some 15
    times the largest result."""
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make(10, 1, T, H, G, 64, 64, F, F, cu)
    whole = dict(zip(("dx", "ddt", "dA", "db", "dc", "dD", "dbias", "dh0"), backward(gdr, d)))
    R = H // G
    db, dc = torch.zeros_like(whole["db"]), torch.zeros_like(whole["dc"])
    for h in range(H):
        g = h // R
        s = slice(h, h + 1)
        one = dict(zip(("dx", "ddt", "dA", "db", "dc", "dD", "dbias", "dh0"), gdr.ssm_scan_bwd(
            d["x"][:, :, s].contiguous(), d["dt"][..., s].contiguous(), d["A"][s], d["b"][:, :, g:g + 1].contiguous(),
            d["c"][:, :, g:g + 1].contiguous(), d["dy"][:, :, s].contiguous(), d["D"][s], d["dt_bias"][s], d["cu"],
            d["h0"][:, s].contiguous(), d["dht"][:, s].contiguous())))
        db[:, :, g] += one["db"][:, :, 0]
        dc[:, :, g] += one["dc"][:, :, 0]
        for name, part in (("dx", whole["dx"][:, :, s]), ("ddt", whole["ddt"][..., s]), ("dA", whole["dA"][s]),
                           ("dD", whole["dD"][s]), ("dbias", whole["dbias"][s]), ("dh0", whole["dh0"][:, s])):
            scale = one[name].abs().max().item()
            # one head's results do not depend on the others, but its spans may be cut elsewhere: 512 U as above
            assert (part - one[name]).abs().max().item() <= 512 * U * 30 * scale, (name, h)
    for name, want in (("db", db), ("dc", dc)):
        assert (whole[name] - want).abs().max().item() <= 512 * U * 30 * want.abs().max().item(), name
