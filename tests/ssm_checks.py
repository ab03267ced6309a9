"""The state space scan's forward and gradient held to the literal fp64
recurrence, element by element, within what fp32 sums and one rounding of each
output leave.

Tolerances.  Every decay e^-|G| is off by at most 8 U (1 + |G|) of itself, and
|G| e^-|G| <= e^(-|G|/2), so sizes of the terms taken with half the decay
exponents bound the decays' errors too.  fp32 sums: 512 U of the sizes (8 U for
the decay and step, 3 U for the products, one U for each addition on a term's
way).  An operand of a bf16 product that is no input is taken as two bf16
values: the first keeps the top 8 bits, what it leaves out is under 2^-7 and
rounded by half a step of bf16, 2^-8, so it is off by 2^-15 of itself, and each
term has one such operand at most: 2^-15 of the sizes.  Then the output's own
half step of the value, and no other.
"""
from __future__ import annotations

import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step

BF = torch.bfloat16
NAMES = ("dx", "ddt", "dA", "db", "dc", "dD", "dbias", "dh0")


def sizes(c):
    """Absolute values, the steps, and the decays with half their exponents."""
    step = ref.softplus(c["dt"] if c["dt_bias"] is None else c["dt"] + c["dt_bias"])
    a = {k: None if v is None else v.abs() for k, v in c.items()}
    return a, step, torch.exp(step * c["A"] / 2)


def on(c, device):
    return {k: None if v is None else v.to(device) for k, v in c.items()}


def terms(dtype):
    """Of the sizes: fp32 sums, and what two bf16 parts leave out."""
    return 512 * U + (2.0 ** -15 if dtype == BF else 0)


def check_forward(got, c, cu, dtype, device="cuda"):
    """`got` (y, ht) against the doubles `c` of a call's inputs."""
    c = on(c, device)
    ry, rh, _ = ref.ssm(c["x"], c["dt"], c["A"], c["b"], c["c"], c["D"], c["dt_bias"], cu, c["h0"])
    a, step, dec = sizes(c)
    my, mh = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], cu, a["h0"])
    half = half_step(dtype) if dtype == BF else 0
    check("y", got[0], ry.cpu(), (terms(dtype) * my + half * ry.abs()).cpu())
    check("ht", got[1], rh.cpu(), (512 * U * mh).cpu())


def check_backward(got, c, cu, dtype, gate, device="cuda"):
    """`got`, the eight gradients, against the doubles `c` of a call's inputs."""
    got, c = dict(zip(NAMES, got)), on(c, device)
    B, T, H, p = c["x"].shape
    G, n = c["b"].shape[2:]
    seqs = ref.bounds(cu, B, T)
    zero = c["x"].new_zeros(len(seqs), H, n, p)
    extras = c["D"] is not None
    names = ["x", "dt", "A", "b", "c", "h0"] + (["D", "dt_bias"] if extras else [])
    leaf = {k: (zero if c[k] is None else c[k]).clone().requires_grad_() for k in names}
    y, ht, _ = ref.ssm(leaf["x"], leaf["dt"], leaf["A"], leaf["b"], leaf["c"], leaf.get("D"), leaf.get("dt_bias"), cu, leaf["h0"])
    dht = zero if c["dht"] is None else c["dht"]
    r = dict(zip(names, torch.autograd.grad((y * c["dy"]).sum() + (ht * dht).sum(), list(leaf.values()))))
    del y, ht

    # the same on absolute values, with the steps and decays as leaves of their own
    a, step, dec = sizes(c)
    m = dict(x=a["x"], st=step, dec=dec, b=a["b"], c=a["c"], h0=zero if a["h0"] is None else a["h0"])
    m = {k: v.clone().requires_grad_() for k, v in m.items()}
    ym, hm = ref.ssm_walk(m["x"], m["st"], m["dec"], m["b"], m["c"], a["D"], cu, m["h0"])
    s = dict(zip(m, torch.autograd.grad((ym * a["dy"]).sum() + (hm * dht.abs()).sum(), list(m.values()))))
    half = half_step(dtype) if dtype == BF else 0
    k = 512 * U
    for name, key in (("dx", "x"), ("db", "b"), ("dc", "c")):
        check(name, got[name], r[key].cpu(), (terms(dtype) * s[key] + half * r[key].abs()).cpu())
    check("dh0", got["dh0"], r["h0"].cpu(), (k * s["h0"]).cpu())
    # the gradient of a decay's logarithm is a sum over the rest of the chunk: what its tokens read of earlier
    # writes, and what later ones read of theirs (not a token's read of its own write), and <E, S> at its end
    R = H // G
    a["bh"], a["ch"] = a["b"].repeat_interleave(R, 2), a["c"].repeat_interleave(R, 2)
    own = step * (a["bh"] * a["ch"]).sum(-1) * (a["x"] * a["dy"]).sum(-1)
    reads = torch.zeros_like(own)
    for i, (b0, e0) in enumerate(seqs):   # |c|^T |S| |dy| of each token, head by head
        S = m["h0"].detach()[i]
        for t in range(b0, e0):
            f = lambda v: v.reshape((-1,) + v.shape[2:])[t]   # noqa: E731
            S = f(dec)[:, None, None] * S
            reads.reshape(-1, H)[t] = ((f(a["ch"])[:, :, None] * S).sum(1) * f(a["dy"])).sum(-1)
            S = S + (f(step)[:, None] * f(a["bh"]))[:, :, None] * f(a["x"])[:, None]
    per = reads + (step * s["st"] - own).clamp(min=0)
    size = torch.zeros_like(per).reshape(-1, H)
    P_, E_ = per.reshape(-1, H), (dec * s["dec"]).reshape(-1, H)
    tail = (dht.abs() * hm.detach()).sum((2, 3))
    for i, (b0, e0) in enumerate(seqs):
        for t0 in range(b0, e0, 64):
            t1 = min(t0 + 64, e0)
            at_end = E_[t1] if t1 < e0 else tail[i]
            size[t0:t1] = P_[t0:t1].flip(0).cumsum(0).flip(0) + at_end
    size = size.reshape(per.shape)
    tol = k * (s["st"] + c["A"].abs() * size)   # sigmoid <= 1
    gh = half_step(gate) if gate == BF else 0
    check("ddt", got["ddt"], r["dt"].cpu(), (tol + gh * r["dt"].abs()).cpu())
    check("dA", got["dA"], r["A"].cpu(), (k * (step * size).sum((0, 1))).cpu())
    if extras:
        check("dD", got["dD"], r["D"].cpu(), (k * (a["x"] * a["dy"]).sum((0, 1, 3))).cpu())
        check("dbias", got["dbias"], r["dt_bias"].cpu(), (tol.sum((0, 1)) + k * r["dt"].abs().sum((0, 1))).cpu())
    else:
        assert got["dD"] is None and got["dbias"] is None
