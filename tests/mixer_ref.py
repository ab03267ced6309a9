"""Plain fp64 references of the operators around the recurrence, written from
their definitions one token at a time (CPU, torch.double, differentiable), and
the tolerances the tests hold the kernels to."""
from __future__ import annotations

import torch

U = 2.0 ** -24   # half a step of fp32, relative


def half_step(dtype) -> float:
    """Half a step of an output type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def bounds(cu, batch, tokens):
    """[start, end) of each sequence in the flattened tokens."""
    if cu is None:
        return [(i * tokens, (i + 1) * tokens) for i in range(batch)]
    return list(zip(cu[:-1], cu[1:]))


def silu(z):
    return z / (1 + torch.exp(-z))


def conv(x, w, bias, cu, s0, act):
    """x [B, T, ch] double; returns (y, st)."""
    B, T, ch = x.shape
    W = w.shape[1]
    flat = x.reshape(-1, ch)
    ys, sts = [], []
    for n, (s, e) in enumerate(bounds(cu, B, T)):
        old = x.new_zeros(W - 1, ch) if s0 is None else s0[n]
        line = torch.cat([old, flat[s:e]])
        z = sum(line[j:j + e - s] * w[:, j] for j in range(W))
        if bias is not None:
            z = z + bias
        ys.append(silu(z) if act else z)
        sts.append(line[e - s:])
    return torch.cat(ys).reshape(B, T, ch), torch.stack(sts)


def norm_rope(x, weight, cos, sin, pos, rms, eps, interleaved):
    """x [B, T, H, d] double, pos [B, T] long (None without tables)."""
    s = (x * x).sum(-1, keepdim=True)
    if rms:
        s = s / x.shape[-1]
    y = x / torch.sqrt(s + eps)
    if weight is not None:
        y = y * weight
    if cos is None:
        return y
    c, sn = cos[pos][:, :, None], sin[pos][:, :, None]
    half = cos.shape[1]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def softplus(raw):
    return torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))


def ssm_walk(x, step, decay, b, c, D, cu, h0):
    """The literal recurrence, one token at a time, from the steps and decays
    [B, T, H]: (y, ht)."""
    B, T, H, p = x.shape
    G, n = b.shape[2:]
    X, st, dec = x.reshape(-1, H, p), step.reshape(-1, H), decay.reshape(-1, H)
    Bh = b.reshape(-1, G, n).repeat_interleave(H // G, 1)
    Ch = c.reshape(-1, G, n).repeat_interleave(H // G, 1)
    ys, hts = [], []
    for i, (s, e) in enumerate(bounds(cu, B, T)):
        S = x.new_zeros(H, n, p) if h0 is None else h0[i]
        for t in range(s, e):
            S = dec[t][:, None, None] * S + (st[t][:, None] * Bh[t])[:, :, None] * X[t][:, None]
            y = (Ch[t][:, :, None] * S).sum(1)
            ys.append(y if D is None else y + D[:, None] * X[t])
        hts.append(S)
    y = torch.stack(ys) if ys else x.new_zeros(0, H, p)
    return y.reshape(B, T, H, p), torch.stack(hts)


def ssm(x, dt, A, b, c, D, dt_bias, cu, h0):
    """x [B, T, H, p], raw dt [B, T, H], b and c [B, T, G, n], all double; returns (y, ht, steps)."""
    step = softplus(dt if dt_bias is None else dt + dt_bias)
    y, ht = ssm_walk(x, step, torch.exp(step * A), b, c, D, cu, h0)
    return y, ht, step


def check(what, got, ref, tol):
    """|got - ref| <= tol for every element (ref and tol double on the CPU)."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what + ": not finite"
    if got.numel() == 0:
        return
    over = ((got - ref).abs() / tol.clamp(min=1e-300)).max().item()
    print("%s: worst error %.3g of its tolerance" % (what, over), flush=True)
    assert over <= 1, "%s: %.3g times its tolerance" % (what, over)
