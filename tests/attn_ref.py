"""Plain fp64 references of softmax attention, its gradient and the paged step,
sequence by sequence and head by head on the CPU, with the tolerances the tests
hold the kernels to.

Tolerances (U = 2^-24, H half a step of the inputs' type, 0 for f32).  A score
is a sum of d exact products in fp32, times scale: off by e = (d + 8) U scale
sum |q k| + 4 U |s|, at most that of the row's worst key.  A probability's
exponent is a difference of two such, its exponential and the reference value
add 8 U (1 + |lse|): relative E = 2 e + 8 U (1 + |lse|).  bf16 rounds it for the
product: H more.  A sum of n terms adds n U of their absolute values.

  o    (H + E + (n + 16) U) sum p |v| + H |o|
  lse  E + (n + 16) U
  ds   p (E |dp - delta| + (d + 8) U sum |do v| + (H + (d + 8) U) sum |do o|) + (H + 4 U) |ds|
       (delta is taken from o as it is stored.  `few`: from the sum of the row's ds with such a delta, which is off by the
       sum of their own errors, without the last term, and by (n + 16) U of their absolute sum)
  dq   scale (sum |err ds| |k| + (n + 16) U sum |ds k|) + H |dq|; dk likewise over the queries
  dv   (H + E + (n + 16) U) sum p |do| + H |dv|

and 4 U of each result for its last scaling and, in fp32, its rounding.  fp32 has no normal value below 2^-126: a
probability or product below it may be taken for 0, so that every sum of n terms is off by (n + 16) 2^-126 times d
times the largest magnitudes (1 where they are smaller) that its terms are products of.
"""
from __future__ import annotations

import torch

from mixer_ref import U, bounds, half_step


def spans(cu, cuk, batch, tq, tk):
    """(query bounds, key bounds) of every sequence."""
    q = bounds(cu, batch, tq)
    return list(zip(q, bounds(cuk if cuk is not None else cu, batch, tk)))


def sees(lq, lk, causal, window):
    """Whether query i sees key j, [lq, lk]."""
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool)
    behind = torch.arange(lq)[:, None] + (lk - lq) - torch.arange(lk)
    return (behind >= 0) & (behind < window if window else True)


def softmax(s, seen):
    """(p, lse) of scores over the keys that are seen; zeros and -inf where there is none."""
    s = torch.where(seen, s, -torch.inf)
    top = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full(s.shape[:-1] + (1,), -torch.inf)
    top = torch.where(top == -torch.inf, 0.0, top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return torch.where(total == 0, 0.0, e / total), (top + torch.log(total))[..., 0]


def vanishing(n, *values):
    """What n terms below fp32's normal values can add up to."""
    size = values[0].shape[-1]
    for x in values:
        size *= max(1.0, x.abs().max().item()) if x.numel() else 1.0
    return (n + 16) * 2.0 ** -126 * size


def one(q, k, v, seen, scale, H):
    """One head of one sequence: (o, lse), their tolerances, and (p, relative error of p)."""
    n, d = max(1, k.shape[0]), q.shape[1]
    p, lse = softmax(scale * (q @ k.t()), seen)
    size = torch.where(seen, abs(scale) * (q.abs() @ k.abs().t()), 0.0)
    e = (d + 12) * U * (size.amax(-1) if k.shape[0] else size.new_zeros(q.shape[0]))
    E = 2 * e + 8 * U * (1 + torch.where(lse == -torch.inf, 0.0, lse.abs()))
    o = p @ v
    to = (H + E + (n + 16) * U)[:, None] * (p @ v.abs()) + (H + 4 * U) * o.abs() + vanishing(n, v)
    return o, lse, to, E + (n + 16) * U, p, E


def attention(q, k, v, cu=None, cuk=None, causal=True, window=0, scale=None, dtype=torch.float32):
    """q [B, Tq, Hq, d], k and v [B, Tk, Hk, d] double: (o, lse, tolerance of o, of lse); rows outside every sequence
    are NaN."""
    B, Tq, Hq, d = q.shape
    Hk, H = k.shape[2], half_step(dtype) if dtype != torch.float32 else 0.0
    scale = d ** -0.5 if scale is None else scale
    Q, K, V = (x.flatten(0, 1) for x in (q, k, v))
    o, to = torch.full_like(Q, torch.nan), torch.zeros_like(Q)
    lse, tl = Q.new_full(Q.shape[:2], torch.nan), Q.new_zeros(Q.shape[:2])
    for (a, b), (e, f) in spans(cu, cuk, B, Tq, k.shape[1]):
        seen = sees(b - a, f - e, causal, window)
        for h in range(Hq):
            g = h // (Hq // Hk)
            o[a:b, h], lse[a:b, h], to[a:b, h], tl[a:b, h], _, _ = one(Q[a:b, h], K[e:f, g], V[e:f, g], seen, scale, H)
    return o.reshape(q.shape), lse.reshape(q.shape[:3]), to.reshape(q.shape), tl.reshape(q.shape[:3])


def gradient(q, k, v, do, cu=None, cuk=None, causal=True, window=0, scale=None, dtype=torch.float32, few=False):
    """((dq, dk, dv), their tolerances) by the formulas; rows outside every sequence are NaN."""
    B, Tq, Hq, d = q.shape
    Hk, H = k.shape[2], half_step(dtype) if dtype != torch.float32 else 0.0
    scale = d ** -0.5 if scale is None else scale
    Q, K, V, DO = (x.flatten(0, 1) for x in (q, k, v, do))
    got = [torch.full_like(x, torch.nan) for x in (Q, K, V)]
    tol = [torch.zeros_like(x) for x in (Q, K, V)]
    for (a, b), (e, f) in spans(cu, cuk, B, Tq, k.shape[1]):
        seen = sees(b - a, f - e, causal, window)
        n, m = max(1, f - e), max(1, (b - a) * (Hq // Hk))
        for x in got[1:]:
            x[e:f] = 0
        for h in range(Hq):
            g = h // (Hq // Hk)
            qs, ks, vs, dos = Q[a:b, h], K[e:f, g], V[e:f, g], DO[a:b, h]
            o, _, _, _, p, E = one(qs, ks, vs, seen, scale, H)
            dp, delta = dos @ vs.t(), (dos * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            off = E[:, None] * (dp - delta).abs() + (d + 8) * U * (dos.abs() @ vs.abs().t())
            shift = (H + (d + 8) * U) * (dos * o).abs().sum(-1, keepdim=True)    # of delta
            if few:
                worst = (dp - delta).abs() + shift
                shift = (p * (off + E[:, None] * shift + (n + 16) * U * worst)).sum(-1, keepdim=True)
            err = p * (off + shift) + (H + 4 * U) * ds.abs()
            got[0][a:b, h] = scale * (ds @ ks)
            tiny = vanishing(n + m, qs, ks, vs, dos) * max(1.0, abs(scale))
            tol[0][a:b, h] = abs(scale) * ((err + (n + 16) * U * ds.abs()) @ ks.abs()) + tiny
            got[1][e:f, g] += scale * (ds.t() @ qs)
            tol[1][e:f, g] += abs(scale) * ((err + (m + 16) * U * ds.abs()).t() @ qs.abs()) + tiny
            got[2][e:f, g] += p.t() @ dos
            tol[2][e:f, g] += (p * (H + E[:, None] + (m + 16) * U)).t() @ dos.abs() + tiny
    tol = [t + (H + 4 * U) * x.abs() for t, x in zip(tol, got)]
    return [x.reshape(y.shape) for x, y in zip(got, (q, k, v))], [x.reshape(y.shape) for x, y in zip(tol, (q, k, v))]


def paged(q, kp, vp, table, lens, window=0, scale=None, dtype=torch.float32):
    """q [N, Hq, d], pages [P, page, Hk, d] double, table [N, M] and lens [N] lists: (o, tolerance)."""
    P, page, Hk, d = kp.shape
    group = q.shape[1] // Hk
    H = half_step(dtype) if dtype != torch.float32 else 0.0
    o, to = torch.zeros_like(q), torch.zeros_like(q)
    for n, (pages, length) in enumerate(zip(table, lens)):
        length = max(0, min(length, len(pages) * page))
        keys = [(pages[j // page], j % page) for j in range(max(0, length - window) if window else 0, length)]
        keys = [x for x in keys if 0 <= x[0] < P]
        if not keys:
            continue
        at = torch.tensor(keys)
        for h in range(q.shape[1]):
            k, v = (x[at[:, 0], at[:, 1], h // group] for x in (kp, vp))
            y = one(q[n, h][None], k, v, torch.ones(1, len(keys), dtype=torch.bool), d ** -0.5 if scale is None else scale, H)
            o[n, h], to[n, h] = y[0][0], y[2][0]
    return o, to


def plan(past, new, free, table, page, tokens):
    """The plan of lists of ints, one token at a time: (table, cu, lens, positions, slots, used)."""
    table = [list(row) for row in table]
    cu, lens, positions, slots, taken, count = [0], [], [], [], 0, 0
    for n, (p, x) in enumerate(zip(past, new)):
        p, x = max(0, p), max(0, x)
        held, want = -(-p // page), -(-(p + x) // page)
        for e in range(held, want):
            if e < len(table[n]):
                table[n][e] = free[taken] if taken < len(free) else -1
            taken += 1
        for t in range(p, p + x):
            e = t // page
            at = table[n][e] if e < len(table[n]) else -1
            positions.append(t)
            slots.append(at * page + t % page if at >= 0 else -1)
        count += x
        cu.append(min(count, tokens))
        lens.append(p + x)
    pad = max(0, tokens - count)
    return table, cu, lens, (positions + [0] * pad)[:tokens], (slots + [-1] * pad)[:tokens], [count, taken]
