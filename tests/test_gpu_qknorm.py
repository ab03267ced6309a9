"""GPU: the query/key norm with rotation (forward, gradient) against the plain
fp64 evaluation of its definition.

Tolerances.  The sum of d squares is off by at most d U of itself (halved by
the root), the root and divide by 4 U, the products and the rotation's two
terms by 4 U of (|a| + |b|): (d / 2 + 16) U (|a| + |b|) in all, plus half a
step of bf16.  The gradient adds the dot product over d: (d + 32) U of
r (|g w| + |x| r^2 sum |g w x| / m).
"""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, check, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32

CASES = [
    # B, T, hq, hk, d, rot, dtype, kind, weight, interleaved, positions
    (1, 1, 1, 1, 64, 0, BF, "l2", False, False, False),
    (1, 1, 4, 1, 128, 128, F, "rms", True, True, True),
    (2, 7, 6, 3, 128, 64, BF, "rms", True, False, True),
    (3, 33, 5, 2, 64, 16, BF, "l2", True, False, True),
    (1, 65, 3, 3, 256, 256, F, "rms", True, False, True),
    (1, 130, 17, 1, 128, 96, BF, "rms", False, True, False),
    (2, 31, 2, 1, 256, 48, BF, "l2", True, False, True),
    (1, 300, 48, 16, 64, 64, F, "l2", False, True, False),
]


def make(B, T, hq, hk, d, rot, dtype, weight, positions, seed=1, wide=False):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g).to(dtype)

    c = dict(q=r(B, T, hq, d), k=r(B, T, hk, d), doq=r(B, T, hq, d), dok=r(B, T, hk, d),
             wq=(1 + 0.3 * r(d).float()).to(dtype) if weight else None,
             wk=(1 + 0.3 * r(d).float()).to(dtype) if weight else None, cos=None, sin=None, pos=None)
    if rot:
        table = T + 40
        ang = torch.arange(table)[:, None].double() * 100.0 ** (-torch.arange(rot // 2).double() / (rot // 2))
        c["cos"], c["sin"] = ang.cos().float(), ang.sin().float()
        if positions:
            c["pos"] = torch.randint(0, table, (B, T), generator=g, dtype=torch.int32)
    dev = {k: None if v is None else v.cuda() for k, v in c.items()}
    if wide:   # q and k as columns of one projection
        both = torch.cat([dev["q"], dev["k"], dev["q"]], 2)
        dev["q"], dev["k"] = both[:, :, :hq], both[:, :, hq:hq + hk]
    dbl = {k: None if v is None else v.double() for k, v in c.items()}
    p = None if not rot else (c["pos"].long() if positions else torch.arange(T).repeat(B, 1))
    return dev, dbl, p


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("B,T,hq,hk,d,rot,dtype,kind,weight,inter,positions", CASES)
def test_norm_forward(B, T, hq, hk, d, rot, dtype, kind, weight, inter, positions, wide):
    import chunked_gated_delta_fwd_amd as gdr
    dv, c, p = make(B, T, hq, hk, d, rot, dtype, weight, positions, wide=wide)
    oq, ok = gdr.qk_norm_rope_fwd(dv["q"], dv["k"], dv["wq"], dv["wk"], dv["cos"], dv["sin"], dv["pos"], norm=kind,
                                  interleaved=inter)
    torch.cuda.synchronize()
    for got, x, w in ((oq, c["q"], c["wq"]), (ok, c["k"], c["wk"])):
        r = ref.norm_rope(x, w, c["cos"], c["sin"], p, kind == "rms", 1e-6, inter)
        n = ref.norm_rope(x, w, None, None, None, kind == "rms", 1e-6, inter).abs()
        size = n if not rot else n + n[..., pair(rot, d, inter)]
        check("norm", got, r, (d / 2 + 16) * U * size + (half_step(dtype) * r.abs() if dtype == BF else 0))


def pair(rot, d, inter):
    """Index of each channel's partner in the rotation."""
    i = torch.arange(d)
    j = torch.where(i % 2 == 0, i + 1, i - 1) if inter else (i + rot // 2) % rot
    return torch.where(i < rot, j, i)


@pytest.mark.parametrize("B,T,hq,hk,d,rot,dtype,kind,weight,inter,positions", CASES)
def test_norm_backward(B, T, hq, hk, d, rot, dtype, kind, weight, inter, positions):
    import chunked_gated_delta_fwd_amd as gdr
    dv, c, p = make(B, T, hq, hk, d, rot, dtype, weight, positions, seed=2)
    got = gdr.qk_norm_rope_bwd(dv["q"], dv["k"], dv["doq"], dv["dok"], dv["wq"], dv["wk"], dv["cos"], dv["sin"], dv["pos"],
                               norm=kind, interleaved=inter)
    torch.cuda.synchronize()
    for i, (x, w, do) in enumerate(((c["q"], c["wq"], c["doq"]), (c["k"], c["wk"], c["dok"]))):
        leaf = [x.clone().requires_grad_()] + ([w.clone().requires_grad_()] if weight else [])
        y = ref.norm_rope(leaf[0], leaf[1] if weight else None, c["cos"], c["sin"], p, kind == "rms", 1e-6, inter)
        rg = torch.autograd.grad(y, leaf, do)
        g = do.abs() if not rot else do.abs() + do.abs()[..., pair(rot, d, inter)]   # |R^T do| <=
        m = d if kind == "rms" else 1
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / m + 1e-6)
        gw = g * (w.abs() if weight else 1)
        size = r * (gw + x.abs() * r * r * (gw * x.abs()).sum(-1, keepdim=True) / m)
        check("dx", got[i], rg[0], (d + 32) * U * size + (half_step(dtype) * rg[0].abs() if dtype == BF else 0))
        if weight:
            terms = (g * x.abs() * r).sum((0, 1, 2))
            check("dw", got[2 + i], rg[1], (d / 2 + 16 + 128) * U * terms)
        else:
            assert got[2 + i] is None


def test_norm_backward_differences():
    import chunked_gated_delta_fwd_amd as gdr
    dv, c, p = make(1, 9, 2, 1, 64, 32, F, True, True, seed=3)
    got = [t.double().cpu() for t in gdr.qk_norm_rope_bwd(dv["q"], dv["k"], dv["doq"], dv["dok"], dv["wq"], dv["wk"],
                                                           dv["cos"], dv["sin"], dv["pos"])]

    def loss(q, w):
        return (ref.norm_rope(q, w, c["cos"], c["sin"], p, True, 1e-6, False) * c["doq"]).sum().item()

    for i, (grad, base) in enumerate(((got[0], c["q"]), (got[2], c["wq"]))):
        v = torch.randn(base.shape, dtype=torch.double, generator=torch.Generator().manual_seed(i))
        at = [c["q"], c["wq"]]
        up, dn = list(at), list(at)
        up[i], dn[i] = base + 1e-5 * v, base - 1e-5 * v
        diff = (loss(*up) - loss(*dn)) / 2e-5
        assert abs(diff - (grad * v).sum().item()) <= (200 * U + 1e-6) * (grad * v).abs().sum().item()


def test_norm_rows_without_values():
    """Zero rows give zeros (eps keeps the root finite), a NaN row stays alone, repeats are bit-identical."""
    import chunked_gated_delta_fwd_amd as gdr
    dv, _, _ = make(1, 20, 4, 2, 128, 64, F, True, True, seed=4)
    dv["q"][0, 3, 1] = 0
    dv["q"][0, 4, 2, 7] = float("nan")
    args = (dv["wq"], dv["wk"], dv["cos"], dv["sin"], dv["pos"])
    oq, ok = gdr.qk_norm_rope_fwd(dv["q"], dv["k"], *args)
    assert (oq[0, 3, 1] == 0).all() and torch.isnan(oq[0, 4, 2]).all()
    assert int(torch.isnan(oq).sum()) == 128 and torch.isfinite(ok).all()
    dv["q"][0, 4, 2, 7] = 0.5
    a = gdr.qk_norm_rope_bwd(dv["q"], dv["k"], dv["doq"], dv["dok"], *args)
    b = gdr.qk_norm_rope_bwd(dv["q"], dv["k"], dv["doq"], dv["dok"], *args)
    assert all(torch.equal(s, t) and torch.isfinite(s).all() for s, t in zip(a, b))


def test_norm_positions_outside_the_table_stay_inside():
    import chunked_gated_delta_fwd_amd as gdr
    dv, _, _ = make(1, 8, 1, 1, 64, 64, F, False, True, seed=5)
    near = dv["pos"].clone()
    dv["pos"][0, 0], dv["pos"][0, 1] = -7, 10 ** 9
    near[0, 0], near[0, 1] = 0, dv["cos"].shape[0] - 1
    a = gdr.qk_norm_rope_fwd(dv["q"], dv["k"], None, None, dv["cos"], dv["sin"], dv["pos"])
    b = gdr.qk_norm_rope_fwd(dv["q"], dv["k"], None, None, dv["cos"], dv["sin"], near)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_outputs():
    """Outputs that are stored past the caches have the bits of their rows computed alone."""
    import chunked_gated_delta_fwd_amd as gdr
    g = torch.Generator(device="cuda").manual_seed(22)
    for dtype, hq in ((torch.bfloat16, 28), (torch.float32, 12)):
        q = torch.randn(2, 8192, hq, 128, generator=g, device="cuda").to(dtype)
        k = torch.randn(2, 8192, 4, 128, generator=g, device="cuda").to(dtype)
        cos, sin = torch.randn(2, 8192, 32, generator=g, device="cuda")
        wq = torch.randn(128, generator=g, device="cuda").to(dtype)
        oq, ok = gdr.qk_norm_rope_fwd(q, k, wq, None, cos, sin)
        assert (oq.numel() + ok.numel()) * oq.element_size() >= 1 << 27
        dq, dk, _, _ = gdr.qk_norm_rope_bwd(q, k, oq, ok, wq, None, cos, sin)
        for i in range(2):
            s = slice(i, i + 1)
            a, b = gdr.qk_norm_rope_fwd(q[s], k[s], wq, None, cos, sin)
            assert torch.equal(a[0], oq[i]) and torch.equal(b[0], ok[i])
            a, b, _, _ = gdr.qk_norm_rope_bwd(q[s], k[s], oq[s], ok[s], wq, None, cos, sin)
            assert torch.equal(a[0], dq[i]) and torch.equal(b[0], dk[i])
