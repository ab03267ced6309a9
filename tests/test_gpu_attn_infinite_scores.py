"""GPU: the gradient of attention where every score of a row is -inf.  Such a
row counts as one that sees no key (o 0, lse -inf): it puts nothing on dk and dv,
and its dq is zero where the keys are finite."""
import pytest
import torch

from test_gpu_attn import BF, F, ints, make, sound

pytestmark = pytest.mark.gpu

SHAPES = [   # lengths, hq, hk, d, dtype, causal, window
    ([1], 1, 1, 64, BF, True, 0),
    ([40], 2, 1, 64, BF, False, 0),
    ([33, 0, 128], 4, 2, 128, BF, True, 0),        # few keys: delta from the sum of ds
    ([300], 2, 1, 128, BF, True, 0),
    ([300], 2, 1, 64, BF, True, 40),
    ([40], 2, 1, 64, F, True, 0),
    ([33, 129], 2, 2, 128, F, False, 0),
    ([900], 2, 1, 128, F, True, 0),                # blocks are shared
    ([1100], 2, 1, 64, BF, False, 0),
]


def gradients(x, cu, **kw):
    import chunked_gated_delta_fwd_amd as gdr
    o, lse = gdr.attn_fwd(x["q"], x["k"], x["v"], cu, **kw)
    return o, lse, gdr.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], cu, **kw)


def rows_of(lens):
    """The first, a middle and the last row of every sequence."""
    start, rows = 0, []
    for n in lens:
        rows += sorted({start, start + n // 2, start + n - 1}) if n else []
        start += n
    return rows


@pytest.mark.parametrize("scale", [None, -0.1])
@pytest.mark.parametrize("lens,hq,hk,d,dtype,causal,window", SHAPES)
def test_products_that_overflow(lens, hq, hk, d, dtype, causal, window, scale):
    """Finite q and k whose products are all below fp32's lowest value.  The other rows' scores do not hold the channel,
    and a row with q and do of zero puts exact zeros on every gradient: all are the same as with such rows, from the same o
    and lse of the others (a wave's rows move their reference values together, so that a forward's last bits hang on
    neighbouring rows)."""
    import chunked_gated_delta_fwd_amd as gdr
    T, rows = sum(lens), rows_of(lens)
    dev, _ = make(1, T, T, hq, hk, d, dtype, seed=51)
    cu = ints([sum(lens[:i]) for i in range(len(lens) + 1)])
    dev["q"][..., 0] = 0
    dev["k"][..., 0] = 1e20 if scale else -1e20
    low, none = dict(dev, q=dev["q"].clone()), dict(dev, q=dev["q"].clone(), do=dev["do"].clone())
    low["q"][:, rows, :, 0] = 1e30
    kw = dict(causal=causal, window=window, scale=scale)
    o, lse, got = gradients(low, cu, **kw)
    assert (lse[:, rows] == -torch.inf).all() and not o[:, rows].any()
    for x in (none["q"], none["do"], lse):
        x[:, rows] = 0
    want = gdr.attn_bwd(none["q"], dev["k"], dev["v"], o, lse, none["do"], cu, **kw)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        assert sound(a).all(), name
        assert torch.equal(a, b), name
    assert not got[0][:, rows].any()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,d", [(1, 64), (40, 128), (300, 64), (300, 128)])
def test_a_first_row_that_sees_a_key_of_infinity_alone(T, d, dtype):
    """Causal: row 0 sees key 0 alone, whose scores are -inf, the others see it among finite ones.  dk and dv are those of a
    key whose probabilities vanish in fp32 (e^-884 and less) and a row 0 without do."""
    dev, _ = make(1, T, T, 2, 1, d, dtype, seed=52)
    dev["q"][..., 0] = 1.0
    x = dict(dev, k=dev["k"].clone())
    x["k"][0, 0, 0, 0] = -float("inf")
    o, lse, (_, dk, dv) = gradients(x, None)
    assert (lse[0, 0] == -torch.inf).all() and not o[0, 0].any()
    assert sound(o).all() and sound(lse[:, 1:]).all() and sound(dk).all() and sound(dv).all()
    assert not dk[0, 0].any() and not dv[0, 0].any()
    x = dict(dev, k=dev["k"].clone(), do=dev["do"].clone())
    x["k"][0, 0, 0, 0] = -1e4
    x["do"][0, 0] = 0
    o2, lse2, (_, dk2, dv2) = gradients(x, None)
    for a, b in ((o[:, 1:], o2[:, 1:]), (lse[:, 1:], lse2[:, 1:]), (dk, dk2), (dv, dv2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [BF, F])
def test_scores_of_2_to_the_28(dtype, sign):
    """Exact and all alike, so that o is the mean of the values that are seen, by the forward and by one token over pages.
    Tolerance: sums of n terms, (n + 16) 2^-24 of the mean |v| for the sums and the quotient, half a step of bf16 for each
    probability and for o; lse is rounded to fp32 twice (2^-23 of it)."""
    import chunked_gated_delta_fwd_amd as gdr
    n, d = 300, 64
    g = torch.Generator().manual_seed(53)
    q, k = torch.zeros(1, n, 2, d), torch.zeros(1, n, 1, d)
    q[..., 0], k[..., 0] = 2.0 ** 17, sign * 2.0 ** 14
    v = torch.randn(1, n, 1, d, generator=g).to(dtype)
    q, k = q.to(dtype).cuda(), k.to(dtype).cuda()
    o, lse = gdr.attn_fwd(q, k, v.cuda())
    count = torch.arange(1, n + 1).double()[None, :, None, None]
    mean, size = (x.double().cumsum(1) / count for x in (v, v.abs()))
    H = 2.0 ** -8 if dtype == BF else 0.0
    tol = (H + (n + 16) * 2.0 ** -24) * size + H * mean.abs()
    assert ((o.double().cpu() - mean).abs() <= tol).all()
    assert (lse.double().cpu() - (sign * 2.0 ** 28 + count[..., 0].log())).abs().max() <= 2.0 ** -23 * 2.0 ** 28
    kp, vp = (torch.zeros(3, 100, 1, d, dtype=dtype, device="cuda") for _ in range(2))
    gdr.page_store(k, v.cuda(), torch.arange(n, device="cuda").int(), kp, vp)
    got = gdr.attn_paged_step(q[:, -1], kp, vp, ints([[0, 1, 2]]), ints([n]))
    assert ((got.double().cpu() - mean[:, -1]).abs() <= tol[:, -1]).all()
