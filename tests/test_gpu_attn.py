"""GPU: softmax attention and its gradient against the plain fp64 evaluation of
their definitions (attn_ref.py derives the tolerances)."""
import pytest
import torch

import attn_ref as ref
from mixer_ref import check

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32

# lengths of queries, of keys (None: the same), hq, hk, d, dtype, causal, window
PACKED = [
    ([1], None, 1, 1, 64, BF, True, 0),
    ([1, 0, 2, 0], None, 2, 1, 128, F, True, 0),
    ([31, 32, 33], None, 3, 3, 64, BF, False, 0),
    ([127, 0, 128, 129], None, 4, 2, 128, BF, True, 0),
    ([65, 300], None, 7, 1, 64, F, True, 0),
    ([200, 1, 77], None, 6, 2, 128, BF, True, 1),
    ([260, 0, 0, 140], None, 2, 2, 64, BF, True, 64),
    ([150, 131], None, 2, 1, 128, F, True, 33),
    ([5, 64, 3], [90, 200, 3], 4, 1, 128, BF, True, 0),
    ([1, 1, 1], [1, 70, 257], 8, 2, 64, F, True, 0),
    ([140, 9, 20], [13, 0, 19], 2, 1, 64, BF, True, 0),       # the first queries see no key
    ([100, 40], [30, 50], 3, 1, 128, F, True, 7),
    ([0, 6], [50, 40], 2, 2, 64, BF, False, 0),               # keys that no query sees
    ([33, 257], [129, 66], 2, 1, 128, BF, False, 0),
]
ROWS = [   # B, Tq, Tk, hq, hk, d, dtype, causal, window
    (3, 96, 96, 4, 4, 64, BF, True, 0),
    (2, 129, 129, 5, 1, 128, F, False, 0),
    (8, 70, 70, 2, 1, 128, BF, True, 16),
    (5, 1, 190, 6, 3, 64, BF, True, 0),
    (2, 40, 10, 2, 1, 64, F, True, 0),
    (3, 33, 0, 2, 1, 64, BF, True, 0),
]


def offsets(lens):
    return None if lens is None else [sum(lens[:i]) for i in range(len(lens) + 1)]


def make(B, Tq, Tk, hq, hk, d, dtype, seed=1, wide=False):
    """q, k, v, do on the GPU and as doubles; wide: q, k and v are columns of a wider projection."""
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g).to(dtype)

    c = dict(q=r(B, Tq, hq, d) * 2, k=r(B, Tk, hk, d), v=r(B, Tk, hk, d), do=r(B, Tq, hq, d))
    dev = {n: x.cuda() for n, x in c.items()}
    if wide:
        for n in ("q", "k", "v", "do"):
            x = dev[n]
            dev[n] = torch.cat([x.new_full(x.shape[:2] + (1, d), torch.nan), x, x.new_full(x.shape[:2] + (2, d), torch.nan)],
                               2)[:, :, 1:1 + x.shape[2]]
    return dev, {n: x.double() for n, x in c.items()}


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def run(dev, dbl, cu, cuk, dtype, scale=None, **kw):
    """Forward and gradient, checked; rows outside every sequence keep what the outputs held."""
    import chunked_gated_delta_fwd_amd as gdr
    C, CK = ints(cu), ints(cuk)
    o0, l0 = torch.full_like(dev["q"].contiguous(), 7), torch.full(dev["q"].shape[:3], 7.0, device="cuda")
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], C, CK, scale=scale, o=o0, lse=l0, **kw)
    torch.cuda.synchronize()
    ro, rl, to, tl = ref.attention(dbl["q"], dbl["k"], dbl["v"], cu, cuk, scale=scale, dtype=dtype, **kw)


    def held(r, t):
        return torch.where(r.isnan(), 7.0, r), torch.where(r.isnan(), 0.0, t)

    check("o", o, *held(ro, to))
    empty = rl == -torch.inf
    assert torch.equal(lse.cpu() == -torch.inf, empty)
    check("lse", lse.cpu().masked_fill(empty, 0), *held(rl.masked_fill(empty, 0), tl))
    # the gradient from o and lse as the definition gives them, rounded to what the forward stores
    gave = ro.nan_to_num().to(dtype).cuda(), rl.nan_to_num(neginf=-torch.inf).float().cuda()
    if not dev["q"].is_contiguous():   # o as rows of something wider too
        gave = torch.cat([gave[0], gave[0]], 2)[:, :, :gave[0].shape[2]], gave[1]
    outs = [torch.full_like(dev[n].contiguous(), 7) for n in ("q", "k", "v")]
    grads = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], *gave, dev["do"], C, CK, scale=scale, dq=outs[0], dk=outs[1],
                         dv=outs[2], **kw)
    torch.cuda.synchronize()
    rg, tg = ref.gradient(dbl["q"], dbl["k"], dbl["v"], dbl["do"], cu, cuk, scale=scale, dtype=dtype, **kw)
    for name, got, r, t in zip(("dq", "dk", "dv"), grads, rg, tg):
        check(name, got, *held(r, t))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", PACKED)
def test_packed(lq, lk, hq, hk, d, dtype, causal, window, wide):
    tail = 3 if wide else 0   # tokens behind the last sequence
    dev, dbl = make(1, sum(lq) + tail, sum(lk or lq) + tail, hq, hk, d, dtype, wide=wide)
    run(dev, dbl, offsets(lq), offsets(lk), dtype, causal=causal, window=window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("B,Tq,Tk,hq,hk,d,dtype,causal,window", ROWS)
def test_rows(B, Tq, Tk, hq, hk, d, dtype, causal, window, wide):
    dev, dbl = make(B, Tq, Tk, hq, hk, d, dtype, seed=2, wide=wide)
    run(dev, dbl, None, None, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", [BF, F])
def test_every_type_and_width_with_a_longer_row(dtype):
    for d in (64, 128):
        dev, dbl = make(1, 700, 700, 2, 1, d, dtype, seed=3)
        run(dev, dbl, None, None, dtype)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (4, 4), (8, 8), (16, 16), (6, 3), (40, 5)])
def test_blocks_of_every_head_count(hq, hk):
    """Blocks are spread over the XCDs by the number of key heads: dividing 8, divided by it, neither."""
    dev, dbl = make(1, 290, 290, hq, hk, 64, BF, seed=4)
    run(dev, dbl, [0, 130, 131, 290], None, BF)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-6, 3.0])
def test_scales(scale):
    for dtype in (BF, F):
        dev, dbl = make(1, 150, 150, 2, 1, 64, dtype, seed=5)
        run(dev, dbl, [0, 150], None, dtype, scale=scale)


def test_many_sequences():
    """More sequences than a wave has lanes, and empty ones among them."""
    lens = [(7 * i) % 5 for i in range(300)]
    dev, dbl = make(1, sum(lens), sum(lens), 2, 1, 64, BF, seed=6)
    run(dev, dbl, offsets(lens), None, BF)


def test_growing_scores():
    """Every key's score is above the last one's: the running maximum changes in every tile."""
    dev, dbl = make(1, 400, 400, 1, 1, 64, F, seed=7)
    up = torch.linspace(-30, 30, 400)
    for x in (dev, dbl):
        x["q"][:] = 0
        x["q"][..., 0] = 8
        x["k"][0, :, 0, 0] = up.to(x["k"])
    dbl["k"][0, :, 0, 0] = up.float().double()
    run(dev, dbl, None, None, F, causal=False)


@pytest.mark.parametrize("lens,window,d", [([2, 3, 9, 30], 0, 64), ([150, 180], 2, 128), ([192], 0, 64), ([500], 40, 128)])
def test_few_keys_do_not_carry_the_rounding_of_o(lens, window, d):
    """Where a block sees at most 192 keys, dq and dk carry the rounding of ds and their own, and not o's."""
    import chunked_gated_delta_fwd_amd as gdr
    T = sum(lens)
    dev, dbl = make(1, T, T, 4, 2, d, BF, seed=20)
    cu = offsets(lens)
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), window=window)
    grads = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints(cu), window=window)
    rg, tg = ref.gradient(*(dbl[n] for n in ("q", "k", "v", "do")), cu, window=window, dtype=BF, few=True)
    for name, got, r, t in zip(("dq", "dk", "dv"), grads, rg, tg):
        check(name, got, r, t)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 20)])
def test_gradient_against_differences(causal, window):
    """<gradient, u> against central differences of the plain forward along u.  The differences are off by h^2 times
    the third derivative: with h = 1e-4 in fp64, far below the fp32 kernel's own tolerance."""
    import chunked_gated_delta_fwd_amd as gdr
    dev, dbl = make(1, 90, 90, 2, 1, 64, F, seed=8)
    cu = [0, 37, 90]
    kw = dict(causal=causal, window=window)
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), **kw)
    grads = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints(cu), **kw)
    _, tol = ref.gradient(*(dbl[n] for n in ("q", "k", "v", "do")), cu, **kw)
    g = torch.Generator().manual_seed(9)
    for name, grad, t in zip(("q", "k", "v"), grads, tol):
        u = torch.randn(dbl[name].shape, generator=g).double()
        loss = []
        for h in (1e-4, -1e-4):
            x = dict(dbl, **{name: dbl[name] + h * u})
            loss.append((ref.attention(x["q"], x["k"], x["v"], cu, **kw)[0] * dbl["do"]).sum())
        want = (loss[0] - loss[1]) / 2e-4
        allowed = (t * u.abs()).sum() + 1e-6 * want.abs() + 1e-6
        assert (grad.double().cpu() * u).sum().sub(want).abs() <= allowed, name


def bits(x):
    return x.contiguous().view(torch.int16 if x.dtype == BF else torch.int32)


@pytest.mark.parametrize("dtype", [BF, F])
def test_repeated_calls_give_the_same_bits(dtype):
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 900, 900, 8, 1, 64, dtype, seed=10)
    cu = ints([0, 333, 900])
    first = None
    for _ in range(3):
        o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], cu)
        got = [o, lse] + list(gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], cu))
        first = first or [x.clone() for x in got]
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(first, got))


def sound(x):
    return torch.isfinite(x.float())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("window", [0, 40])
def test_values_that_are_not_finite_reach_who_sees_them(dtype, value, window):
    """A key, a value, a query and an output gradient that are not finite: every row that does not see them is what it is
    without them, and the rows that do see a NaN are not finite.  What lies behind the last sequence reaches nobody."""
    import chunked_gated_delta_fwd_amd as gdr
    T, cu, at = 330, [0, 150, 300], 210
    dev, dbl = make(1, T, T, 2, 1, 64, dtype, seed=11)
    for n in dev:
        dev[n][:, 300:] = float("nan")
    kw = dict(window=window)

    def both(**x):
        x = dict(dev, **x)
        o, lse = gdr.attn_fwd(x["q"], x["k"], x["v"], ints(cu), o=torch.zeros_like(dev["q"]), lse=torch.zeros(1, T, 2, device="cuda"), **kw)
        z = [torch.zeros_like(dev[n]) for n in "qkv"]
        g = gdr.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], ints(cu), dq=z[0], dk=z[1], dv=z[2], **kw)
        return [o, lse[..., None]] + list(g)

    ro, rl, to, tl = ref.attention(dbl["q"], dbl["k"], dbl["v"], cu, dtype=dtype, **kw)
    rg, tg = ref.gradient(*(dbl[n] for n in ("q", "k", "v", "do")), cu, dtype=dtype, **kw)
    clean = [(x.nan_to_num(), t.nan_to_num()) for x, t in zip([ro, rl[..., None]] + rg, [to, tl[..., None]] + tg)]
    for what, a, (r, t) in zip(("o", "lse", "dq", "dk", "dv"), both(), clean):
        check("clean " + what, a, r, t)
    i = torch.arange(T, device="cuda")
    sees = (i >= at) & (i < 300) & (i - at < (window or T))          # queries that see key `at`
    seen = (i <= at) & (i >= 150) & (at - i < (window or T))         # keys that query `at` sees
    linked = torch.zeros(T, dtype=torch.bool, device="cuda")         # keys that share a query with key `at`
    for row in range(at, 300):
        if sees[row]:
            linked |= (i <= row) & (i >= 150) & (row - i < (window or T))
    none = torch.zeros_like(sees)
    touched = dict(k=(sees, sees, sees, linked, linked), v=(sees, none, sees, linked, none),
                   q=(i == at, i == at, i == at, seen, seen), do=(none, none, i == at, seen, seen))
    for name, rows in touched.items():
        x = dev[name].clone()
        x[0, at, :, 5] = value
        got = both(**{name: x})
        for what, a, (b, t), r in zip(("o", "lse", "dq", "dk", "dv"), got, clean, rows):
            there = ~r.cpu()
            check("%s, beside a %s" % (what, name), a[0, ~r], b[0, there], t[0, there])
            if value != value:   # a NaN is not swallowed
                assert not sound(a[0, r]).all(-1).any(), (name, what)


@pytest.mark.parametrize("lq", [1, 33, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_key_of_infinity_that_nothing_is_put_on(dtype, d, lq):
    """Scores of -inf are probabilities of 0, and gradients of 0 for that key, in tiles that the queries end in too: dk and dv
    are what a score far below the others gives, to the bit."""
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, lq, 40, 2, 1, d, dtype, seed=17)
    dev["q"][..., 0] = 1.0
    got = []
    for value in (-1e30, -float("inf")):
        k = dev["k"].clone()
        k[0, 7, 0, 0] = value
        o, lse = gdr.attn_fwd(dev["q"], k, dev["v"], causal=False)
        dq, dk, dv = gdr.attn_bwd(dev["q"], k, dev["v"], o, lse, dev["do"], causal=False)
        assert all(sound(x).all() for x in (o, lse, dk, dv))
        assert not dk[0, 7].any() and not dv[0, 7].any()
        got.append([bits(x) for x in (o, lse, dk, dv)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_offsets_that_break_the_rules_stay_inside():
    """Whatever cu_seqlens holds, nothing outside the tensors is touched (guards around every output keep their bytes)."""
    import chunked_gated_delta_fwd_amd as gdr
    T, hq, d = 300, 2, 64
    dev, _ = make(1, T, T, hq, 1, d, BF, seed=12)
    for cu in ([0, -5, 400, 300], [50, 20, 10, 0], [2 ** 31 - 1, -2 ** 31, 7, 2 ** 31 - 1], [-9, -8, -7, -6], [299, 300, 301, 302],
               [0, 300, 0, 300]):
        pads = [torch.full((3,) + tuple(dev[n].shape[1:]), 7, dtype=BF, device="cuda") for n in ("q", "q", "k", "v")]
        outs = [p[1:2] for p in pads]
        lse = torch.full((3, T, hq), 7.0, device="cuda")
        gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), ints(cu[::-1]), o=outs[0], lse=lse[1:2])
        gdr.attn_bwd(dev["q"], dev["k"], dev["v"], outs[0], lse[1:2], dev["do"], ints(cu), ints(cu[::-1]), dq=outs[1],
                     dk=outs[2], dv=outs[3])
        torch.cuda.synchronize()
        for p in pads + [lse]:
            assert (p[0] == 7).all() and (p[2] == 7).all(), cu


def test_without_a_sequence():
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 50, 50, 2, 1, 64, BF, seed=13)
    o, lse = torch.full_like(dev["q"], 7), torch.full((1, 50, 2), 7.0, device="cuda")
    gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints([0]), o=o, lse=lse)
    outs = [torch.full_like(dev[n], 7) for n in "qkv"]
    gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints([0]), dq=outs[0], dk=outs[1], dv=outs[2])
    assert all((x == 7).all() for x in [o, lse] + outs)
    none = dev["q"][:0]
    assert gdr.attn_fwd(none, dev["k"][:0], dev["v"][:0])[0].shape == none.shape
    gdr.attn_fwd(dev["q"][:, :0], dev["k"], dev["v"])


def test_lse_is_optional():
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 50, 50, 2, 1, 64, BF, seed=13)
    a, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"])
    b, none = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], output_lse=False)
    assert none is None and torch.equal(a, b) and lse.dtype == F


def test_graph_on_another_stream():
    """Forward and gradient captured on a stream of their own and replayed, with eager calls of other sizes between."""
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 260, 260, 4, 1, 64, BF, seed=14)
    other, _ = make(2, 300, 300, 8, 2, 128, BF, seed=15)
    cu = ints([0, 100, 260])

    def call(x, c):
        o, lse = gdr.attn_fwd(x["q"], x["k"], x["v"], c)
        return [o, lse] + list(gdr.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], c))

    want = [x.clone() for x in call(dev, cu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(dev, cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(dev, cu)
    for _ in range(4):
        for x in got:
            x.zero_()
        eager = call(other, None)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
        assert all(sound(x).all() for x in eager)


def test_two_graphs_that_share_memory():
    """Calls whose blocks are shared and joined, captured in two graphs of one memory pool and replayed in turn: neither reads
    what the other left."""
    import chunked_gated_delta_fwd_amd as gdr
    sets = [make(1, tq, tk, 2, 1, d, BF, seed=41)[0] for tq, tk, d in ((600, 600, 128), (40, 3000, 64))]

    def call(x):
        o, lse = gdr.attn_fwd(x["q"], x["k"], x["v"])
        return [o, lse] + list(gdr.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"]))

    want = [[x.clone() for x in call(x)] for x in sets]
    torch.cuda.synchronize()
    pool, graphs, got = torch.cuda.graph_pool_handle(), [], []
    for x in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            got.append(call(x))
    for _ in range(3):
        for graph, a, b in zip(graphs, got, want):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(bits(y), bits(z)) for y, z in zip(a, b))


def test_calls_on_two_streams():
    """The library's workspace is handed from one stream's call to the other's in order."""
    import chunked_gated_delta_fwd_amd as gdr
    sets = [make(1, 700, 700, 8, 1, 128, BF, seed=s)[0] for s in (21, 22)]

    def call(x):
        o, lse = gdr.attn_fwd(x["q"], x["k"], x["v"])
        return [o, lse] + list(gdr.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"]))

    want = [call(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(call(x))
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        for run_ in runs:
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(run_, w))


def test_few_queries_over_many_keys():
    """The keys are split in runs (one of them without a key that a row sees) and joined, NaN and all."""
    import chunked_gated_delta_fwd_amd as gdr
    for dtype in (BF, F):
        for cu, cuk, kw in (([0, 5, 6], [0, 3000, 3900], dict()), (None, None, dict(causal=False)), ([0, 0, 64], [0, 100, 2600], dict(window=900))):
            Tq, Tk = (cu[-1], cuk[-1]) if cu else (9, 4000)
            dev, dbl = make(1, Tq, Tk, 4, 2, 64, dtype, seed=23)
            o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), ints(cuk), **kw)
            ro, rl, to, tl = ref.attention(dbl["q"], dbl["k"], dbl["v"], cu, cuk, dtype=dtype, **kw)
            check("o", o, ro, to)
            check("lse", lse, rl, tl)
            v = dev["v"].clone()
            v[0, Tk - 1, 0, 3] = float("nan")            # seen by the last row alone where causal
            bad, _ = gdr.attn_fwd(dev["q"], dev["k"], v, ints(cu), ints(cuk), **kw)
            rows = slice(Tq - 1, Tq) if kw.get("causal", True) else slice(0, Tq)
            assert not torch.isfinite(bad[0, rows, :2, 3]).any()
            bad[0, rows, :2, 3] = o[0, rows, :2, 3]
            check("o beside a NaN", bad, ro, to)


LAST = [   # lengths of queries, of keys, hq, hk, d, dtype, causal: some more blocks of one length than the chip holds at once
    ([3451], [1500], 20, 5, 128, BF, False),
    ([1111, 1, 2300, 788], [600, 0, 600, 600], 8, 2, 64, F, False),
    ([2176, 2176], [9000, 9001], 24, 8, 64, BF, True),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal", LAST)
def test_keys_of_the_last_blocks_alone_are_split(lq, lk, hq, hk, d, dtype, causal):
    """Where some blocks are left when the chip was full: on one head of each group (the reference's time), o and lse."""
    import chunked_gated_delta_fwd_amd as gdr
    cu, cuk = offsets(lq), offsets(lk)
    dev, dbl = make(1, cu[-1], cuk[-1], hq, hk, d, dtype, seed=29)
    dev["v"][0, -1, 0, 3] = dbl["v"][0, -1, 0, 3] = 0.0
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), ints(cuk), causal=causal)
    heads = [g * (hq // hk) + g % (hq // hk) for g in range(hk)]
    for g, h in list(enumerate(heads))[::3]:
        ro, rl, to, tl = ref.attention(dbl["q"][:, :, h:h + 1], dbl["k"][:, :, g:g + 1], dbl["v"][:, :, g:g + 1], cu, cuk,
                                       causal=causal, dtype=dtype)
        check("o", o[:, :, h:h + 1], ro, to)
        none = rl == -torch.inf                          # a sequence without keys
        got = lse[:, :, h:h + 1].cpu()
        assert torch.equal(got == -torch.inf, none)
        check("lse", got[~none], rl[~none], tl[~none])
    # every other head: the same rows in a call of its own, whose blocks are split otherwise
    for h in range(hq):
        g = h // (hq // hk)
        alone, _ = gdr.attn_fwd(dev["q"][:, :, h:h + 1].contiguous(), dev["k"][:, :, g:g + 1].contiguous(),
                                dev["v"][:, :, g:g + 1].contiguous(), ints(cu), ints(cuk), causal=causal)
        # each within its tolerance of the value, with the largest |v| for the sums of p |v| and of o, and 30 for those of
        # scale |q k|, whose mean is 15 at most
        H, U = (2.0 ** -8 if dtype == BF else 0.0), 2.0 ** -24
        E = 2 * (d + 12) * U * 30 + 8 * U * (1 + 30)
        assert ((o[:, :, h:h + 1] - alone).float().abs() <= 2 * (2 * H + E + (max(lk) + 20) * U) * 6).all()
    bad = dev["v"].clone()
    bad[0, -1, 0, 3] = float("nan")                      # the last sequence's last key: its rows, of the first group's heads
    got, _ = gdr.attn_fwd(dev["q"], dev["k"], bad, ints(cu), ints(cuk), causal=causal)
    rows = slice(cu[-1] - 1, cu[-1]) if causal else slice(cu[-2], cu[-1])
    assert not torch.isfinite(got[0, rows, :hq // hk, 3]).any()
    got[0, rows, :hq // hk, 3] = o[0, rows, :hq // hk, 3]
    assert sound(got).all()


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", [
    ([900], None, 2, 1, 128, F, True, 0),
    ([1300], None, 3, 3, 64, F, True, 300),
    ([700, 0, 1200], None, 4, 2, 64, BF, True, 0),
    ([1500], None, 2, 1, 128, BF, False, 0),
    ([200, 900], [1900, 900], 2, 2, 128, BF, True, 0),
    ([1025], [70], 2, 1, 64, BF, False, 0),             # many queries over few keys
])
def test_gradients_of_few_blocks(lq, lk, hq, hk, d, dtype, causal, window):
    """Runs of a block's queries, or of its keys, in blocks of their own, joined in order; behind the last sequence nothing is
    written."""
    import chunked_gated_delta_fwd_amd as gdr
    cu, cuk = offsets(lq), offsets(lk)
    Tq, Tk = cu[-1] + 9, (cuk or cu)[-1] + 9
    dev, dbl = make(1, Tq, Tk, hq, hk, d, dtype, seed=31)
    kw = dict(causal=causal, window=window)
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), ints(cuk), **kw)
    full = [torch.full_like(dev[n], 7.0) for n in "qkv"]
    got = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints(cu), ints(cuk), dq=full[0], dk=full[1], dv=full[2], **kw)
    rg, tg = ref.gradient(*(dbl[n] for n in ("q", "k", "v", "do")), cu, cuk, dtype=dtype, **kw)
    for name, a, r, t, end in zip(("dq", "dk", "dv"), got, rg, tg, (cu[-1], (cuk or cu)[-1], (cuk or cu)[-1])):
        check(name, a[:, :end], r[:, :end], t[:, :end])
        assert (a[:, end:] == 7.0).all()
    again = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints(cu), ints(cuk), **kw)
    assert all(torch.equal(bits(a[:, :end]), bits(b[:, :end])) for a, b, end in
               zip(got, again, (cu[-1], (cuk or cu)[-1], (cuk or cu)[-1])))


def test_rows_far_apart():
    """Keys 4 MiB apart: their places pass 2^31 bytes within one sequence."""
    import chunked_gated_delta_fwd_amd as gdr
    T, d, wide = 700, 64, 1 << 21
    dev, dbl = make(1, T, T, 1, 1, d, BF, seed=16)
    far = torch.empty(1, T, wide, dtype=BF, device="cuda")
    k, v = far[:, :, :d].unflatten(-1, (1, d)), far[:, :, wide - d:].unflatten(-1, (1, d))
    k.copy_(dev["k"])
    v.copy_(dev["v"])
    dev.update(k=k, v=v)
    run(dev, dbl, None, None, BF)


def test_content_check():
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 40, 60, 2, 1, 64, BF, seed=17)
    gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 1)
    try:
        gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints([0, 40]), ints([0, 60]))
        with pytest.raises(gdr.GdrError, match="must equal the 40 tokens"):
            gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints([0, 41]), ints([0, 60]))
        with pytest.raises(gdr.GdrError, match="must equal the 60 tokens"):
            gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints([0, 40]), ints([0, 50]))
    finally:
        gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 0)


def test_failed_launch_reports():
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 40, 40, 2, 1, 64, BF, seed=18)
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"])
    for call in (lambda: gdr.attn_fwd(dev["q"], dev["k"], dev["v"]),
                 lambda: gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"])):
        gdr.debug_set(gdr.GDR_DEBUG_FAIL_LAUNCHES, 1)
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.status == -7
        call()


@pytest.mark.parametrize("what,text", [
    (dict(cu_seqlens=lambda: torch.tensor([0, 20], dtype=torch.int64, device="cuda")), "unsupported dtype"),
    (dict(cu_seqlens=lambda: torch.tensor([0, 20], dtype=torch.int32)), "one GPU"),
    (dict(cu_seqlens=lambda: torch.zeros(0, dtype=torch.int32, device="cuda")), "at least one offset"),
    (dict(cu_seqlens_k=lambda: ints([0, 20])), "cu_seqlens_k without"),
    (dict(cu_seqlens=lambda: ints([0, 20]), cu_seqlens_k=lambda: ints([0, 1, 20])), "cu_seqlens_k: shape"),
    (dict(window=lambda: -1), "window"),
    (dict(window=lambda: 5, causal=lambda: False), "window needs causal"),
    (dict(scale=lambda: float("inf")), "scale"),
])
def test_refusals(what, text):
    import chunked_gated_delta_fwd_amd as gdr
    dev, _ = make(1, 20, 20, 2, 1, 64, BF, seed=19)
    lse = torch.zeros(1, 20, 2, device="cuda")
    for call in (lambda **k: gdr.attn_fwd(dev["q"], dev["k"], dev["v"], **k),
                 lambda **k: gdr.attn_bwd(dev["q"], dev["k"], dev["v"], dev["q"], lse, dev["do"], **k)):
        with pytest.raises(gdr.GdrError, match=text):
            call(**{k: v() for k, v in what.items()})
