"""GPU: values of x that are not finite, in the state space scan's forward.  Each
reaches its own column of y from its own token on, and that column of the state,
as in the recurrence; earlier tokens (of its chunk too), other columns, heads and
sequences keep their values (tolerances in ssm_checks.py, where the fp64
recurrence is finite)."""
import pytest
import torch

import mixer_ref as ref
from mixer_ref import U, half_step
from ssm_checks import on, sizes, terms
from test_gpu_ssm_scan import BF, F, forward, make

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def compare(what, got, want, tol):
    """Within `tol` where `want` is finite, not finite elsewhere."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), what
    assert bool(((got - want).abs() <= tol)[fine].all()), what


def check_with(gdr, d, c, cu, dtype):
    y, ht = forward(gdr, d)
    clean = on(c, "cuda")
    a, step, dec = sizes({k: None if v is None else v.nan_to_num(0, 0, 0) for k, v in clean.items()})
    my, mh = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], cu, a["h0"])
    ry, rh, _ = ref.ssm(clean["x"], clean["dt"], clean["A"], clean["b"], clean["c"], clean["D"], clean["dt_bias"], cu, clean["h0"])
    compare("y", y, ry, terms(dtype) * my + (half_step(dtype) * ry.abs() if dtype == BF else 0))
    compare("ht", ht, rh, 512 * U * mh)
    inf = torch.isinf(rh)
    assert torch.equal(ht.double()[inf], rh[inf])   # infinite states stay infinite, with their sign
    return ry, rh


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,p", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [150, 1200])   # walked whole, and in spans
def test_x(T, n, p, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    cu = [0, T - 70, T]
    d, c = make(91, 1, T, 2, 1, n, p, dtype, F, cu)
    for t, h, at, v in ((T - 72, 0, 3, INF), (T - 90, 1, 20, -INF), (T - 1, 0, p - 1, NAN), (T - 20, 1, 40, INF), (5, 0, 9, NAN)):
        for x in (d["x"], c["x"]):
            x[0, t, h, at] = v
    ry, rh = check_with(gdr, d, c, cu, dtype)
    assert torch.isfinite(ry[0, :T - 72, 0, 3]).all() and torch.isinf(rh).any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_rows_whose_tail_holds_anything(dtype):
    """Rows padded on the right with NaN: the tokens before it are not touched."""
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(92, 3, 100, 2, 2, 64, 64, dtype, F, None)
    for t in (d, c):
        for k in ("x", "b", "c", "dt"):
            for i, n in enumerate((100, 33, 70)):
                t[k][i, n:] = NAN
    y, ht = forward(gdr, d)
    good = {k: None if v is None else v.nan_to_num(0) for k, v in on(c, "cuda").items()}
    ry, _, _ = ref.ssm(good["x"], good["dt"], good["A"], good["b"], good["c"], good["D"], good["dt_bias"], None, good["h0"])
    a, step, dec = sizes(good)
    my, _ = ref.ssm_walk(a["x"], step, dec, a["b"], a["c"], a["D"], None, a["h0"])
    tol = terms(dtype) * my + (half_step(dtype) * ry.abs() if dtype == BF else 0)
    for i, n in enumerate((100, 33, 70)):
        assert bool(((y[i, :n].double() - ry[i, :n]).abs() <= tol[i, :n]).all()), i


@pytest.mark.parametrize("dtype", [BF, F])
def test_infinite_state(dtype):
    """An infinite state decays to an infinite one."""
    import chunked_gated_delta_fwd_amd as gdr
    d, c = make(93, 1, 130, 2, 1, 64, 64, dtype, F, None)
    for t in (d, c):
        t["h0"][0, 0, 7, 11], t["h0"][0, 1, 8, 50] = INF, -INF
    check_with(gdr, d, c, None, dtype)
