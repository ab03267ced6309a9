"""GPU: the operators around the recurrence keep inside their tensors whatever
cu_seqlens holds, and the opt-in check of its content reports it.

Every tensor that a call reads or writes lies between two margins of 4096 bytes
that have to keep their fill; the margins of the inputs are NaN, which the
convolution's outputs would show."""
import pytest
import torch

from test_gpu_conv import make as make_conv
from test_gpu_ssm_scan import make as make_scan

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
BAD = {
    "past the end": lambda T: [0, 100, 100000, T],
    "all past the end": lambda T: [T + 1000, T + 2000, T + 3000, T + 4000],
    "negative": lambda T: [-500, -3, 70, T],
    "decreasing": lambda T: [0, T - 50, 30, T],
    "overlapping": lambda T: [0, T, 0, T, 0, T, 0, T],
    "largest": lambda T: [0, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1],
    "short": lambda T: [0, 64, 65, 200],
}
MARGIN = 4096


class Fenced:
    """Tensors in the middle of buffers whose ends are watched."""

    def __init__(self):
        self.kept = []

    def __call__(self, shape, dtype, fill):
        n = torch.Size(shape).numel()
        m = MARGIN // torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((n + 2 * m,), fill, dtype=dtype, device="cuda")
        self.kept.append((buf, m, n, fill))
        return buf[m:m + n].view(shape)

    def copy(self, t):
        if t is None:
            return None
        out = self(t.shape, t.dtype, float("nan") if t.is_floating_point() else -12345)
        out.copy_(t)
        return out

    def intact(self):
        for buf, m, n, fill in self.kept:
            for edge in (buf[:m], buf[m + n:]):
                good = torch.isnan(edge) if fill != fill else edge == fill
                if not bool(good.all()):
                    return False
        return True


@pytest.mark.parametrize("name", list(BAD))
@pytest.mark.parametrize("T", [300, 1300])   # 1300: the scan is split into spans
def test_bad_offsets_stay_inside(name, T):
    import chunked_gated_delta_fwd_amd as gdr
    cu, heads = BAD[name](T), 2
    N = len(cu) - 1
    for op in ("conv", "scan"):
        f = Fenced()
        if op == "conv":
            d, _ = make_conv(41, 1, T, 24 * heads, 4, BF, cu=cu)
            d = {k: f.copy(v) for k, v in d.items()}
            ch = 24 * heads
            y, dx = f((1, T, ch), BF, 5.0), f((1, T, ch), BF, 5.0)
            st, ds0 = f((N, 3, ch), BF, 5.0), f((N, 3, ch), BF, 5.0)
            dw, db = f((ch, 4), F, 5.0), f((ch,), F, 5.0)
            gdr.short_conv_fwd(d["x"], d["w"], d["bias"], d["cu"], d["s0"], y=y, st=st)
            gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"], d["s0"], d["dst"], dx=dx, dw=dw, db=db, ds0=ds0)
            outs = (y, st, dx, dw, db, ds0)
        else:
            d, _ = make_scan(42, 1, T, heads, 1, 64, 64, BF, F, cu=cu)
            d = {k: f.copy(v) for k, v in d.items()}
            y, dx = f((1, T, heads, 64), BF, 5.0), f((1, T, heads, 64), BF, 5.0)
            ht, dh0 = f((N, heads, 64, 64), F, 5.0), f((N, heads, 64, 64), F, 5.0)
            ddt, db, dc = f((1, T, heads), F, 5.0), f((1, T, 1, 64), BF, 5.0), f((1, T, 1, 64), BF, 5.0)
            dA, dD, dbias = (f((heads,), F, 5.0) for _ in range(3))
            args = [d[k] for k in ("x", "dt", "A", "b", "c")]
            gdr.ssm_scan_fwd(*args, d["D"], d["dt_bias"], d["cu"], d["h0"], y=y, ht=ht)
            gdr.ssm_scan_bwd(*args, d["dy"], d["D"], d["dt_bias"], d["cu"], d["h0"], d["dht"], dx=dx, ddt=ddt, dA=dA, db=db,
                             dc=dc, dD=dD, ddt_bias=dbias, dh0=dh0)
            outs = ()   # wrong numbers, from states that no walk stored
        torch.cuda.synchronize()
        assert f.intact(), op
        assert all(torch.isfinite(t).all() for t in outs), op


@pytest.mark.parametrize("name", [n for n in BAD])
def test_the_check_reports_them(name):
    import chunked_gated_delta_fwd_amd as gdr
    T = 300
    cu = BAD[name](T)
    d, _ = make_conv(43, 1, T, 24, 4, BF, cu=cu)
    s, _ = make_scan(44, 1, T, 2, 1, 64, 64, BF, F, cu=cu)
    args = [s[k] for k in ("x", "dt", "A", "b", "c")]
    calls = [
        lambda: gdr.short_conv_fwd(d["x"], d["w"], d["bias"], d["cu"], d["s0"]),
        lambda: gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"], d["s0"], d["dst"]),
        lambda: gdr.ssm_scan_fwd(*args, s["D"], s["dt_bias"], s["cu"], s["h0"]),
        lambda: gdr.ssm_scan_bwd(*args, s["dy"], s["D"], s["dt_bias"], s["cu"], s["h0"], s["dht"]),
    ]
    gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 1)
    try:
        for c in calls:
            with pytest.raises(gdr.GdrError, match="cu_seqlens"):
                c()
    finally:
        gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 0)
    torch.cuda.synchronize()
