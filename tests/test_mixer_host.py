"""Host-only checks of the operators around the recurrence: every refusal, on
descriptors with fake addresses that are never dereferenced (a call that passes
validation stops at the device check, or at the workspace query)."""
import ctypes

import pytest

import chunked_gated_delta_fwd_amd as gdr
from chunked_gated_delta_fwd_amd import GDR_BF16, GDR_F32, GDR_I32
from test_abi_host import Alloc, lib  # noqa: F401

def has_gpu():
    import torch
    return torch.cuda.is_available()


# the addresses are not memory: a call that passes validation must find no device
pytestmark = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")

ESHAPE, EDTYPE, ESTRIDE, EALIAS, EINVAL, EDEVICE = -2, -3, -4, -5, -1, -6


def call(lib, name, descs, *rest):
    args = [None if d is None else ctypes.addressof(d.t) for d in descs]
    status = getattr(lib, "gdr_" + name)(*args, *rest, None)
    return status, lib.gdr_last_error().decode()


def conv_fwd(dt=GDR_BF16, B=1, T=20, ch=48, W=4, N=3):
    A = Alloc()
    return dict(x=A(dt, [B, T, ch]), w=A(dt, [ch, W]), bias=A(dt, [ch]), cu=A(GDR_I32, [N + 1]), s0=A(dt, [N, W - 1, ch]),
                y=A(dt, [B, T, ch]), st=A(dt, [N, W - 1, ch]))


CONV_FWD = [
    (lambda d, A: d.update(x=None), EINVAL, "x: descriptor is NULL"),
    (lambda d, A: d.update(x=A(GDR_I32, [1, 20, 48])), EDTYPE, "x: dtype"),
    (lambda d, A: d.update(w=A(GDR_F32, [48, 4])), EDTYPE, "w: dtype"),
    (lambda d, A: d.update(w=A(GDR_BF16, [48, 5])), ESHAPE, "2, 3 or 4 taps"),
    (lambda d, A: d.update(w=A(GDR_BF16, [48, 1])), ESHAPE, "2, 3 or 4 taps"),
    (lambda d, A: d.update(w=A(GDR_BF16, [47, 4])), ESHAPE, "w: shape"),
    (lambda d, A: d.update(bias=A(GDR_BF16, [47])), ESHAPE, "bias: shape"),
    (lambda d, A: d.update(s0=A(GDR_BF16, [3, 4, 48])), ESHAPE, "s0: shape"),
    (lambda d, A: d.update(s0=A(GDR_F32, [3, 3, 48])), EDTYPE, "s0: dtype"),
    (lambda d, A: d.update(y=A(GDR_BF16, [1, 20, 40])), ESHAPE, "y: shape"),
    (lambda d, A: d.update(y=A(GDR_F32, [1, 20, 48])), EDTYPE, "y: dtype"),
    (lambda d, A: d.update(st=A(GDR_BF16, [2, 3, 48])), ESHAPE, "st: shape"),
    (lambda d, A: d.update(y=d["x"]), EALIAS, "y overlaps x"),
    (lambda d, A: d.update(st=d["s0"]), EALIAS, "st overlaps s0"),
    (lambda d, A: d.update(cu=A(GDR_F32, [4])), EDTYPE, "cu_seqlens"),
    (lambda d, A: d.update(cu=A(GDR_I32, [0])), ESHAPE, "at least one offset"),
    (lambda d, A: d.update(x=A(GDR_BF16, [2, 10, 48]), y=A(GDR_BF16, [2, 10, 48])), ESHAPE, "B == 1"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1, 20, 48], [960, 48, 2])), ESTRIDE, "row must be compact"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1, 20, 48], [960, 40, 1])), ESTRIDE, "x: rows"),
    (lambda d, A: d.update(y=A(GDR_BF16, [1, 20, 48], [2000, 100, 1])), ESTRIDE, "y: strides"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1, 20, 48], misalign=1)), EINVAL, "aligned"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1 << 16, 1 << 16, 1]), cu=None), ESHAPE, "2^31"),
]


@pytest.mark.parametrize("change,status,text", CONV_FWD)
def test_conv_forward_refusals(lib, change, status, text):  # noqa: F811
    d = conv_fwd()
    change(d, Alloc2())
    got = call(lib, "short_conv_fwd", list(d.values()), 1)
    assert got[0] == status and text in got[1], got


class Alloc2(Alloc):
    """Addresses apart from Alloc's."""

    def __init__(self):
        self.next = 1 << 44


def test_conv_activation_is_checked(lib):  # noqa: F811
    got = call(lib, "short_conv_fwd", list(conv_fwd().values()), 7)
    assert got[0] == EINVAL and "activation" in got[1]


def test_evenly_spaced_rows_are_accepted(lib):  # noqa: F811
    """A slice of a wider projection passes validation (and stops at the device check without a GPU)."""
    d = conv_fwd(B=2, T=10)
    d["cu"] = None
    A = Alloc2()
    d["s0"], d["st"] = A(GDR_BF16, [2, 3, 48]), A(GDR_BF16, [2, 3, 48])
    d["x"] = A(GDR_BF16, [2, 10, 48], [1000, 100, 1])
    assert query(lib, d) > 0
    d["x"] = A(GDR_BF16, [2, 10, 48], [1001, 100, 1])
    assert "evenly spaced" in query(lib, d)


def conv_bwd(d, ch=48, W=4):
    A = Alloc2()
    A.next = 1 << 45
    N, B, T = d["st"].t.shape[0], d["y"].t.shape[0], d["y"].t.shape[1]
    return dict(x=d["x"], w=d["w"], bias=d["bias"], cu=d["cu"], s0=d["s0"], dy=A(GDR_BF16, [B, T, ch]),
                dst=A(GDR_BF16, [N, W - 1, ch]), dx=A(GDR_BF16, [B, T, ch]), dw=A(GDR_F32, [ch, W]), db=A(GDR_F32, [ch]),
                ds0=A(GDR_BF16, [N, W - 1, ch]))


def query(lib, d):  # noqa: F811
    """The workspace size of the backward call on these forward descriptors, or its message."""
    size = ctypes.c_int64(-1)
    status, text = call(lib, "short_conv_bwd", list(conv_bwd(d).values()), 1, None, ctypes.addressof(size))
    return size.value if status == 0 else text


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(dw=A(GDR_BF16, [48, 4])), EDTYPE, "dw"),
    (lambda d, A: d.update(db=A(GDR_F32, [40])), ESHAPE, "db"),
    (lambda d, A: d.update(dst=A(GDR_F32, [3, 3, 48])), EDTYPE, "dst"),
    (lambda d, A: d.update(dx=d["dy"]), EALIAS, "dx overlaps dy"),
    (lambda d, A: d.update(ds0=d["s0"]), EALIAS, "ds0 overlaps s0"),
    (lambda d, A: d.update(dy=A(GDR_BF16, [1, 19, 48])), ESHAPE, "dy"),
    (lambda d, A: d.update(dx=None), EINVAL, "dx"),
])
def test_conv_backward_refusals(lib, change, status, text):  # noqa: F811
    d = conv_bwd(conv_fwd())
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "short_conv_bwd", list(d.values()), 1, None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert size.value == -1


def test_workspace_arguments(lib):  # noqa: F811
    assert query(lib, conv_fwd()) == 1 * 48 * 5 * 4   # one block row of W + 1 sums a channel
    d = conv_bwd(conv_fwd())
    small = ctypes.c_int64(16)
    got = call(lib, "short_conv_bwd", list(d.values()), 1, 1 << 50, ctypes.addressof(small))
    assert got[0] in (EINVAL, EDEVICE)   # without a GPU the device check comes first


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(state=A(GDR_BF16, [5, 4, 48])), ESHAPE, "state"),
    (lambda d, A: d.update(state=A(GDR_F32, [5, 3, 48])), EDTYPE, "state"),
    (lambda d, A: d.update(y=A(GDR_BF16, [4, 48])), ESHAPE, "y"),
    (lambda d, A: d.update(y=d["x"]), EALIAS, "y overlaps x"),
    (lambda d, A: d.update(x=A(GDR_BF16, [5, 1, 48])), ESHAPE, "x: expected 2 dimensions"),
])
def test_conv_step_refusals(lib, change, status, text):  # noqa: F811
    A = Alloc()
    d = dict(x=A(GDR_BF16, [5, 48]), state=A(GDR_BF16, [5, 3, 48]), w=A(GDR_BF16, [48, 4]), bias=None, y=A(GDR_BF16, [5, 48]))
    change(d, Alloc2())
    got = call(lib, "short_conv_step", list(d.values()), 1)
    assert got[0] == status and text in got[1], got


def norm_descs(d=128, rot=64):
    A = Alloc()
    return dict(q=A(GDR_BF16, [2, 10, 4, d]), k=A(GDR_BF16, [2, 10, 2, d]), wq=A(GDR_BF16, [d]), wk=A(GDR_BF16, [d]),
                cos=A(GDR_F32, [50, rot // 2]), sin=A(GDR_F32, [50, rot // 2]), pos=A(GDR_I32, [2, 10]),
                oq=A(GDR_BF16, [2, 10, 4, d]), ok=A(GDR_BF16, [2, 10, 2, d]))


NORM = [
    (lambda d, A: d.update(q=None), EINVAL, "q: descriptor is NULL"),
    (lambda d, A: d.update(k=None), EINVAL, "k: descriptor is NULL"),
    (lambda d, A: d.update(k=A(GDR_F32, [2, 10, 2, 128])), EDTYPE, "k: dtype"),
    (lambda d, A: d.update(k=A(GDR_BF16, [2, 9, 2, 128])), ESHAPE, "k: shape"),
    (lambda d, A: d.update(q=A(GDR_BF16, [2, 10, 4, 96])), ESHAPE, "head dim"),
    (lambda d, A: d.update(wq=A(GDR_BF16, [64])), ESHAPE, "wq"),
    (lambda d, A: d.update(sin=None), EINVAL, "both tables"),
    (lambda d, A: d.update(sin=A(GDR_F32, [49, 32])), ESHAPE, "sin"),
    (lambda d, A: d.update(cos=A(GDR_BF16, [50, 32])), EDTYPE, "cos"),
    (lambda d, A: d.update(cos=A(GDR_F32, [50, 20]), sin=A(GDR_F32, [50, 20])), ESHAPE, "multiple of 16"),
    (lambda d, A: d.update(cos=A(GDR_F32, [50, 72]), sin=A(GDR_F32, [50, 72])), ESHAPE, "multiple of 16"),
    (lambda d, A: d.update(cos=A(GDR_F32, [0, 32]), sin=A(GDR_F32, [0, 32])), ESHAPE, "rows"),
    (lambda d, A: d.update(cos=A(GDR_F32, [9, 32]), sin=A(GDR_F32, [9, 32]), pos=None), ESHAPE, "9 rows for 10 tokens"),
    (lambda d, A: d.update(cos=None, sin=None), EINVAL, "positions without"),
    (lambda d, A: d.update(pos=A(GDR_F32, [2, 10])), EDTYPE, "positions"),
    (lambda d, A: d.update(pos=A(GDR_I32, [10, 2])), ESHAPE, "positions"),
    (lambda d, A: d.update(oq=d["q"]), EALIAS, "oq overlaps q"),
    (lambda d, A: d.update(ok=d["oq"]), ESHAPE, "ok"),
    (lambda d, A: d.update(q=A(GDR_BF16, [2, 10, 4, 128], [6000, 600, 128, 1])), -99, ""),
    (lambda d, A: d.update(q=A(GDR_BF16, [2, 10, 4, 128], [6010, 601, 128, 1])), ESTRIDE, "16 bytes"),
    (lambda d, A: d.update(q=A(GDR_BF16, [2, 10, 4, 128], [6000, 600, 130, 1])), ESTRIDE, "row must be compact"),
    (lambda d, A: d.update(q=A(GDR_BF16, [2, 10, 4, 128], misalign=8)), EINVAL, "16-byte"),
]


@pytest.mark.parametrize("change,status,text", NORM)
def test_norm_refusals(lib, change, status, text):  # noqa: F811
    d = norm_descs()
    change(d, Alloc2())
    got = call(lib, "qk_norm_rope_fwd", list(d.values()), 1, 1e-6, 0)
    if status == -99:   # accepted: only the device check stops it
        status, text = EDEVICE, ""
    assert got[0] == status and text in got[1], got


@pytest.mark.parametrize("norm,eps,text", [(2, 1e-6, "norm"), (1, -1.0, "eps"), (0, float("nan"), "eps"), (0, float("inf"), "eps")])
def test_norm_scalars(lib, norm, eps, text):  # noqa: F811
    got = call(lib, "qk_norm_rope_fwd", list(norm_descs().values()), norm, eps, 0)
    assert got[0] == EINVAL and text in got[1], got


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(dwq=A(GDR_BF16, [128])), EDTYPE, "dwq"),
    (lambda d, A: d.update(dwk=A(GDR_F32, [64])), ESHAPE, "dwk"),
    (lambda d, A: d.update(doq=A(GDR_BF16, [2, 10, 2, 128])), ESHAPE, "doq"),
    (lambda d, A: d.update(dq=d["doq"]), EALIAS, "dq overlaps doq"),
    (lambda d, A: None, 0, ""),
])
def test_norm_backward_refusals(lib, change, status, text):  # noqa: F811
    f = norm_descs()
    A = Alloc2()
    A.next = 1 << 45
    d = {k: f[k] for k in ("q", "k", "wq", "wk", "cos", "sin", "pos")}
    d.update(doq=A(GDR_BF16, [2, 10, 4, 128]), dok=A(GDR_BF16, [2, 10, 2, 128]), dq=A(GDR_BF16, [2, 10, 4, 128]),
             dk=A(GDR_BF16, [2, 10, 2, 128]), dwq=A(GDR_F32, [128]), dwk=A(GDR_F32, [128]))
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "qk_norm_rope_bwd", list(d.values()), 1, 1e-6, 0, None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert (size.value > 0) == (status == 0)


def step_descs():
    A = Alloc()
    return dict(x=A(GDR_BF16, [3, 8, 64]), dt=A(GDR_F32, [3, 8]), A=A(GDR_F32, [8]), b=A(GDR_BF16, [3, 2, 128]),
                c=A(GDR_BF16, [3, 2, 128]), D=A(GDR_F32, [8]), bias=A(GDR_F32, [8]), h=A(GDR_F32, [3, 8, 128, 64]),
                y=A(GDR_BF16, [3, 8, 64]))


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(x=None), EINVAL, "x: descriptor is NULL"),
    (lambda d, A: d.update(b=None), EINVAL, "b: descriptor is NULL"),
    (lambda d, A: d.update(A=None), EINVAL, "A: descriptor is NULL"),
    (lambda d, A: d.update(x=A(GDR_BF16, [3, 8, 96])), ESHAPE, "p must be"),
    (lambda d, A: d.update(b=A(GDR_BF16, [3, 2, 96])), ESHAPE, "n must be"),
    (lambda d, A: d.update(b=A(GDR_BF16, [3, 3, 128]), c=A(GDR_BF16, [3, 3, 128])), ESHAPE, "multiple of G"),
    (lambda d, A: d.update(c=A(GDR_BF16, [3, 1, 128])), ESHAPE, "c: shape"),
    (lambda d, A: d.update(c=A(GDR_F32, [3, 2, 128])), EDTYPE, "c: dtype"),
    (lambda d, A: d.update(dt=A(GDR_I32, [3, 8])), EDTYPE, "dt: dtype"),
    (lambda d, A: d.update(dt=A(GDR_F32, [3, 7])), ESHAPE, "dt: shape"),
    (lambda d, A: d.update(A=A(GDR_BF16, [8])), EDTYPE, "A: dtype"),
    (lambda d, A: d.update(D=A(GDR_F32, [7])), ESHAPE, "D: shape"),
    (lambda d, A: d.update(h=A(GDR_F32, [3, 8, 64, 128])), ESHAPE, "h: shape"),
    (lambda d, A: d.update(h=A(GDR_BF16, [3, 8, 128, 64])), EDTYPE, "h: dtype"),
    (lambda d, A: d.update(y=d["x"]), EALIAS, "y overlaps x"),
    (lambda d, A: d.update(x=A(GDR_BF16, [3, 8, 64], misalign=4)), EINVAL, "16-byte"),
])
def test_ssm_step_refusals(lib, change, status, text):  # noqa: F811
    d = step_descs()
    change(d, Alloc2())
    got = call(lib, "ssm_step", list(d.values()))
    assert got[0] == status and text in got[1], got


def test_python_choices():
    import torch
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(gdr.GdrError, match="activation"):
        gdr.short_conv_fwd(x, w, activation="relu")
    with pytest.raises(gdr.GdrError, match="norm"):
        gdr.qk_norm_rope_fwd(torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1, 64), norm="layer")
    with pytest.raises(gdr.GdrError, match="one GPU"):   # host memory never reaches a kernel
        gdr.short_conv_fwd(x, w)
    with pytest.raises(AttributeError):
        gdr.no_such_operator


def scan_descs(T=100, H=4, G=2, n=128, p=64, N=3):
    A = Alloc()
    return dict(x=A(GDR_BF16, [1, T, H, p]), dt=A(GDR_F32, [1, T, H]), A=A(GDR_F32, [H]), b=A(GDR_BF16, [1, T, G, n]),
                c=A(GDR_BF16, [1, T, G, n]), D=A(GDR_F32, [H]), bias=A(GDR_F32, [H]), cu=A(GDR_I32, [N + 1]),
                h0=A(GDR_F32, [N, H, n, p]), y=A(GDR_BF16, [1, T, H, p]), ht=A(GDR_F32, [N, H, n, p]))


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(x=None), EINVAL, "x: descriptor is NULL"),
    (lambda d, A: d.update(dt=None), EINVAL, "dt: descriptor is NULL"),
    (lambda d, A: d.update(c=None), EINVAL, "c: descriptor is NULL"),
    (lambda d, A: d.update(y=None), EINVAL, "y: descriptor is NULL"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1, 100, 4, 32])), ESHAPE, "p must be"),
    (lambda d, A: d.update(b=A(GDR_BF16, [1, 100, 2, 256])), ESHAPE, "n must be"),
    (lambda d, A: d.update(b=A(GDR_BF16, [1, 100, 3, 128]), c=A(GDR_BF16, [1, 100, 3, 128])), ESHAPE, "multiple of G"),
    (lambda d, A: d.update(b=A(GDR_BF16, [1, 99, 2, 128])), ESHAPE, "b: shape"),
    (lambda d, A: d.update(dt=A(GDR_F32, [1, 100, 3])), ESHAPE, "dt: shape"),
    (lambda d, A: d.update(h0=A(GDR_F32, [2, 4, 128, 64])), ESHAPE, "h0: shape"),
    (lambda d, A: d.update(ht=A(GDR_BF16, [3, 4, 128, 64])), EDTYPE, "ht: dtype"),
    (lambda d, A: d.update(y=A(GDR_F32, [1, 100, 4, 64])), EDTYPE, "y: dtype"),
    (lambda d, A: d.update(ht=d["h0"]), EALIAS, "ht overlaps h0"),
    (lambda d, A: d.update(cu=A(GDR_BF16, [4])), EDTYPE, "cu_seqlens"),
    (lambda d, A: d.update(x=A(GDR_BF16, [1, 100, 4, 64], [1 << 26, 1 << 25, 64, 1])), ESTRIDE, "bytes apart"),
    (lambda d, A: d.update(b=A(GDR_BF16, [1, 100, 2, 128], [0, 1001, 128, 1])), ESTRIDE, "16 bytes"),
    (lambda d, A: None, 0, ""),
])
def test_scan_refusals(lib, change, status, text):  # noqa: F811
    d = scan_descs()
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "ssm_scan_fwd", list(d.values()), None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert (size.value >= 0) == (status == 0)


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(dx=None), EINVAL, "dx: descriptor is NULL"),
    (lambda d, A: d.update(dA=None), EINVAL, "dA: descriptor is NULL"),
    (lambda d, A: d.update(ddt=A(GDR_BF16, [1, 100, 4])), EDTYPE, "ddt: dtype"),
    (lambda d, A: d.update(db=A(GDR_BF16, [1, 100, 4, 128])), ESHAPE, "db: shape"),
    (lambda d, A: d.update(dht=A(GDR_F32, [3, 4, 64, 128])), ESHAPE, "dht: shape"),
    (lambda d, A: d.update(dh0=d["dht"]), EALIAS, "dh0 overlaps dht"),
    (lambda d, A: d.update(db=d["dc"]), EALIAS, "dc overlaps db"),
    (lambda d, A: None, 0, ""),
])
def test_scan_backward_refusals(lib, change, status, text):  # noqa: F811
    f = scan_descs()
    A = Alloc2()
    A.next = 1 << 45
    d = {k: f[k] for k in ("x", "dt", "A", "b", "c", "D", "bias", "cu", "h0")}
    d.update(dy=A(GDR_BF16, [1, 100, 4, 64]), dht=A(GDR_F32, [3, 4, 128, 64]), dx=A(GDR_BF16, [1, 100, 4, 64]),
             ddt=A(GDR_F32, [1, 100, 4]), dA=A(GDR_F32, [4]), db=A(GDR_BF16, [1, 100, 2, 128]), dc=A(GDR_BF16, [1, 100, 2, 128]),
             dD=A(GDR_F32, [4]), dbias=A(GDR_F32, [4]), dh0=A(GDR_F32, [3, 4, 128, 64]))
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "ssm_scan_bwd", list(d.values()), None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert (size.value > 0) == (status == 0)
