"""Workspaces of the operators around the recurrence, through the C ABI: what is
refused (before any device is touched), a caller's buffer of exactly the queried
size, the library's own in a stream capture and on two streams in turn."""
import ctypes

import pytest

from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import (EDEVICE, EINVAL, GDR_BF16, GDR_F32, Alloc2, call, conv_bwd, conv_fwd, has_gpu, norm_descs,
                             scan_descs)

no_gpu = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")


def scan_bwd():
    f = scan_descs()
    A = Alloc2()
    A.next = 1 << 45
    d = {k: f[k] for k in ("x", "dt", "A", "b", "c", "D", "bias", "cu", "h0")}
    d.update(dy=A(GDR_BF16, [1, 100, 4, 64]), dht=A(GDR_F32, [3, 4, 128, 64]), dx=A(GDR_BF16, [1, 100, 4, 64]),
             ddt=A(GDR_F32, [1, 100, 4]), dA=A(GDR_F32, [4]), db=A(GDR_BF16, [1, 100, 2, 128]), dc=A(GDR_BF16, [1, 100, 2, 128]),
             dD=A(GDR_F32, [4]), dbias=A(GDR_F32, [4]), dh0=A(GDR_F32, [3, 4, 128, 64]))
    return d


def norm_bwd():
    f = norm_descs()
    A = Alloc2()
    A.next = 1 << 45
    d = {k: f[k] for k in ("q", "k", "wq", "wk", "cos", "sin", "pos")}
    d.update(doq=A(GDR_BF16, [2, 10, 4, 128]), dok=A(GDR_BF16, [2, 10, 2, 128]), dq=A(GDR_BF16, [2, 10, 4, 128]),
             dk=A(GDR_BF16, [2, 10, 2, 128]), dwq=A(GDR_F32, [128]), dwk=A(GDR_F32, [128]))
    return d


CALLS = {   # name of the entry, its descriptors, what stands between them and the workspace
    "short_conv_bwd": (lambda: conv_bwd(conv_fwd()), (1,)),
    "qk_norm_rope_bwd": (norm_bwd, (1, 1e-6, 0)),
    "ssm_scan_fwd": (lambda: scan_descs(T=5000), ()),
    "ssm_scan_bwd": (scan_bwd, ()),
}


@no_gpu
@pytest.mark.parametrize("name", list(CALLS))
def test_refused_workspaces(lib, name):  # noqa: F811
    make, more = CALLS[name]
    descs = list(make().values())
    size = ctypes.c_int64(-1)
    assert call(lib, name, descs, *more, None, ctypes.addressof(size))[0] == 0 and size.value > 0
    at = 1 << 50
    for given, nbytes, text in ((at, size.value - 1, "%d needed" % size.value), (at, 0, "needed"), (at, -1, "needed"),
                                (at + 8, size.value, "16-byte"), (at, None, "size is missing")):
        n = None if nbytes is None else ctypes.c_int64(nbytes)
        got = call(lib, name, descs, *more, given, None if n is None else ctypes.addressof(n))
        assert got[0] == EINVAL and "workspace" in got[1] and text in got[1], (given, nbytes, got)
    # the exact size passes (and finds no device)
    got = call(lib, name, descs, *more, at, ctypes.addressof(size))
    assert got[0] == EDEVICE, got


# --- on the GPU ------------------------------------------------------------------

def inputs(T, H, seed, cu=None):
    import torch
    from test_gpu_ssm_scan import make
    return make(seed, 1, T, H, 1, 64, 64, torch.bfloat16, torch.float32, cu)[0]


def scan_gradient(gdr, d):
    return gdr.ssm_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["dy"], d["D"], d["dt_bias"], d["cu"], d["h0"], d["dht"])


def through_the_abi(gdr, d, workspace, nbytes):
    """The scan's gradient with a workspace given as addresses: (status, gradients)."""
    import torch
    out = [torch.empty_like(d[k]) for k in ("x", "dt", "A", "b", "c", "D", "dt_bias")] + [torch.empty_like(d["dht"])]
    order = [d[k] for k in ("x", "dt", "A", "b", "c", "D", "dt_bias", "cu", "h0", "dy", "dht")] + out
    descs = [gdr._desc(t) for t in order]
    lib = gdr.library()
    status = lib.gdr_ssm_scan_bwd(*[None if d is None else ctypes.addressof(d.t) for d in descs], workspace,
                                  None if nbytes is None else ctypes.addressof(nbytes), torch.cuda.current_stream().cuda_stream)
    return status, out


@pytest.mark.gpu
@pytest.mark.parametrize("T,cu", [(70, None), (1300, [0, 0, 1000, 1300])])
def test_a_workspace_of_exactly_the_queried_size(T, cu):
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    d = inputs(T, 2, 51, cu)
    want = scan_gradient(gdr, d)
    size = ctypes.c_int64(0)
    assert through_the_abi(gdr, d, None, size)[0] == 0 and size.value > 0
    buf = torch.full((size.value + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    at = 4096 - buf.data_ptr() % 16
    status, got = through_the_abi(gdr, d, buf.data_ptr() + at, size)
    assert status == 0
    assert (buf[:at] == 0xA5).all() and (buf[at + size.value:] == 0xA5).all()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_the_librarys_own_is_refused_in_a_capture():
    """The refusal leaves the capture whole."""
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    d = inputs(70, 2, 52)
    scan_gradient(gdr, d)
    x = torch.zeros(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status, _ = through_the_abi(gdr, d, None, None)
        text = gdr.library().gdr_last_error().decode()
        x += 1
    assert status == EINVAL and "capture" in text
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()


@pytest.mark.gpu
def test_two_streams_take_turns():
    """Gradients of two sizes, which share the library's large buffer and make it
    grow, on two streams in turn: the bits of the calls alone."""
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    gdr.free_workspaces()
    cases = [inputs(700, 4, 53), inputs(1500, 6, 54, [0, 1100, 1500])]
    want = [scan_gradient(gdr, d) for d in cases]
    torch.cuda.synchronize()
    gdr.free_workspaces()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(6):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append((i, scan_gradient(gdr, cases[i])))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(want[i], g)), i
