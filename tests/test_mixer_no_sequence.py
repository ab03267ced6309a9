"""Calls with a cu_seqlens of one offset (no sequence) and tokens: every token is
outside all sequences, so nothing is read for them and no row is written, and
sums over the tokens are zero.  On the host, the workspace shows how many tokens
the kernels are told of."""
import ctypes

import pytest

from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import (GDR_BF16, GDR_F32, GDR_I32, Alloc2, call, conv_bwd, conv_fwd, has_gpu,
                             query, scan_descs)

no_gpu = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")


@no_gpu
def test_convolution_gradient_has_no_rows_of_sums(lib):  # noqa: F811
    d = conv_fwd(T=5000)
    A = Alloc2()
    d.update(cu=A(GDR_I32, [1]), s0=A(GDR_BF16, [0, 3, 48]), st=A(GDR_BF16, [0, 3, 48]))
    assert query(lib, d) == 0


@no_gpu
@pytest.mark.parametrize("T", [100, 5000])
def test_scan_gradient_has_no_chunks(lib, T):  # noqa: F811
    f = scan_descs(T=T, N=0)
    A = Alloc2()
    A.next = 1 << 45
    d = {k: f[k] for k in ("x", "dt", "A", "b", "c", "D", "bias", "cu", "h0")}
    d.update(dy=A(GDR_BF16, [1, T, 4, 64]), dht=A(GDR_F32, [0, 4, 128, 64]), dx=A(GDR_BF16, [1, T, 4, 64]),
             ddt=A(GDR_F32, [1, T, 4]), dA=A(GDR_F32, [4]), db=A(GDR_BF16, [1, T, 2, 128]), dc=A(GDR_BF16, [1, T, 2, 128]),
             dD=A(GDR_F32, [4]), dbias=A(GDR_F32, [4]), dh0=A(GDR_F32, [0, 4, 128, 64]))
    size = ctypes.c_int64(-1)
    got = call(lib, "ssm_scan_bwd", list(d.values()), None, ctypes.addressof(size))
    assert got[0] == 0, got
    assert 0 <= size.value < 4096   # the tables' first entries, no chunk and no span


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 5000])
def test_gradients_without_a_sequence(T):
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    from test_gpu_conv import make as conv
    from test_gpu_ssm_scan import make as scan
    BF, F = torch.bfloat16, torch.float32
    d, _ = conv(1, 1, T, 40, 4, BF, cu=[0], state=False)
    dx = torch.full_like(d["x"], 7)
    _, dw, db, ds0 = gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"], dx=dx)
    assert (dx == 7).all() and (dw == 0).all() and (db == 0).all() and ds0.shape[0] == 0
    d, _ = scan(1, 1, T, 2, 1, 64, 64, BF, F, cu=[0], state=False)
    dx = torch.full_like(d["x"], 7)
    got = gdr.ssm_scan_bwd(d["x"], d["dt"], d["A"], d["b"], d["c"], d["dy"], d["D"], d["dt_bias"], d["cu"], dx=dx)
    assert (dx == 7).all() and all((got[i] == 0).all() for i in (2, 5, 6)) and got[7].shape[0] == 0


@pytest.mark.gpu
def test_the_content_check_reports_it():
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    from test_gpu_conv import make
    d, _ = make(1, 1, 40, 40, 4, torch.bfloat16, cu=[0], state=False)
    gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 1)
    try:
        for call_ in (lambda: gdr.short_conv_fwd(d["x"], d["w"], d["bias"], d["cu"]),
                      lambda: gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["cu"])):
            with pytest.raises(gdr.GdrError, match="must equal the 40 tokens"):
                call_()
    finally:
        gdr.debug_set(gdr.GDR_DEBUG_CHECK_CU, 0)
