"""Rows without tokens, more than one of them: an empty tensor's strides say
nothing (torch gives [2, 0, 4, 64] a first stride of 256), states are handed on."""
import pytest

from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import EDEVICE, GDR_BF16, Alloc2, call, conv_fwd, has_gpu


@pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")
def test_strides_of_empty_tensors(lib):  # noqa: F811
    d = conv_fwd()
    A = Alloc2()
    d.update(x=A(GDR_BF16, [2, 0, 48], [48, 48, 1]), y=A(GDR_BF16, [2, 0, 48], [48, 48, 1]), cu=None,
             s0=A(GDR_BF16, [2, 3, 48]), st=A(GDR_BF16, [2, 3, 48]))
    got = call(lib, "short_conv_fwd", list(d.values()), 1)
    assert got[0] == EDEVICE, got   # only the device check stops it


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 2, 5])
def test_states_are_handed_on(B):
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    from test_gpu_conv import make as conv
    from test_gpu_qknorm import make as norm
    from test_gpu_ssm_scan import backward, forward, make as scan
    BF, F = torch.bfloat16, torch.float32
    d, _ = conv(1, B, 0, 48, 4, BF)
    y, st = gdr.short_conv_fwd(d["x"], d["w"], d["bias"], None, d["s0"])
    assert y.numel() == 0 and torch.equal(st, d["s0"])
    _, dw, db, ds0 = gdr.short_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], None, d["s0"], d["dst"])
    assert torch.equal(ds0, d["dst"]) and (dw == 0).all() and (db == 0).all()
    d, _ = scan(2, B, 0, 4, 2, 64, 64, BF, F)
    y, ht = forward(gdr, d)
    assert y.numel() == 0 and torch.equal(ht, d["h0"])
    dx, ddt, dA, db, dc, dD, dbias, dh0 = backward(gdr, d)
    assert torch.equal(dh0, d["dht"]) and all((t == 0).all() for t in (dA, dD, dbias))
    dv, _, _ = norm(B, 0, 2, 1, 64, 64, BF, True, True)
    oq, ok = gdr.qk_norm_rope_fwd(dv["q"], dv["k"], dv["wq"], dv["wk"], dv["cos"], dv["sin"], dv["pos"])
    assert oq.shape == dv["q"].shape and ok.shape == dv["k"].shape
    _, _, dwq, dwk = gdr.qk_norm_rope_bwd(dv["q"], dv["k"], dv["doq"], dv["dok"], dv["wq"], dv["wk"], dv["cos"], dv["sin"],
                                          dv["pos"])
    assert (dwq == 0).all() and (dwk == 0).all()
