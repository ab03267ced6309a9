"""Rows of a single token's inputs may be any distance apart: a step reads one
row of each, with 64-bit addresses (the scan's chunks have a limit of 32 MiB)."""
import pytest

from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import EDEVICE, ESTRIDE, GDR_BF16, Alloc2, call, has_gpu, scan_descs, step_descs


@pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")
def test_far_rows_on_the_host(lib):  # noqa: F811
    far = 1 << 26   # elements
    A = Alloc2()
    d = step_descs()
    d["x"] = A(GDR_BF16, [3, 8, 64], [far, 64, 1])
    A.next += 1 << 34
    d["b"] = A(GDR_BF16, [3, 2, 128], [far, 128, 1])
    got = call(lib, "ssm_step", list(d.values()))
    assert got[0] == EDEVICE, got
    d = scan_descs()
    d["x"] = A(GDR_BF16, [1, 100, 4, 64], [100 * far, far, 64, 1])
    got = call(lib, "ssm_scan_fwd", list(d.values()), None, None)
    assert got[0] == ESTRIDE and "bytes apart" in got[1], got


@pytest.mark.gpu
def test_far_rows_on_the_gpu():
    """One token out of a long prompt's projections: rows 48 MiB apart give the bits of compact ones."""
    import torch
    import chunked_gated_delta_fwd_amd as gdr
    from test_gpu_ssm_step import make
    d, _ = make(3, 4, 2, 128, 64, torch.bfloat16, torch.float32)
    far = {}
    for k in ("x", "b", "c"):
        one = d[k][:, 0].contiguous()
        buf = torch.zeros(3, 24 << 20, dtype=torch.bfloat16, device="cuda")
        at = buf[:, 4096:4096 + one[0].numel()].unflatten(-1, one.shape[1:])
        at.copy_(one)
        far[k] = (one, at)
    out = []
    for i in range(2):
        h = d["h"].clone()
        y = gdr.ssm_step(far["x"][i], d["dt"][:, 0], d["A"], far["b"][i], far["c"][i], h, d["D"], d["dt_bias"])
        out.append((y, h))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
