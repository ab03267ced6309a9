"""GPU: what the Python calls of the operators around the recurrence refuse ends
in the library's own error, also where they make the outputs themselves."""
import pytest
import torch

from test_gpu_conv import make as make_conv
from test_gpu_ssm_scan import make as make_scan

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("cu,text", [
    (lambda: torch.zeros(0, dtype=torch.int32, device="cuda"), "at least one offset"),
    (lambda: torch.tensor(20, dtype=torch.int32, device="cuda"), "expected 1 dimensions"),
    (lambda: torch.zeros(1, 2, dtype=torch.int32, device="cuda"), "expected 1 dimensions"),
    (lambda: torch.tensor([0, 20], dtype=torch.int64, device="cuda"), "unsupported dtype"),
    (lambda: torch.tensor([0, 20], dtype=torch.int32), "one GPU"),
])
def test_offsets(cu, text):
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make_conv(1, 1, 20, 24, 4, BF, state=False)
    s, _ = make_scan(1, 1, 20, 2, 1, 64, 64, BF, F, state=False)
    args = [s[k] for k in ("x", "dt", "A", "b", "c")]
    for call in (lambda: gdr.short_conv_fwd(d["x"], d["w"], cu_seqlens=cu()),
                 lambda: gdr.short_conv_bwd(d["x"], d["w"], d["dy"], cu_seqlens=cu()),
                 lambda: gdr.ssm_scan_fwd(*args, cu_seqlens=cu()),
                 lambda: gdr.ssm_scan_bwd(*args, s["dy"], cu_seqlens=cu())):
        with pytest.raises(gdr.GdrError, match=text):
            call()


def test_taps():
    import chunked_gated_delta_fwd_amd as gdr
    d, _ = make_conv(1, 1, 20, 24, 4, BF, state=False)
    for taps in (0, 1, 5):
        w = torch.zeros(24, taps, dtype=BF, device="cuda")
        for call in (lambda: gdr.short_conv_fwd(d["x"], w), lambda: gdr.short_conv_bwd(d["x"], w, d["dy"])):
            with pytest.raises(gdr.GdrError, match="2, 3 or 4 taps" if taps else "w: "):
                call()
