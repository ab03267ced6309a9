"""GPU: attention gradients of keys that stand before no query at all: zero, with
rows behind the last sequence left as they were; and queries without any key."""
import pytest
import torch

from test_gpu_attn import BF, F, ints, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_keys_without_a_query(dtype, d, causal):
    import chunked_gated_delta_fwd_amd as gdr
    for cu, cuk, B, Tq, Tk in ((None, None, 2, 0, 150), ([0, 0], [0, 300], 1, 0, 303), ([0, 0, 0], [0, 70, 200], 1, 4, 200)):
        dev, _ = make(B, Tq, Tk, 4, 2, d, dtype, seed=71)
        C, CK = (None if x is None else ints(x) for x in (cu, cuk))
        o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], C, CK, causal=causal, o=torch.full_like(dev["q"], 7),
                              lse=torch.full(dev["q"].shape[:3], 7.0, device="cuda"))
        assert (o == 7).all() and (lse == 7).all()
        outs = [torch.full_like(dev[n], 7) for n in "qkv"]
        dq, dk, dv = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], C, CK, causal=causal, dq=outs[0], dk=outs[1],
                                  dv=outs[2])
        end = cuk[-1] if cuk else Tk
        assert not dk[:, :end].any() and not dv[:, :end].any()
        assert (dq == 7).all() and (dk[:, end:] == 7).all() and (dv[:, end:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_queries_without_a_key(dtype):
    import chunked_gated_delta_fwd_amd as gdr
    for cu, cuk, B, Tq, Tk in ((None, None, 2, 130, 0), ([0, 200], [0, 0], 1, 203, 0), ([0, 70, 200], [0, 0, 0], 1, 200, 5)):
        dev, _ = make(B, Tq, Tk, 4, 2, 64, dtype, seed=72)
        C, CK = (None if x is None else ints(x) for x in (cu, cuk))
        o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], C, CK, o=torch.full_like(dev["q"], 7),
                              lse=torch.full(dev["q"].shape[:3], 7.0, device="cuda"))
        end = cu[-1] if cu else Tq
        assert not o[:, :end].any() and (lse[:, :end] == -torch.inf).all() and (o[:, end:] == 7).all()
        outs = [torch.full_like(dev[n], 7) for n in "qkv"]
        dq, dk, dv = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], C, CK, dq=outs[0], dk=outs[1], dv=outs[2])
        assert not dq[:, :end].any() and (dq[:, end:] == 7).all() and (dk == 7).all() and (dv == 7).all()
