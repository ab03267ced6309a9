"""Host-only: calls of more blocks than a launch holds are refused by name.  A
launch has fewer than 2^32 threads along x, 2^24 - 1 blocks of 256."""
import ctypes

import pytest

from chunked_gated_delta_fwd_amd import GDR_BF16, GDR_F32, GDR_I32
from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import EDEVICE, ESHAPE, call, has_gpu

pytestmark = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")

BF, H, D = GDR_BF16, 16, 64


def refused(got, status):
    assert got[0] == status, got
    assert status != ESHAPE or "blocks" in got[1], got


@pytest.mark.parametrize("n,status", [((1 << 20) - 1, 0), (1 << 20, ESHAPE), (1 << 24, ESHAPE)])
def test_attention(lib, n, status):  # noqa: F811
    A, size = Alloc(), ctypes.c_int64(-1)
    q, k, v, o, do, dq, dk, dv = (A(BF, [n, 1, H, D]) for _ in range(8))
    lse = A(GDR_F32, [n, 1, H])
    refused(call(lib, "attn_fwd", [q, k, v, None, None, o, lse], 1, 0, 1.0, None, ctypes.addressof(size)), status)
    refused(call(lib, "attn_bwd", [q, k, v, None, None, o, lse, do, dq, dk, dv], 1, 0, 1.0, None, ctypes.addressof(size)), status)


@pytest.mark.parametrize("n,status", [((1 << 20) - 1, 0), (1 << 20, ESHAPE)])
def test_step(lib, n, status):  # noqa: F811
    A, size = Alloc(), ctypes.c_int64(-1)
    d = [A(BF, [n, H, D]), A(BF, [9, 16, H, D]), A(BF, [9, 16, H, D]), A(GDR_I32, [n, 1]), A(GDR_I32, [n]), A(BF, [n, H, D])]
    refused(call(lib, "attn_paged_step", d, 0, 1.0, None, ctypes.addressof(size)), status)


@pytest.mark.parametrize("tokens,status", [((1 << 24) - 1, EDEVICE), (1 << 24, ESHAPE)])
def test_store(lib, tokens, status):  # noqa: F811
    A = Alloc()
    k, v = (A(BF, [1, tokens, 1, 1024]) for _ in range(2))
    kp, vp = (A(BF, [9, 16, 1, 1024]) for _ in range(2))
    refused(call(lib, "page_store", [k, v, A(GDR_I32, [1, tokens]), kp, vp]), status)
