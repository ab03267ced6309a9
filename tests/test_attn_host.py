"""Host-only checks of attention and its paged cache: every refusal, on
descriptors with fake addresses that are never dereferenced, and workspaces."""
import ctypes

import pytest

import chunked_gated_delta_fwd_amd as gdr
from chunked_gated_delta_fwd_amd import GDR_BF16, GDR_F32, GDR_I32
from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import EALIAS, EDEVICE, EDTYPE, EINVAL, ESHAPE, ESTRIDE, Alloc2, call, has_gpu

pytestmark = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")

BF = GDR_BF16
T, S, HQ, HK, D, N = 20, 30, 4, 2, 64, 3


def fwd():
    A = Alloc()
    return dict(q=A(BF, [1, T, HQ, D]), k=A(BF, [1, S, HK, D]), v=A(BF, [1, S, HK, D]), cu=A(GDR_I32, [N + 1]),
                cuk=A(GDR_I32, [N + 1]), o=A(BF, [1, T, HQ, D]), lse=A(GDR_F32, [1, T, HQ]))


def bwd():
    A, f = Alloc2(), fwd()
    A.next = 1 << 45
    f.update(do=A(BF, [1, T, HQ, D]), dq=A(BF, [1, T, HQ, D]), dk=A(BF, [1, S, HK, D]), dv=A(BF, [1, S, HK, D]))
    return f


INPUTS = [
    (lambda d, A: d.update(q=None), EINVAL, "q: descriptor is NULL"),
    (lambda d, A: d.update(k=None), EINVAL, "k: descriptor is NULL"),
    (lambda d, A: d.update(v=None), EINVAL, "v: descriptor is NULL"),
    (lambda d, A: d.update(q=A(GDR_I32, [1, T, HQ, D])), EDTYPE, "q: dtype"),
    (lambda d, A: d.update(k=A(GDR_F32, [1, S, HK, D])), EDTYPE, "k: dtype"),
    (lambda d, A: d.update(v=A(GDR_F32, [1, S, HK, D])), EDTYPE, "v: dtype"),
    (lambda d, A: d.update(q=A(BF, [1, T, HQ, 96])), ESHAPE, "head dim"),
    (lambda d, A: d.update(q=A(BF, [T, HQ, D])), ESHAPE, "q: expected 4"),
    (lambda d, A: d.update(k=A(BF, [1, S, 3, D])), ESHAPE, "multiple of Hk"),
    (lambda d, A: d.update(k=A(BF, [1, S, 0, D])), ESHAPE, "head counts"),
    (lambda d, A: d.update(k=A(BF, [1, S, HK, 128])), ESHAPE, "k: shape"),
    (lambda d, A: d.update(v=A(BF, [1, S + 1, HK, D])), ESHAPE, "v: shape"),
    (lambda d, A: d.update(v=A(BF, [1, S, 1, D])), ESHAPE, "v: shape"),
    (lambda d, A: d.update(cuk=None), ESHAPE, "need cu_seqlens_k"),
    (lambda d, A: d.update(cu=None), EINVAL, "cu_seqlens_k without"),
    (lambda d, A: d.update(cu=A(GDR_F32, [N + 1])), EDTYPE, "cu_seqlens"),
    (lambda d, A: d.update(cuk=A(GDR_F32, [N + 1])), EDTYPE, "cu_seqlens_k"),
    (lambda d, A: d.update(cuk=A(GDR_I32, [N])), ESHAPE, "cu_seqlens_k: shape"),
    (lambda d, A: d.update(cu=A(GDR_I32, [0])), ESHAPE, "at least one offset"),
    (lambda d, A: d.update(q=A(BF, [2, T, HQ, D])), ESHAPE, "B == 1"),
    (lambda d, A: d.update(q=A(BF, [1, T, HQ, D], [0, 260, D, 1])), ESTRIDE, "16 bytes"),
    (lambda d, A: d.update(k=A(BF, [1, S, HK, D], [0, 200, 100, 1])), ESTRIDE, "row must be compact"),
    (lambda d, A: d.update(k=A(BF, [1, S, HK, D], [0, 1 << 25, D, 1])), ESTRIDE, "32 MiB apart"),
    (lambda d, A: d.update(v=A(BF, [1, S, HK, D], misalign=8)), EINVAL, "16-byte"),
]
FORWARD = [
    (lambda d, A: d.update(o=None), EINVAL, "o: descriptor is NULL"),
    (lambda d, A: d.update(o=A(GDR_F32, [1, T, HQ, D])), EDTYPE, "o: dtype"),
    (lambda d, A: d.update(o=A(BF, [1, T, HK, D])), ESHAPE, "o: shape"),
    (lambda d, A: d.update(lse=A(BF, [1, T, HQ])), EDTYPE, "lse: dtype"),
    (lambda d, A: d.update(lse=A(GDR_F32, [1, HQ, T])), ESHAPE, "lse: shape"),
    (lambda d, A: d.update(o=d["q"]), EALIAS, "o overlaps q"),
    (lambda d, A: d.update(o=A(BF, [1, T, HQ, D], [0, 512, D, 1])), ESTRIDE, "o: strides"),
    (lambda d, A: d.update(lse=None), EDEVICE, ""),
    (lambda d, A: d.update(q=A(BF, [1, T, HQ, D], [0, 512, D, 1])), EDEVICE, ""),
    (lambda d, A: None, EDEVICE, ""),
]


@pytest.mark.parametrize("change,status,text", INPUTS + FORWARD)
def test_forward_refusals(lib, change, status, text):  # noqa: F811
    d = fwd()
    change(d, Alloc2())
    got = call(lib, "attn_fwd", list(d.values()), 1, 0, 1.0, None, None)
    assert got[0] == status and text in got[1], got


@pytest.mark.parametrize("causal,window,scale,text", [
    (1, -1, 1.0, "window must not"), (0, 4, 1.0, "window needs"), (1, 0, float("nan"), "scale"), (1, 0, float("inf"), "scale")])
def test_scalars(lib, causal, window, scale, text):  # noqa: F811
    got = call(lib, "attn_fwd", list(fwd().values()), causal, window, scale, None, None)
    assert got[0] == EINVAL and text in got[1], got
    got = call(lib, "attn_bwd", list(bwd().values()), causal, window, scale, None, None)
    assert got[0] == EINVAL and text in got[1], got


def test_tokens_of_a_call(lib):  # noqa: F811
    A, d = Alloc2(), fwd()
    d.update(q=A(BF, [1, 1 << 30, 1, D]), k=A(BF, [1, (1 << 30) + 1, 1, D]), v=A(BF, [1, (1 << 30) + 1, 1, D]))
    got = call(lib, "attn_fwd", list(d.values()), 1, 0, 1.0, None, None)
    assert got[0] == ESHAPE and "2^30" in got[1], got


@pytest.mark.parametrize("B", [0, 1])
def test_calls_without_a_token(lib, B):  # noqa: F811
    """No batch, or rows of no token: nothing is divided by, and only the device check stops the call."""
    A, size = Alloc2(), ctypes.c_int64(-1)
    q, k = (A(BF, [B, 0, h, D]) for h in (HQ, HK))
    got = call(lib, "attn_fwd", [q, k, k, None, None, q, None], 1, 0, 1.0, None, None)
    assert got[0] == EDEVICE, got
    lse = A(GDR_F32, [B, 0, HQ])
    got = call(lib, "attn_bwd", [q, k, k, None, None, q, lse, q, q, k, k], 1, 0, 1.0, None, ctypes.addressof(size))
    assert got[0] == 0 and size.value == 0, got
    d = dict(q=A(BF, [0, HQ, D]), kp=A(BF, [0, 16, HK, D]), vp=A(BF, [0, 16, HK, D]), table=A(GDR_I32, [0, 0]),
             lens=A(GDR_I32, [0]), o=A(BF, [0, HQ, D]))
    assert call(lib, "attn_paged_step", list(d.values()), 0, 1.0, None, None)[0] == EDEVICE


def test_blocks_of_a_call(lib):  # noqa: F811
    A, n = Alloc2(), 1 << 22
    d = dict(q=A(BF, [n, 1, 1024, D]), k=A(BF, [n, 1, 1024, D]), v=A(BF, [n, 1, 1024, D]), cu=None, cuk=None,
             o=A(BF, [n, 1, 1024, D]), lse=None)
    got = call(lib, "attn_fwd", list(d.values()), 1, 0, 1.0, None, None)
    assert got[0] == ESHAPE and "blocks" in got[1], got


def test_forward_workspace(lib):  # noqa: F811
    """None where the blocks of a call fill the chip or their keys are few; for the runs of every block where a few queries
    stand before many keys; for those of the last ones where 540 blocks of one length come to 512 at a time."""
    def need(Tq, Tk, hq, hk, d):
        A, size = Alloc2(), ctypes.c_int64(-1)
        got = call(lib, "attn_fwd", [A(BF, [1, Tq, hq, d]), A(BF, [1, Tk, hk, d]), A(BF, [1, Tk, hk, d]), None, None,
                                     A(BF, [1, Tq, hq, d]), None], 0, 0, 1.0, None, ctypes.addressof(size))
        assert got[0] == 0, got
        return size.value
    assert need(T, S, HQ, HK, D) == 0
    assert need(128 * 64, 8192, 16, 4, 128) == 0                       # 1024 blocks
    assert need(1, 8192, 16, 4, 128) >= 2 * 4 * (128 + 2) * 16         # two runs at least, of every row
    last = need(128 * 27, 8192, 20, 5, 128)
    assert 2 * 28 * 128 * 4 * (128 + 2) <= last < 540 * 128 * 4 * (128 + 2)


@pytest.mark.parametrize("change,status,text", INPUTS + [
    (lambda d, A: d.update(o=None), EINVAL, "o: descriptor is NULL"),
    (lambda d, A: d.update(lse=None), EINVAL, "lse: descriptor is NULL"),
    (lambda d, A: d.update(do=None), EINVAL, "do: descriptor is NULL"),
    (lambda d, A: d.update(dk=None), EINVAL, "dk: descriptor is NULL"),
    (lambda d, A: d.update(o=A(GDR_F32, [1, T, HQ, D])), EDTYPE, "o: dtype"),
    (lambda d, A: d.update(do=A(BF, [1, T, HK, D])), ESHAPE, "do: shape"),
    (lambda d, A: d.update(dq=A(BF, [1, S, HQ, D])), ESHAPE, "dq: shape"),
    (lambda d, A: d.update(dk=A(BF, [1, S, HQ, D])), ESHAPE, "dk: shape"),
    (lambda d, A: d.update(dv=A(GDR_F32, [1, S, HK, D])), EDTYPE, "dv: dtype"),
    (lambda d, A: d.update(do=A(BF, [1, T, HQ, D], [0, 1 << 25, D, 1])), ESTRIDE, "32 MiB apart"),
    (lambda d, A: d.update(dq=d["do"]), EALIAS, "dq overlaps do"),
    (lambda d, A: d.update(dv=d["dk"]), EALIAS, "dv overlaps dk"),
    (lambda d, A: d.update(o=A(BF, [1, T, HQ, D], [0, 512, D, 1]), do=A(BF, [1, T, HQ, D], [0, 320, D, 1])), 0, ""),
    (lambda d, A: None, 0, ""),
])
def test_backward_refusals(lib, change, status, text):  # noqa: F811
    d = bwd()
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "attn_bwd", list(d.values()), 1, 0, 1.0, None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert (size.value > 0) == (status == 0)


def test_backward_workspace(lib):  # noqa: F811
    size = ctypes.c_int64(-1)
    assert call(lib, "attn_bwd", list(bwd().values()), 1, 0, 1.0, None, ctypes.addressof(size))[0] == 0
    need = size.value
    assert need >= 8 * T * HQ
    for given, address, text in ((need - 1, 1 << 50, "needed"), (need, (1 << 50) + 8, "16-byte")):
        size.value = given
        got = call(lib, "attn_bwd", list(bwd().values()), 1, 0, 1.0, address, ctypes.addressof(size))
        assert got[0] == EINVAL and text in got[1], got
    got = call(lib, "attn_bwd", list(bwd().values()), 1, 0, 1.0, 1 << 50, None)
    assert got[0] == EINVAL and "size is missing" in got[1], got
    # without a sequence no token is looked at
    A, d = Alloc2(), bwd()
    d.update(cu=A(GDR_I32, [1]), cuk=A(GDR_I32, [1]))
    assert call(lib, "attn_bwd", list(d.values()), 1, 0, 1.0, None, ctypes.addressof(size))[0] == 0 and size.value == 0


def test_backward_workspace_of_few_blocks(lib):  # noqa: F811
    """8 bytes a query and head where the blocks fill the chip; sums of shared blocks beside them where they are few."""
    def need(B, Tn, hq, hk, d):
        A, size = Alloc2(), ctypes.c_int64(-1)
        q, k = [A(GDR_F32, [B, Tn, hq, d]) for _ in range(4)], [A(GDR_F32, [B, Tn, hk, d]) for _ in range(4)]
        got = call(lib, "attn_bwd", [q[0], k[0], k[1], None, None, q[1], A(GDR_F32, [B, Tn, hq]), q[2], q[3], k[2], k[3]], 1, 0, 1.0,
                   None, ctypes.addressof(size))
        assert got[0] == 0, got
        return size.value
    assert need(64, 512, 4, 4, 64) == 8 * 64 * 512 * 4               # 1024 blocks
    assert need(1, 900, 2, 1, 128) >= 8 * 900 * 2 + 2 * 8 * 128 * 900 * 2 + 2 * 4 * 128 * 900 * 2


def step(P=9, page=16, M=5):
    A = Alloc()
    return dict(q=A(BF, [N, HQ, D]), kp=A(BF, [P, page, HK, D]), vp=A(BF, [P, page, HK, D]), table=A(GDR_I32, [N, M]),
                lens=A(GDR_I32, [N]), o=A(BF, [N, HQ, D]))


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(q=None), EINVAL, "q: descriptor is NULL"),
    (lambda d, A: d.update(kp=None), EINVAL, "k_pages: descriptor is NULL"),
    (lambda d, A: d.update(lens=None), EINVAL, "lens: descriptor is NULL"),
    (lambda d, A: d.update(q=A(BF, [N, HQ, 32])), ESHAPE, "head dim"),
    (lambda d, A: d.update(q=A(BF, [N, 3, D])), ESHAPE, "multiple of Hk"),
    (lambda d, A: d.update(kp=A(GDR_F32, [9, 16, HK, D])), EDTYPE, "k_pages: dtype"),
    (lambda d, A: d.update(kp=A(BF, [9, 16, HK, 128])), ESHAPE, "k_pages: shape"),
    (lambda d, A: d.update(vp=A(BF, [9, 8, HK, D])), ESHAPE, "v_pages: shape"),
    (lambda d, A: d.update(kp=A(BF, [9, 0, HK, D])), ESHAPE, "pages of 1 to 65536"),
    (lambda d, A: d.update(kp=A(BF, [1 << 27, 16, HK, D]), vp=A(BF, [1 << 27, 16, HK, D])), ESHAPE, "2^31 - 1 tokens"),
    (lambda d, A: d.update(table=A(GDR_I32, [N, 1 << 27])), ESHAPE, "2^30 tokens"),
    (lambda d, A: d.update(table=A(GDR_F32, [N, 5])), EDTYPE, "block_table"),
    (lambda d, A: d.update(table=A(GDR_I32, [N + 1, 5])), ESHAPE, "block_table: shape"),
    (lambda d, A: d.update(lens=A(GDR_I32, [N + 1])), ESHAPE, "lens: shape"),
    (lambda d, A: d.update(o=A(BF, [N, HK, D])), ESHAPE, "o: shape"),
    (lambda d, A: d.update(o=d["q"]), EALIAS, "o overlaps q"),
    (lambda d, A: d.update(kp=A(BF, [9, 16, HK, D], [4096, 256, 64, 1])), ESTRIDE, "k_pages: strides"),
    (lambda d, A: None, 0, ""),
    (lambda d, A: d.update(q=A(BF, [N, HQ, D], [1000, D, 1])), 0, ""),
])
def test_step_refusals(lib, change, status, text):  # noqa: F811
    d = step()
    change(d, Alloc2())
    size = ctypes.c_int64(-1)
    got = call(lib, "attn_paged_step", list(d.values()), 0, 1.0, None, ctypes.addressof(size))
    assert got[0] == status and text in got[1], got
    assert (size.value >= 0) == (status == 0)


def test_step_workspace(lib):  # noqa: F811
    size = ctypes.c_int64(-1)
    for M, window, some in ((1, 0, False), (300, 0, True), (300, 10, False)):   # one chunk needs none
        got = call(lib, "attn_paged_step", list(step(M=M).values()), window, 1.0, None, ctypes.addressof(size))
        assert got[0] == 0 and (size.value > 0) == some, (M, size.value)
    for window, scale, text in ((-1, 1.0, "window"), (0, float("nan"), "scale")):
        got = call(lib, "attn_paged_step", list(step().values()), window, scale, None, None)
        assert got[0] == EINVAL and text in got[1], got


@pytest.mark.parametrize("change,status,text", [
    (lambda d, A: d.update(k=None), EINVAL, "k: descriptor is NULL"),
    (lambda d, A: d.update(slots=None), EINVAL, "slots: descriptor is NULL"),
    (lambda d, A: d.update(v=A(BF, [2, 6, HK, D])), ESHAPE, "v: shape"),
    (lambda d, A: d.update(v=A(GDR_F32, [2, 5, HK, D])), EDTYPE, "v: dtype"),
    (lambda d, A: d.update(slots=A(GDR_I32, [5, 2])), ESHAPE, "slots: shape"),
    (lambda d, A: d.update(slots=A(GDR_F32, [2, 5])), EDTYPE, "slots: dtype"),
    (lambda d, A: d.update(kp=A(BF, [9, 16, HK, 128])), ESHAPE, "k_pages: shape"),
    (lambda d, A: d.update(vp=A(GDR_F32, [9, 16, HK, D])), EDTYPE, "v_pages: dtype"),
    (lambda d, A: d.update(k=A(BF, [1, 1, 1, 12]), v=A(BF, [1, 1, 1, 12])), ESHAPE, "multiple of 16 bytes"),
    (lambda d, A: d.update(vp=d["kp"]), EALIAS, "v_pages overlaps k_pages"),
    (lambda d, A: d.update(k=A(BF, [2, 5, HK, D], [1500, 300, D, 1])), ESTRIDE, "16 bytes"),
    (lambda d, A: d.update(k=A(BF, [2, 5, HK, D], [2000, 400, D, 1])), EDEVICE, ""),
])
def test_store_refusals(lib, change, status, text):  # noqa: F811
    A = Alloc()
    d = dict(k=A(BF, [2, 5, HK, D]), v=A(BF, [2, 5, HK, D]), slots=A(GDR_I32, [2, 5]), kp=A(BF, [9, 16, HK, D]),
             vp=A(BF, [9, 16, HK, D]))
    change(d, Alloc2())
    got = call(lib, "page_store", list(d.values()))
    assert got[0] == status and text in got[1], got


@pytest.mark.parametrize("change,page,status,text", [
    (lambda d, A: d.update(past=None), 16, EINVAL, "past: descriptor is NULL"),
    (lambda d, A: d.update(new=A(GDR_I32, [N + 1])), 16, ESHAPE, "new: shape"),
    (lambda d, A: d.update(new=A(GDR_F32, [N])), 16, EDTYPE, "new: dtype"),
    (lambda d, A: d.update(table=A(GDR_I32, [N + 1, 5])), 16, ESHAPE, "block_table: shape"),
    (lambda d, A: d.update(cu=A(GDR_I32, [N])), 16, ESHAPE, "cu_seqlens: shape"),
    (lambda d, A: d.update(lens=A(GDR_I32, [N + 1])), 16, ESHAPE, "lens: shape"),
    (lambda d, A: d.update(positions=A(GDR_I32, [2, 50])), 16, ESHAPE, "positions: shape"),
    (lambda d, A: d.update(slots=A(GDR_I32, [1, 49])), 16, ESHAPE, "slots: shape"),
    (lambda d, A: d.update(used=A(GDR_I32, [1])), 16, ESHAPE, "used: shape"),
    (lambda d, A: None, 0, ESHAPE, "1 to 65536"),
    (lambda d, A: None, 65537, ESHAPE, "1 to 65536"),
    (lambda d, A: d.update(table=A(GDR_I32, [N, 1 << 27])), 16, ESHAPE, "2^30 tokens"),
    (lambda d, A: d.update(lens=d["past"]), 16, EALIAS, "lens overlaps past"),
    (lambda d, A: d.update(slots=d["positions"]), 16, EALIAS, "slots overlaps positions"),
    (lambda d, A: d.update(pool=A(GDR_I32, [0])), 16, EDEVICE, ""),
    (lambda d, A: None, 16, EDEVICE, ""),
])
def test_plan_refusals(lib, change, page, status, text):  # noqa: F811
    A = Alloc()
    d = dict(past=A(GDR_I32, [N]), new=A(GDR_I32, [N]), pool=A(GDR_I32, [20]), table=A(GDR_I32, [N, 5]), cu=A(GDR_I32, [N + 1]),
             lens=A(GDR_I32, [N]), positions=A(GDR_I32, [1, 50]), slots=A(GDR_I32, [1, 50]), used=A(GDR_I32, [2]))
    change(d, Alloc2())
    got = call(lib, "page_plan", list(d.values()), page)
    assert got[0] == status and text in got[1], got


def test_python_calls_refuse_host_memory():
    import torch
    x = torch.zeros(1, 4, 2, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    for f in (lambda: gdr.attn_fwd(x, x, x), lambda: gdr.attn_bwd(x, x, x, x, x[..., 0], x),
              lambda: gdr.attn_paged_step(x[0], x, x, i, i[0]), lambda: gdr.page_store(x, x, i, x, x),
              lambda: gdr.page_plan(i[0], i[0], i[0], i, 16, 4)):
        with pytest.raises(gdr.GdrError, match="one GPU"):
            f()
