"""Slots and positions of packed tokens without the row of a batch, [tokens]:
what the store takes and the plan fills."""
import pytest

from chunked_gated_delta_fwd_amd import GDR_BF16, GDR_F32, GDR_I32
from test_abi_host import Alloc, lib  # noqa: F401
from test_mixer_host import EDEVICE, EDTYPE, ESHAPE, call, has_gpu

BF, T = GDR_BF16, 50
host = pytest.mark.skipif(has_gpu(), reason="fake addresses, for a machine without a GPU")


@host
@pytest.mark.parametrize("B,shape,dtype,status,text", [
    (1, [5], GDR_I32, EDEVICE, ""), (2, [10], GDR_I32, EDEVICE, ""), (2, [5], GDR_I32, ESHAPE, "slots: shape"),
    (1, [6], GDR_I32, ESHAPE, "slots: shape"), (1, [5], GDR_F32, EDTYPE, "slots: dtype"),
    (1, [1, 1, 5], GDR_I32, ESHAPE, "slots: expected 2")])
def test_store_shapes(lib, B, shape, dtype, status, text):  # noqa: F811
    A = Alloc()
    d = [A(BF, [B, 5, 2, 64]), A(BF, [B, 5, 2, 64]), A(dtype, shape), A(BF, [9, 16, 2, 64]), A(BF, [9, 16, 2, 64])]
    got = call(lib, "page_store", d)
    assert got[0] == status and text in got[1], got


@host
@pytest.mark.parametrize("positions,slots,status,text", [
    ([T], [T], EDEVICE, ""), ([1, T], [T], EDEVICE, ""), ([T], [1, T], EDEVICE, ""), ([T], [T - 1], ESHAPE, "slots: shape"),
    ([T], [1, T - 1], ESHAPE, "slots: shape"), ([1, T, 1], [T], ESHAPE, "positions: expected 2")])
def test_plan_shapes(lib, positions, slots, status, text):  # noqa: F811
    A = Alloc()
    i = lambda *s: A(GDR_I32, list(s))  # noqa: E731
    got = call(lib, "page_plan", [i(3), i(3), i(20), i(3, 5), i(4), i(3), i(*positions), i(*slots), i(2)], 16)
    assert got[0] == status and text in got[1], got


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3])
def test_tokens_are_planned_and_stored_as_in_rows(B):
    import torch

    import chunked_gated_delta_fwd_amd as gdr

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    past, new = ints([3, 0, 17]), ints([6, 11, 4])
    table = [torch.full((3, 8), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    rows = gdr.page_plan(past, new, torch.arange(40, 20, -1, device="cuda").int(), table[0], 4, 21)
    flat = gdr.page_plan(past, new, torch.arange(40, 20, -1, device="cuda").int(), table[1], 4, 21,
                         positions=torch.full((21,), 7, dtype=torch.int32, device="cuda"),
                         slots=torch.full((21,), 7, dtype=torch.int32, device="cuda"))
    assert torch.equal(*table) and flat[2].shape == flat[3].shape == (21,)
    for a, b in zip(rows, flat):
        assert torch.equal(a.flatten(), b)
    k, v = (torch.randn(B, 21 // B, 2, 64, device="cuda") for _ in range(2))
    pages = [torch.zeros(41, 4, 2, 64, device="cuda") for _ in range(4)]
    gdr.page_store(k, v, flat[3].reshape(B, -1), *pages[:2])
    gdr.page_store(k, v, flat[3], *pages[2:])
    assert torch.equal(pages[0], pages[2]) and torch.equal(pages[1], pages[3]) and pages[0].any()
