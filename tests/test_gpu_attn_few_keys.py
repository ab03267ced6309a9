"""GPU: which blocks of the bf16 gradient leave out the rounding of o.  It goes
by the keys that a block's queries see, wherever these lie in the kernel's tiles."""
import pytest
import torch

import attn_ref as ref
from mixer_ref import check
from test_gpu_attn import BF, ints, make, offsets

pytestmark = pytest.mark.gpu


# a block of 128 queries sees window + 127 keys, which begin at 128 i + Lk - Lq + 1 - window
@pytest.mark.parametrize("lq,lk,window,d", [
    ([256], [286], 40, 64),             # 167 keys, in four tiles of 64
    ([384], [384 + 63], 65, 128),       # 192 keys, the most, from a tile's last row on
    ([250, 128], [250 + 17, 128 + 190], 5, 64),
    ([512], [513], 64, 128),
])
def test_few_keys_at_any_place(lq, lk, window, d):
    import chunked_gated_delta_fwd_amd as gdr
    cu, cuk = offsets(lq), offsets(lk)
    dev, dbl = make(1, cu[-1], cuk[-1], 4, 2, d, BF, seed=61)
    o, lse = gdr.attn_fwd(dev["q"], dev["k"], dev["v"], ints(cu), ints(cuk), window=window)
    grads = gdr.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], ints(cu), ints(cuk), window=window)
    rg, tg = ref.gradient(*(dbl[n] for n in ("q", "k", "v", "do")), cu, cuk, window=window, dtype=BF, few=True)
    for name, got, r, t in zip(("dq", "dk", "dv"), grads, rg, tg):
        check(name, got, r, t)
