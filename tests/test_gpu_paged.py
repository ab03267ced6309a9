"""GPU: one token over the paged cache against the plain fp64 evaluation
(attn_ref.py derives the tolerances); page plans and stores, exactly."""
import random

import pytest
import torch

import attn_ref as ref
from mixer_ref import check

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32

STEPS = [   # lens, page, hq, hk, d, dtype, window
    ([1], 16, 1, 1, 64, BF, 0),
    ([0, 1, 2], 1, 2, 1, 128, F, 0),
    ([31, 32, 33, 0, 64, 65], 24, 6, 3, 64, BF, 0),
    ([700, 3, 129], 16, 16, 2, 128, BF, 0),
    ([700, 64, 0], 7, 8, 8, 64, F, 0),
    ([500, 20, 41], 64, 33, 1, 64, BF, 0),          # more than 32 query heads on a key head
    ([300, 2000], 128, 70, 1, 128, F, 0),
    ([900, 30, 100], 24, 7, 1, 128, BF, 1),
    ([900, 30, 100], 24, 4, 2, 64, BF, 100),
    ([9000, 5000], 100, 4, 1, 128, BF, 0),
]


def pages_of(lens, page, hk, d, dtype, seed=1, spare=2):
    """(k, v pages with NaN where no key is, table as lists): pages in a random order."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + spare
    order = torch.randperm(P, generator=g).tolist()
    kp, vp = (torch.full((P, page, hk, d), torch.nan, dtype=dtype) for _ in range(2))
    width, table, used = max(1, max(counts, default=0)), [], 0
    for n, count in zip(lens, counts):
        row = order[used:used + count]
        used += count
        for i, p in enumerate(row):
            rows = min(page, n - i * page)
            for x in (kp, vp):
                x[p, :rows] = torch.randn(rows, hk, d, generator=g).to(dtype)
        table.append(row + [-1] * (width - count))
    return kp, vp, table


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(n, hq, d, dtype, seed=2):
    return (2 * torch.randn(n, hq, d, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("lens,page,hq,hk,d,dtype,window", STEPS)
def test_step(lens, page, hq, hk, d, dtype, window):
    import chunked_gated_delta_fwd_amd as gdr
    kp, vp, table = pages_of(lens, page, hk, d, dtype)
    q = queries(len(lens), hq, d, dtype)
    wide = torch.cat([q, q.new_full((len(lens), 3, d), torch.nan)], 1).cuda()   # a slice of a wider projection
    o = gdr.attn_paged_step(wide[:, :hq], kp.cuda(), vp.cuda(), ints(table), ints(lens), window=window)
    torch.cuda.synchronize()
    check("o", o, *ref.paged(q.double(), kp.double(), vp.double(), table, lens, window, dtype=dtype))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("dtype", [BF, F])
def test_step_scales(dtype, scale):
    import chunked_gated_delta_fwd_amd as gdr
    lens = [40, 200]
    kp, vp, table = pages_of(lens, 16, 2, 64, dtype)
    q = queries(2, 4, 64, dtype)
    o = gdr.attn_paged_step(q.cuda(), kp.cuda(), vp.cuda(), ints(table), ints(lens), scale=scale)
    check("o", o, *ref.paged(q.double(), kp.double(), vp.double(), table, lens, scale=scale, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, F])
def test_pages_that_are_not_there_and_lengths_out_of_range(dtype):
    """Entries outside the pool stand for pages without keys; lens past the table or below zero end at its bounds."""
    import chunked_gated_delta_fwd_amd as gdr
    lens = [150, 150, 96, 60, 10]
    kp, vp, table = pages_of(lens, 16, 1, 64, dtype)
    table[0][3] = -1
    table[0][7] = 10 ** 6
    table[1] = [-5] * len(table[1])
    table[2][0] = 2 ** 31 - 1
    asked = [150, 150, 2 ** 31 - 1, -7, 10]
    for row, n in ((2, 96), (4, 10)):
        table[row] = table[row][:-(-n // 16)] + [-1] * (len(table[row]) - -(-n // 16))
    q = queries(5, 3, 64, dtype)
    for window in (0, 70):
        o = gdr.attn_paged_step(q.cuda(), kp.cuda(), vp.cuda(), ints(table), ints(asked), window=window)
        torch.cuda.synchronize()
        r, t = ref.paged(q.double(), kp.double(), vp.double(), table, asked, window, dtype=dtype)
        check("o", o, r, t)
        assert (o[1] == 0).all() and (o[3] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_one_sequence_does_not_reach_another(dtype):
    import chunked_gated_delta_fwd_amd as gdr
    lens = [100, 100, 100]
    kp, vp, table = pages_of(lens, 24, 2, 64, dtype)
    q = queries(3, 4, 64, dtype).cuda()
    args = ints(table), ints(lens)
    want = gdr.attn_paged_step(q, kp.cuda(), vp.cuda(), *args)
    assert torch.isfinite(want).all()
    for x in (kp, vp):
        y = x.clone()
        y[table[1][2], 5] = float("nan")
        got = gdr.attn_paged_step(q, (y if x is kp else kp).cuda(), (y if x is vp else vp).cuda(), *args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and not torch.isfinite(got[1]).all(-1).any()


def test_step_is_the_last_row_of_the_forward():
    """A prompt's keys stored in pages: the step of its last token is attn_fwd's last row."""
    import chunked_gated_delta_fwd_amd as gdr
    g = torch.Generator().manual_seed(3)
    T, hq, hk, d = 333, 8, 2, 128
    q, k, v = (torch.randn(1, T, h, d, generator=g).cuda() for h in (hq, hk, hk))
    for window in (0, 50):
        o, _ = gdr.attn_fwd(q, k, v, window=window)
        kp, vp = (torch.full((30, 16, hk, d), torch.nan, device="cuda") for _ in range(2))
        table = torch.full((1, 25), -1, dtype=torch.int32, device="cuda")
        _, lens, _, slots, _ = gdr.page_plan(ints([0]), ints([T]), ints(random.Random(1).sample(range(30), 30)), table, 16, T)
        gdr.page_store(k, v, slots, kp, vp)
        got = gdr.attn_paged_step(q[:, -1], kp, vp, table, lens, window=window)
        # both are within the fp32 tolerance of the same values
        t = ref.paged(q[:, -1].double().cpu(), kp.double().cpu(), vp.double().cpu(), table.tolist(), [T], window)[1]
        check("o", got, o[:, -1].double().cpu(), 2 * t)


def test_cache_past_4_gib():
    """Rows of the pages past 2^32 bytes."""
    import chunked_gated_delta_fwd_amd as gdr
    hk, d, page, P = 8, 128, 64, 40000   # 128 KiB a page: 5.2 GB each
    kp, vp = (torch.empty(P, page, hk, d, dtype=BF, device="cuda") for _ in range(2))
    rows = [39999, 0, 33000, 39000]
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(1, 4 * page, hk, d, generator=g).to(BF) for _ in range(2))
    slots = torch.cat([torch.arange(p * page, (p + 1) * page) for p in rows]).int()[None]
    gdr.page_store(k.cuda(), v.cuda(), slots.cuda(), kp, vp)
    for i, p in enumerate(rows):
        assert torch.equal(kp[p].cpu(), k[0, i * page:(i + 1) * page]) and torch.equal(vp[p].cpu(), v[0, i * page:(i + 1) * page])
    q = queries(1, 8, d, BF)
    o = gdr.attn_paged_step(q.cuda(), kp, vp, ints([rows]), ints([250]))
    small = [x[0].reshape(4, page, hk, d).double() for x in (k, v)]
    check("o", o, *ref.paged(q.double(), *small, [[0, 1, 2, 3]], [250], dtype=BF))


def test_step_in_a_graph_follows_its_lengths():
    """Captured once; lengths, table and pages change between replays, and eager calls use the library's workspace."""
    import chunked_gated_delta_fwd_amd as gdr
    page, hk, d = 16, 2, 128
    kp, vp, table = pages_of([600, 600, 600], page, hk, d, BF, seed=5)
    q = queries(3, 8, d, BF)
    K, V, Q, Tb, L = kp.cuda(), vp.cuda(), q.cuda(), ints(table), ints([600, 600, 600])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdr.attn_paged_step(Q, K, V, Tb, L)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdr.attn_paged_step(Q, K, V, Tb, L)
    for lens in ([600, 600, 600], [0, 33, 599], [64, 65, 1], [600, 600, 600]):
        L.copy_(ints(lens))
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        kept = o.clone()
        eager = gdr.attn_paged_step(Q, K, V, Tb, L)
        assert torch.equal(kept, eager)
        check("o", o, *ref.paged(q.double(), kp.double(), vp.double(), table, lens, dtype=BF))


PLANS = [   # past, new, free pages, width, page, tokens past the last
    ([0], [1], 1, 1, 16, 0),
    ([0, 16, 15, 17, 0], [0, 1, 1, 1, 0], 5, 4, 16, 3),
    ([5, 0, 100, 31], [40, 129, 1, 0], 20, 8, 24, 0),
    ([5, 0, 100], [40, 129, 1], 3, 8, 24, 0),            # pages run out
    ([5, 0, 100], [40, 129, 1], 20, 4, 24, 5),           # the table is too narrow
    ([-4, 3], [2, -8], 4, 3, 4, 1),
    ([7] * 9, [1] * 9, 9, 10, 1, 0),
    ([], [], 2, 3, 16, 4),
    ([3, 4], [5, 6], 0, 2, 8, 0),
    ([1000], [3000], 50, 70, 64, 0),
    ([i % 50 for i in range(2500)], [i % 3 for i in range(2500)], 900, 8, 8, 7),
]


@pytest.mark.parametrize("past,new,free,width,page,more", PLANS)
def test_plan(past, new, free, width, page, more):
    import chunked_gated_delta_fwd_amd as gdr
    r = random.Random(5)
    pool = r.sample(range(4000), free)
    table = [[r.randrange(4000, 9000) for _ in range(width)] for _ in past]
    tokens = sum(max(0, x) for x in new) + more
    for capacity in (tokens, tokens // 2):               # all tokens, and fewer than there are
        T = torch.tensor(table, dtype=torch.int32).reshape(len(past), width).cuda()
        cu, lens, positions, slots, used = gdr.page_plan(ints(past), ints(new), ints(pool), T, page, capacity)
        want = ref.plan(past, new, pool, table, page, capacity)
        got = (T.tolist(), cu.tolist(), lens.tolist(), positions[0].tolist(), slots[0].tolist(), used.tolist())
        assert positions.shape == slots.shape == (1, capacity)
        for what, a, b in zip(("table", "cu", "lens", "positions", "slots", "used"), got, want):
            assert a == b, what


def test_plan_of_one_long_prompt():
    """Blocks share a long prompt's tokens; sums past 2^31 stay at it."""
    import chunked_gated_delta_fwd_amd as gdr
    n = 200000
    table = torch.full((1, 3200), -1, dtype=torch.int32, device="cuda")
    _, _, positions, slots, used = gdr.page_plan(ints([10]), ints([n]), torch.arange(3200, 0, -1, device="cuda").int(), table, 64, n)
    at = torch.arange(10, 10 + n, device="cuda")
    assert torch.equal(positions[0], at.int()) and used.tolist() == [n, -(-(n + 10) // 64) - 1]
    page = torch.where(at // 64 == 0, -1, 3200 - (at // 64 - 1))
    assert torch.equal(slots[0], torch.where(page < 0, -1, page * 64 + at % 64).int())
    big = 2 ** 31 - 1
    table = torch.full((2, 4), 3, dtype=torch.int32, device="cuda")
    cu, lens, _, slots, used = gdr.page_plan(ints([big, 0]), ints([big, big]), ints([1, 2]), table, 65536, 5)
    # sequence 0 has more tokens than its row of the table has places: nowhere to go
    assert lens.tolist() == [big, big] and used.tolist() == [big, 65536] and cu.tolist() == [0, 5, 5]
    assert slots.tolist() == [[-1] * 5] and table.tolist() == [[3] * 4, [-1] * 4]


@pytest.mark.parametrize("B,T,hk,d,page,dtype", [(1, 1, 1, 64, 16, BF), (2, 37, 3, 128, 24, F), (1, 1000, 8, 64, 1, BF),
                                                 (3, 5, 1, 24, 7, BF)])
def test_store(B, T, hk, d, page, dtype):
    import chunked_gated_delta_fwd_amd as gdr
    g = torch.Generator().manual_seed(6)
    P = -(-B * T // page) + 2
    wide = torch.randn(B, T, 2 * hk, d, generator=g).to(dtype).cuda()
    wide[0, 0, 0, 0] = float("nan")                       # copied as it is
    k, v = wide[:, :, :hk], wide[:, :, hk:]
    slots = torch.randperm(P * page, generator=g)[:B * T].int()
    slots[1::7] = -1
    slots[2::7] = P * page
    slots[3::11] = -2 ** 31
    kp, vp = (torch.randn(P, page, hk, d, generator=g).to(dtype).cuda() for _ in range(2))
    want = [x.clone() for x in (kp, vp)]
    gdr.page_store(k, v, slots.reshape(B, T).cuda(), kp, vp)
    there = (slots >= 0) & (slots < P * page)
    for x, pages, w in ((k, kp, want[0]), (v, vp, want[1])):
        w.flatten(0, 1)[slots[there].long().cuda()] = x.flatten(0, 1)[there.cuda()]
        assert torch.equal(pages.view(torch.int16), w.view(torch.int16))


def test_plan_into_given_tensors():
    import chunked_gated_delta_fwd_amd as gdr
    want = gdr.page_plan(ints([3, 0]), ints([2, 5]), ints([7, 8, 9]), torch.full((2, 4), 1, dtype=torch.int32, device="cuda"), 4, 7)
    outs = [torch.full_like(x, 77) for x in want]
    for given in (dict(zip(("cu_seqlens", "lens", "positions", "slots", "used"), outs)), dict(lens=outs[1], slots=outs[3])):
        got = gdr.page_plan(ints([3, 0]), ints([2, 5]), ints([7, 8, 9]), torch.full((2, 4), 1, dtype=torch.int32, device="cuda"),
                            4, 7, **given)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert got[1].data_ptr() == outs[1].data_ptr() and all(x.is_contiguous() for x in got)
    some = dict(cu_seqlens=outs[0], lens=outs[1], used=outs[4])
    got = gdr.page_plan(ints([3, 0]), ints([0, 0]), ints([7]), torch.full((2, 4), 1, dtype=torch.int32, device="cuda"), 4, 0, **some)
    assert got[2].shape == got[3].shape == (1, 0) and got[4].tolist() == [0, 0]


def test_refusals():
    import chunked_gated_delta_fwd_amd as gdr
    kp, vp, table = pages_of([40], 16, 2, 64, BF)
    kp, vp, q = kp.cuda(), vp.cuda(), queries(1, 4, 64, BF).cuda()
    T, L = ints(table), ints([40])
    for call, text in (
            (lambda: gdr.attn_paged_step(q, kp, vp, T.long(), L), "unsupported dtype"),
            (lambda: gdr.attn_paged_step(q, kp, vp, T, L.cpu()), "one GPU"),
            (lambda: gdr.attn_paged_step(q, kp, vp[:, :, :1], T, L), "v_pages"),
            (lambda: gdr.attn_paged_step(q, kp.float(), vp, T, L), "k_pages: dtype"),
            (lambda: gdr.attn_paged_step(q[:, :3], kp, vp, T, L), "multiple of Hk"),
            (lambda: gdr.attn_paged_step(q, kp, vp, T, L, window=-1), "window"),
            (lambda: gdr.attn_paged_step(q, kp, vp, T, L, scale=float("nan")), "scale"),
            (lambda: gdr.attn_paged_step(q, kp, vp, T, L, o=q), "o overlaps q"),
            (lambda: gdr.page_store(kp[:1], vp[:1], ints([[0] * 16]), kp, vp), "overlaps"),
            (lambda: gdr.page_store(q[None], q[None], ints([[0]]), kp, vp), "k_pages: shape"),
            (lambda: gdr.page_plan(L, ints([1, 2]), L, T, 16, 4), "new: shape"),
            (lambda: gdr.page_plan(L, ints([1]), T[0], T, 16, 4), "block_table overlaps free_pages"),
            (lambda: gdr.page_plan(L, ints([1]), L, T, 0, 4), "page"),
            (lambda: gdr.page_plan(L, ints([1]), L, T, 2 ** 32 + 16, 4), "page"),
            (lambda: gdr.page_plan(L, ints([1]), L, T, 16, -1), "tokens"),
            (lambda: gdr.page_plan(L, ints([1]), L, T, 16, 2 ** 40), "tokens")):
        with pytest.raises(gdr.GdrError, match=text):
            call()
