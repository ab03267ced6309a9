"""Cases, plain forms and exact values of softmax attention as it stands beside
the recurrent layers of a stack, and of the paged key-value cache it decodes from:

* ``attn``: attention over packed or equal rows with shared key heads, causal,
  with a window or neither (forward, gradient);
* ``token``: one new token of every sequence over keys and values in pages;
* ``plan``: page tables, slots and positions of new tokens from lengths;
* ``store``: new keys and values into the pages.

Where ``own`` is false, ``run`` computes them from elementary torch operations
in fp32; where it is true, it calls the framework's kernels.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


# --- cases ---------------------------------------------------------------------

def listed():
    return [
        # two long prompts, 32 query heads on 4 key heads
        dict(name="attn_prompt_2x8192", op="attn", way="fwd", dtype=BF16, batch=2, tokens=8192, n_seq=2, ghosts=0, past=0,
             hq=32, hk=4, d=128, causal=True, window=0, cut=0),
        # the next 512 tokens or so of each of 8 prompts, behind some 4000 earlier keys
        dict(name="attn_piece_8x512", op="attn", way="fwd", dtype=BF16, batch=0, tokens=4096, n_seq=8, ghosts=1, past=4000,
             hq=16, hk=2, d=128, causal=True, window=0, cut=1),
        # fp32, ragged, some sequences with fewer keys than queries: their first rows see none
        dict(name="attn_odd_f32", op="attn", way="fwd", dtype=F32, batch=0, tokens=701, n_seq=9, ghosts=2, past=-60,
             hq=6, hk=3, d=64, causal=True, window=0, cut=2),
        # a training step on fixed rows
        dict(name="attn_train_4x4096", op="attn", way="bwd", dtype=BF16, batch=4, tokens=4096, n_seq=4, ghosts=0, past=0,
             hq=32, hk=4, d=128, causal=True, window=0, cut=0),
        # a training step on packed documents, 64-channel heads that look 512 tokens back
        dict(name="attn_train_packed", op="attn", way="bwd", dtype=BF16, batch=0, tokens=8191, n_seq=7, ghosts=2, past=0,
             hq=16, hk=4, d=64, causal=True, window=512, cut=3),
        # a decode step of 64 requests, 4096 to 8192 tokens each (0.8 GB of keys and values)
        dict(name="token_64x8192", op="token", dtype=BF16, n_seq=64, least=4096, longest=8192, hq=32, hk=4, d=128, page=64,
             window=0, cut=4),
        # one request with a long past
        dict(name="token_1x131072", op="token", dtype=BF16, n_seq=1, least=131072, longest=131072, hq=16, hk=2, d=128,
             page=128, window=0, cut=5),
        # a few short requests in fp32, pages that end inside a tile
        dict(name="token_7x400_f32", op="token", dtype=F32, n_seq=7, least=0, longest=400, hq=8, hk=4, d=64, page=24,
             window=0, cut=6),
        # the tables of a step of 256 requests: prompts of some of them, one token of the others
        dict(name="plan_256_mixed", op="plan", n_seq=256, past=8192, prompts=12, prompt=4096, page=64, cut=7),
        # the tables of a decode step of 8 requests
        dict(name="plan_8_tokens", op="plan", n_seq=8, past=2000, prompts=0, prompt=0, page=16, cut=8),
        # keys and values of 16384 prompt tokens into the cache
        dict(name="store_16384", op="store", dtype=BF16, tokens=16384, hk=8, d=128, page=64, dropped=0, cut=9),
        # those of one token of each of 64 requests, some of them without a page
        dict(name="store_64", op="store", dtype=BF16, tokens=64, hk=4, d=128, page=16, dropped=3, cut=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["attn", "attn", "attn", "token", "token", "plan", "store"])
    cut = rng.randrange(1 << 20)
    dtype = rng.choice([BF16, BF16, BF16, F32])
    hk = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128])
    if op == "plan":
        return dict(op=op, n_seq=_log_int(rng, 1, 512), past=_log_int(rng, 1, 8192), prompts=rng.choice([0, 1, 5]),
                    prompt=_log_int(rng, 1, 4096), page=rng.choice([16, 24, 64, 128]), cut=cut)
    if op == "store":
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 16384), hk=hk, d=d, page=rng.choice([1, 16, 24, 64, 128]),
                    dropped=rng.choice([0, 0, 1]), cut=cut)
    group = rng.choice([1, 2, 4, 7, 8])
    if op == "token":
        n, hk = _log_int(rng, 1, 64), min(hk, 4)
        longest = _log_int(rng, 1, min(131072, (400000 if dtype == BF16 else 200000) // n))
        return dict(op=op, dtype=dtype, n_seq=n, least=rng.choice([0, longest // 2, longest]), longest=longest, hq=hk * group,
                    hk=hk, d=d, page=rng.choice([16, 24, 64, 128]), window=rng.choice([0, 0, 0, 100, 4096]), cut=cut)
    way = rng.choice(["fwd", "bwd"])
    causal = rng.random() < 0.8
    most = 4096 if way == "fwd" else 3000
    if rng.random() < 0.5:
        b = rng.randrange(1, 4)
        rows = dict(batch=b, tokens=_log_int(rng, 16, most // b), n_seq=b, ghosts=0, past=0)
    else:
        tokens = _log_int(rng, 16, 2500)
        rows = dict(batch=0, tokens=tokens, n_seq=_log_int(rng, 1, max(1, min(16, tokens // 8))), ghosts=rng.randrange(0, 3),
                    past=rng.choice([0, 0, 0, -20, 1000]))
    return dict(op=op, way=way, dtype=dtype, hq=hk * group, hk=hk, d=d, causal=causal,
                window=rng.choice([0, 0, 2, 100, 700]) if causal else 0, cut=cut, **rows)


# --- inputs --------------------------------------------------------------------

def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _lengths(case):
    """(queries, keys) of every sequence of an attention case: equal rows, or tokens cut at random places with empty
    sequences among them; keys are queries and `past` earlier ones, give or take a half (fewer than queries where negative)."""
    if case["batch"]:
        return [case["tokens"]] * case["batch"], [case["tokens"]] * case["batch"]
    r = random.Random(case["cut"])
    n, tokens, past = case["n_seq"], case["tokens"], case["past"]
    cuts = sorted(r.randrange(1, max(2, tokens)) for _ in range(n - 1))
    if past > 0:                                             # pieces of about one length
        cuts = [tokens * (i + 1) // n + r.randrange(-tokens // (8 * n), tokens // (8 * n) + 1) for i in range(n - 1)]
    lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    for _ in range(case["ghosts"]):
        lens.insert(r.randrange(0, len(lens) + 1), 0)
    return lens, [max(0, x + int(past * r.uniform(0.5, 1.5))) for x in lens]


def _context(case):
    r = random.Random(case["cut"])
    return [r.randint(case["least"], case["longest"]) for _ in range(case["n_seq"])]


def _requests(case):
    """(tokens so far, new tokens) of every request of a plan case."""
    r = random.Random(case["cut"])
    n = case["n_seq"]
    past = [r.randint(0, case["past"]) for _ in range(n)]
    new = [1] * n
    for i in r.sample(range(n), min(n, case["prompts"])):
        past[i], new[i] = r.choice([0, 0, past[i]]), r.randint(1, case["prompt"])
    if n > 4:
        new[r.randrange(n)] = 0
    return past, new


def _starts(lens):
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    return starts


def prepare(case, seed):
    """The tensors a caller holds before the call, drawn from the seed."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape, dtype):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=dev).int()

    s = dict(case=case)
    if case["op"] == "plan":
        past, new = _requests(case)
        page = case["page"]
        held = [-(-a // page) for a in past]
        want = sum(-(-(a + b) // page) - h for a, b, h in zip(past, new, held))
        pages = shuffled(sum(held) + want + 5)
        width = max(-(-(a + b) // page) for a, b in zip(past, new)) + 1
        table = torch.full((case["n_seq"], width), -1, dtype=torch.int32, device=dev)
        rows = torch.arange(width, device=dev)[None] < torch.tensor(held, device=dev)[:, None]
        table[rows] = pages[:sum(held)]
        return dict(s, past=ints(past), new=ints(new), free=pages[sum(held):].clone(), table=table, tokens=sum(new))
    dt = _dt(case["dtype"])
    if case["op"] == "store":
        t, hk, d, page = case["tokens"], case["hk"], case["d"], case["page"]
        pages = -(-t // page) + 3
        s["slots"] = shuffled(pages * page)[:t].clone()
        s["slots"][:case["dropped"]] = -1
        s["k"], s["v"] = randn(1, t, hk, d, dtype=dt), randn(1, t, hk, d, dtype=dt)
        s["kp"], s["vp"] = randn(pages, page, hk, d, dtype=dt), randn(pages, page, hk, d, dtype=dt)
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "token":
        lens, page = _context(case), case["page"]
        width = max(1, -(-max(lens) // page))
        pages = sum(-(-x // page) for x in lens) + 3
        table = torch.full((case["n_seq"], width), -1, dtype=torch.int32, device=dev)
        rows = torch.arange(width, device=dev)[None] < torch.tensor([-(-x // page) for x in lens], device=dev)[:, None]
        table[rows] = shuffled(pages)[:pages - 3]
        return dict(s, q=randn(case["n_seq"], hq, d, dtype=dt), kp=randn(pages, page, hk, d, dtype=dt),
                    vp=randn(pages, page, hk, d, dtype=dt), table=table, lens=ints(lens), longest=max(lens))
    lq, lk = _lengths(case)
    b, t = case["batch"] or 1, case["tokens"]
    s["q"] = randn(b, t, hq, d, dtype=dt)
    tk = t if case["batch"] else sum(lk)
    s["k"], s["v"] = randn(b, tk, hk, d, dtype=dt), randn(b, tk, hk, d, dtype=dt)
    s["cu"] = None if case["batch"] else ints(_starts(lq))
    s["cuk"] = None if case["batch"] or lq == lk else ints(_starts(lk))
    s["lq"], s["lk"] = lq, lk
    if case["way"] == "bwd":
        s["o"], s["lse"] = _plain_attn(s, "fwd")             # what the forward of the same step left
        s["do"] = randn(b, t, hq, d, dtype=dt)
    return s


# --- one pass ------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "attn":
        return _plain_attn(state, state["case"]["way"])
    return {"token": _plain_token, "plan": _plain_plan, "store": _plain_store}[op](state)


def _own(s):
    import chunked_gated_delta_fwd_amd as gdr
    case = s["case"]
    if case["op"] == "attn":
        kw = dict(causal=case["causal"], window=case["window"])
        if case["way"] == "fwd":
            return gdr.attn_fwd(s["q"], s["k"], s["v"], s["cu"], s["cuk"], **kw)
        return gdr.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["cu"], s["cuk"], **kw)
    if case["op"] == "token":
        return gdr.attn_paged_step(s["q"], s["kp"], s["vp"], s["table"], s["lens"], window=case["window"])
    if case["op"] == "plan":
        cu, lens, positions, slots, used = gdr.page_plan(s["past"], s["new"], s["free"], s["table"], case["page"], s["tokens"])
        return s["table"], (cu, lens, positions[0], slots[0], used)
    gdr.page_store(s["k"], s["v"], s["slots"][None], s["kp"], s["vp"])
    return s["kp"], s["vp"]


def _seen(case, lq, lk, i, j):
    """Whether query i of a sequence of lq sees key j of its lk."""
    seen = (j >= 0) & (j < lk)
    if case["causal"]:
        seen = seen & (j <= i + lk - lq)
        if case["window"]:
            seen = seen & (j > i + lk - lq - case["window"])
    return seen


def _plain_attn(s, way):
    """Every sequence padded to the longest; key heads with their group of query heads as one product."""
    case = s["case"]
    dt, hk, d = _dt(case["dtype"]), case["hk"], case["d"]
    g = case["hq"] // hk
    dev = s["q"].device
    scale = d ** -0.5
    lq, lk = torch.tensor(s["lq"], device=dev), torch.tensor(s["lk"], device=dev)
    n, mq, mk = len(s["lq"]), max(s["lq"]), max(1, max(s["lk"]))

    def pad(x, lens, most):                       # [tokens, h, d] -> [n, most, h, d] fp32
        x = x.flatten(0, 1)
        at = torch.arange(most, device=dev)[None]
        place = (torch.cumsum(lens, 0) - lens)[:, None] + at
        out = torch.cat([x, x.new_zeros((1,) + x.shape[1:])])[torch.where(at < lens[:, None], place, x.shape[0])]
        return out.float()

    def back(x, lens, shape):                     # the other way
        at = torch.arange(int(math.prod(shape[:2])), device=dev)
        ends = torch.cumsum(lens, 0)
        seq = torch.searchsorted(ends, at, right=True)
        return x[seq, at - (ends - lens)[seq]].reshape(shape)

    def by_key_head(x):                           # [n, mq, hq, d] -> [n hk, g mq, d]
        return x.reshape(n, mq, hk, g, -1).permute(0, 2, 3, 1, 4).reshape(n * hk, g * mq, -1)

    def by_token(x):                              # the other way
        return x.reshape(n, hk, g, mq, -1).permute(0, 3, 1, 2, 4).reshape(n, mq, hk * g, -1)

    q = by_key_head(pad(s["q"], lq, mq))
    k, v = (pad(s[x], lk, mk).transpose(1, 2).reshape(n * hk, mk, d) for x in ("k", "v"))
    i, j = torch.arange(mq, device=dev)[:, None], torch.arange(mk, device=dev)
    hidden = ~_seen(case, lq[:, None, None], lk[:, None, None], i, j)                       # [n, mq, mk]
    score = (q * scale) @ k.transpose(1, 2).contiguous()
    score.view(n, hk * g, mq, mk).masked_fill_(hidden[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if way == "fwd":
        o = (p @ v).div_(total.clamp(min=1e-37))
        lse = top + total.log()
        return (back(by_token(o), lq, s["q"].shape).to(dt), back(by_token(lse), lq, s["q"].shape[:3] + (1,))[..., 0])
    p.div_(total.clamp(min=1e-37))
    do = by_key_head(pad(s["do"], lq, mq))
    dv = p.transpose(1, 2).contiguous() @ do
    ds = do @ v.transpose(1, 2).contiguous()
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k).mul_(scale)
    dk = (ds.transpose(1, 2).contiguous() @ q).mul_(scale)
    dk, dv = (x.reshape(n, hk, mk, d).transpose(1, 2) for x in (dk, dv))
    return (back(by_token(dq), lq, s["q"].shape).to(dt), back(dk, lk, s["k"].shape).to(dt), back(dv, lk, s["v"].shape).to(dt))


def _plain_token(s):
    case = s["case"]
    hk, d, page = case["hk"], case["d"], case["page"]
    g, n, most = case["hq"] // hk, case["n_seq"], max(1, s["longest"])
    at = torch.arange(most, device=s["q"].device)
    rows = s["table"].long()[:, at // page].clamp(min=0) * page + at % page                  # [n, most]
    k, v = (s[x].flatten(0, 1)[rows].float().transpose(1, 2) for x in ("kp", "vp"))          # [n, hk, most, d]
    lens = s["lens"].long()[:, None]
    seen = at < lens
    if case["window"]:
        seen = seen & (at >= lens - case["window"])
    score = (s["q"].float().reshape(n, hk, g, d) * d ** -0.5) @ k.transpose(2, 3).contiguous()
    score.masked_fill_(~seen[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = (p @ v.contiguous()) / p.sum(-1, keepdim=True).clamp(min=1e-37)
    return o.reshape(n, hk * g, d).to(_dt(case["dtype"]))


def _plain_plan(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    past, new = s["past"].long(), s["new"].long()
    width = table.shape[1]
    held = (past + page - 1) // page
    need = (past + new + page - 1) // page - held
    first = torch.cumsum(need, 0) - need
    ends = torch.cumsum(new, 0)
    place = torch.arange(width, device=table.device)[None]
    take = (first - held)[:, None] + place
    fresh = (place >= held[:, None]) & (place < (held + need)[:, None])
    page_of = torch.where(take < free.shape[0], free[take.clamp(0, free.shape[0] - 1)], -1)
    table.copy_(torch.where(fresh, page_of, table))
    token = torch.arange(s["tokens"], device=table.device)
    seq = torch.searchsorted(ends, token, right=True)
    position = past[seq] + token - (ends - new)[seq]
    which = table[seq, position // page].long()
    slots = torch.where(which >= 0, which * page + position % page, -1)
    cu = torch.cat([ends.new_zeros(1), ends])
    used = torch.stack([ends[-1], need.sum()])
    return table, tuple(x.int() for x in (cu, past + new, position, slots, used))


def _plain_store(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    for pages, x in (("kp", "k"), ("vp", "v")):
        s[pages].flatten(0, 1)[at] = s[x][0][keep]
    return s["kp"], s["vp"]


# --- what a pass cannot do without ---------------------------------------------

def _pairs(case):
    """How many (query, key) pairs of one head are visible."""
    total = 0
    for lq, lk in zip(*_lengths(case)):
        if not case["causal"]:
            total += lq * lk
            continue
        for i in range(lq):
            last = i + lk - lq
            total += max(0, last + 1 - (max(0, last + 1 - case["window"]) if case["window"] else 0))
    return total


def work(case):
    if case["op"] == "plan":
        past, new = _requests(case)
        page = case["page"]
        fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(past, new))
        return dict(bytes=4 * (4 * case["n_seq"] + 2 * fresh + 2 * sum(new)), flops=4 * sum(new) + 4 * case["n_seq"])
    e = 2 if case["dtype"] == BF16 else 4
    row = case["hk"] * case["d"] * e
    if case["op"] == "store":
        return dict(bytes=case["tokens"] * (4 * row + 4), flops=0)
    hq, d = case["hq"], case["d"]
    if case["op"] == "token":
        keys = sum(min(x, case["window"]) if case["window"] else x for x in _context(case))
        return dict(bytes=2 * keys * row + 2 * case["n_seq"] * hq * d * e, flops=4 * keys * hq * d)
    lq, lk = (sum(x) for x in _lengths(case))
    pairs = _pairs(case) * hq
    if case["way"] == "fwd":
        return dict(bytes=lq * hq * (2 * d * e + 4) + 2 * lk * row, flops=4 * d * pairs)
    return dict(bytes=lq * hq * (4 * d * e + 4) + 4 * lk * row, flops=10 * d * pairs)


# --- the definitions in 64 bits ------------------------------------------------

def exact(case, seed):
    """Sequence by sequence and key head by key head in float64, from the definitions."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "store":
        got = []
        for pages, x in (("kp", "k"), ("vp", "v")):
            flat = s[pages].double().flatten(0, 1)
            for slot, row in zip(s["slots"].tolist()[:case["dropped"]], s[x][0].double()[:case["dropped"]]):
                assert slot < 0
            at = s["slots"][case["dropped"]:].long()[:, None, None].expand(-1, case["hk"], case["d"])
            got.append(flat.scatter(0, at, s[x][0, case["dropped"]:].double()).reshape(s[pages].shape))
        return tuple(got)
    return _exact_token(s, case) if case["op"] == "token" else _exact_attn(s, case)


def _softmax64(score):
    """Probabilities and logarithm of the sum; rows of -inf alone give zeros and -inf."""
    top = score.max(-1, keepdim=True).values
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), (top + torch.log(total))[..., 0]


def _exact_token(s, case):
    hk, d, page = case["hk"], case["d"], case["page"]
    g = case["hq"] // hk
    o = torch.zeros(case["n_seq"], case["hq"], d, dtype=torch.float64, device=s["q"].device)
    for n, length in enumerate(s["lens"].tolist()):
        first = max(0, length - case["window"]) if case["window"] else 0
        if length == first:
            continue
        at = torch.arange(first, length, device=o.device)
        pages = s["table"][n].long()[torch.div(at, page, rounding_mode="floor")]
        k, v = (s[x][pages, at % page].double() for x in ("kp", "vp"))               # [keys, hk, d]
        for h in range(hk):
            p, _ = _softmax64(s["q"][n, h * g:(h + 1) * g].double() @ k[:, h].t() / math.sqrt(d))
            o[n, h * g:(h + 1) * g] = p @ v[:, h]
    return o


def _exact_attn(s, case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    g, scale = hq // hk, 1 / math.sqrt(d)
    f8 = torch.float64
    q, k, v = (s[x].flatten(0, 1) for x in ("q", "k", "v"))
    grad = case["way"] == "bwd"
    o, lse = torch.zeros(q.shape, dtype=f8, device=q.device), torch.full(q.shape[:2], -math.inf, dtype=f8, device=q.device)
    dq, dk, dv = (torch.zeros(x.shape, dtype=f8, device=q.device) for x in (q, k, v))
    q0 = k0 = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        if lq and lk:
            i = torch.arange(lq, device=q.device)[:, None]
            hidden = ~_seen(case, lq, lk, i, torch.arange(lk, device=q.device))
            for h in range(hq):
                qs, ks, vs = q[q0:q0 + lq, h].to(f8), k[k0:k0 + lk, h // g].to(f8), v[k0:k0 + lk, h // g].to(f8)
                p, each = _softmax64((scale * (qs @ ks.t())).masked_fill(hidden, -math.inf))
                if not grad:
                    o[q0:q0 + lq, h], lse[q0:q0 + lq, h] = p @ vs, each
                    continue
                do = s["do"].flatten(0, 1)[q0:q0 + lq, h].to(f8)
                dv[k0:k0 + lk, h // g] += p.t() @ do
                dp = do @ vs.t()
                ds = scale * p * (dp - (do * (p @ vs)).sum(-1, keepdim=True))
                dq[q0:q0 + lq, h] = ds @ ks
                dk[k0:k0 + lk, h // g] += ds.t() @ qs
        q0, k0 = q0 + lq, k0 + lk
    if grad:
        return dq.reshape(s["q"].shape), dk.reshape(s["k"].shape), dv.reshape(s["v"].shape)
    return o.reshape(s["q"].shape), lse.reshape(s["q"].shape[:3])
