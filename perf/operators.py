"""Cases, plain forms and exact values of the operators that stand around the
gated delta rule in a token mixer:

* ``conv``: the short causal depthwise convolution over the projected tokens
  (prompt, gradient, single token),
* ``norm``: the norm of every query and key head with the position rotation in
  the same pass (forward, gradient),
* ``scan``: the selective state space scan with one decay per head (prompt,
  gradient, single token).

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
        # the q, k and v projections (16 + 16 + 32 heads of 128) of a packed
        # 64k-token prompt, as the delta rule's benchmark workload has them
        dict(name="conv_prompt_64k", op="conv", way="fwd", dtype=BF16, batch=0, tokens=65536, n_seq=15, ghosts=2,
             channels=8192, width=4, bias=False, silu=True, state=True),
        # a training step on fixed rows, channels of a scan's x, b and c together
        dict(name="conv_train_4x4096", op="conv", way="bwd", dtype=BF16, batch=4, tokens=4096, n_seq=4, ghosts=0,
             channels=4608, width=4, bias=True, silu=True, state=True),
        # a decode step of 256 requests
        dict(name="conv_token_256", op="conv", way="step", dtype=BF16, batch=256, tokens=1, n_seq=256, ghosts=0,
             channels=8192, width=4, bias=False, silu=True, state=True),
        # odd sizes in fp32: short ragged segments, a channel count with no common factor, three taps
        dict(name="conv_odd_f32", op="conv", way="fwd", dtype=F32, batch=0, tokens=1003, n_seq=37, ghosts=5,
             channels=1031, width=3, bias=True, silu=False, state=True),
        # L2-normalised queries and keys of the packed 64k-token prompt (what the delta rule takes)
        dict(name="norm_prompt_64k", op="norm", way="fwd", dtype=BF16, batch=1, tokens=65536, hq=16, hk=16, d=128,
             rot=0, kind="l2", weight=False, interleaved=False, table=0),
        # gradient of RMS-normed, half-rotated queries and keys with shared key heads
        dict(name="norm_train_2x8192", op="norm", way="bwd", dtype=BF16, batch=2, tokens=8192, hq=32, hk=4, d=128,
             rot=64, kind="rms", weight=True, interleaved=False, table=8192),
        # one token of each of 64 requests at far positions
        dict(name="norm_token_64", op="norm", way="fwd", dtype=BF16, batch=64, tokens=1, hq=16, hk=2, d=128,
             rot=128, kind="rms", weight=True, interleaved=True, table=32768),
        # the packed 64k-token prompt on the benchmark workload's heads (16 shared by 32, 128 x 128 states)
        dict(name="scan_prompt_64k", op="scan", way="fwd", dtype=BF16, gate=BF16, batch=0, tokens=65536, n_seq=15,
             ghosts=2, heads=32, groups=16, n=128, p=128, state=True),
        # gradient of a 16k-token packed training row, heads of 64 on one shared b and c
        dict(name="scan_train_16k", op="scan", way="bwd", dtype=BF16, gate=F32, batch=0, tokens=16384, n_seq=4,
             ghosts=0, heads=32, groups=1, n=128, p=64, state=True),
        # a decode step of 256 requests (the state alone is 537 MB)
        dict(name="scan_token_256", op="scan", way="step", dtype=BF16, gate=BF16, batch=256, tokens=1, n_seq=256,
             ghosts=0, heads=32, groups=16, n=128, p=128, state=True),
        # fp32 rows of an odd length
        dict(name="scan_f32_2x1999", op="scan", way="fwd", dtype=F32, gate=F32, batch=2, tokens=1999, n_seq=2,
             ghosts=0, heads=8, groups=2, n=64, p=64, state=True),
        # many short pieces of prompts in one call, empty ones among them
        dict(name="scan_ragged_600", op="scan", way="fwd", dtype=BF16, gate=F32, batch=0, tokens=600, n_seq=37,
             ghosts=5, heads=16, groups=1, n=128, p=64, state=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["conv", "norm", "scan"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op == "conv":
        way = rng.choice(["fwd", "bwd", "step"])
        channels = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            channels = (channels + 7) // 8 * 8
        c = dict(op=op, way=way, dtype=dtype, channels=channels, width=rng.choice([2, 3, 4, 4]),
                 bias=rng.random() < 0.5, silu=rng.random() < 0.7, state=True, ghosts=0)
        if way == "step":
            b = _log_int(rng, 1, 256)
            return dict(c, batch=b, tokens=1, n_seq=b)
        if rng.random() < 0.5:
            t = _log_int(rng, 1, 32768)
            n = _log_int(rng, 1, max(1, min(64, t)))
            return dict(c, batch=0, tokens=t, n_seq=n, ghosts=rng.randrange(0, 4), state=rng.random() < 0.7)
        b = rng.randrange(1, 9)
        return dict(c, batch=b, tokens=_log_int(rng, 1, 32768 // b), n_seq=b, state=rng.random() < 0.7)
    if op == "norm":
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        d = rng.choice([64, 128, 128, 256])
        rot = rng.choice([0, d // 4, d // 2, d])
        b = rng.choice([1, 1, 2, 7, 64])
        c = dict(op=op, way=rng.choice(["fwd", "bwd"]), dtype=dtype, batch=b,
                 tokens=_log_int(rng, 1, 16384 // b), hq=hk * rng.choice([1, 2, 3]), hk=hk, d=d, rot=rot,
                 kind=rng.choice(["l2", "rms"]), weight=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                 table=0)
        return dict(c, table=max(c["tokens"], rng.choice([4096, 32768])) if rot else 0)
    way = rng.choice(["fwd", "bwd", "step"])
    groups = rng.choice([1, 1, 2, 4])
    c = dict(op=op, way=way, dtype=dtype, gate=rng.choice([dtype, F32]), heads=groups * rng.choice([1, 2, 3, 8]),
             groups=groups, n=rng.choice([64, 128]), p=rng.choice([64, 128]), ghosts=0, state=True)
    if way == "step":
        b = _log_int(rng, 1, 256)
        return dict(c, batch=b, tokens=1, n_seq=b)
    most = 8192 if way == "fwd" else 4096
    if rng.random() < 0.6:
        t = _log_int(rng, 1, most)
        n = _log_int(rng, 1, max(1, min(40, t)))
        return dict(c, batch=0, tokens=t, n_seq=n, ghosts=rng.randrange(0, 4), state=rng.random() < 0.7)
    b = rng.randrange(1, 5)
    return dict(c, batch=b, tokens=_log_int(rng, 1, most // b), n_seq=b, state=rng.random() < 0.7)


# --- inputs --------------------------------------------------------------------

def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _lengths(case, seed):
    """Segment lengths: fixed rows, or `tokens` cut at random places with empty segments among them."""
    if case["batch"]:
        return [case["tokens"]] * case["batch"]
    r = random.Random(seed)
    cuts = sorted(r.randrange(1, case["tokens"]) if case["tokens"] > 1 else 1 for _ in range(case["n_seq"] - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
    for _ in range(case["ghosts"]):
        lens.insert(r.randrange(0, len(lens) + 1), 0)
    return lens


def prepare(case, seed):
    """The tensors a caller holds before the call, drawn from the seed."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _dt(case["dtype"])

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    def rand(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case=case)
    if case["op"] == "norm":
        b, t, d = case["batch"], case["tokens"], case["d"]
        s["q"] = randn(b, t, case["hq"], d, dtype=dt)
        s["k"] = randn(b, t, case["hk"], d, dtype=dt)
        s["wq"] = (1 + 0.2 * randn(d)).to(dt) if case["weight"] else None
        s["wk"] = (1 + 0.2 * randn(d)).to(dt) if case["weight"] else None
        s["cos"] = s["sin"] = s["pos"] = None
        if case["rot"]:
            freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
            angle = torch.arange(case["table"], device=dev, dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            first = torch.randint(0, case["table"] - t + 1, (b, 1), generator=gen, device=dev)
            s["pos"] = (first + torch.arange(t, device=dev)).to(torch.int32)
        if case["way"] == "bwd":
            s["doq"], s["dok"] = randn(b, t, case["hq"], d, dtype=dt), randn(b, t, case["hk"], d, dtype=dt)
        return s

    step = case["way"] == "step"
    lens = _lengths(case, seed)
    n_seq = len(lens)
    rows = (case["batch"],) if step else (case["batch"] or 1, case["tokens"])
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    s["cu"] = None if case["batch"] else torch.tensor(starts, dtype=torch.int32, device=dev)
    # the same starts as a host program holds them (fixed rows too)
    s["starts"] = torch.tensor(starts, dtype=torch.int64, device=dev)
    s["n_seq"], s["lens"] = n_seq, lens
    if case["op"] == "conv":
        ch, w = case["channels"], case["width"]
        s["x"] = randn(*rows, ch, dtype=dt)
        s["w"] = rand(ch, w, lo=-w ** -0.5, hi=w ** -0.5).to(dt)
        s["bias"] = randn(ch, dtype=dt, scale=0.1) if case["bias"] else None
        s["s0"] = randn(n_seq, w - 1, ch, dtype=dt) if case["state"] else None
        if case["way"] == "bwd":
            s["dy"] = randn(*rows, ch, dtype=dt)
            s["dst"] = randn(n_seq, w - 1, ch, dtype=dt) if case["state"] else None
        return s
    h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
    s["x"] = randn(*rows, h, p, dtype=dt)
    s["b"] = randn(*rows, g, n, dtype=dt)
    s["c"] = randn(*rows, g, n, dtype=dt)
    s["dt"] = randn(*rows, h, dtype=_dt(case["gate"]), scale=0.5)
    s["A"] = -rand(h, lo=1.0, hi=16.0)
    s["D"] = rand(h, lo=0.5, hi=1.5)
    # softplus(dt_bias) between 0.001 and 0.1, evenly over its logarithm
    s["dt_bias"] = torch.expm1(torch.exp(rand(h, lo=math.log(1e-3), hi=math.log(1e-1)))).log()
    s["h0"] = randn(n_seq, h, n, p, scale=0.3) if case["state"] else None
    if case["way"] == "bwd":
        s["dy"] = randn(*rows, h, p, dtype=dt)
        s["dht"] = randn(n_seq, h, n, p, scale=0.3) if case["state"] else None
    return s


# --- one pass ------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    case = state["case"]
    return {"conv": _plain_conv, "norm": _plain_norm, "scan": _plain_scan}[case["op"]](state, case["way"])


def _own(s):
    import chunked_gated_delta_fwd_amd as gdr
    case = s["case"]
    op, way = case["op"], case["way"]
    if op == "conv":
        act = "silu" if case["silu"] else None
        if way == "fwd":
            return gdr.short_conv_fwd(s["x"], s["w"], s["bias"], s["cu"], s["s0"], activation=act)
        if way == "bwd":
            return gdr.short_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["cu"], s["s0"], s["dst"], activation=act)
        return gdr.short_conv_step(s["x"], s["s0"], s["w"], s["bias"], activation=act), s["s0"]
    if op == "norm":
        kw = dict(cos=s["cos"], sin=s["sin"], positions=s["pos"], norm=case["kind"], eps=1e-6,
                  interleaved=case["interleaved"])
        if way == "fwd":
            return gdr.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], **kw)
        return gdr.qk_norm_rope_bwd(s["q"], s["k"], s["doq"], s["dok"], s["wq"], s["wk"], **kw)
    if way == "fwd":
        return gdr.ssm_scan_fwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"], s["cu"], s["h0"])
    if way == "bwd":
        return gdr.ssm_scan_bwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["dy"], s["D"], s["dt_bias"], s["cu"],
                                s["h0"], s["dht"])
    return gdr.ssm_step(s["x"], s["dt"], s["A"], s["b"], s["c"], s["h0"], s["D"], s["dt_bias"]), s["h0"]


def _spans(s, extra):
    """Sequence, first and last position of every token, and of `extra` places before each sequence."""
    starts = s["starts"]
    total = s["x"].shape[0] * s["x"].shape[1]
    pos = torch.arange(total, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), pos, right=True)
    if extra:
        back = starts[:-1, None] - extra + torch.arange(extra, device=starts.device)
        pos = torch.cat([pos, back.reshape(-1)])
        seq = torch.cat([seq, torch.arange(s["n_seq"], device=starts.device).repeat_interleave(extra)])
    return pos, seq, starts[seq], starts[seq + 1]


def _plain_conv(s, way):
    case = s["case"]
    dt, w = _dt(case["dtype"]), case["width"]
    weight, ch = s["w"].float(), case["channels"]
    bias = 0.0 if s["bias"] is None else s["bias"].float()
    if way == "step":
        window = torch.cat([s["s0"], s["x"][:, None]], 1)
        z = (window.float() * weight.t()).sum(1) + bias
        s["s0"].copy_(window[:, 1:])
        return (z * torch.sigmoid(z) if case["silu"] else z).to(dt), s["s0"]
    x = s["x"].reshape(-1, ch)
    total, n_seq = x.shape[0], s["n_seq"]
    s0 = torch.zeros(n_seq, w - 1, ch, dtype=dt, device=x.device) if s["s0"] is None else s["s0"]
    past = torch.cat([x, s0.reshape(-1, ch)])
    pos, seq, first, end = _spans(s, w - 1)

    def row_of(p, n, start):        # the row of `past` that holds position p of sequence n
        return torch.where(p >= start, p, total + n * (w - 1) + (p - start + w - 1))

    taps = torch.arange(w, device=x.device)
    at = row_of(pos[:total, None] - (w - 1) + taps, seq[:total, None], first[:total, None])
    window = past[at].float()                              # [tokens, taps, channels]
    z = (window * weight.t()).sum(1) + bias
    if way == "fwd":
        y = z * torch.sigmoid(z) if case["silu"] else z
        last = s["starts"][1:, None] - (w - 1) + taps[:-1]
        n = torch.arange(n_seq, device=x.device)[:, None]
        return y.to(dt).reshape(s["x"].shape), past[row_of(last, n, s["starts"][:-1, None])]
    dy = s["dy"].reshape(-1, ch).float()
    sig = torch.sigmoid(z)
    dz = dy * sig * (1 + z * (1 - sig)) if case["silu"] else dy
    dw = (window * dz[:, None]).sum(0).t()
    db = dz.sum(0) if s["bias"] is not None else None
    # what position p gets: dz of the positions p .. p + w - 1 of its sequence, and the final state's gradient
    none = dz.new_zeros(1, ch)
    later = pos[:, None] + taps
    inside = (later >= first[:, None]) & (later < end[:, None])
    dpast = (torch.cat([dz, none])[torch.where(inside, later, total)] * weight.t().flip(0)).sum(1)
    if s["dst"] is not None:
        place = pos - (end - (w - 1))
        dst = torch.cat([s["dst"].reshape(-1, ch).float(), none])
        dpast = dpast + dst[torch.where(place >= 0, seq * (w - 1) + place, n_seq * (w - 1))]
    return (dpast[:total].to(dt).reshape(s["x"].shape), dw, db, dpast[total:].to(dt).reshape(n_seq, w - 1, ch))


def _plain_norm_one(x, weight, s):
    case = s["case"]
    square = x.square().mean(-1, keepdim=True) if case["kind"] == "rms" else x.square().sum(-1, keepdim=True)
    y = x / torch.sqrt(square + 1e-6)
    if weight is not None:
        y = y * weight
    if not case["rot"]:
        return y
    half = case["rot"] // 2
    cos, sin = s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]
    turned, rest = y[..., :case["rot"]], y[..., case["rot"]:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _plain_norm(s, way):
    dt = _dt(s["case"]["dtype"])
    outs, grads = [], []
    pairs = (("q", "wq", "doq"), ("k", "wk", "dok"))
    if way == "fwd":
        return tuple(_plain_norm_one(s[x].float(), None if s[w] is None else s[w].float(), s).to(dt)
                     for x, w, _ in pairs)
    for name, w, do in pairs:
        x = s[name].float().requires_grad_()
        weight = None if s[w] is None else s[w].float().requires_grad_()
        leaves = [x] if weight is None else [x, weight]
        got = torch.autograd.grad(_plain_norm_one(x, weight, s), leaves, s[do].float())
        outs.append(got[0].to(dt))
        grads.append(got[1] if weight is not None else None)
    return outs[0], outs[1], grads[0], grads[1]


def _plain_scan_core(s, x, dt_raw, A, b, c, D, dt_bias, h0):
    """The scan in chunks of 64 tokens that restart with every sequence, states joined by one product."""
    case = s["case"]
    h, g, n, p, size = case["heads"], case["groups"], case["n"], case["p"], 64
    starts = s["starts"]
    total, n_seq, dev = x.shape[0], s["n_seq"], x.device
    count = (starts[1:] - starts[:-1] + size - 1) // size
    first = torch.cumsum(count, 0) - count                 # first chunk of each sequence
    chunks = sum((x + size - 1) // size for x in s["lens"])
    pos = torch.arange(total, device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), pos, right=True)
    slot = first[seq] * size + (pos - starts[seq])          # token -> place in the chunks
    back = torch.full((chunks * size,), total, device=dev).scatter_(0, slot, pos)

    def lay(t):                                            # [tokens, ...] -> [chunks, size, ...], zero elsewhere
        return torch.cat([t, t.new_zeros((1,) + t.shape[1:])])[back].reshape((chunks, size) + t.shape[1:])

    dt = torch.nn.functional.softplus(dt_raw + dt_bias)
    steps = lay(dt).permute(0, 2, 1)                       # [chunks, heads, size]
    logs = torch.cumsum(steps.double() * A.double()[:, None], -1)
    ends = logs[..., -1]                                   # [chunks, heads]
    xs, bs, cs = lay(x).permute(0, 2, 1, 3), lay(b).permute(0, 2, 1, 3), lay(c).permute(0, 2, 1, 3)
    low = torch.ones(size, size, dtype=torch.bool, device=dev).tril()
    gap = (logs[..., :, None] - logs[..., None, :]).masked_fill(~low, -math.inf)
    score = (cs @ bs.transpose(-1, -2)).repeat_interleave(h // g, 1) * gap.exp().float() * steps[..., None, :]
    bh = bs.repeat_interleave(h // g, 1)
    local = (bh * ((ends[..., None] - logs).exp().float() * steps)[..., None]).transpose(-1, -2) @ xs
    # states at chunk starts: every earlier chunk of the same sequence, and its initial state, decayed
    owner = torch.searchsorted(torch.cumsum(count, 0), torch.arange(chunks, device=dev), right=True)
    before = torch.cumsum(ends, 0) - ends                  # [chunks, heads], over all chunks so far
    entry = torch.cat([before, before.new_zeros(1, h)])[first.clamp(max=chunks)]
    place = torch.arange(chunks, device=dev)
    held = (owner[:, None] == owner) & (place < place[:, None])
    since = (before[:, None] - (before + ends)[None]).masked_fill(~held[..., None], -math.inf).exp().float()
    born = (before[:, None] - entry[None]).masked_fill((owner[:, None] != torch.arange(n_seq, device=dev))[..., None],
                                                       -math.inf).exp().float()
    weights = torch.cat([since, born], 1).permute(2, 0, 1)                    # [heads, chunks, chunks + n_seq]
    entries = torch.cat([local, h0], 0).permute(1, 0, 2, 3).reshape(h, chunks + n_seq, n * p)
    state = (weights @ entries).reshape(h, chunks, n, p).permute(1, 0, 2, 3)  # at the start of each chunk
    ch = cs.repeat_interleave(h // g, 1)
    y = score @ xs + (ch @ state) * logs.exp().float()[..., None]
    y = y.permute(0, 2, 1, 3).reshape(chunks * size, h, p)[slot] + D[:, None] * x
    after = state * ends.exp().float()[..., None, None] + local               # at the end of each chunk
    last = torch.where(count > 0, first + count - 1, chunks + torch.arange(n_seq, device=dev))
    return y, torch.cat([after, h0])[last]


def _plain_scan(s, way):
    case = s["case"]
    dt, h, g, n, p = _dt(case["dtype"]), case["heads"], case["groups"], case["n"], case["p"]
    if way == "step":
        step = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
        b, c = (s[k].float().repeat_interleave(h // g, 1) for k in ("b", "c"))
        x, state = s["x"].float(), s["h0"]
        state.mul_((step * s["A"]).exp()[..., None, None]).add_((step[..., None] * b)[..., None] * x[:, :, None])
        y = (c[..., None] * state).sum(2) + s["D"][:, None] * x
        return y.to(dt), state
    rows = s["x"].shape[:2]
    total = rows[0] * rows[1]
    h0 = torch.zeros(s["n_seq"], h, n, p, device=s["x"].device) if s["h0"] is None else s["h0"]
    args = [s["x"].reshape(total, h, p).float(), s["dt"].reshape(total, h).float(), s["A"],
            s["b"].reshape(total, g, n).float(), s["c"].reshape(total, g, n).float(), s["D"], s["dt_bias"], h0]
    if way == "fwd":
        y, ht = _plain_scan_core(s, *args)
        return y.to(dt).reshape(s["x"].shape), ht
    args = [t.detach().requires_grad_() for t in args]
    y, ht = _plain_scan_core(s, *args)
    dht = torch.zeros_like(ht) if s["dht"] is None else s["dht"]
    dx, ddt, dA, db, dc, dD, dbias, dh0 = torch.autograd.grad([y, ht], args, [s["dy"].reshape(y.shape).float(), dht])
    return (dx.to(dt).reshape(s["x"].shape), ddt.to(s["dt"].dtype).reshape(s["dt"].shape), dA,
            db.to(dt).reshape(s["b"].shape), dc.to(dt).reshape(s["c"].shape), dD, dbias, dh0)


# --- what a pass cannot do without ---------------------------------------------

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    tokens = case["tokens"] * max(1, case["batch"])
    if case["op"] == "conv":
        w, ch = case["width"], case["channels"]
        par = ch * (w + (1 if case["bias"] else 0))
        states = (case["n_seq"] + case["ghosts"]) * (w - 1) * ch * e
        if case["way"] == "bwd":
            return dict(bytes=3 * tokens * ch * e + par * (e + 4) + states * (3 if case["state"] else 1),
                        flops=tokens * ch * (6 * w + 12))
        return dict(bytes=2 * tokens * ch * e + par * e + states * (2 if case["state"] else 1),
                    flops=tokens * ch * (2 * w + 4))
    if case["op"] == "norm":
        values = tokens * (case["hq"] + case["hk"]) * case["d"]
        table = min(case["table"], tokens) * case["rot"] * 4 + (tokens * 4 if case["rot"] else 0)
        if case["way"] == "bwd":
            return dict(bytes=3 * values * e + table, flops=values * 14)
        return dict(bytes=2 * values * e + table, flops=values * 7)
    h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
    ge = 2 if case["gate"] == BF16 else 4
    states = (case["n_seq"] + case["ghosts"]) * h * n * p * 4
    io = tokens * (h * p * e + 2 * g * n * e + h * ge)
    if case["way"] == "step":
        return dict(bytes=io + tokens * h * p * e + 2 * states, flops=5 * tokens * h * n * p)
    # in chunks of 64: the scores, their product with x, the state read and written
    pair = 64 * (n + p)
    if case["way"] == "fwd":
        return dict(bytes=io + tokens * h * p * e + states * (2 if case["state"] else 1),
                    flops=tokens * h * (pair + 4 * n * p))
    return dict(bytes=2 * io + tokens * h * p * e + states * (3 if case["state"] else 1),
                flops=tokens * h * (3 * pair + 10 * n * p))


# --- the definitions in 64 bits ------------------------------------------------

def exact(case, seed):
    """Token by token in float64, from the definitions; gradients by their own formulas."""
    if case["op"] == "scan" and max(_lengths(case, seed)) > 40000:
        return None                                        # more than 20 seconds
    s = prepare(case, seed)
    return {"conv": _exact_conv, "norm": _exact_norm, "scan": _exact_scan}[case["op"]](s, case)


def _exact_conv(s, case):
    w, ch = case["width"], case["channels"]
    weight = s["w"].double()
    bias = torch.zeros(ch, dtype=torch.float64, device=weight.device) if s["bias"] is None else s["bias"].double()
    step = case["way"] == "step"
    x = s["x"].reshape(-1, ch).double()
    y, st = torch.zeros_like(x), []
    dx, dw, db, ds0 = torch.zeros_like(x), torch.zeros_like(weight), torch.zeros_like(bias), []
    bounds = list(range(case["batch"] + 1)) if step else s["starts"].tolist()
    for i, (a, e) in enumerate(zip(bounds[:-1], bounds[1:])):
        old = torch.zeros(w - 1, ch, dtype=torch.float64, device=x.device) if s["s0"] is None else s["s0"][i].double()
        line = torch.cat([old, x[a:e]])
        z = bias.expand(e - a, ch).clone()
        for j in range(w):
            z += line[j:j + e - a] * weight[:, j]
        y[a:e] = z / (1 + torch.exp(-z)) if case["silu"] else z
        st.append(line[e - a:])
        if case["way"] == "bwd":
            dz = s["dy"].reshape(-1, ch)[a:e].double()
            if case["silu"]:
                up = torch.exp(-z)
                dz = dz * (1 + up + z * up) / (1 + up) ** 2
            dline = torch.zeros_like(line)
            if s["dst"] is not None:
                dline[e - a:] += s["dst"][i].double()
            for j in range(w):
                dline[j:j + e - a] += dz * weight[:, j]
                dw[:, j] += (dz * line[j:j + e - a]).sum(0)
            db += dz.sum(0)
            dx[a:e], old = dline[w - 1:], dline[:w - 1]
            ds0.append(old)
    if case["way"] == "bwd":
        return dx.reshape(s["x"].shape), dw, None if s["bias"] is None else db, torch.stack(ds0)
    return y.reshape(s["x"].shape), torch.stack(st)


def _exact_norm(s, case):
    rot, d = case["rot"], case["d"]
    if rot:
        index = torch.arange(rot, device=s["q"].device)
        other = index ^ 1 if case["interleaved"] else (index + rot // 2) % rot
        angle = index // 2 if case["interleaved"] else index % (rot // 2)
        low = index % 2 == 0 if case["interleaved"] else index < rot // 2
        cos = s["cos"].double()[s["pos"].long()][:, :, None][..., angle]
        sin = s["sin"].double()[s["pos"].long()][:, :, None][..., angle] * torch.where(low, -1.0, 1.0)

    def turn(t, back):
        if not rot:
            return t
        r = t[..., :rot]
        return torch.cat([r * cos + (-1 if back else 1) * r[..., other] * sin, t[..., rot:]], -1)

    outs, grads = [], []
    for name, w, do in (("q", "wq", "doq"), ("k", "wk", "dok")):
        x = s[name].double()
        weight = torch.ones(d, dtype=torch.float64, device=x.device) if s[w] is None else s[w].double()
        m = d if case["kind"] == "rms" else 1
        inv = ((x * x).sum(-1, keepdim=True) / m + 1e-6) ** -0.5
        if case["way"] == "fwd":
            outs.append(turn(x * inv * weight, False))
            continue
        dn = turn(s[do].double(), True)
        grads.append((dn * x * inv).sum((0, 1, 2)) if s[w] is not None else None)
        dn = dn * weight
        outs.append(inv * dn - x * inv ** 3 * (dn * x).sum(-1, keepdim=True) / m)
    return tuple(outs) if case["way"] == "fwd" else (outs[0], outs[1], grads[0], grads[1])


def _exact_scan(s, case):
    h, g, n, p = case["heads"], case["groups"], case["n"], case["p"]
    f8 = torch.float64
    dev = s["x"].device
    x = s["x"].reshape(-1, h, p).to(f8)
    b = s["b"].reshape(-1, g, n).to(f8).repeat_interleave(h // g, 1)
    c = s["c"].reshape(-1, g, n).to(f8).repeat_interleave(h // g, 1)
    raw = s["dt"].reshape(-1, h).to(f8) + s["dt_bias"].to(f8)
    dt = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    A, D = s["A"].to(f8), s["D"].to(f8)
    decay = torch.exp(dt * A)
    lens, n_seq = s["lens"], s["n_seq"]
    starts = s["starts"].tolist()
    order = sorted(range(n_seq), key=lambda i: -lens[i])   # so that the sequences still running come first
    first = torch.tensor([starts[i] for i in order], device=dev)
    state = torch.zeros(n_seq, h, n, p, dtype=f8, device=dev) if s["h0"] is None else s["h0"].to(f8)[order]
    back = torch.tensor(order, device=dev).argsort()
    running = [sum(1 for v in lens if v > j) for j in range(max(lens) if lens else 0)]
    y = torch.zeros_like(x)
    grad = case["way"] == "bwd"
    kept = torch.zeros(x.shape[0], h, n, p, dtype=f8, device=dev) if grad else None
    for j, k in enumerate(running):
        at = first[:k] + j
        new = decay[at][..., None, None] * state[:k] + (dt[at][..., None] * b[at])[..., None] * x[at][:, :, None]
        if grad:
            kept[at] = state[:k]
        state[:k] = new
        y[at] = (c[at][:, :, None] @ new)[:, :, 0]
    y += D[:, None] * x
    if not grad:
        return y.reshape(s["x"].shape), state[back]
    dy = s["dy"].reshape(-1, h, p).to(f8)
    dstate = torch.zeros_like(state) if s["dht"] is None else s["dht"].to(f8)[order]
    dx, db, dc = torch.zeros_like(x), torch.zeros_like(b), torch.zeros_like(c)
    ddt, dlog = torch.zeros_like(dt), torch.zeros_like(dt)
    for j in range(len(running) - 1, -1, -1):
        k = running[j]
        at = first[:k] + j
        old, xa, ba, da = kept[at], x[at], b[at], dt[at]
        new = decay[at][..., None, None] * old + (da[..., None] * ba)[..., None] * xa[:, :, None]
        dc[at] = (new @ dy[at][..., None])[..., 0]
        ds = dstate[:k] + c[at][..., None] * dy[at][:, :, None]
        bx = (ba[:, :, None] @ ds)[:, :, 0]                # b . dS, over n
        dx[at] = da[..., None] * bx
        db[at] = da[..., None] * (ds @ xa[..., None])[..., 0]
        ddt[at] = (bx * xa).sum(-1)
        dlog[at] = decay[at] * (ds * old).sum((-1, -2))
        dstate[:k] = decay[at][..., None, None] * ds
    ddt = ddt + dlog * A
    dA = (dlog * dt).sum(0)
    dD = (dy * x).sum((0, 2))
    draw_ = ddt / (1 + torch.exp(-raw))
    return ((dx + D[:, None] * dy).reshape(s["x"].shape), draw_.reshape(s["dt"].shape), dA,
            db.reshape(-1, g, h // g, n).sum(2).reshape(s["b"].shape),
            dc.reshape(-1, g, h // g, n).sum(2).reshape(s["c"].shape), dD, draw_.sum(0), dstate[back])
