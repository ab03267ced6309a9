"""A small stack of token mixers: a state space layer and a delta-rule layer,
each behind a short convolution, run as they are used in a model.

    python examples/token_mixer.py [--tokens 4096] [--new 32] [--steps 20]

1. a prompt of packed sequences of several lengths, which leaves every layer's
   state behind (the convolution's last tokens and the recurrence's matrix);
2. single tokens from those states, captured once as a graph and replayed,
   checked against the prompt pass over the longer sequences;
3. a few training steps, gradients through every operator.

Weights and inputs are random; all arithmetic of the operators is in the HIP
kernels of chunked_gated_delta_fwd_amd, the projections are torch's.
"""
import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_fwd_amd as gdr  # noqa: E402

CONV_WIDTH = 4


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, cu):
        ctx.save_for_backward(x, w, bias, cu)
        return gdr.short_conv_fwd(x, w, bias, cu, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, w, bias, cu = ctx.saved_tensors
        dx, dw, db, _ = gdr.short_conv_bwd(x, w, dy.contiguous(), bias, cu, want_ds0=False)
        return dx, dw.to(w.dtype), db.to(bias.dtype), None


class QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, cos, sin, pos):
        ctx.save_for_backward(q, k, cos, sin, pos)
        return gdr.qk_norm_rope_fwd(q, k, cos=cos, sin=sin, positions=pos, norm="l2")

    @staticmethod
    def backward(ctx, doq, dok):
        q, k, cos, sin, pos = ctx.saved_tensors
        dq, dk, _, _ = gdr.qk_norm_rope_bwd(q, k, doq.contiguous(), dok.contiguous(), cos=cos, sin=sin, positions=pos,
                                            norm="l2")
        return dq, dk, None, None, None


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, cu):
        ctx.save_for_backward(q, k, v, g, beta, cu)
        return gdr.chunk_fwd(q, k, v, g, beta, cu, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        q, k, v, g, beta, cu = ctx.saved_tensors
        return gdr.chunk_bwd(q, k, v, g, beta, do.contiguous(), cu, want_dh0=False)[:5] + (None,)


class SsmScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, b, c, D, dt_bias, cu):
        ctx.save_for_backward(x, dt, A, b, c, D, dt_bias, cu)
        return gdr.ssm_scan_fwd(x, dt, A, b, c, D, dt_bias, cu, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, dt, A, b, c, D, dt_bias, cu = ctx.saved_tensors
        return gdr.ssm_scan_bwd(x, dt, A, b, c, dy.contiguous(), D, dt_bias, cu, want_dh0=False)[:7] + (None,)


def positions_of(cu, tokens):
    """Each token's place in its own sequence, int32 [1, tokens]."""
    at = torch.arange(tokens, device=cu.device, dtype=torch.int32)
    return (at - cu[torch.searchsorted(cu, at, right=True) - 1])[None]


class DeltaLayer(torch.nn.Module):
    """projection -> short convolution -> norm and rotation of q and k -> delta rule -> norm -> projection"""

    def __init__(self, width, hk=4, hv=8, d=128, rot=64, table=65536):
        super().__init__()
        self.hk, self.hv, self.d = hk, hv, d
        self.qk, self.vd = 2 * hk * d, hv * d
        self.proj = torch.nn.Parameter(torch.randn(width, self.qk + self.vd + 2 * hv) * width ** -0.5)
        self.conv_w = torch.nn.Parameter(torch.randn(self.qk + self.vd, CONV_WIDTH) * 0.4)
        self.conv_b = torch.nn.Parameter(torch.randn(self.qk + self.vd) * 0.1)
        self.out = torch.nn.Parameter(torch.randn(self.vd, width) * self.vd ** -0.5)
        # computed in fp64: an angle of thousands of radians loses its fraction in fp32
        angle = torch.arange(table, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
        self.tables = angle.cos().float(), angle.sin().float()

    def _apply(self, fn, *args, **kw):   # the tables follow the device and stay fp32
        super()._apply(fn, *args, **kw)
        self.tables = tuple(t.to(self.proj.device) for t in self.tables)
        return self

    def split(self, x):
        z = x @ self.proj
        mixed, gate, beta = z.split([self.qk + self.vd, self.hv, self.hv], -1)
        return mixed, F.logsigmoid(gate.float() + 2), torch.sigmoid(beta.float())

    def heads(self, qk, v):
        q, k = qk.unflatten(-1, (2 * self.hk, self.d)).split(self.hk, -2)
        return q, k, v.unflatten(-1, (self.hv, self.d))

    def finish(self, o):
        return F.rms_norm(o, (self.d,), eps=1e-6).flatten(-2) @ self.out

    def forward(self, x, cu):
        mixed, g, beta = self.split(x)
        n = self.qk   # q and k are convolved apart from v: each result is whole
        qk = ShortConv.apply(mixed[..., :n], self.conv_w[:n], self.conv_b[:n], cu)
        v = ShortConv.apply(mixed[..., n:], self.conv_w[n:], self.conv_b[n:], cu)
        q, k, v = self.heads(qk, v)
        q, k = QkNorm.apply(q, k, *self.tables, positions_of(cu, x.shape[1]))
        return self.finish(DeltaRule.apply(q, k, v, g, beta, cu))

    def prompt(self, x, cu, state=None):
        mixed, g, beta = self.split(x)
        n, old = self.qk, state or (None, None, None)
        qk, s_qk = gdr.short_conv_fwd(mixed[..., :n], self.conv_w[:n], self.conv_b[:n], cu, old[0])
        v, s_v = gdr.short_conv_fwd(mixed[..., n:], self.conv_w[n:], self.conv_b[n:], cu, old[1])
        q, k, v = self.heads(qk, v)
        q, k = gdr.qk_norm_rope_fwd(q, k, cos=self.tables[0], sin=self.tables[1], positions=positions_of(cu, x.shape[1]),
                                    norm="l2")
        o, h = gdr.chunk_fwd(q, k, v, g, beta, cu, old[2])
        return self.finish(o), (s_qk, s_v, h)

    def step(self, x, state, positions):
        mixed, g, beta = self.split(x)
        n = self.qk
        qk = gdr.short_conv_step(mixed[:, :n], state[0], self.conv_w[:n], self.conv_b[:n])
        v = gdr.short_conv_step(mixed[:, n:], state[1], self.conv_w[n:], self.conv_b[n:])
        q, k, v = self.heads(qk, v)
        q, k = gdr.qk_norm_rope_fwd(q[:, None], k[:, None], cos=self.tables[0], sin=self.tables[1],
                                    positions=positions[:, None], norm="l2")
        return self.finish(gdr.decode_step(q[:, 0], k[:, 0], v, g, beta, state[2]))


class SsmLayer(torch.nn.Module):
    """projection -> short convolution -> state space scan -> projection"""

    def __init__(self, width, heads=16, p=64, groups=1, n=128):
        super().__init__()
        self.h, self.p, self.g, self.n = heads, p, groups, n
        self.sizes = [heads * p, groups * n, groups * n]
        self.proj = torch.nn.Parameter(torch.randn(width, sum(self.sizes) + heads) * width ** -0.5)
        self.conv_w = torch.nn.Parameter(torch.randn(sum(self.sizes), CONV_WIDTH) * 0.4)
        self.conv_b = torch.nn.Parameter(torch.randn(sum(self.sizes)) * 0.1)
        self.A = torch.nn.Parameter(-torch.linspace(1, 16, heads))
        self.D = torch.nn.Parameter(torch.ones(heads))
        self.dt_bias = torch.nn.Parameter(torch.linspace(-6, -2, heads))
        self.out = torch.nn.Parameter(torch.randn(heads * p, width) * (heads * p) ** -0.5)

    def split(self, mixed):
        x, b, c = mixed.split(self.sizes, -1)
        return x.unflatten(-1, (self.h, self.p)), b.unflatten(-1, (self.g, self.n)), c.unflatten(-1, (self.g, self.n))

    def head_params(self):   # fp32 whatever the layer's type
        return self.A.float(), self.D.float(), self.dt_bias.float()

    def forward(self, x, cu):
        mixed, dt = (x @ self.proj).split([sum(self.sizes), self.h], -1)
        u, b, c = self.split(ShortConv.apply(mixed, self.conv_w, self.conv_b, cu))
        A, D, bias = self.head_params()
        return SsmScan.apply(u, dt, A, b, c, D, bias, cu).flatten(-2) @ self.out

    def prompt(self, x, cu, state=None):
        old = state or (None, None)
        mixed, dt = (x @ self.proj).split([sum(self.sizes), self.h], -1)
        mixed, s = gdr.short_conv_fwd(mixed, self.conv_w, self.conv_b, cu, old[0])
        u, b, c = self.split(mixed)
        A, D, bias = self.head_params()
        y, h = gdr.ssm_scan_fwd(u, dt, A, b, c, D, bias, cu, old[1])
        return y.flatten(-2) @ self.out, (s, h)

    def step(self, x, state, positions):
        mixed, dt = (x @ self.proj).split([sum(self.sizes), self.h], -1)
        u, b, c = self.split(gdr.short_conv_step(mixed, state[0], self.conv_w, self.conv_b))
        A, D, bias = self.head_params()
        return gdr.ssm_step(u, dt, A, b, c, state[1], D, bias).flatten(-2) @ self.out


class Stack(torch.nn.Module):
    def __init__(self, width=512):
        super().__init__()
        self.layers = torch.nn.ModuleList([SsmLayer(width), DeltaLayer(width)])

    def forward(self, x, cu):
        for layer in self.layers:
            x = x + layer(x, cu)
        return x

    @torch.no_grad()
    def prompt(self, x, cu, states=None):
        """x [1, T, width]: packed sequences.  Returns the outputs and every layer's state."""
        new = []
        for i, layer in enumerate(self.layers):
            y, s = layer.prompt(x, cu, states and states[i])
            x = x + y
            new.append(s)
        return x, new

    @torch.no_grad()
    def step(self, x, states, positions):
        """x [N, width]: one token of each sequence; the states are updated in place."""
        for layer, s in zip(self.layers, states):
            x = x + layer.step(x, s, positions)
        return x


def packed(lengths, device):
    return torch.tensor([0] + lengths, device=device).cumsum(0).int()


class Decoder:
    """Stack.step as one captured graph: the states and positions live in it."""

    def __init__(self, model, states, positions, width, dtype):
        self.x = torch.zeros(len(positions), width, device=positions.device, dtype=dtype)
        start = [[t.clone() for t in s] for s in states]
        self.states, self.positions = states, positions.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # one step before the capture: libraries set themselves up
            model.step(self.x, states, self.positions)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = model.step(self.x, states, self.positions)
            self.positions += 1
        for s, old in zip(states, start):   # what the step before the capture changed
            for t, o in zip(s, old):
                t.copy_(o)
        self.positions.copy_(positions)

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y.clone()


def decode_and_compare(model, lengths, new, dtype, seed=0):
    """The largest relative distance, over the new tokens, between single steps
    and the prompt pass over the longer sequences; and the time of a step."""
    dev = model.layers[0].proj.device
    width = model.layers[0].proj.shape[0]
    gen = torch.Generator(device=dev).manual_seed(seed)
    xs = [torch.randn(n + new, width, device=dev, generator=gen).to(dtype) for n in lengths]
    cu = packed(lengths, dev)
    _, states = model.prompt(torch.cat([x[:n] for x, n in zip(xs, lengths)])[None], cu)
    step = Decoder(model, states, cu.diff().int(), width, dtype)
    got = [step(torch.stack([x[n + i] for x, n in zip(xs, lengths)])) for i in range(new)]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        step.graph.replay()
    torch.cuda.synchronize()
    each = (time.perf_counter() - t0) / 20
    longer = [n + new for n in lengths]
    want, _ = model.prompt(torch.cat(xs)[None], packed(longer, dev))
    want = want[0].split(longer)
    far = 0.0
    for i, y in enumerate(got):
        w = torch.stack([s[n + i] for s, n in zip(want, lengths)]).double()
        far = max(far, ((y.double() - w).norm() / w.norm()).item())
    return far, each


def train(model, cu, steps, lr=1e-3):
    """Losses of a regression onto random targets."""
    dev = model.layers[0].proj.device
    width = model.layers[0].proj.shape[0]
    x, want = (torch.randn(1, int(cu[-1]), width, device=dev).to(model.layers[0].proj.dtype) for _ in range(2))
    opt = torch.optim.Adam(model.parameters(), lr=lr, eps=1e-5)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (model(x, cu).float() - want.float()).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--new", type=int, default=32)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    torch.manual_seed(0)
    t = args.tokens
    lengths = [n for n in (1, t // 3, 63, t - t // 3 - 64) if n > 0]
    model = Stack().cuda().bfloat16()
    far, each = decode_and_compare(model, lengths, args.new, torch.bfloat16)
    print("prompt of %s tokens, then %d single tokens: within %.2g of the whole pass, %.0f us a step"
          % (lengths, args.new, far, each * 1e6))
    losses = train(model, packed(lengths, "cuda"), args.steps)
    print("training: loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], args.steps))


if __name__ == "__main__":
    main()
