"""A stack that alternates a recurrent layer with softmax attention, run as it is
used in a model: the delta-rule layer of token_mixer.py, full attention and
attention with a window, both decoding from a paged key-value cache.

    python examples/hybrid_stack.py [--tokens 4096] [--new 32] [--steps 20]

1. a prompt of packed sequences: keys and values go to pages that are planned on
   the GPU from the lengths;
2. single tokens in a captured graph, which plans their pages, stores their keys
   and attends over the cache, checked against the whole pass over the longer
   sequences;
3. a few training steps, gradients through every operator.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import token_mixer as tm  # noqa: E402
from token_mixer import gdr  # noqa: E402


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu, window):
        o, lse = gdr.attn_fwd(q, k, v, cu, window=window)
        ctx.save_for_backward(q, k, v, o, lse, cu)
        ctx.window = window
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, cu = ctx.saved_tensors
        return gdr.attn_bwd(q, k, v, o, lse, do.contiguous(), cu, window=ctx.window) + (None, None)


class Pages:
    """The page tables that all attention layers share, kept on the GPU: what a call takes from the list of free pages
    leaves it there."""

    def __init__(self, sequences, longest, page, device):
        self.page, width = page, -(-longest // page)
        self.past = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.table = torch.full((sequences, width), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(sequences * width, device=device).int()
        self.at = torch.arange(self.free.numel(), device=device)

    def take(self, new, tokens):
        """Room for `new` tokens of each sequence (`tokens` in all): (cu_seqlens, positions, slots)."""
        cu, lens, positions, slots, used = gdr.page_plan(self.past, new, self.free, self.table, self.page, tokens)
        self.past.copy_(lens)
        at = self.at + used[1]
        self.free.copy_(torch.where(at < at.numel(), self.free[at.clamp(max=at.numel() - 1)], -1))
        return cu, positions, slots


class AttentionLayer(torch.nn.Module):
    """projection -> norm and rotation of q and k -> attention -> projection"""

    def __init__(self, width, hq=8, hk=2, d=64, window=0, table=65536):
        super().__init__()
        self.hq, self.hk, self.d, self.window = hq, hk, d, window
        self.proj = torch.nn.Parameter(torch.randn(width, (hq + 2 * hk) * d) * width ** -0.5)
        self.out = torch.nn.Parameter(torch.randn(hq * d, width) * (hq * d) ** -0.5)
        angle = torch.arange(table, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2).double() / d)
        self.tables = angle.cos().float(), angle.sin().float()

    def _apply(self, fn, *args, **kw):   # the tables follow the device and stay fp32
        super()._apply(fn, *args, **kw)
        self.tables = tuple(t.to(self.proj.device) for t in self.tables)
        return self

    def heads(self, x):   # slices of one projection: the operators take rows as they lie
        return (x @ self.proj).unflatten(-1, (self.hq + 2 * self.hk, self.d)).split([self.hq, self.hk, self.hk], -2)

    def norm(self, q, k, positions):
        return gdr.qk_norm_rope_fwd(q, k, cos=self.tables[0], sin=self.tables[1], positions=positions, norm="l2")

    # normed by length 1, so that a score is the cosine of an angle: the scale lets a row choose
    def forward(self, x, cu):
        q, k, v = self.heads(x)
        q, k = tm.QkNorm.apply(q, k, *self.tables, tm.positions_of(cu, x.shape[1]))
        return Attention.apply(q * self.d ** 0.5, k, v, cu, self.window).flatten(-2) @ self.out

    def cache(self, pages):
        shape = pages.free.numel(), pages.page, self.hk, self.d
        return tuple(torch.zeros(shape, dtype=self.proj.dtype, device=self.proj.device) for _ in range(2))

    def prompt(self, x, plan, cache):
        cu, positions, slots = plan
        q, k, v = self.heads(x)
        q, k = self.norm(q, k, positions)
        gdr.page_store(k, v, slots, *cache)
        return gdr.attn_fwd(q * self.d ** 0.5, k, v, cu, window=self.window, output_lse=False)[0].flatten(-2) @ self.out

    def step(self, x, plan, cache, pages):
        _, positions, slots = plan
        q, k, v = self.heads(x[None])          # [1, N, heads, d]: the new tokens as one packed row
        q, k = self.norm(q, k, positions)
        gdr.page_store(k, v, slots, *cache)
        o = gdr.attn_paged_step(q[0] * self.d ** 0.5, *cache, pages.table, pages.past, window=self.window)
        return o.flatten(-2) @ self.out


class Stack(torch.nn.Module):
    def __init__(self, width=512, window=128):
        super().__init__()
        self.layers = torch.nn.ModuleList([tm.DeltaLayer(width), AttentionLayer(width), AttentionLayer(width, window=window)])

    def forward(self, x, cu):
        for layer in self.layers:
            x = x + layer(x, cu)
        return x

    @torch.no_grad()
    def prompt(self, x, lengths, pages):
        """x [1, T, width]: packed sequences of lengths (on the GPU).  Returns the outputs and every layer's state."""
        plan, states = pages.take(lengths, x.shape[1]), []
        for layer in self.layers:
            if isinstance(layer, AttentionLayer):
                states.append(layer.cache(pages))
                y = layer.prompt(x, plan, states[-1])
            else:
                y, s = layer.prompt(x, plan[0])
                states.append(s)
            x = x + y
        return x, states

    @torch.no_grad()
    def step(self, x, states, pages, one):
        """x [N, width]: one token of each sequence (`one`: N ones); states and pages are updated in place."""
        plan = pages.take(one, x.shape[0])
        for layer, s in zip(self.layers, states):
            x = x + (layer.step(x, plan, s, pages) if isinstance(layer, AttentionLayer) else layer.step(x, s, plan[1][0]))
        return x


class Decoder:
    """Stack.step as one captured graph: states, pages and lengths live in it."""

    def __init__(self, model, states, pages, width, dtype):
        kept = [t for s in states for t in s] + [pages.past, pages.table, pages.free]
        start = [t.clone() for t in kept]
        self.x = torch.zeros(len(pages.past), width, device=pages.past.device, dtype=dtype)
        one = torch.ones_like(pages.past)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # one step before the capture: libraries set themselves up
            model.step(self.x, states, pages, one)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = model.step(self.x, states, pages, one)
        self.kept = kept, one
        for t, o in zip(kept, start):   # what the step before the capture changed
            t.copy_(o)

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y.clone()


def decode_and_compare(model, lengths, new, dtype, page=16, seed=0):
    """The largest relative distance, over the new tokens, between single steps
    and the whole pass over the longer sequences; and the time of a step."""
    dev = model.layers[0].proj.device
    width = model.layers[0].proj.shape[0]
    gen = torch.Generator(device=dev).manual_seed(seed)
    xs = [torch.randn(n + new, width, device=dev, generator=gen).to(dtype) for n in lengths]
    pages = Pages(len(lengths), max(lengths) + new + 24, page, dev)   # 24: the timed steps below
    counts = torch.tensor(lengths, dtype=torch.int32, device=dev)
    _, states = model.prompt(torch.cat([x[:n] for x, n in zip(xs, lengths)])[None], counts, pages)
    step = Decoder(model, states, pages, width, dtype)
    got = [step(torch.stack([x[n + i] for x, n in zip(xs, lengths)])) for i in range(new)]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        step.graph.replay()
    torch.cuda.synchronize()
    each = (time.perf_counter() - t0) / 20
    longer = [n + new for n in lengths]
    with torch.no_grad():
        want = model(torch.cat(xs)[None], tm.packed(longer, dev))[0].split(longer)
    far = 0.0
    for i, y in enumerate(got):
        w = torch.stack([s[n + i] for s, n in zip(want, lengths)]).double()
        far = max(far, ((y.double() - w).norm() / w.norm()).item())
    return far, each


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
    losses = tm.train(model, tm.packed(lengths, "cuda"), args.steps)
    print("training: loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], args.steps))


if __name__ == "__main__":
    main()
