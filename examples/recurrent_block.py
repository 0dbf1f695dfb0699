"""Blocks of a gated linear recurrence over the cells of a map: projections from
the map's layout to token rows and back, the recurrence along the cells, its
output normed by heads and gated, and the norms between blocks together with the
residual stream in 32 bits.

    python examples/recurrent_block.py [--height 32 --width 32 --channels 64 --inner 128 --blocks 2 --dtype bf16]

trains them for a few steps on random maps (the operators' backward passes behind
torch.autograd) and then serves: a map's first rows at once, the rest cell by cell
from the states they left, which must give the same outputs.
"""
import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import selective_state_space_ssm2d_amd as ssm2d  # noqa: E402


class Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, channels_first, out_channels_first):
        args = dict(act=act, channels_first=channels_first, out_channels_first=out_channels_first)
        w = weight.to(x.dtype)
        keep = act is not None
        y = ssm2d.linear_fwd(x, w, bias, residual, return_pre=keep, **args)
        y, pre = y if keep else (y, None)
        ctx.save_for_backward(x, w, pre)
        ctx.args = args
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, pre = ctx.saved_tensors
        _, has_weight, has_bias, has_residual = ctx.needs_input_grad[:4]
        g = ssm2d.linear_bwd(x, w, dy.contiguous(), pre, bias=has_bias, **ctx.args)
        return g["dx"], g["dweight"].float() if has_weight else None, g.get("dbias"), dy if has_residual else None, None, None, None


class BlockNorm(torch.autograd.Function):
    """(out, y) of block_norm_fwd with next_weight, else out."""

    @staticmethod
    def forward(ctx, x, weight, gate, residual, scale, next_weight, groups):
        ctx.save_for_backward(x, weight, gate, residual, scale, next_weight)
        ctx.groups = groups
        return ssm2d.block_norm_fwd(x, weight, gate=gate, residual=residual, scale=scale, next_weight=next_weight, groups=groups)

    @staticmethod
    def backward(ctx, dout, dy=None):
        x, weight, gate, residual, scale, next_weight = ctx.saved_tensors
        dout, dy = (t.contiguous() if t is not None else None for t in (dout, dy))
        g = ssm2d.block_norm_bwd(x, dout, dy, weight, gate=gate, residual=residual, scale=scale, next_weight=next_weight, groups=ctx.groups)
        return (*(g.get(k) for k in ("dx", "dweight", "dgate", "dresidual", "dscale", "dnext_weight")), None)


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g):
        ctx.save_for_backward(x, g)
        return ssm2d.recurrence_fwd(x, g, gates="sigmoid")

    @staticmethod
    def backward(ctx, dh):
        r = ssm2d.recurrence_bwd(*ctx.saved_tensors, dh.contiguous(), gates="sigmoid")
        return r["dx"], r["dg"]


class RecurrentBlocks(torch.nn.Module):
    def __init__(self, channels, inner, blocks, heads=4, device="cuda"):
        super().__init__()
        new = lambda *s, std: torch.nn.Parameter(torch.randn(*s, device=device) * std)  # noqa: E731
        full = lambda n, v=1.0: torch.nn.Parameter(torch.full((n,), v, device=device))  # noqa: E731
        self.heads = heads
        self.embed, self.embed_bias = new(inner, channels, std=channels ** -0.5), full(inner, 0.0)
        self.readout = new(channels, inner, std=0.5 * inner ** -0.5)
        self.blocks = torch.nn.ModuleList()
        for _ in range(blocks):
            b = torch.nn.Module()
            b.pre, b.post, b.head, b.scale = full(inner), full(inner), full(inner), full(inner, 0.5)
            b.w_in = new(3 * inner, inner, std=inner ** -0.5)
            b.b_in = torch.nn.Parameter(torch.cat([torch.zeros(inner), torch.linspace(0, 4, inner), torch.zeros(inner)]).to(device))
            b.w_out = new(inner, inner, std=inner ** -0.5)
            self.blocks.append(b)
        self.last = full(inner)

    def mixed(self, b, y, recurrence):
        """A block's branch of normed tokens: recurrence(x, g), normed by heads, gated, projected."""
        x, g, z = Linear.apply(y, b.w_in, b.b_in, None, None, False, None).chunk(3, -1)
        return Linear.apply(BlockNorm.apply(recurrence(x, g), b.head, z, None, None, None, self.heads), b.w_out, None, None, None, False, None)

    def tokens(self, e, recurrences):
        """Of embedded tokens [..., inner] what the readout sees."""
        stream = e.float()
        _, y = BlockNorm.apply(torch.zeros_like(e), None, None, stream, None, self.blocks[0].pre, 1)
        for i, b in enumerate(self.blocks):
            after = self.blocks[i + 1].pre if i + 1 < len(self.blocks) else self.last
            stream, y = BlockNorm.apply(self.mixed(b, y, recurrences[i]), b.post, None, stream, b.scale, after, 1)
        return y

    def forward(self, x):
        e = Linear.apply(x, self.embed, self.embed_bias, None, "silu", True, False)  # maps to rows
        y = self.tokens(e, [Recurrence.apply] * len(self.blocks))
        return Linear.apply(y, self.readout, None, x.flatten(2), None, False, True).view_as(x)  # and back, added to the map

    @torch.no_grad()
    def serve(self, x, first_rows):
        """forward(x) as a stream: the first rows at once, then cell by cell."""
        batch, channels, height, width = x.shape
        states = [None] * len(self.blocks)

        def first(i):
            def run(u, g):
                h, states[i] = ssm2d.recurrence_fwd(u, g, gates="sigmoid", return_last_state=True)
                return h
            return run

        def step(i):
            return lambda u, g: ssm2d.recurrence_step(u, g, states[i], gates="sigmoid")

        embed, readout = self.embed.to(x.dtype), self.readout.to(x.dtype)
        head = x[:, :, :first_rows]
        e = ssm2d.linear_fwd(head.contiguous(), embed, self.embed_bias, act="silu", channels_first=True, out_channels_first=False)
        y = self.tokens(e, [first(i) for i in range(len(self.blocks))])
        out = [ssm2d.linear_fwd(y, readout, None, head.flatten(2), out_channels_first=True)]
        for cell in range(first_rows * width, height * width):
            at = x.flatten(2)[:, :, cell].contiguous()
            e = ssm2d.linear_fwd(at, embed, self.embed_bias, act="silu")
            y = self.tokens(e, [step(i) for i in range(len(self.blocks))])
            out.append(ssm2d.linear_fwd(y, readout, None, at)[:, :, None])
        return torch.cat(out, 2).view_as(x)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("batch", 2), ("channels", 64), ("inner", 128), ("blocks", 2), ("height", 32), ("width", 32), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="bf16")
    a = ap.parse_args()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype]
    torch.manual_seed(0)
    model = RecurrentBlocks(a.channels, a.inner, a.blocks)
    x = torch.randn(a.batch, a.channels, a.height, a.width, device="cuda").to(dtype)
    target = x.roll(1, -1)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss = F.mse_loss(model(x).float(), target.float())
        opt.zero_grad()
        loss.backward()
        opt.step()
        torch.cuda.synchronize()
        print(f"step {step}: loss {loss.item():.4f}, {1e3 * (time.perf_counter() - t):.2f} ms", flush=True)
    with torch.no_grad():
        full = model(x)
    rows = a.height - 1
    diff = (model.serve(x, rows) - full).abs().max().item()
    print(f"served {rows} rows at once and {a.width} cells one by one: outputs within {diff:.2e} of the whole map's")


if __name__ == "__main__":
    main()
