"""A block over the cells of a map: layer norm of the channels-first map, rotary
positions of rows and columns on queries and keys, the gated delta rule along the
cells, and a residual projection back to the map.

    python examples/map_mixer.py [--height 64 --width 64 --channels 96 --heads 4 --dtype bf16]

trains it for a few steps on random maps (the operators' backward passes behind
torch.autograd) and then serves it: a map's first rows at once, the rest cell by
cell from the state they left, which must give the same outputs.
"""
import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import selective_state_space_ssm2d_amd as ssm2d  # noqa: E402


class MapNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ssm2d.layer_norm_fwd(x, weight, bias, eps, channels_first=True, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = ssm2d.layer_norm_bwd(x, weight, mean, rstd, dy.contiguous(), channels_first=True)
        return g["dx"], g["dweight"], g["dbias"], None


class Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, sections):
        ctx.save_for_backward(positions, inv_freq)
        ctx.sections = sections
        return ssm2d.rope_fwd(q, k, positions, inv_freq, sections)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*ssm2d.rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors, ctx.sections), None, None, None)


class GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return ssm2d.gated_delta_fwd(q, k, v, g, beta)

    @staticmethod
    def backward(ctx, do):
        r = ssm2d.gated_delta_bwd(*ctx.saved_tensors, do.contiguous())
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"]


class MapMixer(torch.nn.Module):
    """``heads`` heads read ``heads_qk`` queries and keys of d_k = 2 * pairs dims;
    the first half of the pairs turns with the row, the other with the column."""

    def __init__(self, channels, heads, heads_qk=None, pairs=16, d_v=32, device="cuda"):
        super().__init__()
        self.heads, self.heads_qk, self.pairs, self.d_v = heads, heads_qk or heads, pairs, d_v
        new = lambda *s, std: torch.nn.Parameter(torch.randn(*s, device=device) * std)  # noqa: E731
        self.norm_weight = torch.nn.Parameter(torch.ones(channels, device=device))
        self.norm_bias = torch.nn.Parameter(torch.zeros(channels, device=device))
        self.wide = 4 * self.heads_qk * pairs + heads * d_v
        self.w_in = new(channels, self.wide + 2 * heads, std=channels ** -0.5)
        self.w_out = new(heads * d_v, channels, std=(heads * d_v) ** -0.5)
        self.sections = (pairs // 2, pairs - pairs // 2)
        freq = [100.0 ** (-i / s) for s in self.sections for i in range(s)]
        self.register_buffer("inv_freq", torch.tensor(freq, device=device))

    def positions(self, rows, width):
        """int32 [2, cells] of the cells of some rows: their row and their column."""
        r = torch.as_tensor(rows, dtype=torch.int32, device=self.inv_freq.device)
        return torch.stack([r.repeat_interleave(width), torch.arange(width, dtype=torch.int32, device=r.device).repeat(len(r))])

    def project(self, y):
        """q, k, v, g, beta of normed cells [batch, cells, channels]."""
        z = y @ self.w_in.to(y.dtype)
        d = 2 * self.pairs
        q, k, v = z[..., :self.wide].split([self.heads_qk * d, self.heads_qk * d, self.heads * self.d_v], -1)
        gate, beta = z[..., self.wide:].float().split(self.heads, -1)
        q, k = (F.normalize(t.float().unflatten(-1, (self.heads_qk, d)), dim=-1).to(y.dtype) for t in (q, k))
        return q, k, v.unflatten(-1, (self.heads, self.d_v)), -0.1 * F.softplus(gate), torch.sigmoid(beta)

    def forward(self, x):
        batch, channels, height, width = x.shape
        y = MapNorm.apply(x, self.norm_weight, self.norm_bias, 1e-5)
        q, k, v, g, beta = self.project(y.flatten(2).transpose(1, 2))
        q, k = Rope.apply(q, k, self.positions(range(height), width), self.inv_freq, self.sections)
        o = GatedDelta.apply(q, k, v, g, beta)
        return x + (o.flatten(2) @ self.w_out.to(x.dtype)).transpose(1, 2).reshape(x.shape)

    @torch.no_grad()
    def serve(self, x, first_rows):
        """forward(x) as a stream: the first rows at once, then cell by cell."""
        batch, channels, height, width = x.shape
        head = x[:, :, :first_rows]
        y = ssm2d.layer_norm_fwd(head.contiguous(), self.norm_weight, self.norm_bias, channels_first=True)
        q, k, v, g, beta = self.project(y.flatten(2).transpose(1, 2))
        q, k = ssm2d.rope_fwd(q, k, self.positions(range(first_rows), width), self.inv_freq, self.sections)
        o, state = ssm2d.gated_delta_fwd(q, k, v, g, beta, return_last_state=True)
        out = [o]
        for row in range(first_rows, height):
            at = self.positions([row], width)
            for col in range(width):
                cell = x[:, :, row, col]
                y = ssm2d.layer_norm_fwd(cell, self.norm_weight, self.norm_bias, channels_first=True)
                q, k, v, g, beta = self.project(y[:, None])
                q, k = ssm2d.rope_fwd(q, k, at[:, col:col + 1], self.inv_freq, self.sections)
                o = ssm2d.gated_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state)
                out.append(o[:, None])
        o = torch.cat(out, 1)
        return x + (o.flatten(2) @ self.w_out.to(x.dtype)).transpose(1, 2).reshape(x.shape)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("batch", 2), ("channels", 96), ("height", 64), ("width", 64), ("heads", 4), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="bf16")
    a = ap.parse_args()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[a.dtype]
    torch.manual_seed(0)
    mixer = MapMixer(a.channels, a.heads)
    x = torch.randn(a.batch, a.channels, a.height, a.width, device="cuda").to(dtype)
    target = x.roll(1, -1)
    opt = torch.optim.Adam(mixer.parameters(), lr=1e-2)
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss = F.mse_loss(mixer(x).float(), target.float())
        opt.zero_grad()
        loss.backward()
        opt.step()
        torch.cuda.synchronize()
        print(f"step {step}: loss {loss.item():.4f}, {1e3 * (time.perf_counter() - t):.2f} ms", flush=True)
    with torch.no_grad():
        full = mixer(x)
    rows = a.height - 1
    diff = (mixer.serve(x, rows) - full).abs().max().item()
    print(f"served {rows} rows at once and {a.width} cells one by one: outputs within {diff:.2e} of the whole map's")


if __name__ == "__main__":
    main()
