"""What the operators around the 2D scan cost: layer norm, rotary positions
with several axes, and the gated delta rule (chunked and recurrent), each with
its plain form in elementary torch operations.

Layer norm:   y = (x - mean) / sqrt(var + eps) * weight + bias over the channels, of token rows [rows, n]
              or of channels-first maps [batch, channels, cells].
Rotary:       pair p of a head's dims turns by positions[axis of p] * inv_freq[p].
Gated delta:  per head, state S [d_k, d_v]:  S' = exp(g) S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = scale S^T q.
"""
import math

import torch

own = False
CHUNK = 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through the norm before a mixer: launch latency
        {"name": "norm one row", "op": "norm", "batch": 1, "n": 768, "cells": 1, "cf": False, "dtype": "bf16", "stats": False},
        # the norm of a stage-1 batch of maps in the scan's own layout (56 x 56, 192 channels)
        {"name": "norm stage maps", "op": "norm", "batch": 32, "n": 192, "cells": 56 * 56, "cf": True, "dtype": "bf16",
         "stats": True},
        # the norm's gradient on rows of 768 channels (64 maps of 14 x 14)
        {"name": "norm rows bwd", "op": "norm_bwd", "batch": 64 * 196, "n": 768, "cells": 1, "cf": False, "dtype": "bf16"},
        # the norm's gradient on the giga-pixel map (384 x 512, 128 channels, fp32)
        {"name": "norm gigapixel bwd", "op": "norm_bwd", "batch": 1, "n": 128, "cells": 384 * 512, "cf": True, "dtype": "f32"},
        # rows and columns as positions of a batch of 56 x 56 maps, 6 heads of 32
        {"name": "rotary maps", "op": "rope", "batch": 32, "frames": 1, "H": 56, "W": 56, "hq": 6, "hk": 6, "d": 32,
         "inter": False, "dtype": "bf16"},
        # time, height and width of short clips of odd size, one shared key head, gradient
        {"name": "rotary clips bwd", "op": "rope_bwd", "batch": 2, "frames": 9, "H": 33, "W": 47, "hq": 5, "hk": 1, "d": 72,
         "inter": True, "dtype": "f32"},
        # one token of one stream
        {"name": "delta step one", "op": "step", "batch": 1, "hk": 8, "h": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # one token of many streams
        {"name": "delta step many", "op": "step", "batch": 128, "hk": 8, "h": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # slides of very different sizes packed in one batch (one empty, one of a single tile), states carried in and out
        {"name": "delta packed slides", "op": "delta", "lens": "5120,1,0,777,4099,64,9973", "batch": 0, "T": 0, "hk": 4, "h": 8,
         "dk": 128, "dv": 128, "dtype": "bf16", "state": True},
        # all cells of the giga-pixel map as one sequence, 128 channels in 4 heads, fp32
        {"name": "delta gigapixel", "op": "delta", "lens": "", "batch": 1, "T": 384 * 512, "hk": 4, "h": 4, "dk": 32, "dv": 32,
         "dtype": "f32", "state": True},
        # training on 64 maps of 14 x 14, 768 channels in 12 heads
        {"name": "delta maps bwd", "op": "delta_bwd", "lens": "", "batch": 64, "T": 196, "hk": 12, "h": 12, "dk": 64, "dv": 64,
         "dtype": "bf16", "state": False},
        # training on long sequences of odd length, two value heads to a key head, states' gradients too
        {"name": "delta long bwd", "op": "delta_bwd", "lens": "", "batch": 2, "T": 4099, "hk": 4, "h": 8, "dk": 128, "dv": 128,
         "dtype": "bf16", "state": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "rope_bwd", "step", "delta", "delta", "delta_bwd", "delta_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_bwd"):
        n = _log(rng, 24, 4096)
        cf = rng.random() < 0.5
        if cf:
            n = min(n, 1536)
            batch = rng.randint(1, 32)
            cells = _log(rng, 49, max(50, min(200000, 20000000 // (n * batch))))
        else:
            batch, cells = _log(rng, 1, max(2, 20000000 // n)), 1
        c = {"op": op, "batch": batch, "n": n, "cells": cells, "cf": cf, "dtype": dtype}
        if op == "norm":
            c["stats"] = rng.random() < 0.5
        return c
    if op in ("rope", "rope_bwd"):
        frames = rng.choice([1, 1, rng.randint(2, 12)])
        H, W = rng.randint(1, 64), rng.randint(1, 64)
        hk = rng.choice([1, 2, 3, 6])
        return {"op": op, "batch": rng.randint(1, 8), "frames": frames, "H": H, "W": W, "hq": hk * rng.choice([1, 2]), "hk": hk,
                "d": 2 * rng.randint(6, 64), "inter": rng.random() < 0.5, "dtype": dtype}
    hk = rng.choice([1, 2, 3, 4, 8])
    h = hk * rng.choice([1, 1, 2, 3])
    dk, dv = rng.choice([32, 64, 96, 128, rng.randint(8, 128)]), rng.choice([32, 64, 96, 128, rng.randint(8, 128)])
    if op == "step":
        return {"op": op, "batch": _log(rng, 1, 128), "hk": hk, "h": h, "dk": dk, "dv": dv, "dtype": dtype}
    c = {"op": op, "lens": "", "batch": 0, "T": 0, "hk": hk, "h": h, "dk": dk, "dv": dv, "dtype": dtype,
         "state": rng.random() < 0.5}
    most = max(64, 5000000 // (h * max(dk, dv)))
    if rng.random() < 0.4:
        lens, left = [], min(most, 20000)
        for _ in range(rng.randint(1, 9)):
            t = 0 if rng.random() < 0.1 else _log(rng, 1, max(2, left // 2))
            lens.append(t)
            left -= t
        if sum(lens) == 0:
            lens.append(rng.randint(1, 64))
        c["lens"] = ",".join(map(str, lens))
    else:
        c["T"] = _log(rng, 2, min(most, 8192))
        c["batch"] = rng.randint(1, max(1, min(64, most // c["T"])))
    return c


# ------------------------------------------------------------------ inputs

def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lens(case):
    return [int(t) for t in case["lens"].split(",")] if case["lens"] else []


def _axes(case):
    """Pairs of each axis: (height, width), or (time, height, width) for clips."""
    half = case["d"] // 2
    if case["frames"] == 1:
        return [half - half // 2, half // 2]
    t = half // 4
    return [t, (half - t) - (half - t) // 2, (half - t) // 2]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, dev = _dt(case), torch.device("cuda")

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op, s = case["op"], {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        n = case["n"]
        shape = (case["batch"], n, case["cells"]) if case["cf"] else (case["batch"], n)
        # activations: a scale and a shift a channel, and a few channels that stand out
        a = torch.exp(0.5 * randn(n)) * torch.where(torch.rand(n, generator=gen, device=dev) < 0.02, 8.0, 1.0)
        b = 0.3 * randn(n)
        x = randn(*shape)
        x = (x * a[:, None] + b[:, None]) if case["cf"] else (x * a + b)
        s.update(x=x.to(dt), weight=1 + 0.2 * randn(n), bias=0.1 * randn(n), eps=1e-5)
        if op == "norm_bwd":
            xf, ax = s["x"].float(), 1
            s["mean"] = xf.mean(ax).contiguous()
            s["rstd"] = torch.rsqrt(xf.var(ax, unbiased=False) + s["eps"]).contiguous()
            s["dy"] = randn(*shape).to(dt)
        return s
    if op in ("rope", "rope_bwd"):
        f, H, W, B = case["frames"], case["H"], case["W"], case["batch"]
        T, d = f * H * W, case["d"]
        t = torch.arange(T, device=dev, dtype=torch.int32)
        pos = [(t // W) % H, t % W] if f == 1 else [t // (H * W), (t // W) % H, t % W]
        sec = _axes(case)
        freq = torch.cat([10000.0 ** (-torch.arange(m, device=dev, dtype=torch.float64) / max(m, 1)) for m in sec]).float()
        s.update(q=randn(B, T, case["hq"], d).to(dt), k=randn(B, T, case["hk"], d).to(dt),
                 positions=torch.stack(pos).to(torch.int32).contiguous(), inv_freq=freq, sections=tuple(sec))
        return s
    hk, h, dk, dv = case["hk"], case["h"], case["dk"], case["dv"]
    lens = _lens(case) if op != "step" else []
    B, T = (1, sum(lens)) if lens else (case["batch"], 1 if op == "step" else case["T"])

    def unit(x):
        # queries and keys as a mixer makes them: SiLU, then unit length a head
        x = x * torch.sigmoid(x)
        return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)

    q, k = unit(randn(B, T, hk, dk)).to(dt), unit(randn(B, T, hk, dk)).to(dt)
    v = randn(B, T, h, dv).to(dt)
    # log decay -A softplus(step): A in [1, 16] a head, steps around 0.01
    A = torch.exp(torch.rand(h, generator=gen, device=dev) * math.log(16.0))
    g = -A * torch.nn.functional.softplus(randn(B, T, h) - 4.0)
    beta = torch.sigmoid(randn(B, T, h))
    if op == "step":
        s.update(q=q[:, 0], k=k[:, 0], v=v[:, 0], g=g[:, 0], beta=beta[:, 0], state=0.3 * randn(B, h, dk, dv))
        return {key: t.contiguous() if isinstance(t, torch.Tensor) else t for key, t in s.items()}
    nseq = len(lens) or B
    s.update(q=q, k=k, v=v, g=g.contiguous(), beta=beta.contiguous(), h_init=None, cu=None, lens=lens)
    if lens:
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        s["cu"] = cu.to(dev)
    if case["state"]:
        s["h_init"] = 0.3 * randn(nseq, h, dk, dv)
    if op == "delta_bwd":
        s["do"] = randn(B, T, h, dv).to(dt)
        s["dh_last"] = randn(nseq, h, dk, dv) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _norm(x, w, b, eps, cf):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + eps)
    if cf:
        w, b = w[:, None], b[:, None]
    return xc * rstd * w + b, mean.squeeze(1), rstd.squeeze(1)


def _norm_bwd(x, w, mean, rstd, dy, cf):
    x, dy = x.float(), dy.float()
    mean, rstd = mean.unsqueeze(1), rstd.unsqueeze(1)
    xh = (x - mean) * rstd
    gw = dy * (w[:, None] if cf else w)
    dx = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    red = (0, 2) if cf else (0,)
    return dx, (dy * xh).sum(red), dy.sum(red)


def _rotate(x, positions, inv_freq, sections, inter, sign):
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device))
    ang = positions[axis].t().float() * inv_freq  # [T, pairs]
    c, s = torch.cos(ang)[None, :, None], sign * torch.sin(ang)[None, :, None]
    xf, half = x.float(), inv_freq.numel()
    if inter:
        x1, x2 = xf[..., 0 : 2 * half : 2], xf[..., 1 : 2 * half : 2]
        return torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2).to(x.dtype)
    x1, x2 = xf[..., :half], xf[..., half : 2 * half]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1).to(x.dtype)


def _unit_lower_inverse(L):
    """(I + L)^-1 for strictly lower L [..., CHUNK, CHUNK], by halves: [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']]."""
    T = torch.eye(CHUNK, device=L.device).expand(L.shape).clone()
    b = 1
    while b < CHUNK:
        m = CHUNK // (2 * b)
        Tb, Lb = T.unflatten(-1, (m, 2 * b)).unflatten(-3, (m, 2 * b)), L.unflatten(-1, (m, 2 * b)).unflatten(-3, (m, 2 * b))
        i = torch.arange(m, device=L.device)
        t, low = Tb[..., i, :, i, :], Lb[..., i, :, i, :]  # [m, ..., 2b, 2b]
        off = -(t[..., b:, b:] @ low[..., b:, :b] @ t[..., :b, :b])
        t = torch.cat([t[..., :b, :], torch.cat([off, t[..., b:, b:]], -1)], -2)
        Tn = torch.zeros_like(Tb)
        Tn[..., i, :, i, :] = t
        T = Tn.flatten(-4, -3).flatten(-2, -1)
        b *= 2
    return T


def _delta(q, k, v, g, beta, scale, h_init, lens):
    """o and the last states: chunks of 64 tokens, the chunks' states by a doubling scan over their transitions."""
    B, T, h, dv = v.shape
    q, k = (t.float().repeat_interleave(h // t.shape[2], 2) for t in (q, k))
    v, g, beta = v.float(), g.float(), beta.float()
    dk = q.shape[-1]
    dev = v.device
    # place of each token in whole chunks; first and last chunk of each sequence
    if lens:
        n = [-(-t // CHUNK) for t in lens]
        first = torch.tensor([0] + n, device=dev).cumsum(0)
        ln = torch.tensor(lens, device=dev)
        start = ln.cumsum(0) - ln
        seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), ln)
        at = first[seq] * CHUNK + torch.arange(T, device=dev) - start[seq]
        N = int(sum(n))
    else:
        N = -(-T // CHUNK)
        at = torch.arange(T, device=dev)

    def chunks(t):
        out = torch.zeros((B, N * CHUNK) + tuple(t.shape[2:]), device=dev)
        out = out.index_copy(1, at, t)
        out = out.unflatten(1, (N, CHUNK))
        return out.permute(0, 3, 1, 2, 4) if t.dim() == 4 else out.permute(0, 3, 1, 2)

    q, k, v, g, beta = (chunks(t) for t in (q, k, v, g, beta))  # [B, h, N, CHUNK(, d)]
    G = g.cumsum(-1)
    i = torch.arange(CHUNK, device=dev)
    low = i[:, None] >= i
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], torch.full((), -1e30, device=dev)))
    kT = k.transpose(-1, -2).contiguous()
    L = beta[..., None] * decay * (k @ kT) * (i[:, None] > i)
    Tm = _unit_lower_inverse(L)
    eG = torch.exp(G)[..., None]
    u0 = Tm @ (beta[..., None] * v)
    w = Tm @ (beta[..., None] * eG * k)
    last = torch.exp(G[..., -1:] - G)[..., None]
    kl = (k * last).transpose(-1, -2).contiguous()
    a = torch.exp(G[..., -1])[..., None, None] * torch.eye(dk, device=dev) - kl @ w  # S1 = a S0 + b
    b = kl @ u0
    # a state carried in enters ahead of its sequence's first chunk
    if lens:
        nz = [j for j in range(len(lens)) if lens[j]]
        f = first[torch.tensor(nz, device=dev)]
        keep = torch.ones(N, device=dev).index_fill(0, f, 0.0)[None, None, :, None, None]
        enter = torch.zeros((1, h, N, dk, dv), device=dev)
        if h_init is not None:
            enter = enter.index_copy(2, f, h_init[nz].float().permute(1, 0, 2, 3)[None])
    else:
        keep = torch.ones(N, device=dev).index_fill(0, torch.zeros(1, dtype=torch.long, device=dev), 0.0)[None, None, :, None, None]
        enter = torch.zeros((B, h, N, dk, dv), device=dev)
        if h_init is not None:
            enter = torch.cat([h_init.float()[:, :, None], enter[:, :, 1:]], 2)
    b = b + a @ enter
    a = a * keep
    step = 1
    while step < N:
        b = torch.cat([b[:, :, :step], b[:, :, step:] + a[:, :, step:] @ b[:, :, :-step]], 2)
        if 2 * step < N:
            a = torch.cat([a[:, :, :step], a[:, :, step:] @ a[:, :, :-step]], 2)
        step *= 2
    S1 = b
    S0 = torch.cat([torch.zeros_like(S1[:, :, :1]), S1[:, :, :-1]], 2) * keep + enter
    u = u0 - w @ S0
    o = scale * (eG * (q @ S0) + (decay * low * (q @ kT)) @ u)
    o = o.permute(0, 2, 3, 1, 4).reshape(B, N * CHUNK, h, dv)[:, at]
    if lens:
        e = torch.tensor([sum(n[: j + 1]) - 1 for j in nz], device=dev)
        S = h_init.float().clone() if h_init is not None else torch.zeros((len(lens), h, dk, dv), device=dev)
        S = S.index_copy(0, torch.tensor(nz, device=dev), S1[0, :, e].transpose(0, 1))
    else:
        S = S1[:, :, -1]
    return o, S


def _delta_bwd(s, scale):
    names = ["q", "k", "v", "g", "beta"] + (["h_init"] if s["h_init"] is not None else [])
    leaf = {n: s[n].detach().float().requires_grad_(True) for n in names}
    with torch.enable_grad():
        o, S = _delta(*(leaf[n] for n in ("q", "k", "v", "g", "beta")), scale, leaf.get("h_init"), s["lens"])
        loss = (o * s["do"].float()).sum()
        if s["dh_last"] is not None:
            loss = loss + (S * s["dh_last"]).sum()
        grads = torch.autograd.grad(loss, [leaf[n] for n in names])
    return {"d" + n: x.to(s[n].dtype) for n, x in zip(names, grads)}


def _step(s, scale):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (t.float().repeat_interleave(rep, 1) for t in (s["q"], s["k"]))
    S = s["state"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"].copy_(S)
    return scale * (S * q[..., None]).sum(-2)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import selective_state_space_ssm2d_amd as ssm2d
    if op == "norm":
        if own:
            y = ssm2d.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"], channels_first=case["cf"],
                                     return_stats=case["stats"])
            return {"y": y[0], "mean": y[1], "rstd": y[2]} if case["stats"] else {"y": y}
        y, mean, rstd = _norm(s["x"], s["weight"], s["bias"], s["eps"], case["cf"])
        y = y.to(s["x"].dtype)
        return {"y": y, "mean": mean, "rstd": rstd} if case["stats"] else {"y": y}
    if op == "norm_bwd":
        if own:
            return ssm2d.layer_norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], channels_first=case["cf"])
        dx, dw, db = _norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], case["cf"])
        return {"dx": dx.to(s["x"].dtype), "dweight": dw, "dbias": db}
    if op in ("rope", "rope_bwd"):
        args = (s["positions"], s["inv_freq"], s["sections"])
        if own:
            f = ssm2d.rope_fwd if op == "rope" else ssm2d.rope_bwd
            q, k = f(s["q"], s["k"], *args, interleaved=case["inter"])
        else:
            q, k = (_rotate(t, *args, case["inter"], 1.0 if op == "rope" else -1.0) for t in (s["q"], s["k"]))
        return {"q": q, "k": k}
    scale = case["dk"] ** -0.5
    if op == "step":
        if own:
            o = ssm2d.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=scale)
        else:
            o = _step(s, scale).to(s["v"].dtype)
        return {"o": o, "state": s["state"]}
    if op == "delta":
        if own:
            r = ssm2d.gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=scale, h_init=s["h_init"],
                                      cu_seqlens=s["cu"], return_last_state=case["state"])
            return {"o": r[0], "h_last": r[1]} if case["state"] else {"o": r}
        o, S = _delta(s["q"], s["k"], s["v"], s["g"], s["beta"], scale, s["h_init"], s["lens"])
        o = o.to(s["v"].dtype)
        return {"o": o, "h_last": S} if case["state"] else {"o": o}
    if own:
        return ssm2d.gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], scale=scale, h_init=s["h_init"],
                                     dh_last=s["dh_last"], cu_seqlens=s["cu"])
    return _delta_bwd(s, scale)


# ------------------------------------------------------------------ work

def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_bwd"):
        rows = case["batch"] * case["cells"]
        m = rows * case["n"]
        if op == "norm":
            return {"bytes": 2 * m * e + 8 * case["n"] + (8 * rows if case["stats"] else 0), "flops": 8 * m}
        return {"bytes": 3 * m * e + 12 * case["n"] + 8 * rows, "flops": 14 * m}
    if op in ("rope", "rope_bwd"):
        T = case["frames"] * case["H"] * case["W"]
        m = case["batch"] * T * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * m * e + T * 4 * len(_axes(case)) + 2 * case["d"], "flops": 3 * m}
    hk, h, dk, dv = case["hk"], case["h"], case["dk"], case["dv"]
    lens = _lens(case) if op != "step" else []
    tok = sum(lens) if lens else case["batch"] * (1 if op == "step" else case["T"])
    nseq = len(lens) or case["batch"]
    st = nseq * h * dk * dv * 4
    qk, vv, gb = tok * hk * dk * e, tok * h * dv * e, tok * h * 4
    if op == "delta_bwd":
        return {"bytes": 4 * qk + 3 * vv + 4 * gb + (3 * st if case["state"] else 0), "flops": 18 * tok * h * dk * dv}
    return {"bytes": 2 * qk + 2 * vv + 2 * gb + (2 * st if op == "step" or case["state"] else 0), "flops": 6 * tok * h * dk * dv}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for k, t in s.items()}
    op = case["op"]
    if op == "norm":
        x, w, b = d["x"], d["weight"], d["bias"]
        if case["cf"]:
            x = x.permute(0, 2, 1)
        mean = x.sum(-1) / case["n"]
        var = ((x - mean[..., None]) ** 2).sum(-1) / case["n"]
        y = (x - mean[..., None]) / torch.sqrt(var + s["eps"])[..., None] * w + b
        out = {"y": y.permute(0, 2, 1) if case["cf"] else y}
        if case["stats"]:
            out.update(mean=mean, rstd=1 / torch.sqrt(var + s["eps"]))
        return out
    if op == "norm_bwd":
        x, dy, mean, rstd = d["x"], d["dy"], d["mean"], d["rstd"]
        if case["cf"]:
            x, dy = x.permute(0, 2, 1), dy.permute(0, 2, 1)
        xh = (x - mean[..., None]) * rstd[..., None]
        dxh = dy * d["weight"]
        n = case["n"]
        dx = rstd[..., None] / n * (n * dxh - dxh.sum(-1, keepdim=True) - xh * (dxh * xh).sum(-1, keepdim=True))
        xh, dy = xh.reshape(-1, n), dy.reshape(-1, n)
        return {"dx": dx.permute(0, 2, 1) if case["cf"] else dx, "dweight": (xh * dy).sum(0), "dbias": dy.sum(0)}
    if op in ("rope", "rope_bwd"):
        out, sec, sign = {}, s["sections"], 1.0 if op == "rope" else -1.0
        ang = torch.cat([s["positions"][a].double()[:, None] * d["inv_freq"][sum(sec[:a]) : sum(sec[: a + 1])] for a in range(len(sec))], 1)
        turn = torch.polar(torch.ones_like(ang), sign * ang)[None, :, None]
        half = case["d"] // 2
        for name in ("q", "k"):
            x = d[name]
            z = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) if case["inter"] else torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
            z = z * turn
            out[name] = torch.view_as_real(z).flatten(-2) if case["inter"] else torch.cat([z.real, z.imag], -1)
        return out
    scale, h, hk, dk, dv = case["dk"] ** -0.5, case["h"], case["hk"], case["dk"], case["dv"]
    if op == "step":
        o, S, _ = _tokens(d["q"][:, None], d["k"][:, None], d["v"][:, None], d["g"][:, None], d["beta"][:, None], scale, d["state"])
        return {"o": o[:, 0], "state": S}
    parts = s["lens"] or [case["T"]]
    if sum(parts) > 220000 or (op == "delta_bwd" and sum(parts) * (1 if s["lens"] else case["batch"]) * h * dk * dv * 8 > 40e9):
        return None
    got, at = [], 0
    for j, t in enumerate(parts):
        x = [d[n][:, at : at + t] for n in ("q", "k", "v", "g", "beta")]
        S0 = torch.zeros((x[0].shape[0], h, dk, dv), device=x[0].device, dtype=torch.float64)
        if d["h_init"] is not None:
            S0 = d["h_init"][j : j + 1] if s["lens"] else d["h_init"]
        if op == "delta":
            o, S, _ = _tokens(*x, scale, S0)
            got.append({"o": o, "h_last": S})
        else:
            D = torch.zeros_like(S0)
            if d["dh_last"] is not None:
                D = d["dh_last"][j : j + 1] if s["lens"] else d["dh_last"]
            got.append(_tokens_bwd(*x, scale, S0, d["do"][:, at : at + t], D))
        at += t
    out = {n: torch.cat([p[n] for p in got], 0 if n in ("h_last", "dh_init") else 1) for n in got[0]}
    if not case["state"]:
        out.pop("h_last" if op == "delta" else "dh_init")
    return out


def _tokens(q, k, v, g, beta, scale, S, keep=False):
    """The recurrence, token by token; `keep`: the state before each token, and each token's u before beta."""
    rep = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    a = torch.exp(g)[..., None, None]
    o = torch.zeros(v.shape, device=v.device, dtype=torch.float64)
    hist = torch.zeros((v.shape[1],) + tuple(S.shape), device=v.device, dtype=torch.float64) if keep else None
    for t in range(v.shape[1]):
        if keep:
            hist[t] = S
        S = a[:, t] * S
        e = v[:, t] - (S * k[:, t, :, :, None]).sum(2)
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        o[:, t] = scale * (S * q[:, t, :, :, None]).sum(2)
    return o, S, hist


def _tokens_bwd(q, k, v, g, beta, scale, S0, do, D):
    """Its derivative, token by token from the last."""
    B, T, h, dv = v.shape
    hk, dk = q.shape[2], q.shape[3]
    hist = _tokens(q, k, v, g, beta, scale, S0, keep=True)[2]
    q, k = q.repeat_interleave(h // hk, 2), k.repeat_interleave(h // hk, 2)
    r = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v), "dg": torch.zeros_like(g), "dbeta": torch.zeros_like(beta)}
    for t in range(T - 1, -1, -1):
        a, kt, qt, b = torch.exp(g[:, t])[..., None, None], k[:, t, :, :, None], q[:, t, :, :, None], beta[:, t, :, None]
        Sd = a * hist[t]
        e = v[:, t] - (Sd * kt).sum(2)
        S = Sd + kt * (b * e)[:, :, None]
        r["dq"][:, t] = scale * (S * do[:, t, :, None]).sum(-1)
        D = D + scale * qt * do[:, t, :, None]
        du = (D * kt).sum(2)
        r["dbeta"][:, t] = (du * e).sum(-1)
        r["dv"][:, t] = b * du
        r["dk"][:, t] = (D * (b * e)[:, :, None]).sum(-1) - (Sd * (b * du)[:, :, None]).sum(-1)
        D = D - kt * (b * du)[:, :, None]
        r["dg"][:, t] = (D * Sd).sum((-1, -2))
        D = a * D
    for n in ("dq", "dk"):
        r[n] = r[n].unflatten(2, (hk, h // hk)).sum(3)
    r["dh_init"] = D
    return r
