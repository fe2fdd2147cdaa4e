"""What is measured of the 8-bit token mixer's operators and of the norms around it: the cases,
their inputs, each operator in plain torch, and the calls a user makes of the library's kernels.

Operators:
    linear_i8      out = (x_q w_q^T) scaled per token and per channel, + bias, + addend
    quantize_rows  the 8-bit codes and the scale of each row
    gate_norm_i8   y SiLU(z), RMS-normalised per channel group, as 8-bit codes and row scales
    block_norm     the norms before and after a block with its modulation, gate and residual scale

The widths are the block's: model width 2560, 80 x 64 SSD channels, 20 x 128 attention channels,
10,448 in_proj rows; the token counts are those of its grids (32,768 = 32x32x32, 131,072 = 128x32x32,
2 x 73,728 = two of 32x48x48), of the ragged 7 x 11 x 15 grid, and of a conditioning vector (one row
per video).
"""
import math

import torch

own = False

_D = 2560            # model width
_MA = 5120           # MA-branch channels, 80 heads x 64
_IN = 10448          # in_proj rows: z 5120, x|B|C 5248, dt 80
_BF, _F32 = "bf16", "f32"
_DT = {_BF: torch.bfloat16, _F32: torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the modulation vectors (shift, scale, gate) of a layer from the conditioning of two videos
        dict(name="linear modulation 2 rows", op="linear", M=2, K=_D, N=3 * _D, out=_F32, bias=True, addend=False),
        # a projection of a short clip's ragged grid (7 x 11 x 15 tokens)
        dict(name="linear ragged 1155", op="linear", M=1155, K=_D, N=_D, out=_BF, bias=False, addend=False),
        # the composition of a 32x32x32 grid: the MA branch added to the TE branch's projection
        dict(name="linear compose 32k", op="linear", M=32768, K=_MA, N=_D, out=_BF, bias=False, addend=True),
        # in_proj of the 128x32x32 grid: the block's largest matrix product
        dict(name="linear in_proj 131k", op="linear", M=131072, K=_D, N=_IN, out=_BF, bias=False, addend=False),
        # the conditioning vectors of two videos, ahead of the modulation product
        dict(name="quantize 2 rows", op="quant", M=2, K=_D),
        # the TE-branch output of the 128x32x32 grid, ahead of its projection
        dict(name="quantize 131k", op="quant", M=131072, K=_D),
        # the MA-branch output side of the ragged grid, two channel groups
        dict(name="gate_norm ragged 1155", op="gate", M=1155, C=_MA, groups=2),
        # the MA-branch output side of the 128x32x32 grid
        dict(name="gate_norm 131k", op="gate", M=131072, C=_MA, groups=1),
        # one token of each of two videos, layer norm ahead of the first block
        dict(name="norm before, 1 token", op="norm", B=2, n=1, C=_D, kind="layer", x=_BF, post=False, y=False, h=_BF),
        # three ragged grids, residual stream in fp32: the norm after one block and before the next
        dict(name="norm after+before 3x1155", op="norm", B=3, n=1155, C=_D, kind="rms", x=_F32, post=True, y=True,
             h=_BF),
        # between two 8-bit blocks on the 128x32x32 grid: after one, before the next, codes out
        dict(name="norm after+before i8 131k", op="norm", B=1, n=131072, C=_D, kind="rms", x=_BF, post=True, y=True,
             h="i8"),
        # after the last block of two 32x48x48 grids: the gated residual alone
        dict(name="norm after 2x73728", op="norm", B=2, n=73728, C=_D, kind="rms", x=_BF, post=True, y=True, h=None),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "quant", "gate", "norm", "norm"])
    M = _log(rng, 1, 131072)
    if op == "linear":
        K, N = 16 * _log(rng, 4, 480), 8 * _log(rng, 8, 1306)
        out = rng.choice([_BF, _BF, _F32])
        addend = rng.random() < 0.3
        # no more work and no more bytes than the in_proj of the 128x32x32 grid
        size = lambda m: max(m * K * N / (131072 * _D * _IN),  # noqa: E731
                             m * (K + N * (4 if out == _F32 else 2) * (1 + addend)) / (131072 * (_D + 2 * _IN)))
        while size(M) > 1:
            M = M * 3 // 4
        return dict(op=op, M=M, K=K, N=N, out=out, bias=rng.random() < 0.5, addend=addend)
    if op == "quant":
        return dict(op=op, M=M, K=16 * _log(rng, 4, 640) if M < 32768 else _D)
    if op == "gate":
        g = rng.choice([1, 2, 4])
        return dict(op=op, M=M, C=g * 16 * _log(rng, 4, 320 // g), groups=g)
    B = min(M, rng.choice([1, 1, 2, 3, 4]))
    y = rng.random() < 0.7
    return dict(op=op, B=B, n=M // B, C=8 * _log(rng, 8, 320), kind=rng.choice(["rms", "layer"]),
                x=rng.choice([_BF, _BF, _F32]), post=y and rng.random() < 0.7, y=y,
                h=rng.choice([_BF, "i8", "i8"] + ([None] if y else [])))


# ------------------------------------------------------------------ inputs
def _codes(v):
    """8-bit codes and scales of fp32 rows, as a user's program holds them before a product."""
    s = v.abs().amax(1) / 127
    return torch.round(v / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op = case, case["op"]

    def rn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        xq, xs = _codes(rn(M, K))
        wq, ws = _codes(rn(N, K) / math.sqrt(K))
        return dict(op=op, xq=xq, xs=xs, wq=wq, ws=ws, out=_DT[c["out"]],
                    bias=rn(N) / 10 if c["bias"] else None,
                    addend=rn(M, N).to(_DT[c["out"]]) if c["addend"] else None)
    if op == "quant":
        return dict(op=op, x=(rn(c["M"], c["K"]) * torch.exp(0.5 * rn(c["K"]))).to(torch.bfloat16))
    if op == "gate":
        M, C = c["M"], c["C"]
        return dict(op=op, y=rn(M, C).to(torch.bfloat16), z=rn(M, C).to(torch.bfloat16), w=1 + rn(C) / 10,
                    group=C // c["groups"], eps=1e-5)
    B, n, C = c["B"], c["n"], c["C"]
    x = (rn(B, n, C) * torch.exp(0.5 * rn(C)) + rn(C) / 4).to(_DT[c["x"]])
    y = rn(B, n, C).to(torch.bfloat16) if c["y"] else None
    mod = rn(B, 3 * C) / 4  # shift, scale and gate of each video, as the modulation product leaves them
    return dict(op=op, x=x, y=y, shift=mod[:, :C], scale=mod[:, C:2 * C], gate=mod[:, 2 * C:], w_post=1 + rn(C) / 10,
                w_pre=1 + rn(C) / 10, kind=c["kind"], post=c["post"], h=c["h"], alpha=0.875, eps=1e-6)


# ------------------------------------------------------------------ plain forms
def _plain_norm(v, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def _values(q, s):
    """What the codes of each row stand for, as the model's activations."""
    return torch.mul(q, s[..., None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))


def _plain_quant(v):
    """Codes and scales of rows: the code's border is one half, so it is found in 64 bits."""
    amax = v.abs().amax(-1, keepdim=True)
    q = torch.round(v.double() * 127 / amax.double().clamp_min(1e-300)).to(torch.int8)
    return q, (amax / 127).squeeze(-1)


def _plain(st):
    op = st["op"]
    if op == "linear":
        out = st["xq"].float() @ st["wq"].float().T
        out *= st["xs"][:, None]
        out *= st["ws"]
        if st["bias"] is not None:
            out += st["bias"]
        if st["addend"] is not None:
            out += st["addend"]
        return out.to(st["out"])
    if op == "quant":
        q, s = _plain_quant(st["x"].float())
        return _values(q, s), s
    if op == "gate":
        z = st["z"].float()
        v = st["y"].float() * (z / (1 + torch.exp(-z)))
        v = _plain_norm(v.view(v.shape[0], -1, st["group"]), "rms", st["eps"]).flatten(1) * st["w"]
        q, s = _plain_quant(v)
        return _values(q, s), s
    r, out = st["x"].float(), []
    if st["y"] is not None:
        y = st["y"].float()
        if st["post"]:
            y = _plain_norm(y, st["kind"], st["eps"]) * st["w_post"]
        r = st["alpha"] * r + st["gate"][:, None] * y
        out.append(r.to(st["x"].dtype))
    if st["h"] is not None:
        h = _plain_norm(r, st["kind"], st["eps"]) * st["w_pre"] * (1 + st["scale"][:, None]) + st["shift"][:, None]
        if st["h"] == "i8":
            q, s = _plain_quant(h)
            out += [_values(q, s), s]
        else:
            out.append(h.to(torch.bfloat16))
    return out


# ------------------------------------------------------------------ the library's calls
def _own(st):
    import linear_complexity_video_b200 as mate

    op = st["op"]
    if op == "linear":
        return mate.linear_i8(st["xq"], st["xs"], st["wq"], st["ws"], bias=st["bias"], addend=st["addend"],
                              out_dtype=st["out"])
    if op == "quant":
        q, s = mate.quantize_rows(st["x"])
        return _values(q, s), s
    if op == "gate":
        q, s = mate.gate_norm_i8(st["y"], st["z"], st["w"], st["group"], st["eps"])
        return _values(q, s), s
    post = dict(y=st["y"], gate=st["gate"], residual_scale=st["alpha"], post_norm=st["post"]) if st["y"] is not None \
        else {}
    if st["post"]:
        post["w_post"] = st["w_post"]
    pre = dict(w_pre=st["w_pre"], scale=st["scale"], shift=st["shift"]) if st["h"] is not None else {}
    r, h = mate.block_norm(st["x"], **post, **pre, norm=st["kind"], eps=st["eps"],
                           h_dtype={None: None, _BF: torch.bfloat16, "i8": torch.int8}[st["h"]])
    out = [] if r is None else [r]
    if st["h"] == "i8":
        out += [_values(*h), h[1]]
    elif h is not None:
        out.append(h)
    return out


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_norm(v, kind, eps):
    if kind == "layer":
        var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
        return (v - mean) / (var + eps).sqrt()
    return v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + eps).sqrt()


def _exact_codes(v):
    step = v.abs().amax(-1, keepdim=True) / 127
    return (v / step).round() * step, step.squeeze(-1)


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = st["op"], torch.float64
    if op == "linear":
        out = torch.mm(st["xq"].to(f64), st["wq"].to(f64).t()) * torch.outer(st["xs"].to(f64), st["ws"].to(f64))
        for more in (st["bias"], st["addend"]):
            if more is not None:
                out = out + more.to(f64)
        return out
    if op == "quant":
        x = st["x"].to(f64)
        amax = x.abs().amax(-1, keepdim=True)
        return (127 * x / amax).round() * amax / 127, amax.squeeze(-1) / 127
    if op == "gate":
        y, z = st["y"].to(f64), st["z"].to(f64)
        v = torch.stack([_exact_norm(part, "rms", st["eps"]) for part in (y * z * torch.sigmoid(z)).split(st["group"], 1)],
                        1).flatten(1)
        return _exact_codes(v * st["w"].to(f64))
    x, out = st["x"].to(f64), []
    if st["y"] is not None:
        y = st["y"].to(f64)
        if st["post"]:
            y = _exact_norm(y, st["kind"], st["eps"]) * st["w_post"].to(f64)
        x = x * st["alpha"] + y * st["gate"].to(f64).unsqueeze(1)
        out.append(x)
    if st["h"] is not None:
        h = _exact_norm(x, st["kind"], st["eps"])
        h = h * ((st["scale"].to(f64) + 1) * st["w_pre"].to(f64)).unsqueeze(1) + st["shift"].to(f64).unsqueeze(1)
        out += list(_exact_codes(h)) if st["h"] == "i8" else [h]
    return out


# ------------------------------------------------------------------ what no form can do without
def work(case):
    c, op = case, case["op"]
    if op == "linear":
        M, K, N, e = c["M"], c["K"], c["N"], 4 if c["out"] == _F32 else 2
        return {"bytes": M * K + N * K + 4 * (M + N) + (4 * N if c["bias"] else 0) + M * N * e * (2 if c["addend"] else 1),
                "flops": 2 * M * N * K}
    if op == "quant":
        M, K = c["M"], c["K"]
        return {"bytes": 3 * M * K + 4 * M, "flops": 4 * M * K}
    if op == "gate":
        M, C = c["M"], c["C"]
        return {"bytes": 5 * M * C + 4 * M + 4 * C, "flops": 16 * M * C}
    B, C = c["B"], c["C"]
    M, e = B * c["n"], 4 if c["x"] == _F32 else 2
    n = e * M * C + (M * C * (2 + e) + 4 * (B + c["post"]) * C if c["y"] else 0)
    if c["h"] is not None:
        n += 4 * (1 + 2 * B) * C + (M * C + 4 * M if c["h"] == "i8" else 2 * M * C)
    return {"bytes": n, "flops": (8 if c["y"] else 0) * M * C + (12 if c["h"] else 0) * M * C}
