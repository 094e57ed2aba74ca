"""The transformer block's operators around the attention: what they compute, on which sizes, and how a user calls them.

Three operators of the video DiT block that surround the block-sparse attention:

  norm    residual_norm: the gated residual of a block's output (with an optional norm of that output) and the
          adaptively modulated norm that feeds the next block, in one pass over the residual stream;
  linear  token_quantize / residual_norm(quantize=True) and int8_linear: the block's projections as products of 8-bit
          integers with one scale a token and one a channel, with bias, activation, gate and residual;
  rotary  rotary: rotary positions, interleaved or half layout, part of the head, several axes, scaled for longer clips.

`run` computes each in elementary torch operations (`own` false) or by the framework's calls (`own` true).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the norm of the "tiny" workload's tokens (2 heads of 64 channels): a launch-bound call
        dict(name="norm_tiny", op="norm", B=1, N=1024, C=128, G=1, x="bf16", y="", norm="layer", post="", weight=False,
             gate=False, modulate=True, indexed=False, ragged=False, params="fp32"),
        # one rank's rows of a sequence-sharded step, its tokens of two noise levels (modulation chosen by index)
        dict(name="norm_indexed", op="norm", B=1, N=4722, C=5376, G=2, x="bf16", y="bf16", norm="rms", post="",
             weight=True, gate=True, modulate=True, indexed=True, ragged=False, params="bf16"),
        # the long clip's ragged batch of two, a norm after and before the block, residual stream kept in fp32
        dict(name="norm_sandwich_long", op="norm", B=2, N=53824, C=4096, G=2, x="fp32", y="bf16", norm="rms", post="rms",
             weight=True, gate=True, modulate=False, indexed=False, ragged=True, params="fp32"),
        # the 720p workload's tokens between attention and feed-forward
        dict(name="norm_720p", op="norm", B=1, N=75600, C=5120, G=1, x="bf16", y="bf16", norm="layer", post="",
             weight=False, gate=True, modulate=True, indexed=False, ragged=False, params="fp32"),
        # the six modulation vectors of a block from two samples' conditioning vectors: single tokens, weight-bound
        dict(name="linear_modulation", op="linear", feed="tokens", B=1, N=2, K=4096, M=24576, H=0, x="bf16", out="fp32",
             bias=True, act="", gate=False, residual=False),
        # key projection of a few hundred conditioning tokens, an odd count
        dict(name="linear_context", op="linear", feed="tokens", B=1, N=333, K=4096, M=5120, H=0, x="fp16", out="fp16",
             bias=True, act="", gate=False, residual=False),
        # one rank's feed-forward down projection, gated onto the residual stream
        dict(name="linear_down_rank", op="linear", feed="tokens", B=1, N=4722, K=21504, M=5376, H=0, x="bf16",
             out="bf16", bias=True, act="", gate=True, residual=True),
        # 720p: modulated norm, then the query projection straight into the attention's head layout
        dict(name="linear_norm_heads_720p", op="linear", feed="norm", B=1, N=75648, K=5120, M=5120, H=40, x="bf16",
             out="bf16", bias=True, act="", gate=False, residual=False),
        # 480p token count: feed-forward up projection with its GELU
        dict(name="linear_up_gelu_480p", op="linear", feed="tokens", B=1, N=32760, K=5120, M=20480, H=0, x="bf16",
             out="bf16", bias=True, act="gelu_tanh", gate=False, residual=False),
        # long clip: the attention's output from its head layout through the output projection, gated onto the residual
        dict(name="linear_heads_out_long", op="linear", feed="heads", B=2, N=53824, K=4096, M=4096, H=32, x="bf16",
             out="bf16", bias=False, act="", gate=True, residual=True),
        # the "tiny" workload's queries, half layout in fp32
        dict(name="rotary_tiny", op="rotary", B=1, H=2, N=1024, D=64, rope=64, axes=1, layout="half", order="heads",
             x="fp32", scaling="", factor=1.0, first=0, inverse=False),
        # 720p queries: three axes on 96 of 128 channels, adjacent pairs
        dict(name="rotary_720p", op="rotary", B=1, H=40, N=75648, D=128, rope=96, axes=3, layout="interleaved",
             order="heads", x="bf16", scaling="", factor=1.0, first=0, inverse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "rotary"])
    if op == "norm":
        x, y = rng.choice([("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "")])
        C = _log(rng, 64, 8192)
        C = C if rng.random() < 0.4 else -(-C // 64) * 64
        B = rng.randint(1, 3)
        N = _log(rng, 1, max(1, min(75600, 380_000_000 // (B * C))))
        indexed = rng.random() < 0.3
        return dict(op="norm", B=B, N=N, C=C, G=rng.randint(1, 4) if indexed else B, x=x, y=y,
                    norm=rng.choice(["layer", "rms"]), post=rng.choice(["", "", "layer", "rms"]) if y else "",
                    weight=rng.random() < 0.5, gate=bool(y) and rng.random() < 0.8, modulate=rng.random() < 0.7,
                    indexed=indexed, ragged=rng.random() < 0.4, params="fp32" if rng.random() < 0.6 else (y or x))
    if op == "linear":
        feed = rng.choice(["tokens", "tokens", "norm", "heads"])
        H = 0
        if feed == "heads":
            H = _log(rng, 2, 40)
            K = 128 * H
        else:
            K = _log(rng, 64, 20480)
        M = _log(rng, 32, 20480)
        if feed == "norm":
            H = _log(rng, 1, 40)
            M = 128 * H
        B = rng.randint(1, 2)
        top = min(75600 // B, int(3.3e12 / (K * M)) // B, int(1.5e9 / max(K, M)) // B)
        N = _log(rng, 1, max(1, top))
        x = rng.choice(["bf16", "bf16", "fp16"])
        plain = feed != "norm"
        return dict(op="linear", feed=feed, B=B, N=N, K=K, M=M, H=H, x=x, out=x, bias=rng.random() < 0.7,
                    act=rng.choice(["", "gelu_tanh", "silu"]) if plain else "", gate=plain and rng.random() < 0.4,
                    residual=plain and rng.random() < 0.5)
    D = rng.choice([64, 128])
    axes = rng.choice([1, 1, 3])
    rope = rng.choice([D, D // 2]) if axes == 1 else rng.choice([48, 60])
    H = _log(rng, 1, 40)
    B = rng.randint(1, 2)
    N = _log(rng, 1, max(1, min(131072, 380_000_000 // (B * H * D))))
    return dict(op="rotary", B=B, H=H, N=N, D=D, rope=rope, axes=axes, layout=rng.choice(["interleaved", "half"]),
                order=rng.choice(["heads", "tokens"]), x=rng.choice(["bf16", "fp16", "fp32"]),
                scaling=rng.choice(["", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0]),
                first=rng.choice([0, 1000, 1_000_000]), inverse=rng.random() < 0.3)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _stream(g, *shape, dtype):
    """A residual stream: channels of unequal spread and offset, as they stand between blocks."""
    C = shape[-1]
    spread = torch.exp(0.5 * torch.randn(C, generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * spread
            + 0.3 * torch.randn(C, generator=g, device="cuda")).to(dtype)


def _pad16(n):
    return -(-n // 16) * 16


def _table_plan(case):
    """The framework's frequency table, as a user's program keeps it."""
    import video_dit_block_b200 as sba
    return sba.rope_frequencies(case["rope"], axes=case["axes"], base=10000.0, scaling=case["scaling"] or None,
                                factor=case["factor"], original_length=4096)


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rotary":  # each side's frequency table, made once by a user's program
        s["t_freq"], s["t_axis"], s["amp"] = _frequencies(case, "cuda")
        s["table"] = _table_plan(case) if own else None
    return s


def _inputs(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["x"]]
    s = dict(case)
    if case["op"] == "norm":
        B, N, C, G = (case[k] for k in "BNCG")
        s["t_x"] = _stream(g, B, N, C, dtype=dt)
        pt = DTYPES[case["params"]]
        s["t_y"] = _randn(g, B, N, C, dtype=DTYPES[case["y"]]) if case["y"] else None
        s["t_gate"] = _randn(g, G, C, dtype=pt, std=0.5) if case["gate"] else None
        s["t_scale"] = _randn(g, G, C, dtype=pt, std=0.3) if case["modulate"] else None
        s["t_shift"] = _randn(g, G, C, dtype=pt, std=0.3) if case["modulate"] else None
        s["t_weight"] = (1 + _randn(g, C, std=0.2)).to(pt) if case["weight"] else None
        s["t_bias"] = _randn(g, C, dtype=pt, std=0.1) if case["weight"] and case["norm"] == "layer" else None
        s["t_post"] = (1 + _randn(g, C, std=0.2)).to(pt) if case["post"] else None
        s["t_index"] = (torch.randint(0, G, (B, N), generator=g, device="cuda", dtype=torch.int32)
                        if case["indexed"] else None)
        s["t_len"] = None
        if case["ragged"]:
            s["t_len"] = torch.randint(max(1, N - max(1, N // 400)), N + 1, (B,), generator=g, device="cuda",
                                       dtype=torch.int32)
        return s
    if case["op"] == "linear":
        B, N, K, M, H = (case[k] for k in "BNKMH")
        if case["feed"] == "heads":
            s["t_x"] = _randn(g, B, H, N, K // H, dtype=dt)
        else:
            s["t_x"] = _stream(g, B, N, K, dtype=dt)
        w = _randn(g, M, K, std=K ** -0.5)
        s["t_ws"] = w.abs().amax(1) / 127
        s["t_w"] = torch.zeros(M, _pad16(K), dtype=torch.int8, device="cuda")
        s["t_w"][:, :K] = torch.round(w / s["t_ws"][:, None]).to(torch.int8)
        s["t_bias"] = _randn(g, M, std=0.1) if case["bias"] else None
        s["t_gate"] = _randn(g, B, M, std=0.5) if case["gate"] else None
        s["t_res"] = _stream(g, B, N, M, dtype=DTYPES[case["out"]]) if case["residual"] else None
        if case["feed"] == "norm":
            s["t_scale"], s["t_shift"] = _randn(g, B, K, std=0.3), _randn(g, B, K, std=0.3)
        return s
    B, H, N, D, A = (case[k] for k in ("B", "H", "N", "D", "axes"))
    x = _randn(g, B, N, H, D, dtype=dt) if case["order"] == "tokens" else _randn(g, B, H, N, D, dtype=dt)
    s["t_x"] = x.transpose(1, 2) if case["order"] == "tokens" else x
    n = torch.arange(N, device="cuda", dtype=torch.int32)
    if A == 1:
        p = (n + case["first"])[:, None]
    else:  # a lattice of 45 x 80 tokens a frame, in raster order
        p = torch.stack([n // 3600 + case["first"], n // 80 % 45, n % 80], 1)
    s["t_pos"] = p[None].repeat(B, 1, 1).contiguous()
    return s


# ---------------------------------------------------------------- plain forms

def _normed(v, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _rows(t, s):
    """A [G, C] parameter as it meets the rows of [B, N, C]."""
    return t.float()[s["t_index"].long()] if s["t_index"] is not None else t.float()[:, None, :]


def _plain_norm(s):
    x, y = s["t_x"].float(), s["t_y"]
    if y is not None:
        z = y.float()
        if s["post"]:
            z = _normed(z, s["post"]) * s["t_post"].float()
        if s["gate"]:
            z = z * _rows(s["t_gate"], s)
        x = x + z
    h = _normed(x, s["norm"])
    if s["t_weight"] is not None:
        h = h * s["t_weight"].float()
    if s["t_bias"] is not None:
        h = h + s["t_bias"].float()
    if s["modulate"]:
        h = h * (1 + _rows(s["t_scale"], s)) + _rows(s["t_shift"], s)
    if s["t_len"] is not None:
        live = torch.arange(s["N"], device="cuda") < s["t_len"][:, None]
        h = torch.where(live[:, :, None], h, 0.0)
        x = torch.where(live[:, :, None], x, 0.0) if y is not None else x
    out = {"h": h.to(DTYPES[s["y"] or s["x"]])}
    if y is not None:
        out["x"] = x.to(DTYPES[s["x"]])
    return out


def _codes(v):
    """[.., K] fp32 -> codes as fp32 whole numbers, and the scale a token."""
    top = v.abs().amax(-1, keepdim=True)
    inv = torch.where(top > 0, 127.0 / top, 0.0)
    return torch.round(v * inv), top / 127.0


def _plain_linear(s):
    x = s["t_x"].float()
    if s["feed"] == "heads":
        x = x.transpose(1, 2).reshape(s["B"], s["N"], s["K"])
    elif s["feed"] == "norm":
        x = _normed(x, "layer") * (1 + s["t_scale"][:, None]) + s["t_shift"][:, None]
    a, sa = _codes(x)
    v = torch.matmul(a, s["t_w"][:, :s["K"]].float().t()) * sa * s["t_ws"]
    if s["bias"]:
        v = v + s["t_bias"]
    if s["act"] == "gelu_tanh":
        v = 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    elif s["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    if s["gate"]:
        v = v * s["t_gate"][:, None]
    if s["residual"]:
        v = v + s["t_res"].float()
    v = v.to(DTYPES[s["out"]])
    if s["feed"] == "norm":
        v = v.view(s["B"], s["N"], s["H"], -1).transpose(1, 2).contiguous()
    return v


def _frequencies(case, device):
    """Radians a position of each pair, in 64 bits; the axis of each; the factor on the result."""
    A, da = case["axes"], case["rope"] // case["axes"]
    i = torch.arange(da // 2, dtype=torch.float64, device=device)
    base, f, scale = 10000.0, case["factor"], 1.0
    if case["scaling"] == "ntk":
        base = base * f ** (da / (da - 2))
    freq = base ** (-2 * i / da)
    if case["scaling"] == "linear":
        freq = freq / f
    elif case["scaling"] == "yarn":
        lo, hi = (da * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), da - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        freq = freq / f * (1 - keep) + freq * keep
        scale = 0.1 * math.log(f) + 1
    return freq.repeat(A), torch.arange(A, device=device).repeat_interleave(da // 2), scale


def _plain_rotary(s):
    x = s["t_x"].float()
    angle = s["t_pos"].double()[:, :, s["t_axis"]] * s["t_freq"]  # far positions: 64 bits
    c, sn = (torch.cos(angle) * s["amp"]).float()[:, None], (torch.sin(angle) * s["amp"]).float()[:, None]
    if s["inverse"]:
        sn = -sn
    r = s["rope"]
    out = x.clone()
    if s["layout"] == "half":
        u, v = x[..., :r // 2], x[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = u * c - v * sn, u * sn + v * c
    else:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = u * c - v * sn, u * sn + v * c
    return out.to(DTYPES[s["x"]])


# ---------------------------------------------------------------- the framework's calls

def _own_norm(s):
    import video_dit_block_b200 as sba
    x, h = sba.residual_norm(s["t_x"], s["t_y"], gate=s["t_gate"], post_norm=s["post"] or None, post_weight=s["t_post"],
                             norm=s["norm"], weight=s["t_weight"], bias=s["t_bias"], scale=s["t_scale"],
                             shift=s["t_shift"], index=s["t_index"], valid_len=s["t_len"], eps=EPS)
    return {"h": h, "x": x} if s["t_y"] is not None else {"h": h}


def _own_linear(s):
    import video_dit_block_b200 as sba
    if s["feed"] == "norm":
        _, a, sa = sba.residual_norm(s["t_x"], norm="layer", scale=s["t_scale"], shift=s["t_shift"], eps=EPS,
                                     quantize=True)
    else:
        a, sa = sba.token_quantize(s["t_x"])
    return sba.int8_linear(a, sa, s["t_w"], s["t_ws"], bias=s["t_bias"], activation=s["act"] or None, gate=s["t_gate"],
                           residual=s["t_res"], out_dtype=DTYPES[s["out"]],
                           heads=s["H"] if s["feed"] == "norm" else None)


def _own_rotary(s):
    import video_dit_block_b200 as sba
    return sba.rotary(s["t_x"], s["t_pos"], s["table"], layout=s["layout"], inverse=s["inverse"])


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "rotary": _own_rotary}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "rotary": _plain_rotary}[op](state)


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "": 0}
    if case["op"] == "norm":
        n = case["B"] * case["N"] * case["C"]
        xs, ys = size[case["x"]], size[case["y"]]
        both = n * (2 * xs + 2 * ys) if ys else n * 2 * xs
        params = size[case["params"]] * case["C"] * (
            case["G"] * (case["gate"] + 2 * case["modulate"]) + 2 * case["weight"] + bool(case["post"]))
        return {"bytes": both + params + 4 * case["B"] * case["N"] * case["indexed"], "flops": 12 * n}
    if case["op"] == "linear":
        rows, K, M = case["B"] * case["N"], case["K"], case["M"]
        b = rows * K * size[case["x"]] + K * M + 4 * M + rows * M * size[case["out"]] * (1 + case["residual"])
        b += 4 * M * case["bias"] + 4 * case["B"] * M * case["gate"] + 8 * case["B"] * K * (case["feed"] == "norm")
        return {"bytes": b, "flops": 2 * rows * K * M}
    n = case["B"] * case["H"] * case["N"] * case["D"]
    return {"bytes": 2 * n * size[case["x"]] + 4 * case["B"] * case["N"] * case["axes"], "flops": 3 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s):
    """Sample by sample, row statistics through sums of the values and of their squared distances."""
    hs, xs = [], []
    for b in range(s["B"]):
        n = s["N"] if s["t_len"] is None else int(s["t_len"][b])
        row = (lambda t: t.double()[s["t_index"][b, :n].long()]) if s["t_index"] is not None else (
            lambda t: t.double()[b].expand(n, -1))
        stat = lambda v, kind: ((v - v.sum(1, True) / s["C"]) if kind == "layer" else v)  # noqa: E731
        r = s["t_x"][b, :n].double()
        if s["t_y"] is not None:
            z = s["t_y"][b, :n].double()
            if s["post"]:
                z = stat(z, s["post"])
                z = z / torch.sqrt(z.pow(2).sum(1, True) / s["C"] + EPS) * s["t_post"].double()
            r = torch.addcmul(r, row(s["t_gate"]), z) if s["gate"] else r + z
        h = stat(r, s["norm"])
        h = h / torch.sqrt(h.pow(2).sum(1, True) / s["C"] + EPS)
        if s["t_weight"] is not None:
            h = h * s["t_weight"].double()
        if s["t_bias"] is not None:
            h = h + s["t_bias"].double()
        if s["modulate"]:
            h = h + h * row(s["t_scale"]) + row(s["t_shift"])
        hs.append(torch.nn.functional.pad(h, (0, 0, 0, s["N"] - n)))
        if s["t_y"] is not None:
            xs.append(torch.nn.functional.pad(r, (0, 0, 0, s["N"] - n)))
    return {"h": torch.stack(hs), "x": torch.stack(xs)} if xs else {"h": torch.stack(hs)}


def _exact_linear(s):
    """codes = the nearest whole numbers to fp32(x * fp32(127 / max|x|)), ties to even, as the operator defines them."""
    outs = []
    for b in range(s["B"]):
        x = s["t_x"][b].double()
        if s["feed"] == "heads":
            x = x.permute(1, 0, 2).reshape(s["N"], s["K"])
        elif s["feed"] == "norm":
            x = x - x.sum(1, True) / s["K"]
            x = x / torch.sqrt(x.pow(2).sum(1, True) / s["K"] + EPS)
            x = x + x * s["t_scale"][b].double() + s["t_shift"][b].double()
        top = x.abs().amax(1, True)
        inv = torch.where(top > 0, 127 / top, top).float().double()
        a = (x * inv).float().double().round()
        v = (a @ s["t_w"][:, :s["K"]].double().t()) * (top / 127) * s["t_ws"].double()
        if s["bias"]:
            v += s["t_bias"].double()
        if s["act"] == "gelu_tanh":
            v *= torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        elif s["act"] == "silu":
            v *= torch.sigmoid(v)
        if s["gate"]:
            v *= s["t_gate"][b].double()
        if s["residual"]:
            v += s["t_res"][b].double()
        if s["feed"] == "norm":
            v = v.view(s["N"], s["H"], -1).permute(1, 0, 2)
        outs.append(v)
    return torch.stack(outs)


def _exact_rotary(s):
    """Each pair as a complex number times e^(i angle), head by head."""
    r, A = s["rope"], s["axes"]
    da = r // A
    freq, scale = [], 1.0
    for i in range(da // 2):
        w = 10000.0 ** (-2 * i / da)
        if s["scaling"] == "linear":
            w /= s["factor"]
        elif s["scaling"] == "ntk":
            w = (10000.0 * s["factor"] ** (da / (da - 2))) ** (-2 * i / da)
        elif s["scaling"] == "yarn":
            at = lambda turns: da * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
            lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), da - 1)
            part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / s["factor"] * part + w * (1 - part)
            scale = 0.1 * math.log(s["factor"]) + 1
        freq.append(w)
    sign = -1.0 if s["inverse"] else 1.0
    pos = s["t_pos"].double()
    theta = torch.cat([pos[:, :, a, None] * torch.tensor(freq, dtype=torch.float64, device=pos.device)
                       for a in range(A)], -1)
    turn = torch.polar(torch.full_like(theta, scale), sign * theta)
    out = s["t_x"].double()
    out = out.clone(memory_format=torch.contiguous_format)
    for h in range(s["H"]):
        v = out[:, h]
        pair = (v[..., 0:r:2], v[..., 1:r:2]) if s["layout"] == "interleaved" else (v[..., :r // 2], v[..., r // 2:r])
        z = torch.complex(pair[0].contiguous(), pair[1].contiguous()) * turn
        pair[0].copy_(z.real)
        pair[1].copy_(z.imag)
    return out


def exact(case, seed):
    return {"norm": _exact_norm, "linear": _exact_linear, "rotary": _exact_rotary}[case["op"]](_inputs(case, seed))
