"""The block's operators -- residual_norm, token_quantize, int8_linear, rotary -- against
their formulas in 64 bits.

Tolerances.  u = 2^-24 is a rounding in fp32; a result of type t is rounded once more, by at
most eps(t) / 2 of itself (or half the smallest step of fp16's subnormals, 2^-25).

  rotary    sin and cos are off by at most pi u (the angle's conversion to fp32) + 2^-30 (its
            dropped bits) + 2 units in the last place + 1 rounding of the amplitude, together
            below 8 u; each product and sum adds u: |error| <= 11 u amp (|u| + |v|).
  norm      a sum over a row is at most d = 90 additions deep (64 in a thread, 5 across a warp,
            16 warps).  The mean is off by d u mean|r|; the squares' mean by (d + 3) u relatively,
            its root by half of that and 3 roundings; r by 2 u of its terms, and by a post
            norm's error, bounded the same way.  With S = |w (1 + scale)| inv max_row(|x| + |g z|)
            + |b (1 + scale)| + |shift| as the size of the terms, all of it is below
            4 (d + 10) u S = 400 u S.
  linear    the sum is exact; its conversion, the scales' product, the product and the bias
            are 4 roundings: 4 u (|acc sa sw| + |bias|).  The activations' slopes are below
            1.13; their own error is at most (2 + 1.16 |t|) 2^-23 (exponential) + 3 |t| u (its
            argument) + 2^-22 (division) + 2 u of the result.  Gate and residual: one rounding
            each.
"""
import math
import zlib

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def sba():
    import video_dit_block_b200 as m
    return m


@pytest.fixture(autouse=True)
def clean_status(sba):
    yield
    assert sba.device_status() == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=SF, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def rounding(ref, dtype):
    """Half a step of `dtype` at each value of ref (fp32 results carry u in their own bounds)."""
    if dtype == SF:
        return torch.zeros_like(ref)
    return ref.abs() * torch.finfo(dtype).eps / 2 + (2.0 ** -25 if dtype == HF else 0.0)


def close(got, ref, tol, dtype):
    """|got - ref| <= tol, then a rounding of the value the kernel had."""
    bound = tol + rounding(ref.abs() + tol, dtype)
    err = (got.double() - ref).abs()
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, f"error {err.max().item():.3e}, {worst:.3e} over its bound"


# ------------------------------------------------------------------------------ rotary

def rotary_ref(x, pos, table, layout, inverse):
    """In 64 bits, the angles taken modulo a turn in 80-bit arithmetic."""
    B, H, N, D = x.shape
    r = table.rope_dim
    p = pos.cpu().numpy().reshape(B, N, -1)[:, :, list(table.axis)].astype(np.longdouble)
    turns = p * np.array(table.inv_freq, dtype=np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    turns -= np.rint(turns)
    th = torch.from_numpy((2 * np.pi * turns.astype(np.float64))).to(x.device)[:, None]
    c, s = torch.cos(th) * table.amplitude, torch.sin(th) * table.amplitude * (-1 if inverse else 1)
    out = x.double().clone(memory_format=torch.contiguous_format)
    tol = torch.zeros_like(out)
    a, b = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2)))
    u, v = x.double()[..., a], x.double()[..., b]
    out[..., a], out[..., b] = u * c - v * s, u * s + v * c
    tol[..., a] = tol[..., b] = 11 * U * table.amplitude * (u.abs() + v.abs())
    return out, tol


ROTARY = [
    # B, H, N, D, rope_dim, axes, layout, type, first position
    (1, 2, 1, 64, 64, 1, "half", BF, 0),
    (1, 1, 1, 2, 2, 1, "interleaved", SF, 5),
    (2, 3, 257, 128, 96, 3, "interleaved", BF, 0),
    (2, 3, 257, 128, 96, 3, "half", HF, 0),
    (1, 9, 130, 128, 128, 1, "half", SF, 2 ** 31 - 200),
    (1, 8, 65, 128, 128, 1, "interleaved", SF, -2 ** 31),
    (1, 17, 33, 64, 32, 1, "half", HF, 1_000_000),
    (1, 5, 77, 80, 60, 3, "interleaved", BF, 0),     # pairs that are no multiple of 8
    (1, 5, 77, 80, 60, 3, "half", SF, 0),
    (3, 2, 50, 75, 30, 1, "half", BF, 7),            # odd head dimension
    (3, 2, 50, 75, 30, 1, "interleaved", HF, 7),
    (1, 2, 40, 256, 256, 1, "half", BF, 100),
    (1, 1, 3, 1024, 256, 2, "interleaved", BF, 100),
]


@pytest.mark.parametrize("order", ["heads", "tokens", "slice"])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary(sba, case, order):
    B, H, N, D, rope, axes, layout, dt, first = case
    g = gen(zlib.crc32(str(case).encode()))
    if order == "heads":
        x = randn(g, B, H, N, D, dtype=dt)
    elif order == "tokens":
        x = randn(g, B, N, H, D, dtype=dt).transpose(1, 2)
    else:  # queries of a packed projection, rows at an odd offset
        x = randn(g, B, N, 3 * H * D + 1, dtype=dt)[:, :, 1 + H * D:1 + 2 * H * D].unflatten(2, (H, D)).transpose(1, 2)
    pos = torch.randint(0, 300, (B, N, axes), generator=g, device=DEV) + torch.arange(N, device=DEV)[:, None] + first
    pos = pos.clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32)
    table = sba.rope_frequencies(rope, axes=axes)
    out = sba.rotary(x, pos, table, layout=layout)
    ref, tol = rotary_ref(x, pos, table, layout, False)
    close(out, ref, tol, dt)
    back = sba.rotary(x, pos, table, layout=layout, inverse=True)
    ref, tol = rotary_ref(x, pos, table, layout, True)
    close(back, ref, tol, dt)


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_scaled(sba, scaling, layout):
    g = gen(5)
    x = randn(g, 1, 4, 200, 128)
    pos = (torch.arange(200, device=DEV) * 997).to(torch.int32)[None]
    table = sba.rope_frequencies(128, scaling=scaling, factor=8.0, original_length=2048)
    ref, tol = rotary_ref(x, pos, table, layout, False)
    close(sba.rotary(x, pos, table, layout=layout), ref, tol, SF)


@pytest.mark.parametrize("rope,dt", [(96, BF), (128, HF), (30, SF)])
def test_rotary_in_place_and_gaps(sba, rope, dt):
    """In place, and into a strided output whose other elements stay as they were."""
    g = gen(6)
    x = randn(g, 2, 3, 70, 128, dtype=dt)
    pos = torch.randint(0, 5000, (2, 70), generator=g, device=DEV, dtype=torch.int32)
    table = sba.rope_frequencies(rope)
    want = sba.rotary(x, pos, table)
    wide = torch.full((2, 3, 70, 160), 7.0, dtype=dt, device=DEV)
    sba.rotary(x, pos, table, out=wide[..., 16:144])
    assert torch.equal(wide[..., 16:144], want)
    assert (wide[..., :16] == 7).all() and (wide[..., 144:] == 7).all()
    y = x.clone()
    assert sba.rotary(y, pos, table, out=y) is y
    assert torch.equal(y, want)


def test_rotary_inverse_is_the_gradient(sba):
    """<rotary(x), g> = <x, inverse(g)>, and differences of the loss along a direction."""
    g = gen(7)
    x, go, d = (randn(g, 1, 2, 64, 128) for _ in range(3))
    pos = torch.randint(0, 5000, (1, 64, 3), generator=g, device=DEV, dtype=torch.int32)
    table = sba.rope_frequencies(96, axes=3)
    grad = sba.rotary(go, pos, table, inverse=True).double()
    loss = lambda t: (rotary_ref(t, pos, table, "interleaved", False)[0] * go.double()).sum()
    diff = (loss(x.double() + 1e-3 * d.double()) - loss(x.double() - 1e-3 * d.double())) / 2e-3
    size = (go.double().abs() * d.double().abs()).sum().item()
    # 11 u (|u| + |v|) each, |u| + |v| at most twice the larger; the loss is linear in x
    assert abs((grad * d.double()).sum().item() - diff.item()) <= 1e-5 * size


def test_rotary_agrees_with_the_producer_step(sba):
    """On values the producer's norm leaves as they are, its rotation and this one agree to a
    step of bf16."""
    g = gen(8)
    sign = torch.randint(0, 2, (1, 2, 128, 128), generator=g, device=DEV) * 2 - 1
    x = sign.to(BF)  # mean square 1: the norm divides by sqrt(1 + 1e-6), which rounds back
    pos = torch.randint(0, 80, (1, 128, 3), generator=g, device=DEV, dtype=torch.int32)
    a, _ = sba.qk_norm_rope_pool(x, torch.ones(128, dtype=BF, device=DEV), pos)
    b = sba.rotary(x, pos, sba.rope_frequencies(96, axes=3))
    assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs() + 2e-5).all()


# ------------------------------------------------------------------------------ norms

def norm_ref(x, y, gate, norm, weight, bias, scale, shift, index, post, post_weight, valid_len, eps):
    """(r, h, tolerance of r, tolerance of h) in 64 bits."""
    B, N, C = x.shape
    row = lambda t: t.double()[index.long()] if index is not None else t.double()[:B, None]
    stat = lambda v, k: v - v.mean(-1, keepdim=True) if k == "layer" else v
    inv = lambda v: torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)
    r = x.double()
    terms = r.abs()
    rtol = torch.zeros_like(r)
    if y is not None:
        z = y.double()
        if post:
            c = stat(z, post)
            i = inv(c)
            zs = i * z.abs().amax(-1, keepdim=True)
            z = c * i
            if post_weight is not None:
                z, zs = z * post_weight.double(), zs * post_weight.double().abs()
            zs = zs.expand_as(z)
        else:
            zs = z.abs()
        g = row(gate) if gate is not None else torch.ones_like(r)
        r = r + g * z
        rtol = (200 if post else 3) * U * (terms + (g * zs).abs())
        terms = terms + (g * zs).abs()
    h = tol = None
    if norm:
        c = stat(r, norm)
        i = inv(c)
        h, size = c * i, i * terms.amax(-1, keepdim=True)
        m = torch.ones_like(r)
        if weight is not None:
            m = m * weight.double()
        h, size = h * m, size * m.abs()
        if bias is not None:
            h, size = h + bias.double(), size + bias.double().abs()
        if scale is not None:
            h, size = h * (1 + row(scale)), size * (1 + row(scale).abs())
        if shift is not None:
            h, size = h + row(shift), size + row(shift).abs()
        tol = 400 * U * size
    if valid_len is not None:
        dead = (torch.arange(N, device=x.device) >= valid_len[:, None])[:, :, None]
        if y is not None:
            r, rtol = r.masked_fill(dead, 0), rtol.masked_fill(dead, 0)
        if norm:
            h, tol = h.masked_fill(dead, 0), tol.masked_fill(dead, 0)
    return r, h, rtol, tol


def norm_inputs(g, B, N, C, xt, yt, pt, G, parts, offset=0.0):
    """`parts`: letters of what is given -- y, g(ate), w(eight), b(ias), m(odulation), i(ndex),
    p(ost weight)."""
    par = lambda *s, mean=0.0, std=0.4: (mean + randn(g, *s, std=std)).to(pt)
    spread = torch.exp(0.5 * torch.randn(C, generator=g, device=DEV))
    x = (randn(g, B, N, C) * spread + offset).to(xt)
    kw = dict(y=randn(g, B, N, C, dtype=yt) if "y" in parts else None)
    kw["gate"] = par(G, C) if "g" in parts else None
    kw["weight"] = par(C, mean=1.0) if "w" in parts else None
    kw["bias"] = par(C) if "b" in parts else None
    kw["scale"], kw["shift"] = (par(G, C), par(G, C)) if "m" in parts else (None, None)
    kw["index"] = torch.randint(0, G, (B, N), generator=g, device=DEV, dtype=torch.int32) if "i" in parts else None
    kw["post_weight"] = par(C, mean=1.0) if "p" in parts else None
    return x, kw


def check_norm(sba, x, kw, norm, post, valid_len=None, eps=1e-6):
    r, h = sba.residual_norm(x, norm=norm, post_norm=post, valid_len=valid_len, eps=eps, **kw)
    rr, hr, rt, ht = norm_ref(x, kw["y"], kw["gate"], norm, kw["weight"], kw["bias"], kw["scale"], kw["shift"],
                              kw["index"], post, kw["post_weight"], valid_len, eps)
    if kw["y"] is not None:
        assert r.dtype == x.dtype
        close(r, rr, rt, x.dtype)
    else:
        assert r is x
    if norm:
        close(h, hr, ht, h.dtype)
    return r, h


NORM = [
    # B, N, C, x, y, parameters, parts, norm, post
    (1, 1, 8, BF, BF, SF, "", "layer", None),
    (1, 1, 1, SF, SF, SF, "ygwbm", "rms", None),
    (2, 3, 7, BF, BF, BF, "ygwbm", "layer", None),
    (1, 33, 64, HF, HF, HF, "ygm", "rms", None),
    (2, 17, 128, BF, BF, SF, "ygm", "layer", None),
    (1, 9, 257, SF, SF, SF, "ygwm", "layer", "rms"),
    (2, 5, 512, SF, BF, SF, "ygwp", "rms", "rms"),
    (2, 5, 640, SF, HF, HF, "ygwbmp", "layer", "layer"),
    (1, 6, 1000, BF, BF, BF, "yw", "rms", "rms"),
    (1, 6, 1024, BF, BF, SF, "m", "layer", None),
    (3, 4, 1032, HF, HF, SF, "ygmi", "layer", None),
    (1, 5, 2048, BF, BF, SF, "ygmi", "rms", None),
    (1, 5, 2561, SF, BF, SF, "ygmi", "rms", "layer"),
    (2, 3, 4096, SF, BF, SF, "ygwp", "rms", "rms"),
    (1, 3, 4097, BF, BF, SF, "ygm", "layer", None),
    (1, 5, 5120, BF, BF, SF, "ygm", "layer", None),
    (1, 5, 5376, BF, BF, BF, "ygwmi", "rms", None),
    (1, 3, 6000, HF, HF, HF, "ywb", "layer", "rms"),
    (1, 3, 8192, SF, SF, SF, "ygm", "layer", None),
    (1, 2, 8200, BF, BF, SF, "ygm", "layer", None),
    (1, 2, 16384, BF, BF, SF, "yg", "rms", None),
    (1, 2, 20000, SF, BF, SF, "ygm", "layer", "rms"),
    (1, 2, 32768, SF, SF, SF, "ygwbm", "layer", "layer"),
    (1, 2, 32767, BF, BF, SF, "ygwbm", "layer", "layer"),
    (1, 9, 320, BF, BF, SF, "yg", None, None),
    (2, 9, 321, SF, HF, SF, "yp", None, "rms"),
]


@pytest.mark.parametrize("case", NORM)
def test_residual_norm(sba, case):
    B, N, C, xt, yt, pt, parts, norm, post = case
    g = gen(zlib.crc32(str(case).encode()))
    x, kw = norm_inputs(g, B, N, C, xt, yt, pt, 3 if "i" in parts else B, parts)
    check_norm(sba, x, kw, norm, post)


@pytest.mark.parametrize("C", [96, 1001, 5120])
@pytest.mark.parametrize("lens", [(0, 1), (5, 2), (40, 39)])
def test_residual_norm_ragged(sba, C, lens):
    """Padding rows come out as zeros whatever they hold, and are not read."""
    g = gen(11)
    x, kw = norm_inputs(g, 2, 40, C, BF, BF, SF, 2, "ygm")
    vl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    xn, kn = x.clone(), dict(kw, y=kw["y"].clone())
    r, h = check_norm(sba, x, kw, "layer", None, vl)
    for b in range(2):
        xn[b, lens[b]:], kn["y"][b, lens[b]:] = float("nan"), float("inf")
    r2, h2 = sba.residual_norm(xn, norm="layer", valid_len=vl, **kn)
    assert torch.equal(r, r2) and torch.equal(h, h2)
    _, codes, scales = sba.residual_norm(xn, norm="layer", valid_len=vl, quantize=True, **kn)
    for b in range(2):
        assert not codes[b, lens[b]:].any() and not scales[b, lens[b]:].any()


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("C", [100, 4096])
def test_residual_norm_hard_rows(sba, C, norm):
    """Constant rows, zero rows, a large common offset, tiny and huge values."""
    g = gen(12)
    x = randn(g, 1, 6, C)
    x[0, 0] = 0
    x[0, 1] = 3.5
    x[0, 2] += 3000.0
    x[0, 3] *= 1e-12
    x[0, 4] *= 1e15
    kw = dict(y=None, gate=None, weight=None, bias=None, scale=None, shift=None, index=None, post_weight=None)
    # a constant row's distances from its mean are the mean's own rounding, which eps outweighs
    check_norm(sba, x, kw, norm, None, eps=1e-5)


def test_residual_norm_strides_and_in_place(sba):
    g = gen(13)
    B, N, C = 2, 19, 256
    wide = randn(g, B, N + 3, 2 * C + 8, dtype=BF)
    x, y = wide[:, 2:N + 2, 8:C + 8], wide[:, 1:N + 1, C + 8:]
    gate = randn(g, B, C)
    r0, h0 = sba.residual_norm(x.contiguous(), y.contiguous(), gate=gate)
    r, h = sba.residual_norm(x, y, gate=gate)
    assert torch.equal(r, r0) and torch.equal(h, h0)
    # one row for all tokens, by a stride of 0
    r, h = sba.residual_norm(x[:, :1].expand(B, N, C), y, gate=gate)
    r1, h1 = sba.residual_norm(x[:, :1].expand(B, N, C).contiguous(), y.contiguous(), gate=gate)
    assert torch.equal(r, r1) and torch.equal(h, h1)
    # at an odd element offset (single-element accesses)
    odd = torch.empty(B * N * C + 1, dtype=BF, device=DEV)[1:].view(B, N, C)
    odd.copy_(x)
    r, h = sba.residual_norm(odd, y, gate=gate)
    close(r, r0.double(), 3 * U * (x.double().abs() + y.double().abs() * gate.double()[:, None].abs()), BF)
    xi, yi = x.contiguous(), y.contiguous()
    r, h = sba.residual_norm(xi, yi, gate=gate, x_out=xi, out=yi)
    assert r is xi and h is yi and torch.equal(xi, r0) and torch.equal(yi, h0)
    out = torch.full((B, N + 4, C + 16), 5.0, dtype=BF, device=DEV)
    sba.residual_norm(x, y, gate=gate, out=out[:, :N, :C])
    assert torch.equal(out[:, :N, :C], h0) and (out[:, N:] == 5).all() and (out[:, :, C:] == 5).all()


def test_residual_norm_bad_index(sba):
    g = gen(14)
    x, kw = norm_inputs(g, 1, 6, 64, BF, BF, SF, 2, "ygmi")
    kw["index"][0, 2], kw["index"][0, 4] = 2, -1
    r, _ = sba.residual_norm(x, **kw)
    assert sba.device_status() == 6
    kw["index"] = kw["index"].clone()
    kw["index"][0, 2] = kw["index"][0, 4] = 0
    r0, _ = sba.residual_norm(x, **kw)
    assert torch.equal(r, r0)


# ------------------------------------------------------------------------------ quantised rows

def codes_ref(rows):
    """The definition on the host: fp32 steps, rounded to the nearest, ties to even."""
    v = rows.float().cpu().numpy().astype(np.float32)
    top = np.abs(v).max(-1, keepdims=True)
    live = top >= np.float32(2.0 ** -100)
    inv = np.where(live, np.float32(127) / np.where(live, top, np.float32(1)), np.float32(0)).astype(np.float32)
    scale = np.where(live, top / np.float32(127), np.float32(0)).astype(np.float32)[..., 0]
    return np.rint(v * inv).astype(np.int8), scale


@pytest.mark.parametrize("dt", [BF, HF, SF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 16), (5, 17), (3, 128), (2, 3, 1000), (7, 1024), (2, 3, 5120), (3, 8184),
                                   (2, 20480), (2, 32768), (1, 32761), (2, 3, 9, 64), (1, 5, 4, 75), (1, 1, 6, 128),
                                   (2, 40, 3, 128)])
def test_token_quantize(sba, shape, dt):
    g = gen(20)
    x = randn(g, *shape, dtype=dt)
    rows = x.transpose(1, 2).flatten(2) if x.dim() == 4 else x
    K = rows.shape[-1]
    codes, scales = sba.token_quantize(x)
    ref, sref = codes_ref(rows)
    assert codes.shape == (*rows.shape[:-1], -(-K // 16) * 16) and scales.shape == rows.shape[:-1]
    np.testing.assert_array_equal(codes[..., :K].cpu().numpy(), ref)
    np.testing.assert_array_equal(scales.cpu().numpy(), sref)
    assert not codes[..., K:].any()


def test_token_quantize_hard_rows(sba):
    g = gen(21)
    x = randn(g, 8, 333)
    x[0] = 0
    x[1] = -0.0
    x[2] *= 1e-30
    x[3] *= 1e-34          # below 2^-100: counts as zero
    x[4] *= 1e37
    x[5] = 1.0
    x[6] = torch.arange(333, device=DEV) % 255 - 127 + 0.5   # halves between codes
    x[6, 0] = 127.0
    codes, scales = sba.token_quantize(x)
    ref, sref = codes_ref(x)
    np.testing.assert_array_equal(codes[:, :333].cpu().numpy(), ref)
    np.testing.assert_array_equal(scales.cpu().numpy(), sref)
    assert not codes[3].any() and scales[3] == 0


@pytest.mark.parametrize("shape", [(7, 40), (7, 333), (7, 1024), (7, 5120), (7, 5121), (7, 20480), (2, 3, 5, 64)])
@pytest.mark.parametrize("dt", [BF, SF])
def test_token_quantize_shows_nan_and_infinities(sba, shape, dt):
    """They become the row's scale, and the other rows stay as they are."""
    g = gen(23)
    x = randn(g, *shape, dtype=dt)
    rows = x.transpose(1, 2).flatten(2).flatten(0, 1) if x.dim() == 4 else x
    ref, sref = codes_ref(rows)
    N = 5 if x.dim() == 4 else 7

    def put(i, c, v):
        if x.dim() == 4:
            x[i // N, c // 64, i % N, c % 64] = v
        else:
            x[i, c] = v

    K = rows.shape[1]
    put(1, K - 1, float("nan"))
    put(2, 0, float("inf"))
    put(3, K // 2, float("-inf"))
    put(5, 3, float("nan"))
    put(5, K // 2, float("inf"))
    codes, scales = sba.token_quantize(x)
    codes, scales = codes.flatten(0, -2), scales.flatten()
    assert scales[[1, 5]].isnan().all() and (scales[[2, 3]] == float("inf")).all()
    for i in (0, 4, 6):
        np.testing.assert_array_equal(codes[i, :K].cpu().numpy(), ref[i])
        assert scales[i].item() == sref[i]
    w, ws = sba.token_quantize(randn(g, 32, K))
    y = sba.int8_linear(codes, scales, w, ws)
    assert not y[[1, 2, 3, 5]].isfinite().any() and y[[0, 4, 6]].isfinite().all()


def test_token_quantize_strides(sba):
    g = gen(22)
    x = randn(g, 2, 5, 3, 3 * 64, dtype=BF)
    for v in (x[..., 64:128], x.transpose(1, 2), x[:, ::2], x[..., 1:65]):
        a, s = sba.token_quantize(v)
        b, t = sba.token_quantize(v.contiguous())
        assert torch.equal(a, b) and torch.equal(s, t)
    flat = randn(g, 9, 100, dtype=HF)[::2, 3:60]
    a, s = sba.token_quantize(flat)
    b, t = sba.token_quantize(flat.contiguous())
    assert torch.equal(a, b) and torch.equal(s, t)


@pytest.mark.parametrize("C", [64, 250, 1000, 4096, 5120, 5376])
def test_residual_norm_quantized(sba, C):
    """Codes are the nearest to h's own value within h's error; the scale is max|h| / 127."""
    g = gen(23)
    x, kw = norm_inputs(g, 2, 21, C, BF, BF, SF, 2, "ygm")
    r, codes, scales = sba.residual_norm(x, norm="layer", quantize=True, **kw)
    rr, h, rt, ht = norm_ref(x, kw["y"], kw["gate"], "layer", None, None, kw["scale"], kw["shift"], None, None, None,
                             None, 1e-6)
    close(r, rr, rt, BF)
    top, off = h.abs().amax(-1), ht.amax(-1)
    assert ((scales.double() * 127 - top).abs() <= off + 2 * U * top).all()
    step = (top / 127)[..., None]
    assert ((codes[..., :C].double() - h / step).abs() <= 0.5 + 3 * off[..., None] / step + 127 * 4 * U).all()
    assert not codes[..., C:].any()


# ------------------------------------------------------------------------------ int8 products

def linear_ref(a, sa, w, sw, bias, act, gate, index, residual):
    """(out, tolerance) in 64 bits; a [B, N, K]."""
    B = a.shape[0]
    acc = a.double() @ w.double().t()
    v = acc * sa.double()[..., None] * sw.double()
    tol = 4 * U * v.abs()
    if bias is not None:
        v, tol = v + bias.double(), tol + 4 * U * bias.double().abs()
    if act:
        t = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        f = v * torch.sigmoid(t)
        tol = 1.13 * tol + f.abs() * ((2 + 1.16 * t.abs()) * 2 * U + 3 * t.abs() * U + 6 * U)
        v = f
    if gate is not None:
        gr = gate.double()[index.long()] if index is not None else gate.double()[:B, None]
        v, tol = v * gr, (tol + U * v.abs()) * gr.abs()
    if residual is not None:
        v, tol = v + residual.double(), tol + U * (v.abs() + residual.double().abs())
    return v, tol + U * v.abs()


def linear_inputs(g, B, N, K, M):
    Kp = -(-K // 16) * 16
    a = torch.randint(-127, 128, (B, N, Kp), generator=g, device=DEV).to(torch.int8)
    w = torch.randint(-127, 128, (M, Kp), generator=g, device=DEV).to(torch.int8)
    sa = torch.rand(B, N, generator=g, device=DEV) * 0.01 + 1e-4
    sw = (torch.rand(M, generator=g, device=DEV) + 0.5) * 0.01 / math.sqrt(Kp)
    return a, sa, w, sw


LINEAR = [
    # B, N, K, M, out, parts (b(ias), g(ate), i(ndex), r(esidual)), activation, parameters
    (1, 1, 16, 1, SF, "", None, SF),
    (1, 1, 16, 8, BF, "b", None, BF),
    (1, 1, 4096, 6144, SF, "b", None, SF),
    (1, 2, 1000, 333, HF, "bgr", "silu", SF),
    (3, 1, 5120, 512, BF, "bgr", None, BF),
    (1, 7, 128, 64, BF, "", "gelu_tanh", SF),
    (1, 9, 144, 65, SF, "bgr", None, SF),
    (2, 60, 2000, 200, HF, "bgir", None, HF),
    (1, 127, 512, 320, BF, "r", None, SF),
    (1, 128, 272, 256, BF, "b", "silu", SF),
    (1, 129, 640, 130, SF, "bg", "gelu_tanh", SF),
    (1, 333, 4096, 1024, HF, "b", None, SF),
    (2, 300, 1024, 700, BF, "bgr", None, SF),
    (1, 1500, 384, 2304, BF, "b", "gelu_tanh", BF),     # many tiles of 256 x 256 from here on
    (1, 2049, 1040, 1536, BF, "bgr", None, SF),
    (3, 700, 512, 1400, HF, "bgir", "silu", HF),
    (1, 1537, 2064, 1601, SF, "bgr", None, SF),
    (1, 5000, 16, 1000, BF, "", None, SF),
]


@pytest.mark.parametrize("case", LINEAR)
def test_int8_linear(sba, case):
    B, N, K, M, ot, parts, act, pt = case
    g = gen(zlib.crc32(str(case).encode()))
    a, sa, w, sw = linear_inputs(g, B, N, K, M)
    G = 4 if "i" in parts else B
    bias = randn(g, M, dtype=pt, std=0.5) if "b" in parts else None
    gate = randn(g, G, M, dtype=pt) if "g" in parts else None
    index = torch.randint(0, G, (B, N), generator=g, device=DEV, dtype=torch.int32) if "i" in parts else None
    res = randn(g, B, N, M, dtype=ot) if "r" in parts else None
    out = sba.int8_linear(a, sa, w, sw, bias=bias, activation=act, gate=gate, index=index, residual=res, out_dtype=ot)
    ref, tol = linear_ref(a, sa, w, sw, bias, act, gate, index, res)
    assert out.shape == (B, N, M) and out.dtype == ot
    close(out, ref, tol, ot)
    if res is not None:  # onto the residual itself
        again = sba.int8_linear(a, sa, w, sw, bias=bias, activation=act, gate=gate, index=index, residual=res,
                                out_dtype=ot, out=res)
        assert again is res and torch.equal(res, out)


@pytest.mark.parametrize("N,K", [(3, 131056), (300, 131056), (2600, 16384)])
def test_int8_linear_sums_are_exact(sba, N, K):
    """Sums near the largest, and ones where single units decide: powers of two as scales keep
    every step exact that fp32 can hold."""
    M = 2560 if N > 1000 else 80
    a = torch.full((1, N, K), 127, dtype=torch.int8, device=DEV)
    w = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
    one_a, one_w = torch.ones(1, N, device=DEV), torch.ones(M, device=DEV)
    a[0, ::3] = -127
    out = sba.int8_linear(a, one_a, w, one_w, out_dtype=SF)
    want = torch.tensor(127 * 127 * K, dtype=torch.float64, device=DEV).float()
    assert (out[0, 1::3] == want).all() and (out[0, ::3] == -want).all()
    # cancelling halves leave what stands at one place
    a[:, :, 1::2] = -a[:, :, 0::2]
    a[0, :, 0] = torch.arange(N, device=DEV).remainder(127).to(torch.int8)
    a[0, :, 1] = 0
    out = sba.int8_linear(a, one_a, w, one_w, out_dtype=SF)
    assert torch.equal(out[0], (a[0, :, 0].float() * 127)[:, None].expand(N, M))


@pytest.mark.parametrize("B,N,K,H,D", [(1, 5, 256, 3, 64), (2, 130, 512, 4, 128), (2, 1000, 512, 10, 128),
                                       (1, 2048, 128, 24, 64), (1, 64, 128, 2, 32)])
def test_int8_linear_heads(sba, B, N, K, H, D):
    g = gen(31)
    a, sa, w, sw = linear_inputs(g, B, N, K, H * D)
    bias = randn(g, H * D)
    rows = sba.int8_linear(a, sa, w, sw, bias=bias)
    heads = sba.int8_linear(a, sa, w, sw, bias=bias, heads=H)
    assert heads.shape == (B, H, N, D) and heads.is_contiguous()
    assert torch.equal(heads, rows.view(B, N, H, D).transpose(1, 2))
    big = torch.full((B, H, N + 8, D), 3.0, dtype=BF, device=DEV)
    sba.int8_linear(a, sa, w, sw, bias=bias, heads=H, out=big[:, :, :N])
    assert torch.equal(big[:, :, :N], heads) and (big[:, :, N:] == 3).all()


def test_int8_linear_strided_out_and_rows(sba):
    g = gen(32)
    for N, M in ((11, 96), (900, 2560)):
        a, sa, w, sw = linear_inputs(g, 1, N, 256, M)
        res = randn(g, 1, N, M + 40, dtype=BF)
        want = sba.int8_linear(a, sa, w, sw, residual=res[..., 8:M + 8].contiguous())
        for off in (8, 3):
            r = torch.zeros_like(res)
            r[..., off:off + M] = res[..., 8:M + 8]
            out = torch.full((1, N + 2, M + 24), 9.0, dtype=BF, device=DEV)
            got = sba.int8_linear(a, sa, w, sw, residual=r[..., off:off + M], out=out[:, :N, off:off + M])
            close(got, want.double(), want.double().abs() * 2.0 ** -8, BF)  # one step between the two paths
            assert (out[:, N:] == 9).all() and (out[:, :N, :off] == 9).all() and (out[:, :N, off + M:] == 9).all()
        two = sba.int8_linear(a[0], sa[0], w, sw)
        assert torch.equal(two, sba.int8_linear(a, sa, w, sw)[0])


def test_int8_linear_bad_index(sba):
    g = gen(33)
    for N, M in ((20, 64), (1000, 2560)):
        a, sa, w, sw = linear_inputs(g, 1, N, 64, M)
        gate = randn(g, 2, M)
        index = torch.zeros(1, N, dtype=torch.int32, device=DEV)
        want = sba.int8_linear(a, sa, w, sw, gate=gate, index=index)
        index[0, 3], index[0, 7] = 2, -5
        got = sba.int8_linear(a, sa, w, sw, gate=gate, index=index)
        assert sba.device_status() == 6
        assert torch.equal(got, want)


@pytest.mark.parametrize("N,M", [(40, 128), (40, 8192), (1500, 2560)])
def test_int8_linear_wait_limit(sba, N, M):
    """A wait that runs out is a device status, and the next call is right."""
    g = gen(34)
    a, sa, w, sw = linear_inputs(g, 1, N, 2048, M)
    want = sba.int8_linear(a, sa, w, sw)
    assert sba.device_status() == 0
    sba.set_wait_limit(1)
    try:
        sba.int8_linear(a, sa, w, sw)
        assert sba.device_status() == 5
    finally:
        sba.set_wait_limit(0)
    assert torch.equal(sba.int8_linear(a, sa, w, sw), want)


# ------------------------------------------------------------------------------ streams, graphs, refusals

def calls(sba, g):
    """One call of each operator on fixed inputs, as functions that return their outputs."""
    x, kw = norm_inputs(g, 2, 300, 512, BF, BF, SF, 2, "ygm")
    a, sa, w, sw = linear_inputs(g, 2, 300, 512, 2048)
    t = sba.rope_frequencies(96, axes=3)
    q = randn(g, 2, 4, 300, 128, dtype=BF)
    pos = torch.randint(0, 80, (2, 300, 3), generator=g, device=DEV, dtype=torch.int32)
    return [lambda s=None: sba.residual_norm(x, norm="layer", stream=s, **kw),
            lambda s=None: sba.residual_norm(x, norm="rms", quantize=True, stream=s, **kw),
            lambda s=None: sba.token_quantize(q, stream=s),
            lambda s=None: (sba.int8_linear(a, sa, w, sw, stream=s),),
            lambda s=None: (sba.int8_linear(a[:, :3].contiguous(), sa[:, :3].contiguous(), w, sw, stream=s),),
            lambda s=None: (sba.rotary(q, pos, t, stream=s),)]


def test_other_streams(sba):
    fs = calls(sba, gen(40))
    want = [f() for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in fs]
    got = [[f(s) for f, s in zip(fs, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for again in got:
        for u, v in zip(again, want):
            assert all(torch.equal(p, q) for p, q in zip(u, v))


def test_captured_and_replayed(sba):
    fs = calls(sba, gen(41))
    want = [f() for f in fs]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [f() for f in fs]
        graphs.append((graph, got))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        for u, v in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(u, v))


def test_calls_from_two_threads(sba):
    """Products of other sizes, and the other calls, at once from two host threads."""
    import threading
    g = gen(42)
    sizes = [(2, 64, 512), (40, 2048, 1024), (700, 4096, 256), (5, 320, 8192)]
    ins = [linear_inputs(g, 1, n, k, m) for n, m, k in sizes]
    more = calls(sba, g)
    want = [sba.int8_linear(*i) for i in ins], [f() for f in more]
    torch.cuda.synchronize()
    wrong = []

    def work(which):
        try:
            s = torch.cuda.Stream()
            for i in range(100):
                j = (i + which) % len(ins)
                got = sba.int8_linear(*ins[j], stream=s)
                rest = more[i % len(more)](s)
                s.synchronize()
                if not torch.equal(got, want[0][j]) or not all(map(torch.equal, rest, want[1][i % len(more)])):
                    wrong.append((which, i))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(w,)) for w in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


@pytest.mark.parametrize("C", [256, 251])
@pytest.mark.parametrize("far", ["samples", "tokens"])
def test_offsets_past_32_bits(sba, C, far):
    """Rows 2^31 elements apart."""
    g = gen(43)
    big = torch.empty((1 << 31) + (1 << 20), dtype=BF, device=DEV)
    shape = (2, 3, C) if far == "samples" else (1, 2, C)
    strides = (1 << 31, 2 * C + 5 if C % 8 else 2 * C, 1) if far == "samples" else (1 << 31, 1 << 31, 1)
    place = lambda at: big.as_strided(shape, strides, at)
    x, y, out = place(0), place(C + (8 - C % 8) % 8), place(1 << 16)
    xs, ys = randn(g, *shape, dtype=BF), randn(g, *shape, dtype=BF)
    x.copy_(xs)
    y.copy_(ys)
    gate = randn(g, shape[0], C)
    r0, h0 = sba.residual_norm(xs, ys, gate=gate)
    r, h = sba.residual_norm(x, y, gate=gate, out=out)
    assert h.data_ptr() == out.data_ptr() and torch.equal(r, r0)  # (no sums in r)
    # rows that start elsewhere on the 16-byte grid are summed in another order: two results within
    # 400 u S and a rounding each of the same value
    size = xs.double().abs() + ys.double().abs() * gate.double()[:, None].abs()
    S = size.amax(-1, keepdim=True) / (xs.double() + ys.double() * gate.double()[:, None]).std(-1, keepdim=True, correction=0)
    assert ((h.double() - h0.double()).abs() <= 800 * U * S + 2 * rounding(h0.double().abs() + 800 * U * S, BF)).all()
    r, h = sba.residual_norm(xs, ys, gate=gate, x_out=out)
    assert torch.equal(out, r0)
    assert all(map(torch.equal, sba.token_quantize(x), sba.token_quantize(xs)))
    a, s = sba.token_quantize(xs)
    w, ws = sba.token_quantize(randn(g, C, 96 if C % 8 else 128))
    a = a[..., :1].expand(*shape[:2], w.shape[1]).contiguous()
    res = sba.int8_linear(a, s, w, ws, residual=xs)
    assert torch.equal(sba.int8_linear(a, s, w, ws, residual=x, out=out), res)
    table = sba.rope_frequencies(64 if C % 8 == 0 else 62)
    pos = torch.arange(shape[1], device=DEV, dtype=torch.int32).expand(shape[:2]).contiguous()
    want = sba.rotary(xs[:, None], pos, table)
    got = sba.rotary(x[:, None], pos, table, out=out[:, None])
    assert torch.equal(got, want)


def test_empty_batches(sba):
    x = torch.empty(2, 0, 64, dtype=BF, device=DEV)
    r, h = sba.residual_norm(x, x)
    assert r.shape == h.shape == x.shape
    codes, scales = sba.token_quantize(x)
    assert codes.shape == (2, 0, 64) and scales.shape == (2, 0)
    w = torch.ones(32, 64, dtype=torch.int8, device=DEV)
    assert sba.int8_linear(codes, scales, w, torch.ones(32, device=DEV)).shape == (2, 0, 32)
    q = torch.empty(1, 2, 0, 64, dtype=BF, device=DEV)
    assert sba.rotary(q, torch.empty(1, 0, dtype=torch.int32, device=DEV), sba.rope_frequencies(64)).shape == q.shape


def test_refusals(sba):
    x = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    f = torch.zeros(2, 64, device=DEV)
    a, s = sba.token_quantize(x)
    w, ws = a[0], s[0]
    q, pos, t = x[None], torch.zeros(1, 4, dtype=torch.int32, device=DEV), sba.rope_frequencies(64)
    bad = [
        lambda: sba.residual_norm(x[0]), lambda: sba.residual_norm(x.double()), lambda: sba.residual_norm(x, x.half()),
        lambda: sba.residual_norm(x, x.float()), lambda: sba.residual_norm(x, x[:, :3]),
        lambda: sba.residual_norm(x.transpose(1, 2)), lambda: sba.residual_norm(x, norm="batch"),
        lambda: sba.residual_norm(x, norm=None), lambda: sba.residual_norm(x, scale=f[:1]),
        lambda: sba.residual_norm(x, scale=f.half()), lambda: sba.residual_norm(x, scale=f, shift=f.bfloat16()),
        lambda: sba.residual_norm(x, scale=f[:, :32]), lambda: sba.residual_norm(x, index=pos),
        lambda: sba.residual_norm(x, scale=f, index=pos.long()), lambda: sba.residual_norm(x, x_out=x),
        lambda: sba.residual_norm(x, out=x[:, :1].expand(2, 4, 64)), lambda: sba.residual_norm(x, out_dtype=torch.int8),
        lambda: sba.residual_norm(x, valid_len=pos), lambda: sba.residual_norm(x, out=x.cpu()),
        lambda: sba.residual_norm(x, x, norm=None, quantize=True), lambda: sba.residual_norm(x, out_scale=s),
        lambda: sba.token_quantize(x.long()), lambda: sba.token_quantize(x.transpose(1, 2)),
        lambda: sba.token_quantize(x, codes=a[:1]),
        lambda: sba.int8_linear(a, s[:1], w, ws), lambda: sba.int8_linear(a, s, w[:, :32], ws),
        lambda: sba.int8_linear(a, s, w, ws, activation="relu"), lambda: sba.int8_linear(a, s, w, ws, heads=3),
        lambda: sba.int8_linear(a, s, w, ws, out_dtype=torch.int8), lambda: sba.int8_linear(a, s, w, ws, index=pos),
        lambda: sba.int8_linear(a, s, w, ws, residual=x), lambda: sba.int8_linear(a.float(), s, w, ws),
        lambda: sba.int8_linear(a, s, w, ws, gate=f), lambda: sba.int8_linear(a, s, w.t(), ws),
        lambda: sba.rotary(x, pos, t), lambda: sba.rotary(q, pos.long(), t), lambda: sba.rotary(q, pos[:, :3], t),
        lambda: sba.rotary(q, pos, t, layout="thirds"), lambda: sba.rotary(q, pos, sba.rope_frequencies(128)),
        lambda: sba.rotary(q, pos, sba.rope_frequencies(60, axes=3)),
        lambda: sba.rotary(q, pos, t, out=q[..., :32]), lambda: sba.rotary(q[..., ::2], pos, t),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was accepted")
    with pytest.raises(sba.SbaError):
        sba.residual_norm(x, gate=torch.zeros(2, 64, device=DEV))  # nothing to gate


# ------------------------------------------------------------------------------ together

def test_block_around_the_attention(sba):
    """A whole attention sub-block from the residual stream and back onto it, on a ragged batch:
    modulated norm in 8 bits, projections into the head layout, rotary positions, routed
    attention, its output in 8 bits, the output projection gated onto the residual, and the
    norm of what results.  The first four steps and the last three are held to a 64-bit
    evaluation of their own inputs; the attention between them is tested elsewhere."""
    g = gen(50)
    B, N, H, D = 2, 320, 3, 128
    C = H * D
    lens = torch.tensor([320, 203], dtype=torch.int32, device=DEV)
    x = randn(g, B, N, C, dtype=BF)
    scale, shift, gate = (randn(g, B, C, std=0.3) for _ in range(3))
    ws = [sba.token_quantize(randn(g, C, C, std=C ** -0.5)) for _ in range(4)]
    pos = torch.stack([torch.arange(N, device=DEV) // 80, torch.arange(N, device=DEV) // 10 % 8,
                       torch.arange(N, device=DEV) % 10], 1).to(torch.int32)[None].repeat(B, 1, 1)
    table = sba.rope_frequencies(96, axes=3)

    r, codes, scales = sba.residual_norm(x, scale=scale, shift=shift, valid_len=lens, quantize=True)
    assert r is x
    q, k, v = (sba.int8_linear(codes, scales, *w, heads=H) for w in ws[:3])
    for t, w in zip((q, k, v), ws):
        ref, tol = linear_ref(codes, scales, *w, None, None, None, None, None)
        close(t, ref.view(B, N, H, D).transpose(1, 2), tol.view(B, N, H, D).transpose(1, 2), BF)
    ref, tol = rotary_ref(q, pos, table, "interleaved", False)
    q = sba.rotary(q, pos, table, out=q)
    close(q, ref, tol, BF)
    k = sba.rotary(k, pos, table, out=k)
    o, lse, _, _ = sba.sparse_attention(q, k, v, lens, sparsity=0.5)
    oc, os = sba.token_quantize(o)
    for b in range(B):  # padding rows of the attention are zeros, so their codes are
        assert not oc[b, lens[b]:].any() and not os[b, lens[b]:].any()
    x2 = sba.int8_linear(oc, os, *ws[3], gate=gate, residual=x)
    ref, tol = linear_ref(oc, os, *ws[3], None, None, gate, None, x)
    close(x2, ref, tol, BF)
    _, h = sba.residual_norm(x2, scale=scale, shift=shift, valid_len=lens)
    _, href, _, ht = norm_ref(x2, None, None, "layer", None, None, scale, shift, None, None, None, lens, 1e-6)
    close(h, href, ht, BF)
    # the gate as the norm's step in place of the product's: the same stream within two roundings
    y = sba.int8_linear(oc, os, *ws[3])
    x3, h3 = sba.residual_norm(x, y, gate=gate, scale=scale, shift=shift, valid_len=lens)
    live = torch.arange(N, device=DEV) < lens[:, None]
    err = (x3.double() - x2.double()).abs()[live]
    step = (x.double().abs() + 3 * (y.double() * gate.double()[:, None]).abs())[live] * 2.0 ** -8
    assert (err <= 2 * step).all()
    assert torch.isfinite(lse[0]).all()
