"""The block's operators at sizes whose kernels go round their loops: more rows than CTAs are
resident, more tiles than clusters, more heads than a thread has in flight.  The formulas and
tolerances are those of test_gpu_block.py, whose sizes mostly end after one turn (its three
products marked as many tiles of 256 x 256 have tiles of 256 x 192, one a cluster)."""
import ctypes
import math
import zlib

import numpy as np
import pytest
import torch

from test_gpu_block import (BF, DEV, HF, SF, clean_status, close, codes_ref, gen, linear_inputs, linear_ref,  # noqa: F401
                            norm_inputs, norm_ref, randn, rotary_ref, sba)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(DEV).multi_processor_count


def lengths(g, B, N):
    """Samples that end anywhere, one of them empty, the last one whole."""
    vl = torch.randint(0, N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    vl[0], vl[1], vl[B - 1] = N // 2, 0, N
    return vl


# ------------------------------------------------------------------------------ rows

def resident(C, vec):
    """The most rows that are in work at once: four a CTA of 128 threads up to 1024 channels, one a
    CTA above, and an SM holds 2048 threads and 32 CTAs."""
    chunks = -(-C // 8) if vec else -(-C // 8) + 2
    if chunks <= 128:
        return sms() * 16 * 4
    threads = -(-chunks // (32 * (4 if chunks <= 1024 else 9))) * 32
    return sms() * min(32, 2048 // threads)


ROWS = [
    # B, N, C, x, y, parameters, parts (as norm_inputs), norm, post
    (3, 7001, 128, BF, BF, SF, "ygm", "layer", None),
    (70, 301, 128, HF, HF, HF, "ygmi", "rms", None),
    (3, 7001, 250, BF, BF, SF, "ygm", "layer", None),
    (70, 301, 250, SF, BF, SF, "ygwp", "rms", "rms"),
    (3, 3500, 1000, BF, BF, BF, "wb", "layer", None),
    (50, 211, 1001, SF, SF, SF, "ygm", "rms", None),
    (3, 1301, 5120, BF, BF, SF, "m", "layer", None),
    (50, 77, 5120, HF, HF, HF, "m", "rms", None),
    (50, 77, 5120, BF, BF, BF, "ygm", "layer", None),
    (3, 1301, 5120, SF, HF, SF, "ygmi", "rms", None),
    (50, 77, 5120, SF, BF, SF, "ygwp", "rms", "rms"),
    (3, 1301, 5120, BF, BF, SF, "yw", "rms", None),
    (50, 77, 5120, SF, SF, SF, "ygm", "layer", None),
    (3, 1301, 5121, BF, BF, SF, "ygm", "layer", None),
    (50, 77, 5121, SF, BF, SF, "ygwp", "rms", "rms"),
    (3, 801, 8200, BF, BF, SF, "ygm", "layer", None),
    (3, 401, 20000, SF, BF, SF, "ygmi", "layer", "rms"),
    (30, 49, 20001, BF, BF, SF, "ygm", "rms", None),
]


@pytest.mark.parametrize("case", ROWS)
def test_residual_norm_of_many_rows(sba, case):
    B, N, C, xt, yt, pt, parts, norm, post = case
    assert B * N > resident(C, C % 8 == 0)
    g = gen(zlib.crc32(str(case).encode()))
    x, kw = norm_inputs(g, B, N, C, xt, yt, pt, 5 if "i" in parts else B, parts)
    vl = lengths(g, B, N)
    r, h = sba.residual_norm(x, norm=norm, post_norm=post, valid_len=vl, **kw)
    for b0 in range(0, B, max(1, B // 3)):  # in slices: the reference is in 64 bits
        b = slice(b0, b0 + max(1, B // 3))
        cut = lambda t: t[b] if t is not None else None
        tables = (lambda t: t) if "i" in parts else cut
        rr, hr, rt, ht = norm_ref(x[b], cut(kw["y"]), tables(kw["gate"]), norm, kw["weight"], kw["bias"],
                                  tables(kw["scale"]), tables(kw["shift"]), cut(kw["index"]), post, kw["post_weight"],
                                  vl[b], 1e-6)
        close(h[b], hr, ht, yt)
        if kw["y"] is not None:
            close(r[b], rr, rt, xt)
    # in 8 bits: the codes and scales of a row are those of a call on a few rows at its place
    _, codes, scales = sba.residual_norm(x, norm=norm, post_norm=post, valid_len=vl, quantize=True, **kw)
    live = (torch.arange(N, device=DEV) < vl[:, None])
    assert not codes[~live].any() and not scales[~live].any()
    for b in sorted({0, B // 2, B - 1}):
        n = min(N, 40)
        for n0 in sorted({0, (N - n) // 2, N - n}):
            rows = slice(n0, n0 + n)
            few = {k: v if v is None or k in ("weight", "bias", "post_weight") else
                   v[b:b + 1, rows] if k == "y" else
                   v[b:b + 1, rows].contiguous() if k == "index" else
                   v if "i" in parts else v[b:b + 1] for k, v in kw.items()}
            rf, cf, sf = sba.residual_norm(x[b:b + 1, rows], norm=norm, post_norm=post, quantize=True, **few)
            at = live[b, rows]
            assert torch.equal(codes[b, rows][at], cf[0][at]) and torch.equal(scales[b, rows][at], sf[0][at])
            if kw["y"] is not None:
                assert torch.equal(r[b, rows][at], rf[0][at])
    # in place
    if kw["y"] is not None:
        x2, y2 = x.clone(), kw["y"].clone()
        r2, h2 = sba.residual_norm(x2, y2, norm=norm, post_norm=post, valid_len=vl, x_out=x2, out=y2,
                                   **{k: v for k, v in kw.items() if k != "y"})
        assert r2 is x2 and h2 is y2 and torch.equal(x2, r) and torch.equal(y2, h)
    else:
        x2 = x.clone()
        _, h2 = sba.residual_norm(x2, norm=norm, valid_len=vl, out=x2, **kw)
        assert torch.equal(h2, h)


@pytest.mark.parametrize("dt", [BF, SF])
@pytest.mark.parametrize("shape", [(21_000, 128), (3, 7000, 250), (10_500, 1001), (4000, 5120), (3, 1300, 5121),
                                   (2500, 8200), (1100, 20_001), (2, 40, 1100, 128), (3, 5, 4001, 75)])
def test_token_quantize_of_many_rows(sba, shape, dt):
    g = gen(70)
    x = randn(g, *shape, dtype=dt)
    x[..., 0] *= torch.rand(x.shape[:-1], generator=g, device=DEV) * 30  # (scales that differ widely)
    rows = x.transpose(1, 2).flatten(2) if x.dim() == 4 else x
    K = rows.shape[-1]
    assert math.prod(rows.shape[:-1]) > resident(K, K % 8 == 0)
    codes, scales = sba.token_quantize(x)
    ref, sref = codes_ref(rows)
    np.testing.assert_array_equal(codes[..., :K].cpu().numpy(), ref)
    np.testing.assert_array_equal(scales.cpu().numpy(), sref)
    assert not codes[..., K:].any()


# ------------------------------------------------------------------------------ products

def plan(sba, rows, channels, codes):
    columns, splits = ctypes.c_int(), ctypes.c_int()
    assert sba.lib().sba_int8_linear_plan(rows, channels, codes, sms(), ctypes.byref(columns), ctypes.byref(splits)) == 0
    return columns.value, splits.value


def many_tiles(sba, rows, channels, codes):
    """The pair kernel's widest tile, and four of them at least for every cluster."""
    assert plan(sba, rows, channels, codes) == (256, 0)
    assert -(-rows // 256) * -(-channels // 256) >= 4 * (sms() // 2)


LINEAR = [
    # B, N, K, M, out, parts (b(ias), g(ate), i(ndex), r(esidual)), activation, parameters
    (1, 9000, 144, 2305, BF, "bgr", None, SF),         # columns off the 16-byte grid
    (3, 3001, 400, 2307, SF, "bgir", "silu", SF),
    (1, 4700, 144, 4104, BF, "bgr", "gelu_tanh", BF),  # on it, 8 columns past the last whole piece
    (2, 2650, 272, 4104, HF, "bgir", None, HF),
    (2, 2650, 272, 4100, SF, "bgir", "silu", SF),
    (1, 5300, 2064, 4100, SF, "gr", None, SF),
    (1, 5299, 2064, 4096, BF, "b", None, SF),
]


@pytest.mark.parametrize("case", LINEAR)
def test_int8_linear_of_many_tiles(sba, case):
    B, N, K, M, ot, parts, act, pt = case
    many_tiles(sba, B * N, M, K)
    g = gen(zlib.crc32(str(case).encode()))
    a, sa, w, sw = linear_inputs(g, B, N, K, M)
    G = 4 if "i" in parts else B
    bias = randn(g, M, dtype=pt, std=0.5) if "b" in parts else None
    gate = randn(g, G, M, dtype=pt) if "g" in parts else None
    index = torch.randint(0, G, (B, N), generator=g, device=DEV, dtype=torch.int32) if "i" in parts else None
    res = randn(g, B, N, M, dtype=ot) if "r" in parts else None
    out = sba.int8_linear(a, sa, w, sw, bias=bias, activation=act, gate=gate, index=index, residual=res, out_dtype=ot)
    ref, tol = linear_ref(a, sa, w, sw, bias, act, gate, index, res)
    close(out, ref, tol, ot)
    if res is not None:  # onto the residual itself
        again = sba.int8_linear(a, sa, w, sw, bias=bias, activation=act, gate=gate, index=index, residual=res,
                                out_dtype=ot, out=res)
        assert again is res and torch.equal(res, out)


@pytest.mark.parametrize("ot", [BF, SF])
def test_int8_linear_into_heads_of_many_tiles(sba, ot):
    B, N, K, H, D = 2, 2650, 272, 33, 128
    many_tiles(sba, B * N, H * D, K)
    g = gen(71)
    a, sa, w, sw = linear_inputs(g, B, N, K, H * D)
    bias = randn(g, H * D)
    out = sba.int8_linear(a, sa, w, sw, bias=bias, out_dtype=ot, heads=H)
    ref, tol = linear_ref(a, sa, w, sw, bias, None, None, None, None)
    split = lambda t: t.unflatten(2, (H, D)).transpose(1, 2)
    close(out, split(ref), split(tol), ot)


# ------------------------------------------------------------------------------ rotary

ROTARY = [
    # B, H, N, D, rope_dim, axes, layout, type
    (1, 9, 20_011, 128, 96, 3, "interleaved", BF),
    (1, 13, 20_011, 128, 128, 1, "half", SF),
    (2, 8, 10_007, 128, 96, 3, "half", HF),
    (1, 40, 19_003, 128, 64, 1, "half", BF),
    (1, 11, 38_001, 64, 32, 1, "interleaved", SF),
    (1, 13, 2_700, 75, 30, 1, "half", BF),          # any width
    (1, 9, 8_001, 80, 60, 3, "interleaved", SF),
]


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary_of_many_tokens(sba, case, order):
    B, H, N, D, rope, axes, layout, dt = case
    # eight heads a thread: the launch keeps them where that leaves four CTAs an SM
    vector = D % 16 == 0 and rope // 2 % (8 if layout == "half" else 4) == 0
    assert N * (D // 16 if vector else D - rope // 2) // 256 * B * -(-H // 8) >= 4 * sms()
    g = gen(zlib.crc32(str(case).encode()))
    x = randn(g, B, H, N, D, dtype=dt) if order == "heads" else randn(g, B, N, H, D, dtype=dt).transpose(1, 2)
    pos = torch.randint(0, 3000, (B, N, axes), generator=g, device=DEV, dtype=torch.int32)
    table = sba.rope_frequencies(rope, axes=axes)
    out = sba.rotary(x, pos, table, layout=layout)
    for h in range(0, H, 7):
        ref, tol = rotary_ref(x[:, h:h + 7], pos, table, layout, False)
        close(out[:, h:h + 7], ref, tol, dt)
    assert sba.rotary(x, pos, table, layout=layout, out=x) is x
    assert torch.equal(x, out)
