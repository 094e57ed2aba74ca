"""The block's operators at the ends of the ranges they document: products of more row tiles
than a grid's second dimension holds, rotary frequencies of many turns a position, parameters
at the alignment of their element only."""
from fractions import Fraction

import pytest
import torch

from test_gpu_block import (BF, DEV, HF, SF, U, clean_status, close, gen, linear_inputs, linear_ref, norm_inputs,  # noqa: F401
                            norm_ref, randn, rotary_ref, sba)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N", [(1, 65535 * 128), (1, 65535 * 128 + 1), (3, 2_900_000)])
def test_int8_linear_of_millions_of_rows(sba, B, N):
    """Up to 65535 row tiles and past them: the same results, in the row layout and in heads."""
    g = gen(60)
    K, M = 16, 64
    a = torch.randint(-127, 128, (B, N, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    sa = torch.rand(B, N, generator=g, device=DEV) * 0.01 + 1e-4
    sw = torch.rand(M, generator=g, device=DEV) * 0.01 + 1e-3
    bias = randn(g, M)
    out = sba.int8_linear(a, sa, w, sw, bias=bias)
    for n in range(0, N, 1 << 20):  # in slices: the reference is in 64 bits
        part = slice(n, min(N, n + (1 << 20)))
        ref, tol = linear_ref(a[:, part], sa[:, part], w, sw, bias, None, None, None, None)
        close(out[:, part], ref, tol, BF)
    heads = sba.int8_linear(a, sa, w, sw, bias=bias, heads=2)
    for h in range(2):
        assert torch.equal(heads[:, h], out[..., 32 * h:32 * h + 32])


# 2 pi to 60 digits
TWO_PI = Fraction(62831853071795864769252867665590057683943387987502116419499, 10 ** 58)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_of_many_turns_a_position(sba, layout):
    """Frequencies up to the largest accepted, at positions up to the largest: the angle, taken modulo
    a turn in exact arithmetic, is as exact as any (the bound of test_gpu_block.py)."""
    g = gen(61)
    freq = [1e9, -1e9, 999_999_937.0, 123_456_789.123, 1e6 / 3, 6.283185307179586, 1e3, 1.0,
            0.1, 1e-3, 2.0 ** -20, 1e-9, 2.0 ** 29, 3.0 ** 18, -12_345.678, 1e-300]
    pos = [0, 1, -1, 2, 1000, 65537, 2 ** 31 - 1, -2 ** 31, 1_234_567_890, -987_654_321]
    table = sba.RopeTable(freq)
    turns = [[Fraction(p) * Fraction(f) / TWO_PI for f in freq] for p in pos]
    th = torch.tensor([[2 * torch.pi * float(t - round(t)) for t in row] for row in turns], dtype=torch.float64, device=DEV)
    c, s = th.cos(), th.sin()
    x = randn(g, 1, 3, len(pos), 48)  # 16 channels are copied
    r = sba.rotary(x, torch.tensor(pos, dtype=torch.int32, device=DEV)[None], table, layout=layout)
    one, two = (slice(0, 16), slice(16, 32)) if layout == "half" else (slice(0, 32, 2), slice(1, 32, 2))
    ref, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    u, v = x.double()[..., one], x.double()[..., two]
    ref[..., one], ref[..., two] = u * c - v * s, u * s + v * c
    tol[..., one] = tol[..., two] = 11 * U * (u.abs() + v.abs())
    close(r, ref, tol, SF)


def at_odd_address(t):
    """The same values one element past a multiple of 16 bytes."""
    if t is None:
        return None
    moved = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    return moved.copy_(t)


@pytest.mark.parametrize("C", [64, 512, 1024, 5120, 5121])
@pytest.mark.parametrize("xt,yt,pt", [(BF, BF, SF), (SF, HF, HF), (SF, SF, SF)])
def test_residual_norm_parameters_at_any_alignment(sba, C, xt, yt, pt):
    g = gen(62)
    x, kw = norm_inputs(g, 2, 9, C, xt, yt, pt, 3, "ygwbmip")
    want = norm_ref(x, kw["y"], kw["gate"], "layer", kw["weight"], kw["bias"], kw["scale"], kw["shift"], kw["index"], "rms",
                    kw["post_weight"], None, 1e-6)
    for odd in ("gate", "weight", "bias", "scale", "shift", "index", "post_weight", None):
        moved = {k: at_odd_address(v) if k != "y" and odd in (k, None) else v for k, v in kw.items()}
        r, h = sba.residual_norm(x, norm="layer", post_norm="rms", **moved)
        close(r, want[0], want[2], xt)
        close(h, want[1], want[3], yt)


@pytest.mark.parametrize("N,M", [(20, 320), (1500, 2560)])
@pytest.mark.parametrize("ot,pt", [(BF, SF), (HF, HF), (SF, SF)])
def test_int8_linear_parameters_at_any_alignment(sba, N, M, ot, pt):
    g = gen(63)
    a, sa, w, sw = linear_inputs(g, 2, N, 144, M)
    bias, gate, res = randn(g, M, dtype=pt), randn(g, 3, M, dtype=pt), randn(g, 2, N, M, dtype=ot)
    index = torch.randint(0, 3, (2, N), generator=g, device=DEV, dtype=torch.int32)
    ref, tol = linear_ref(a, sa, w, sw, bias, "silu", gate, index, res)
    for odd in range(7):
        t = [at_odd_address(v) if odd in (i, 6) else v for i, v in enumerate((sa, sw, bias, gate, index, res))]
        out = sba.int8_linear(a, t[0], w, t[1], bias=t[2], activation="silu", gate=t[3], index=t[4], residual=t[5],
                              out_dtype=ot)
        close(out, ref, tol, ot)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_positions_at_any_alignment(sba, layout):
    g = gen(64)
    x, pos = randn(g, 2, 3, 50, 128, dtype=BF), torch.randint(0, 999, (2, 50, 3), generator=g, device=DEV, dtype=torch.int32)
    table = sba.rope_frequencies(96, axes=3)
    ref, tol = rotary_ref(x, pos, table, layout, False)
    close(sba.rotary(x, at_odd_address(pos), table, layout=layout), ref, tol, BF)
