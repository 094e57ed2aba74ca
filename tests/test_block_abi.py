"""C-ABI checks of the block's operators that need no GPU: bad arguments come back as a
status before any CUDA call, the binding refuses what it can see, and the frequency tables
follow their formulas."""
import ctypes
import math

import pytest

A = ctypes.c_void_p(0x10000)     # 16-byte aligned
M8 = ctypes.c_void_p(0x10008)    # 8-byte aligned
M2 = ctypes.c_void_p(0x10002)    # 2-byte aligned
M1 = ctypes.c_void_p(0x10001)
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from video_dit_block_b200 import build
    build.build()
    import video_dit_block_b200 as sba
    return sba.lib()


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def norm(lib, x=A, y=A, r=A, h=A, hs=None, xt=BF16, t=BF16, B=2, N=8, C=64, st=None, vl=None, kind=1, w=None, b=None,
         post=0, pw=None, gate=None, scale=None, shift=None, pt=FP32, G=2, index=None, eps=1e-6):
    st = i64(*(st or [512, 64] * 4))
    return lib.sba_residual_norm(x, y, r, h, hs, xt, t, B, N, C, st, vl, kind, w, b, post, pw, gate, scale, shift, pt, G,
                                 index, eps, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(r=None), 1), (dict(h=None), 1), (dict(B=0), 1), (dict(N=-1), 1), (dict(C=0), 1),
    (dict(xt=3), 1), (dict(t=-1), 1), (dict(pt=7), 1), (dict(kind=3), 1), (dict(kind=-1), 1), (dict(post=5), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(st=[-1, 64] * 4), 1),
    (dict(y=None, gate=A), 1), (dict(y=None, post=1), 1), (dict(pw=A), 1),
    (dict(kind=0, y=None), 1), (dict(kind=0, w=A), 1), (dict(kind=0, scale=A), 1), (dict(kind=0, hs=A), 1),
    (dict(gate=A, G=0), 1), (dict(gate=A, G=1), 1),
    (dict(C=32769), 2), (dict(B=65536, N=65536), 2), (dict(xt=BF16, t=FP16), 2), (dict(xt=BF16, t=FP32), 2),
    (dict(scale=A, pt=FP16), 2),
    (dict(x=M1), 3), (dict(xt=FP32, x=M2), 3), (dict(y=M1), 3), (dict(gate=M2), 3), (dict(w=M2), 3),
    (dict(h=M8, hs=A), 3), (dict(hs=A, st=[512, 64, 512, 64, 512, 64, 512, 72]), 3), (dict(gate=A, index=M2), 3),
    (dict(vl=M2), 3),
])
def test_residual_norm_rejects(lib, kw, code):
    assert norm(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(t=9), 1),
    (dict(H=257, D=128), 2), (dict(B=65536, N=65536), 2), (dict(x=M1), 3), (dict(c=M8), 3), (dict(s=M2), 3),
])
def test_token_quantize_rejects(lib, kw, code):
    a = dict(x=A, t=BF16, B=1, H=2, N=8, D=64, c=A, s=A) | kw
    assert lib.sba_token_quantize(a["x"], a["t"], a["B"], a["H"], a["N"], a["D"], i64(1, 1, 1), a["c"], a["s"],
                                  None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), 1), (dict(sa=None), 1), (dict(w=None), 1), (dict(sw=None), 1), (dict(out=None), 1),
    (dict(B=0), 1), (dict(K=0), 1), (dict(M=0), 1), (dict(act=3), 1), (dict(ot=5), 1), (dict(pt=-2), 1),
    (dict(heads=3), 1), (dict(heads=-1), 1), (dict(gate=A, G=0), 1), (dict(gate=A, G=1), 1),
    (dict(st=[0, 0, -1, 0, 0]), 1),
    (dict(K=40), 2), (dict(K=131072), 2), (dict(heads=4), 2), (dict(pt=FP16), 2), (dict(B=65536, N=65536), 2),
    (dict(M=1 << 25), 2),
    (dict(a=M8), 3), (dict(w=M8), 3), (dict(sa=M2), 3), (dict(out=M1), 3), (dict(residual=M1), 3), (dict(bias=M2), 3),
])
def test_int8_linear_rejects(lib, kw, code):
    a = dict(a=A, sa=A, w=A, sw=A, B=2, N=8, K=64, M=64, bias=None, gate=None, pt=FP32, G=2, index=None, act=0,
             residual=None, out=A, ot=BF16, heads=0, st=[512, 64, 512, 0, 64]) | kw
    assert lib.sba_int8_linear(a["a"], a["sa"], a["w"], a["sw"], a["B"], a["N"], a["K"], a["M"], a["bias"], a["gate"],
                               a["pt"], a["G"], a["index"], a["act"], a["residual"], a["out"], a["ot"], a["heads"],
                               i64(*a["st"]), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(o=None), 1), (dict(pos=None), 1), (dict(axes=0), 1), (dict(rope=0), 1), (dict(rope=7), 1),
    (dict(rope=130), 1), (dict(layout=2), 1), (dict(t=4), 1), (dict(amp=float("inf")), 1),
    (dict(freq=[float("nan")] * 32), 1), (dict(freq=[2e9] * 32), 1), (dict(axis=[1] * 32), 1), (dict(st=[-1] * 6), 1),
    (dict(D=512, rope=300, freq=[1.0] * 150, axis=[0] * 150), 2), (dict(B=65536), 2), (dict(H=65536), 2),
    (dict(x=M1), 3), (dict(o=M1), 3), (dict(pos=M2), 3), (dict(t=FP32, x=M2), 3),
])
def test_rotary_rejects(lib, kw, code):
    a = dict(x=A, o=A, t=BF16, pos=A, axes=1, B=1, H=2, N=8, D=128, rope=64, layout=0, freq=[1.0] * 32, axis=[0] * 32,
             amp=1.0, st=[0] * 6) | kw
    n = len(a["freq"])
    assert lib.sba_rotary(a["x"], a["o"], a["t"], a["pos"], a["axes"], a["B"], a["H"], a["N"], a["D"], i64(*a["st"]),
                          a["rope"], a["layout"], (ctypes.c_double * n)(*a["freq"]), (ctypes.c_uint8 * n)(*a["axis"]),
                          a["amp"], 0, None) == code


P, Q, R = (ctypes.c_void_p(n) for n in (0x20000, 0x30000, 0x40000))


@pytest.mark.parametrize("kw", [
    dict(x=A, y=P, r=Q, h=Q),                                            # both outputs in one place
    dict(x=A, y=P, r=P, h=Q),                                            # the residual stream over the block's output
    dict(x=A, y=P, r=A, h=Q, st=[512, 64, 512, 64, 1024, 64, 512, 64]),  # in place, other strides
    dict(x=A, y=P, r=A, h=Q, st=[64, 128, 512, 64, 64, 256, 512, 64]),
    dict(x=A, y=P, r=Q, h=P, st=[512, 64, 512, 64, 512, 64, 512, 128]),
    dict(x=A, y=P, r=Q, h=P, hs=R), dict(x=A, y=None, r=None, h=A, hs=R),
    dict(x=A, y=None, r=None, h=A, xt=FP32),
])
def test_residual_norm_rejects_overlaps(lib, kw):
    assert norm(lib, **kw) == 1


def test_others_reject_overlaps(lib):
    for heads, st in ((2, [512, 64, 512, 64, 64]), (0, [512, 64, 1024, 0, 64]), (0, [512, 64, 512, 0, 128])):
        assert lib.sba_int8_linear(A, P, A, P, 2, 8, 64, 64, None, None, FP32, 0, None, 0, Q, Q, BF16, heads, i64(*st),
                                   None) == 1
    for w, out in ((A, P), (P, A)):
        assert lib.sba_int8_linear(w, Q, out, Q, 2, 8, 64, 64, None, None, FP32, 0, None, 0, None, A, BF16, 0,
                                   i64(0, 0, 512, 0, 64), None) == 1
    assert lib.sba_token_quantize(A, BF16, 1, 1, 8, 64, i64(512, 0, 64), A, P, None) == 1
    f, a = (ctypes.c_double * 32)(*[1.0] * 32), (ctypes.c_uint8 * 32)()
    for st in ([0, 1024, 128, 0, 1024, 256], [0, 1024, 128, 0, 128, 128]):
        assert lib.sba_rotary(A, A, BF16, P, 1, 1, 2, 8, 128, i64(*st), 64, 0, f, a, 1.0, 0, None) == 1


def test_binding_refuses_sizes_past_32_bits():
    from video_dit_block_b200 import sba
    sba._counts(1, 0x7fffffff)
    with pytest.raises(ValueError):
        sba._counts(1, 0x80000000)


def test_binding_refuses_cpu_tensors():
    import torch

    import video_dit_block_b200 as sba
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sba.residual_norm(x)
    with pytest.raises(ValueError):
        sba.token_quantize(x)
    with pytest.raises(ValueError):
        sba.int8_linear(x.to(torch.int8), x[..., 0].float(), x[0].to(torch.int8), x[0, :, 0].float())
    with pytest.raises(ValueError):
        sba.rotary(x[None], torch.zeros(1, 4, dtype=torch.int32), sba.rope_frequencies(64))


def test_rope_frequencies():
    import video_dit_block_b200 as sba
    t = sba.rope_frequencies(96, axes=3)
    assert t.rope_dim == 96 and t.axes == 3 and t.amplitude == 1.0
    assert t.axis == (0,) * 16 + (1,) * 16 + (2,) * 16
    assert t.inv_freq[:16] == t.inv_freq[16:32] == t.inv_freq[32:]
    for i, f in enumerate(t.inv_freq[:16]):
        assert f == pytest.approx(10000.0 ** (-2 * i / 32), rel=1e-14)
    lin = sba.rope_frequencies(128, scaling="linear", factor=4.0)
    ref = sba.rope_frequencies(128)
    assert all(a == b / 4 for a, b in zip(lin.inv_freq, ref.inv_freq))
    # ntk: the fastest pair as it was, the slowest slowed by exactly the factor
    ntk = sba.rope_frequencies(128, scaling="ntk", factor=4.0)
    assert ntk.inv_freq[0] == ref.inv_freq[0]
    assert ntk.inv_freq[-1] == pytest.approx(ref.inv_freq[-1] / 4, rel=1e-12)
    # yarn: pairs of at least 32 turns within the length as they were, of at most one turn
    # slowed by the factor, the others between, in order
    y = sba.rope_frequencies(128, scaling="yarn", factor=4.0, original_length=4096)
    assert y.amplitude == pytest.approx(0.1 * math.log(4.0) + 1)
    for f, r in zip(y.inv_freq, ref.inv_freq):
        turns = 4096 * r / (2 * math.pi)
        assert r / 4 * (1 - 1e-12) <= f <= r * (1 + 1e-12)
        if turns > 32 * 1.2:
            assert f == pytest.approx(r, rel=1e-12)
        if turns < 1 / 1.2:
            assert f == pytest.approx(r / 4, rel=1e-12)
    assert list(y.inv_freq) == sorted(y.inv_freq, reverse=True)


@pytest.mark.parametrize("kw", [
    dict(rope_dim=63), dict(rope_dim=0), dict(rope_dim=64, axes=3), dict(rope_dim=64, axes=0), dict(rope_dim=64, base=0.0),
    dict(rope_dim=64, factor=0.0), dict(rope_dim=64, scaling="cubic"), dict(rope_dim=2, scaling="ntk", factor=2.0),
    dict(rope_dim=64, scaling="yarn", factor=2.0, beta_fast=1.0), dict(rope_dim=64, base=float("inf")),
    dict(rope_dim=64, scaling="yarn", factor=2.0, original_length=0),
])
def test_rope_frequencies_rejects(kw):
    import video_dit_block_b200 as sba
    with pytest.raises(ValueError):
        sba.rope_frequencies(**kw)


def test_rope_table_rejects():
    import video_dit_block_b200 as sba
    for bad in (dict(inv_freq=[]), dict(inv_freq=[1.0], axis=[0, 1]), dict(inv_freq=[float("nan")]),
                dict(inv_freq=[1.0], axis=[-1]), dict(inv_freq=[1.0], axis=[255]),
                dict(inv_freq=[1.0], amplitude=float("inf"))):
        with pytest.raises(ValueError):
            sba.RopeTable(**bad)
