"""The block's operators at the ends of the ranges they document: products of more row tiles
than a grid's second dimension holds."""
import pytest
import torch

from test_gpu_block import BF, DEV, clean_status, close, gen, linear_ref, randn, sba  # noqa: F401 (fixtures)

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
