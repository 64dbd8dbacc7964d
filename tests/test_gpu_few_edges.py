"""Values at the edges of the types in the few-token default-maths operators:
infinities beside large finite values, and tokens near the largest value."""
import pytest
import torch

import few_reference as ref
import test_gpu_few_tokens as few
from test_gpu_few_tokens import by_format

pytestmark = pytest.mark.gpu

INF = float("inf")


def same_specials(got, want):
    """NaN where the 64-bit form has NaN, the same infinity where it has one; finite elsewhere."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isposinf(got), torch.isposinf(want)) and torch.equal(torch.isneginf(got), torch.isneginf(want))


def rows_with_infinities(x):
    """Rows 0 .. 3 of x get an infinity, beside finite values of every size and sign."""
    x[0, 3] = INF
    x[1, 7] = -INF
    x[1, ::5] = x[1, ::5] * 1e5
    x[2, 1::3] = -1e5
    x[2, 2::3] = 1e30
    x[2, 11] = INF
    x[3, :] = torch.where(x[3] > 0, 1e-30, -7e4)
    x[3, 0] = -INF
    return x


@pytest.mark.parametrize("M", [4, 8, 16, 40, 200])
def test_product_of_rows_with_an_infinity(metis, M):
    """Every form of the NVFP4 weight-only product (streamed or on the tensor cores) gives the
    infinities of the formula, whatever stands beside them in the row, and leaves the other rows alone."""
    N, K = 512, 1088
    g = few.gen(1000 + M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, sf, gs = few.nvfp4_weights(g, 1, N, K)
    clean = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, clean)
    x = rows_with_infinities(x)
    y = torch.empty_like(clean)
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y)
    assert metis.metis_check_device_status() == 0
    want = x[:4].double() @ ref.nvfp4_values(q, sf, gs)[0].t()
    assert bool(torch.isinf(want).any())
    same_specials(y[:4], want)
    assert torch.equal(y[4:], clean[4:])


@by_format
@pytest.mark.parametrize("T,k", [(5, 1), (5, 4), (60, 4)])
def test_layer_of_tokens_with_an_infinity(metis, fmt, T, k):
    """Positive weights: the infinity of a token's x reaches every output with its sign."""
    d = few.layer(fmt, 1010 + T, T, 256, 384, 8, k)
    d["tw"] = d["tw"].abs() + 0.1
    for p in ("up", "down"):
        q, *rest = d[p]
        # E4M3 codes 1 .. 126; E2M1 codes 1 .. 7 and block scales above zero
        q = q % 126 + 1 if fmt is few.Fp8 else (q & 0x77) | 0x11
        if fmt is few.Nvfp4:
            rest[0] = rest[0] % 126 + 1
        d[p] = (q, *rest)
    clean = few.run(metis, fmt, d)
    d["x"] = rows_with_infinities(d["x"].clone())
    y = few.run(metis, fmt, d)
    assert metis.metis_check_device_status() == 0
    for row, sign in enumerate((INF, -INF, INF, -INF)):
        assert bool((y[row] == sign).all()), row
    assert torch.equal(y[4:], clean[4:])


@by_format
@pytest.mark.parametrize("T,k", [(2, 1), (5, 4), (60, 4)])
def test_layer_of_very_large_tokens(metis, fmt, T, k):
    """Tokens whose outputs are finite while the sums of codes alone, without the weights' scales, are not."""
    d = few.layer(fmt, 1020 + T, T, 256, 256, 8, k)
    d["x"] = (d["x"].float() * 2.0 ** 120).bfloat16()
    y, bound = few.expect(fmt, d)
    assert float(y.abs().max()) < 2.0 ** 127
    got = few.run(metis, fmt, d)
    assert metis.metis_check_device_status() == 0
    ref.assert_within(got, y, bound)


@pytest.mark.parametrize("M", [1, 3, 8])
def test_streamed_product_of_very_large_tokens(metis, M):
    N, K = 512, 1088
    g = few.gen(1030 + M)
    x = (torch.randn(M, K, generator=g, device="cuda") * 2.0 ** 120).bfloat16()
    q, sf, gs = few.nvfp4_weights(g, 1, N, K)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y)
    assert metis.metis_check_device_status() == 0
    want, bound = ref.product(x, ref.nvfp4_values(q, sf, gs)[0])
    assert float(want.abs().max()) < 2.0 ** 127
    ref.assert_within(y, want, bound)
