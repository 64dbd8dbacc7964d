"""The forms of the NVFP4 weight-only product for up to 16 tokens, each known to
have run. The streamed form stages a token as FP16 after a shift: elements below
2^-39 of the token's largest count as zero there, while the tensor cores
multiply them as BF16. One such element beside a weight of zero tells them apart."""
import pytest
import torch

import few_reference as ref
import test_gpu_few_tokens as few

pytestmark = pytest.mark.gpu

NAN = float("nan")


def streamed(metis, M, N, K):
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** 60, 2.0 ** 18           # below 2^-39 of the largest
    q = torch.full((N, K // 2), 0x20, dtype=torch.uint8, device="cuda")  # even elements 0, odd ones 1
    sf = torch.full((N * K // 16,), 0x38, dtype=torch.uint8, device="cuda")  # 1
    y = torch.full((M, N), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q, sf, torch.ones(1, device="cuda"), y)
    assert bool((y == y[0, 0]).all()) and float(y[0, 0]) in (0.0, 2.0 ** 18)
    return float(y[0, 0]) == 0.0


# (tokens, N, K): 8 and 16 warps; 16 columns; one and two jobs (9 tokens in a kernel of 8 columns; rows of
# which 5 fit); the longest rows; and the sizes beside them that the tensor cores take
STREAMED = [(1, 14336, 4096), (5, 14336, 4096), (8, 14336, 4096), (1, 128, 65536), (2, 384, 1088), (7, 2048, 2048),
            (16, 14336, 4096), (9, 9600, 4096), (9, 9600, 8192), (16, 9600, 8192), (6, 9600, 13632)]
TENSOR = [(16, 14336, 4352), (13, 12288, 5632), (9, 14336, 7104), (8, 2048, 6144), (16, 2048, 6144)]


@pytest.mark.parametrize("form,shape", [(True, s) for s in STREAMED] + [(False, s) for s in TENSOR], ids=str)
def test_form_of_a_product(metis, form, shape):
    M, N, K = shape
    assert streamed(metis, M, N, K) == form
    g = few.gen(1200 + M + N + K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, sf, gs = few.nvfp4_weights(g, 1, N, K)
    y = torch.full((M + 1, N), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y[:M])
    assert metis.metis_check_device_status() == 0
    ref.assert_within(y[:M], *ref.product(x, ref.nvfp4_values(q, sf, gs)[0]))
    assert bool(torch.isnan(y[M]).all())
