"""Products that split a tile's K over a cluster, several at once on two streams:
their CTAs compete for the SMs' tensor memory with one another and with the
CTA-pair kernels."""
import pytest
import torch

import test_gpu_few_tokens as few

pytestmark = pytest.mark.gpu


def nvfp4_product(metis, M, N, K, seed):
    g = few.gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, sf, gs = few.nvfp4_weights(g, 1, N, K)
    return lambda y: metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y), M, N


def mxfp4_product(metis, M, N, K, seed):
    g = few.gen(seed)
    rows = (M + 127) // 128 * 128
    qa, qb = (torch.randint(0, 256, (r, K // 2), generator=g, device="cuda", dtype=torch.uint8) for r in (rows, N))
    sa, sb = (torch.randint(121, 127, (r * K // 32,), generator=g, device="cuda", dtype=torch.uint8) for r in (rows, N))
    return lambda y: metis.metis_mxfp4_gemm(qa, sa, qb, sb, y), M, N


# (tokens, N, K): tiles of 32, 64, 128 and 256 tokens, few enough of them that clusters share their K;
# the MXFP4 product split over clusters, and as CTA pairs
ONE = [(nvfp4_product, 20, 1024, 4096), (nvfp4_product, 60, 2048, 6144), (mxfp4_product, 16, 2048, 6144),
       (nvfp4_product, 256, 2048, 6144)]
TWO = [(nvfp4_product, 37, 1024, 8192), (mxfp4_product, 16, 1024, 8192), (nvfp4_product, 100, 1024, 6144),
       (mxfp4_product, 600, 2048, 2048)]


def test_split_products_on_two_streams(metis):
    ops = [[make(metis, M, N, K, 1100 + i) for i, (make, M, N, K) in enumerate(side)] for side in (ONE, TWO)]
    out = [[torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _, M, N in side] for side in ops]
    want = []
    for side, ys in zip(ops, out):
        for (run, _, _), y in zip(side, ys):
            run(y)
        want.append([y.clone() for y in ys])
    assert metis.metis_check_device_status() == 0
    assert all(bool(torch.isfinite(y).all()) for ys in want for y in ys)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for _ in range(10):
            for s, side, ys in zip(streams, ops, out):
                with torch.cuda.stream(s):
                    for (run, _, _), y in zip(side, ys):
                        run(y)
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for ys, ws in zip(out, want) for y, w in zip(ys, ws))
    assert metis.metis_check_device_status() == 0
