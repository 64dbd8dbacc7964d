"""Long rows and matrices past 32-bit offsets in the default-maths operators for
few tokens and in the MXFP4 product."""
import pytest
import torch

import few_reference as ref
import test_gpu_few_tokens as few

pytestmark = pytest.mark.gpu

NAN = float("nan")
N, K = 131200, 65536     # more than 2^32 bytes of codes


@pytest.mark.parametrize("fmt,shape", [(few.Fp8, (25, 8192, 64, 2, 2)), (few.Fp8, (20, 8192, 4096, 2, 1)),
                                       (few.Fp8, (9, 64, 8192, 1, 1)), (few.Nvfp4, (25, 8192, 128, 2, 2)),
                                       (few.Nvfp4, (20, 8192, 4096, 2, 1)), (few.Nvfp4, (9, 128, 8192, 1, 1))], ids=str)
def test_layer_with_several_jobs_of_fewer_than_8_slots(metis, fmt, shape):
    few.check(metis, fmt, few.layer(fmt, 1300 + shape[0] + shape[2], *shape))


def random_bytes(n, seed, lo=0, hi=256):
    return torch.randint(lo, hi, (n,), generator=few.gen(seed), device="cuda", dtype=torch.uint8)


def rows_at_both_ends(n):
    return torch.cat((torch.arange(128, device="cuda"), torch.arange(n - 256, n, device="cuda")))


def scales(sf, rows, chunk):
    """The tiled scale bytes of whole 128-row blocks [rows, 4 * chunks], chunk by chunk."""
    blocks = sf.view(-1, K // chunk * 512)[rows[::128] // 128]
    return ref.untile(blocks, len(rows), K // chunk * 4)


@pytest.mark.parametrize("M", [1, 3, 16, 40, 200, 3001])
def test_nvfp4_product_past_32_bit_offsets(metis, M):
    """Streamed, on the tensor cores and widened: the first and the last channels."""
    q = random_bytes(N * K // 2, 1310).view(N, K // 2)
    sf = random_bytes(N * K // 16, 1311, 0, 127)
    gs = torch.full((1,), 2.0 ** -16, device="cuda")
    x = torch.randn(M, K, generator=few.gen(1312 + M), device="cuda").bfloat16()
    n = metis.metis_workspace_size(metis.METIS_OP_NVFP4_W4A16, M, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    y = torch.full((M, N), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q, sf, gs, y, ws)
    assert metis.metis_check_device_status() == 0
    rows = rows_at_both_ends(N)
    w = ref.e2m1(q[rows]) * ref.e4m3(scales(sf, rows, 64).contiguous()).repeat_interleave(16, dim=1) * gs.double()
    tokens = torch.arange(M, device="cuda")[-40:]
    ref.assert_within(y[tokens][:, rows], *ref.product(x[tokens], w))
    assert bool(torch.isfinite(y).all())


def mxfp4(seed, n):
    q, sf = random_bytes(n * K // 2, seed).view(n, K // 2), random_bytes(n * K // 32, seed + 1, 121, 127)

    def values(rows):
        return ref.e2m1(q[rows]) * ref.e8m0(scales(sf, rows, 128)).repeat_interleave(32, dim=1)
    return q, sf, values


@pytest.mark.parametrize("m,n", [(128, N), (384, N), (N, 384)], ids=["one-cta-B", "pairs-B", "pairs-A"])
def test_mxfp4_product_past_32_bit_offsets(metis, m, n):
    qa, sa, va = mxfp4(1320, m)
    qb, sb, vb = mxfp4(1330, n)
    y = torch.full((m, n), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_mxfp4_gemm(qa, sa, qb, sb, y)
    assert metis.metis_check_device_status() == 0
    ra, rb = (rows_at_both_ends(v) if v > 384 else torch.arange(v, device="cuda") for v in (m, n))
    ref.assert_within(y[ra][:, rb], *ref.product(va(ra), vb(rb)))
    assert bool(torch.isfinite(y).all())
