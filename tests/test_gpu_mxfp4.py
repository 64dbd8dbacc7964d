"""MXFP4 quantisation, reading back and product against plain 64-bit forms."""
import pytest
import torch

import few_reference as ref
from few_reference import assert_within

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quant(metis, x, tiled):
    R, K = x.shape
    rows = (R + 127) // 128 * 128 if tiled else R
    q = torch.full((R, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows * K // 32 + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    metis.metis_quant_mxfp4(x, q, sf, tiled)
    assert bool((sf[rows * K // 32:] == 0xEE).all())
    sf = sf[:rows * K // 32]
    return q, sf, (ref.untile(sf, rows, K // 32) if tiled else sf.view(R, K // 32))


def check_quant(metis, x, tiled):
    R, K = x.shape
    q, raw, sf = quant(metis, x, tiled)
    values, c, code = ref.mxfp4_quant(x)
    assert torch.equal(sf[:R], c)
    assert bool((sf[R:] == 0).all())
    assert torch.equal(torch.stack((q & 15, q >> 4), dim=-1).view(R, K), code)
    y = torch.full((R + 1, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    metis.metis_dequant_mxfp4(q, raw, y[:R], tiled)
    assert metis.metis_check_device_status() == 0
    assert torch.equal(y[:R].double(), values) and bool(torch.isnan(y[R]).all())
    assert torch.equal(torch.signbit(y[:R]), torch.signbit(x))


SIZES = [(1, 32), (1, 64), (3, 96), (7, 2048), (128, 128), (129, 160), (300, 992), (1000, 4096), (2, 65536), (33, 8224)]


@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tiled", [False, True])
def test_quant_and_back(metis, R, K, dtype, tiled):
    if tiled and K % 128:
        K += 128 - K % 128
        if K > 65536:
            pytest.skip("beyond the largest row")
    g = gen(R + K)
    x = torch.randn(R, K, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 30, (R, 1), generator=g, device="cuda").float())
    check_quant(metis, x.to(dtype), tiled)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_ties_zeros_and_the_ends_of_the_range(metis, dtype):
    """Every quarter step between -8 and 8 (all ties among them) at every block exponent; zeros of both
    signs; subnormal and largest values; blocks whose amax is a power of two."""
    steps = torch.arange(-32, 32, device="cuda").double() / 4
    rows = []
    for e in list(range(-133, 126, 7)) + [-126, -127, -128, 0, 1, 2, 125]:
        block = (steps * 2.0 ** e).clamp(-3.3e38, 3.3e38)
        rows.append(block)
    x = torch.stack(rows).to(dtype)
    x[:, 5] = -0.0
    x[3] = 0
    x[4] = -0.0
    x[5, :32] = 2.0 ** -40
    check_quant(metis, x.contiguous(), False)
    if dtype == torch.float32:
        tiny = torch.full((2, 64), 2.0 ** -149, device="cuda")
        tiny[1] = 2.0 ** -127 * 1.5
        check_quant(metis, tiny, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tiled", [False, True])
def test_quant_infinities_and_nans_mark_their_block(metis, dtype, tiled):
    x = torch.randn(4, 256, generator=gen(5), device="cuda").to(dtype)
    clean = quant(metis, x, tiled)
    x[0, 33] = float("inf")
    x[1, 255] = float("-inf")
    x[2, 0] = float("nan")
    q, raw, sf = quant(metis, x, tiled)
    hit = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 7] = hit[2, 0] = True
    assert bool((sf[:4][hit] == 255).all()) and torch.equal(sf[:4][~hit], clean[2][:4][~hit])
    el = hit.repeat_interleave(16, dim=1)
    assert bool((q[el] == 0).all()) and torch.equal(q[~el], clean[0][~el])
    y = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    metis.metis_dequant_mxfp4(q, raw, y, tiled)
    assert torch.equal(torch.isnan(y), hit.repeat_interleave(32, dim=1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_strided_rows(metis, dtype):
    base = torch.randn(20, 512, generator=gen(6), device="cuda").to(dtype)
    check_quant(metis, base[:, 64:64 + 160], False)
    check_quant(metis, base[::3, :384], True)


def test_dequant_every_code_and_scale(metis):
    """Each scale code with each E2M1 code: exact, infinite past BF16's range, NaN for 255."""
    q = torch.arange(16, device="cuda", dtype=torch.uint8)
    q = (q[0::2] | (q[1::2] << 4)).repeat(2).repeat(256, 1).contiguous()
    sf = torch.arange(256, device="cuda", dtype=torch.uint8).view(256, 1)
    y = torch.empty(256, 32, dtype=torch.bfloat16, device="cuda")
    metis.metis_dequant_mxfp4(q, sf.contiguous(), y)
    want = (ref.e2m1(q) * ref.e8m0(sf)).float().bfloat16()
    assert torch.equal(y[:255], want[:255]) and bool(torch.isnan(y[255]).all())


def mx(g, R, K, lo=118, hi=128):
    rows = (R + 127) // 128 * 128
    return (torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(lo, hi, (rows * K // 32,), generator=g, device="cuda", dtype=torch.uint8))


def mx_values(q, sf, R, K):
    return ref.e2m1(q[:R]) * ref.e8m0(ref.untile(sf, R, K // 32)).repeat_interleave(32, dim=1)


GEMM = [(1, 128, 128), (16, 256, 256), (17, 384, 640), (127, 128, 2048), (128, 512, 384), (129, 256, 128),
        (257, 1152, 896), (700, 2176, 1024), (3, 128, 65536), (300, 128, 8320),
        (5, 2048, 6144), (100, 384, 4224), (128, 1280, 8192), (129, 640, 6016), (500, 2048, 6144)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_sizes(metis, M, N, K):
    g = gen(M + N + K)
    (qa, sa), (qb, sb) = mx(g, M, K), mx(g, N, K)
    y = torch.full((M + 1, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    metis.metis_mxfp4_gemm(qa, sa, qb[:N], sb, y[:M])
    assert metis.metis_check_device_status() == 0
    a, b = mx_values(qa, sa, M, K), mx_values(qb, sb, N, K)
    r, bound = ref.product(a, b)
    assert_within(y[:M], r, bound)
    assert bool(torch.isnan(y[M]).all())


def test_gemm_scales_far_apart_and_nan_blocks(metis):
    """Scales of a row over 80 binades, and a NaN scale: only its row of the product is NaN."""
    M, N, K = 200, 256, 512
    g = gen(9)
    (qa, sa), (qb, sb) = mx(g, M, K, 90, 170), mx(g, N, K, 90, 120)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    metis.metis_mxfp4_gemm(qa, sa, qb, sb, y)
    r, bound = ref.product(mx_values(qa, sa, M, K), mx_values(qb, sb, N, K))
    assert_within(y, r, bound)
    bad = sa.clone()
    bad[16 * (130 % 32) + 4 * (130 % 128 // 32) + 512 * (130 // 128 * (K // 128) + 2) + 1] = 255  # row 130, block 9
    z = torch.empty_like(y)
    metis.metis_mxfp4_gemm(qa, bad, qb, sb, z)
    assert metis.metis_check_device_status() == 0
    keep = torch.arange(M, device="cuda") != 130
    assert bool(torch.isnan(z[130]).all()) and torch.equal(z[keep], y[keep])


def test_layer_quantised_end_to_end_captured_and_replayed(metis):
    """As a layer uses them: weights quantised once (tiled), activations per call, the product; captured,
    replayed on new activations, and the same on another stream."""
    M, N, K = 96, 640, 1280
    g = gen(11)
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    qb = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    sb = torch.empty(N * K // 32, dtype=torch.uint8, device="cuda")
    metis.metis_quant_mxfp4(w, qb, sb, tiled=True)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    qa = torch.zeros(128, K // 2, dtype=torch.uint8, device="cuda")
    sa = torch.empty(128 * K // 32, dtype=torch.uint8, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def step():
        metis.metis_quant_mxfp4(x, qa[:M], sa, tiled=True)
        metis.metis_mxfp4_gemm(qa, sa, qb, sb, y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    wv = ref.mxfp4_quant(w)[0]
    for seed in (1, 2):
        x.copy_(torch.randn(M, K, generator=gen(seed), device="cuda"))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_within(y, *ref.product(ref.mxfp4_quant(x)[0], wv))
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            step()
    side.synchronize()
    assert torch.equal(y, want) and metis.metis_check_device_status() == 0


def test_rows_past_32_bit_offsets(metis):
    """More than 2^32 bytes of x and 2^32 codes; checked at both ends."""
    R, K = 65600, 65536
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    ends = torch.cat((torch.arange(40), torch.arange(R - 90, R))).cuda()
    x[ends] = torch.randn(ends.numel(), K, generator=gen(90), device="cuda").bfloat16()
    q = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty((R + 127) // 128 * 128 * K // 32, dtype=torch.uint8, device="cuda")
    metis.metis_quant_mxfp4(x, q, sf, tiled=True)
    want, c, _ = ref.mxfp4_quant(x[ends])
    atoms = K // 128 * 512
    r = ends.unsqueeze(1)
    b = torch.arange(K // 32, device="cuda").unsqueeze(0)
    assert torch.equal(sf[(r // 128) * atoms + b // 4 * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4], c)
    x.fill_(float("nan"))
    metis.metis_dequant_mxfp4(q, sf, x, tiled=True)
    assert torch.equal(x[ends].double(), want)
    assert bool((x[1000:1100] == 0).all()) and metis.metis_check_device_status() == 0


def test_no_rows(metis):
    def empty(*shape, dtype=torch.uint8):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    metis.metis_quant_mxfp4(empty(0, 128, dtype=torch.bfloat16), empty(0, 64), empty(0))
    metis.metis_dequant_mxfp4(empty(0, 64), empty(0), empty(0, 128, dtype=torch.bfloat16))
    metis.metis_mxfp4_gemm(empty(0, 64), empty(0), empty(128, 64), empty(512), empty(0, 128, dtype=torch.bfloat16))
    assert metis.metis_check_device_status() == 0


def test_binding_refuses_what_the_library_cannot_see(metis):
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(4, 128, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(32, dtype=torch.uint8, device="cuda")
    for args in ((x.half(), q, sf), (x, q[:3], sf), (x, q, sf[:31]), (x[:, ::2], q, sf), (x.cpu(), q, sf)):
        with pytest.raises(ValueError, match="metis_quant_mxfp4"):
            metis.metis_quant_mxfp4(*args)
    with pytest.raises(ValueError, match="too small"):
        metis.metis_quant_mxfp4(x, q, sf, tiled=True)
    y = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    b, s = torch.zeros(128, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1024, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="ceil"):
        metis.metis_mxfp4_gemm(q, s, b, s, y)  # qa without the rows past M
    metis.metis_mxfp4_gemm(b, s, b, s, y)
    assert metis.metis_check_device_status() == 0
