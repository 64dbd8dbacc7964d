"""Default maths for few tokens against plain 64-bit forms: the routed layer
with FP8 and NVFP4 experts, and the NVFP4 weight-only product."""
import os
import subprocess
import sys

import pytest
import torch

import few_reference as ref
from few_reference import assert_within

pytestmark = pytest.mark.gpu

NAN = float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def fp8_weights(g, E, N, K):
    """Every E4M3 code but the NaNs, channel scales over three binades."""
    q = torch.randint(0, 254, (E, N, K), generator=g, device="cuda", dtype=torch.int32)
    q = (q + (q >= 127).int()).to(torch.uint8)  # 0 .. 126, 128 .. 254
    s = torch.exp2(torch.randint(-12, -9, (E, N), generator=g, device="cuda").float()) * \
        (1 + torch.rand(E, N, generator=g, device="cuda"))
    return q, s


def nvfp4_weights(g, E, N, K):
    """Every E2M1 code, block scales over all finite E4M3 values, tiled."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(0, 127, ((E * N + 127) // 128 * 128 * K // 16,), generator=g, device="cuda", dtype=torch.uint8)
    return q, sf, torch.rand(E, generator=g, device="cuda") * 1e-4 + 1e-5


class Fp8:
    name, op, step = "metis_moe_w8a16", "METIS_OP_MOE_W8A16", 16
    weights = staticmethod(fp8_weights)
    values = staticmethod(ref.fp8_values)


class Nvfp4:
    name, op, step = "metis_moe_nvfp4_w4a16", "METIS_OP_MOE_NVFP4_W4A16", 128
    weights = staticmethod(nvfp4_weights)
    values = staticmethod(ref.nvfp4_values)


FORMATS = [Fp8, Nvfp4]
by_format = pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: f.__name__)


def layer(fmt, seed, T, H, I, E, k, ids=None):
    g = gen(seed)
    d = dict(T=T, H=H, I=I, E=E, k=k)
    d["x"] = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    if ids is None:
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
    d["ids"] = ids.to(torch.int32).contiguous()
    d["tw"] = torch.randn(T, k, generator=g, device="cuda")
    d["up"], d["down"] = fmt.weights(g, E, I, H), fmt.weights(g, E, H, I)
    return d


def workspace(metis, fmt, d):
    n = metis.metis_workspace_size(getattr(metis, fmt.op), d["T"], d["I"], d["H"], d["k"], d["E"])
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns


def run(metis, fmt, d, ws=None, y=None):
    y = torch.full((d["T"], d["H"]), NAN, dtype=torch.bfloat16, device="cuda") if y is None else y
    ws = workspace(metis, fmt, d) if ws is None else ws
    getattr(metis, fmt.name)(d["x"], d["ids"], d["tw"], *d["up"], *d["down"], y, ws)
    return y


def expect(fmt, d):
    return ref.moe(d["x"], d["ids"], d["tw"], fmt.values(*d["up"]), fmt.values(*d["down"]))


def check(metis, fmt, d, what=""):
    y = run(metis, fmt, d)
    assert metis.metis_check_device_status() == 0
    assert_within(y, *expect(fmt, d), what)
    return y


FP8_SIZES = [(1, 16, 16, 1, 1), (1, 2048, 1024, 64, 8), (3, 80, 48, 5, 2), (8, 272, 144, 8, 8), (9, 1040, 528, 24, 3),
             (17, 256, 512, 4, 4), (64, 512, 256, 16, 4), (128, 128, 128, 8, 8), (2, 8192, 16, 3, 1),
             (2, 16, 8192, 3, 2), (33, 4096, 1040, 6, 2), (5, 8192, 2064, 3, 2), (40, 2048, 1024, 32, 8),
             (1, 1008, 992, 2, 2), (6, 2048, 1040, 1024, 5), (1, 64, 48, 1024, 1024), (1, 128, 112, 65, 65),
             (1, 128, 112, 64, 64), (16, 80, 32, 64, 64), (4, 8192, 8192, 2, 2), (128, 32, 16, 1, 1)]
FP4_SIZES = [(1, 128, 128, 1, 1), (1, 2048, 1024, 64, 8), (5, 384, 256, 7, 3), (17, 640, 896, 4, 4),
             (64, 1024, 512, 16, 4), (128, 128, 128, 8, 8), (2, 8192, 128, 2, 2), (2, 128, 8192, 2, 2),
             (33, 1152, 1664, 6, 2), (40, 2048, 1024, 32, 8), (3, 256, 128, 1024, 7), (1, 128, 256, 1024, 1024),
             (1, 256, 128, 65, 65), (1, 256, 128, 64, 64), (16, 128, 256, 64, 64), (4, 8192, 8192, 2, 2)]


@pytest.mark.parametrize("T,H,I,E,k", FP8_SIZES)
def test_moe_fp8_sizes(metis, T, H, I, E, k):
    check(metis, Fp8, layer(Fp8, 100 + T + H, T, H, I, E, k))


@pytest.mark.parametrize("T,H,I,E,k", FP4_SIZES)
def test_moe_nvfp4_sizes(metis, T, H, I, E, k):
    check(metis, Nvfp4, layer(Nvfp4, 200 + T + H, T, H, I, E, k))


@by_format
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 25, 100])
def test_moe_every_token_on_one_expert(metis, fmt, T):
    """All slots on expert 2 of 4: one long segment, the other experts empty."""
    d = layer(fmt, 300 + T, T, 256, 384, 4, 1, torch.full((T, 1), 2, device="cuda"))
    check(metis, fmt, d)


@by_format
@pytest.mark.parametrize("T,k", [(1, 4), (3, 3), (128, 8)])
def test_moe_expert_named_twice(metis, fmt, T, k):
    """The same expert in several slots of a token: each slot counts with its own weight."""
    ids = torch.arange(T * k, device="cuda").view(T, k) // 2 % 8
    check(metis, fmt, layer(fmt, 400 + T, T, 256, 256, 8, k, ids))


@by_format
def test_moe_ids_of_no_expert(metis, fmt):
    """Ids outside [0, E) drop their slot and are recorded; a token without any expert gets zeros."""
    ids = torch.tensor([[0, -1, 3], [-1, -1, -1], [4, 1, 2], [2 ** 31 - 1, -2 ** 31, 0], [5, 5, 5]], device="cuda")
    d = layer(fmt, 500, 5, 256, 128, 4, 3, ids)
    y = run(metis, fmt, d)
    with pytest.raises(AssertionError):
        assert metis.metis_check_device_status() == 0
    assert metis.metis_check_device_status() == 0  # cleared by the read above
    assert_within(y, *expect(fmt, d))
    assert bool((y[1] == 0).all()) and bool((y[4] == 0).all())


@by_format
def test_moe_no_expert_at_all(metis, fmt):
    d = layer(fmt, 501, 3, 256, 128, 4, 2, torch.full((3, 2), -1, device="cuda"))
    y = run(metis, fmt, d)
    assert metis.metis_check_device_status() == metis.METIS_ERR_INVALID_ARG
    assert bool((y == 0).all())


@by_format
def test_moe_wide_range_and_zero_rows(metis, fmt):
    """Tokens of very different magnitude, elements spread over 60 binades, an all-zero token."""
    d = layer(fmt, 510, 9, 512, 256, 4, 2)
    g = gen(511)
    d["x"] = (d["x"].float() * torch.exp2(torch.randint(-40, 20, (9, 512), generator=g, device="cuda").float())).bfloat16()
    d["x"][3] = 0
    d["x"][4] *= 2.0 ** 80
    d["x"][5] *= 2.0 ** -90
    y = check(metis, fmt, d)
    assert bool((y[3] == 0).all())


@by_format
def test_moe_nonfinite_token_stays_alone(metis, fmt):
    d = layer(fmt, 520, 10, 256, 256, 3, 2)
    clean = run(metis, fmt, d)
    d["x"] = d["x"].clone()
    d["x"][2, 17] = float("inf")
    d["x"][6, 255] = NAN
    y = run(metis, fmt, d)
    assert metis.metis_check_device_status() == 0
    keep = [0, 1, 3, 4, 5, 7, 8, 9]
    assert torch.equal(y[keep], clean[keep])
    assert not bool(torch.isfinite(y[2]).any()) and not bool(torch.isfinite(y[6]).any())


def test_moe_fp8_nan_weight_stays_in_its_channel(metis):
    d = layer(Fp8, 530, 4, 256, 128, 2, 2)
    clean = run(metis, Fp8, d)
    d["down"][0][1, 37, 5] = 0x7F
    y = run(metis, Fp8, d)
    assert bool(torch.isnan(y[:, 37]).all())
    other = torch.arange(256, device="cuda") != 37
    assert torch.equal(y[:, other], clean[:, other])


@by_format
def test_moe_zero_and_infinite_routing_weights(metis, fmt):
    d = layer(fmt, 540, 4, 256, 128, 8, 4)
    d["tw"][1] = 0
    y = check(metis, fmt, d)
    assert bool((y[1] == 0).all())
    d["tw"][2, 0] = NAN
    y = run(metis, fmt, d)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isfinite(y[3]).all())


@by_format
def test_moe_bits_repeat_and_do_not_depend_on_the_workspace(metis, fmt):
    d = layer(fmt, 550, 48, 512, 384, 8, 4)
    a = run(metis, fmt, d)
    ws = workspace(metis, fmt, d).zero_()
    b = run(metis, fmt, d, ws)
    for _ in range(5):
        assert torch.equal(run(metis, fmt, d, ws), a)  # the last call's contents are in it
    assert torch.equal(a, b)


@by_format
def test_moe_leaves_rows_behind_the_last_token(metis, fmt):
    d = layer(fmt, 560, 5, 256, 128, 4, 2)
    buf = torch.full((8, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(metis, fmt, d)
    guard = torch.cat((ws, torch.full((4096,), 0xA5, dtype=torch.uint8, device="cuda")))
    run(metis, fmt, d, guard, buf[:5])
    assert metis.metis_check_device_status() == 0
    assert bool((buf[5:] == 7.0).all()) and bool((guard[ws.numel():] == 0xA5).all())


@by_format
def test_moe_captured_replayed_and_on_two_streams(metis, fmt):
    """A captured call sees new inputs at each replay (other experts, other counts); calls on two
    streams with a workspace each do not disturb one another."""
    a, b = layer(fmt, 570, 6, 512, 256, 8, 2), layer(fmt, 571, 20, 512, 256, 8, 3)
    ya, yb = run(metis, fmt, a), run(metis, fmt, b)
    torch.cuda.synchronize()
    wsa, wsb = workspace(metis, fmt, a), workspace(metis, fmt, b)
    oa, ob = torch.empty_like(ya), torch.empty_like(yb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(metis, fmt, a, wsa, oa)
    c = layer(fmt, 572, 6, 512, 256, 8, 2, torch.tensor([[7, 1]] * 6, device="cuda"))
    yc = run(metis, fmt, {**a, "x": c["x"], "ids": c["ids"], "tw": c["tw"]})
    for x, ids, tw, want in ((a["x"].clone(), a["ids"].clone(), a["tw"].clone(), ya), (c["x"], c["ids"], c["tw"], yc)):
        a["x"].copy_(x), a["ids"].copy_(ids), a["tw"].copy_(tw)
        for _ in range(3):
            oa.fill_(NAN)
            graph.replay()
            assert torch.equal(oa, want)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    want = run(metis, fmt, a)
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            run(metis, fmt, a, wsa, oa)
        with torch.cuda.stream(s2):
            run(metis, fmt, b, wsb, ob)
    torch.cuda.synchronize()
    assert torch.equal(oa, want) and torch.equal(ob, yb)
    assert metis.metis_check_device_status() == 0


def test_moe_router_to_layer_to_projection(metis):
    """As a decode step uses them: router top-k, the routed layer in both formats, a 4-bit projection
    of its output, one stream after another on the same workspace."""
    T, H, I, E, k, N = 12, 512, 256, 16, 4, 384
    g = gen(580)
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, k, device="cuda")
    q, sf, gs = nvfp4_weights(g, 1, N, H)
    for fmt in FORMATS:
        d = layer(fmt, 581, T, H, I, E, k)
        metis.metis_moe_route_topk(logits, ids, tw, bias)
        d["ids"], d["tw"] = ids, tw
        y = run(metis, fmt, d)
        z = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        metis.metis_nvfp4_w4a16_gemm(y, q[0], sf, gs, z)
        assert metis.metis_check_device_status() == 0
        assert torch.equal(ids.long().sort(dim=1).values, (logits + bias).topk(k, dim=1).indices.sort(dim=1).values)
        assert_within(y, *expect(fmt, d), fmt.__name__)
        assert_within(z, *ref.product(y, ref.nvfp4_values(q, sf, gs)[0]), "projection")


@pytest.mark.parametrize("N,K", [(128, 64), (256, 192), (384, 2048), (128, 8192), (256, 12352), (128, 65536),
                                 (2176, 4096), (6144, 320)])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 37, 64, 65, 129, 256, 300])
def test_w4a16_sizes(metis, M, N, K):
    g = gen(600 + M + N)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, sf, gs = nvfp4_weights(g, 1, N, K)
    n = metis.metis_workspace_size(metis.METIS_OP_NVFP4_W4A16, M, N, K)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    y = torch.full((M + 1, N), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y[:M], ws)
    assert metis.metis_check_device_status() == 0
    assert_within(y[:M], *ref.product(x, ref.nvfp4_values(q, sf, gs)[0]))
    assert bool(torch.isnan(y[M]).all())


@pytest.mark.parametrize("M", [3, 40, 200])
def test_w4a16_special_rows_capture_and_streams(metis, M):
    g = gen(700 + M)
    N, K = 512, 1088
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    x[1] = 0
    q, sf, gs = nvfp4_weights(g, 1, N, K)
    n = metis.metis_workspace_size(metis.METIS_OP_NVFP4_W4A16, M, N, K)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    clean = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, clean, ws)
    assert bool((clean[1] == 0).all())
    x[0, 5] = NAN
    y = torch.empty_like(clean)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[0]).all()) and torch.equal(y[1:], clean[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y.zero_(), ws)
    side.synchronize()
    assert torch.equal(y[1:], clean[1:])
    assert metis.metis_check_device_status() == 0


@pytest.mark.parametrize("M", [3000, 3001, 3300])
def test_w4a16_around_the_widening(metis, M):
    """Past 3000 tokens the weights are widened into the workspace; the rows of both forms agree."""
    N, K = 384, 1088
    g = gen(650)
    x = torch.randn(3300, K, generator=g, device="cuda").bfloat16()[:M]
    q, sf, gs = nvfp4_weights(g, 1, N, K)
    n = metis.metis_workspace_size(metis.METIS_OP_NVFP4_W4A16, M, N, K)
    assert (n > 0) == (M > 3000)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    y = torch.full((M + 1, N), NAN, dtype=torch.bfloat16, device="cuda")
    metis.metis_nvfp4_w4a16_gemm(x, q[0], sf, gs, y[:M], ws)
    assert metis.metis_check_device_status() == 0
    assert_within(y[:M], *ref.product(x, ref.nvfp4_values(q, sf, gs)[0]))
    assert bool(torch.isnan(y[M]).all())


@by_format
def test_moe_weights_past_32_bit_offsets(metis, fmt):
    """More than 2^32 codes per projection, the chosen experts at both ends."""
    T, H, I, E, k = 5, 2048, 2176, 1024, 3
    chosen = torch.tensor([0, 1, 511, 1022, 1023], device="cuda")
    g = gen(660)
    pick = torch.rand(T, 5, generator=g, device="cuda").topk(k, dim=1).indices
    small = layer(fmt, 661, T, H, I, 5, k, pick)
    big = {**small, "E": E, "ids": chosen[pick].to(torch.int32).contiguous()}
    for p in ("up", "down"):
        big[p] = tuple(torch.zeros(E * (t.numel() // 5), dtype=t.dtype, device="cuda") for t in small[p])
        big[p] = tuple(t.view(E, *u.shape[1:]) if u.shape[0] == 5 else t for t, u in zip(big[p], small[p]))
        for dst, src in zip(big[p], small[p]):
            dst.view(E, -1)[chosen] = src.view(5, -1)
    y = run(metis, fmt, big)
    assert metis.metis_check_device_status() == 0
    assert_within(y, *expect(fmt, small))


FIRST_CALLS_CAPTURED = """
import torch
from moe_gemm_token_b200 import metis
def u8(*s): return torch.randint(0, 120, s, device="cuda", dtype=torch.uint8)
T, H, I, E, k, N = 3, 256, 128, 4, 2, 384
x = torch.randn(3100, H, device="cuda").bfloat16()
ids = torch.tensor([[0, 1], [2, 3], [1, 1]], dtype=torch.int32, device="cuda")
tw, g, one = torch.ones(T, k, device="cuda"), torch.full((E,), 1e-3, device="cuda"), torch.ones(1, device="cuda")
fp8 = (u8(E, I, H), torch.full((E, I), 1e-3, device="cuda"), u8(E, H, I), torch.full((E, H), 1e-3, device="cuda"))
fp4 = (u8(E, I, H // 2), u8(E * I * H // 16), g, u8(E, H, I // 2), u8(E * H * I // 16), g)
w, wsf = u8(N, H // 2), u8(N * H // 16)
ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
q, sf = torch.zeros(128, H // 2, dtype=torch.uint8, device="cuda"), torch.empty(128 * H // 32, dtype=torch.uint8, device="cuda")
out = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
       for m, n in ((T, H), (T, H), (3, N), (40, N), (3100, N), (40, H), (40, 128))]
metis.load()
def run():
    metis.metis_moe_w8a16(x[:T], ids, tw, *fp8, out[0], ws)
    metis.metis_moe_nvfp4_w4a16(x[:T], ids, tw, *fp4, out[1], ws)
    for y in out[2:5]:
        metis.metis_nvfp4_w4a16_gemm(x[:len(y)], w, wsf, one, y, ws)
    metis.metis_quant_mxfp4(x[:40], q[:40], sf, tiled=True)
    metis.metis_dequant_mxfp4(q[:40], sf, out[5], tiled=True)
    metis.metis_mxfp4_gemm(q, sf, q, sf, out[6])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
for y in out:
    y.fill_(float("nan"))
graph.replay()
torch.cuda.synchronize()
first = [y.clone() for y in out]
run()
assert all(torch.equal(a, b) for a, b in zip(first, out)) and metis.metis_check_device_status() == 0
"""


def test_first_calls_of_a_process_captured_together():
    """Every operator's first call of a process inside one capture; the replay equals the calls after it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@by_format
def test_no_tokens(metis, fmt):
    d = layer(fmt, 670, 0, 256, 128, 4, 2, torch.empty(0, 2, device="cuda"))
    assert run(metis, fmt, d, torch.empty(0, dtype=torch.uint8, device="cuda")).shape == (0, 256)
    q, sf, gs = nvfp4_weights(gen(671), 1, 128, 64)
    metis.metis_nvfp4_w4a16_gemm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), q[0], sf, gs,
                                 torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
    assert metis.metis_check_device_status() == 0


@pytest.mark.parametrize("argv", [["moefew", "3"], ["moe4few", "40"], ["w4a16", "5", "256", "192"],
                                  ["w4a16", "70", "256", "192"], ["quantmx", "9", "256"], ["gemmmx", "9", "256", "384"]],
                         ids=lambda a: "-".join(a))
def test_drive_commands(metis, argv, capsys):
    from moe_gemm_token_b200 import drive
    assert drive.main([*argv, "--calls", "2"]) == 0
    assert "device status 0" in capsys.readouterr().out


@by_format
def test_moe_binding_refuses_what_the_library_cannot_see(metis, fmt):
    d = layer(fmt, 800, 4, 256, 128, 4, 2)
    name = fmt.name
    ws = workspace(metis, fmt, d)
    for key, bad in (("x", d["x"].float()), ("x", d["x"][:, ::2]), ("ids", d["ids"].long()),
                     ("ids", d["ids"][:2]), ("tw", d["tw"].double()), ("x", d["x"].cpu()),
                     ("x", torch.empty(256, 4, dtype=torch.bfloat16, device="cuda").t())):
        with pytest.raises(ValueError, match=name):
            run(metis, fmt, {**d, key: bad}, ws, torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(metis.MetisError):
        run(metis, fmt, d, ws[:-256])
    with pytest.raises(metis.MetisError):
        run(metis, fmt, d, torch.cat((ws, ws))[16:])  # misaligned
