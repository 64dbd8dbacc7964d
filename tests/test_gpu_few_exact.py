"""The few-token routed layers on whole numbers: every product and sum is a
whole number below 2^24, which FP32 holds exactly in any order, so the output
has to be the exact result rounded to BF16 once. h has more bits than a 16-bit
value holds."""
import pytest
import torch

import few_reference as ref
import test_gpu_few_tokens as few

pytestmark = pytest.mark.gpu

# one token and a few (the down-projection's CTAs own output rows); 8 and 16 warps; 8 and 16 slots of
# an expert at a time; rows so long that fewer than 8 slots fit, several passes through an expert
FP8 = [(1, 256, 128, 8, 4), (1, 2048, 1024, 16, 8), (5, 1040, 528, 24, 3), (20, 512, 256, 8, 4), (30, 512, 256, 4, 4),
       (32, 1024, 512, 64, 8), (100, 1024, 512, 48, 8), (6, 128, 4096, 4, 2), (12, 128, 8192, 2, 1), (25, 64, 4096, 2, 2)]
FP4 = [(1, 256, 128, 8, 4), (1, 2048, 1024, 16, 8), (16, 256, 256, 8, 4), (40, 256, 256, 4, 2), (32, 1024, 512, 128, 8),
       (100, 1024, 512, 100, 8), (6, 128, 4096, 4, 2), (12, 128, 8192, 2, 1)]


def whole_layer(fmt, T, H, I, E, k):
    g = few.gen(900 + T + I)
    d = few.layer(fmt, 901 + T + H, T, H, I, E, k)
    d["tw"] = torch.ones(T, k, device="cuda")
    keep = torch.rand(E, H, I, generator=g, device="cuda") < 256 / I  # keeps the sums below 2^24
    if fmt is few.Fp8:
        d["x"] = torch.randint(-127, 128, (T, H), generator=g, device="cuda").bfloat16()
        for p, n, kk, most in (("up", I, H, 8), ("down", H, I, 4)):
            w = torch.randint(-most, most + 1, (E, n, kk), generator=g, device="cuda").float()
            if p == "down":
                w *= keep
            d[p] = (w.to(torch.float8_e4m3fn).view(torch.uint8), torch.ones(E, n, device="cuda"))
    else:
        d["x"] = torch.randint(-63, 64, (T, H), generator=g, device="cuda").bfloat16()
        for p in ("up", "down"):
            q, sf, _ = d[p]
            if p == "down":
                q = q & (15 * keep[..., ::2].byte() + 240 * keep[..., 1::2].byte())
            d[p] = (q, torch.full_like(sf, 0x40), torch.ones(E, device="cuda"))  # block scales of 2
    return d


def check(metis, fmt, shape):
    d = whole_layer(fmt, *shape)
    up, down = fmt.values(*d["up"]), fmt.values(*d["down"])
    y = torch.zeros(d["T"], d["H"], dtype=torch.float64, device="cuda")
    most, h_most = 0.0, 0.0
    for t in range(d["T"]):
        for e in d["ids"][t].tolist():
            x = d["x"][t].double()
            h = up[e] @ x
            y[t] += down[e] @ h
            most = max(most, float((down[e].abs() @ h.abs()).max()), float((up[e].abs() @ x.abs()).max()))
            most, h_most = max(most, float(y[t].abs().max())), max(h_most, float(h.abs().max()))
    assert most < 2 ** 24 and 2 ** 12 < h_most < 2 ** 22
    got = few.run(metis, fmt, d)
    assert metis.metis_check_device_status() == 0
    assert torch.equal(got, y.float().bfloat16())


@pytest.mark.parametrize("shape", FP8, ids=str)
def test_fp8_layer_on_whole_numbers(metis, shape):
    check(metis, few.Fp8, shape)


@pytest.mark.parametrize("shape", FP4, ids=str)
def test_nvfp4_layer_on_whole_numbers(metis, shape):
    check(metis, few.Nvfp4, shape)
