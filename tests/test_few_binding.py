"""The binding refuses codes and scales whose elements are not the bytes that the
kernels read: a check that the C entry points cannot make. The tensors are on
the CPU; what is refused for its type never gets to the check of the device."""
import pytest
import torch

from moe_gemm_token_b200 import metis

T, k, E, H, I, N = 3, 2, 4, 256, 128, 384
WRONG = [torch.bfloat16, torch.int32, torch.float8_e5m2]


def zeros(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=torch.uint8).to(dtype)


def layer(packed, **types):
    """Arguments of a routed layer; `types` gives another type to one of the arrays."""
    bf, f = torch.bfloat16, torch.float32
    d = dict(x=zeros(T, H, dtype=bf), ids=zeros(T, k, dtype=torch.int32), tw=zeros(T, k, dtype=f),
             w_up=zeros(E, I, H // packed), w_down=zeros(E, H, I // packed))
    if packed == 1:
        d.update(s_up=zeros(E, I, dtype=f), s_down=zeros(E, H, dtype=f))
    else:
        d.update(sf_up=zeros(E * I * H // 16), sf_down=zeros(E * H * I // 16), g_up=zeros(E, dtype=f), g_down=zeros(E, dtype=f))
    for name, dtype in types.items():
        d[name] = zeros(*d[name].shape, dtype=dtype)
    y, ws = zeros(T, H, dtype=bf), zeros(1 << 16)
    if packed == 1:
        return metis.metis_moe_w8a16, (d["x"], d["ids"], d["tw"], d["w_up"], d["s_up"], d["w_down"], d["s_down"], y, ws)
    return metis.metis_moe_nvfp4_w4a16, (d["x"], d["ids"], d["tw"], d["w_up"], d["sf_up"], d["g_up"], d["w_down"],
                                         d["sf_down"], d["g_down"], y, ws)


def refused(call):
    fn, args = call
    with pytest.raises(ValueError, match=f"{fn.__name__}.*bytes"):
        fn(*args)


@pytest.mark.parametrize("dtype", WRONG, ids=str)
def test_layers_refuse_codes_of_another_type(dtype):
    for name in ("w_up", "w_down"):
        refused(layer(1, **{name: dtype}))
        refused(layer(2, **{name: dtype}))
    for name in ("sf_up", "sf_down"):
        refused(layer(2, **{name: dtype}))


@pytest.mark.parametrize("dtype", WRONG, ids=str)
def test_products_and_quantizer_refuse_codes_of_another_type(dtype):
    bf = torch.bfloat16
    x, y = zeros(T, H, dtype=bf), zeros(T, N, dtype=bf)
    qb, sfb, g = zeros(N, H // 2), zeros(N * H // 16), zeros(1, dtype=torch.float32)
    refused((metis.metis_nvfp4_w4a16_gemm, (x, zeros(N, H // 2, dtype=dtype), sfb, g, y)))
    refused((metis.metis_nvfp4_w4a16_gemm, (x, qb, zeros(N * H // 16, dtype=dtype), g, y)))
    qa, sfa = zeros(128, H // 2), zeros(128 * H // 32)
    good = (qa, sfa, qb, zeros(N * H // 32), y)
    for i in range(4):
        bad = tuple(zeros(*t.shape, dtype=dtype) if j == i else t for j, t in enumerate(good))
        refused((metis.metis_mxfp4_gemm, bad))
    q, sf, v = zeros(T, H // 2), zeros(T, H // 32), zeros(T, H, dtype=bf)
    for fn, args in ((metis.metis_quant_mxfp4, lambda a, b: (x, a, b)), (metis.metis_dequant_mxfp4, lambda a, b: (a, b, v))):
        refused((fn, args(zeros(T, H // 2, dtype=dtype), sf)))
        refused((fn, args(q, zeros(T, H // 32, dtype=dtype))))


def test_the_types_of_the_formats_are_taken():
    """What is accepted gets to the check of the device (or of a GPU's presence)."""
    for call in (layer(1, w_up=torch.float8_e4m3fn, w_down=torch.float8_e4m3fn), layer(2, sf_up=torch.float8_e4m3fn),
                 (metis.metis_quant_mxfp4, (zeros(T, H, dtype=torch.bfloat16), zeros(T, H // 2),
                                            zeros(T, H // 32).view(torch.float8_e8m0fnu)))):
        with pytest.raises((ValueError, RuntimeError, AssertionError)) as e:
            call[0](*call[1])
        assert "bytes" not in str(e.value)
