"""Refusals of the few-token default-maths operators and of the MXFP4 operators:
argument errors are found on the host before anything is launched, so these
calls need no GPU (and would not survive being launched: the pointers are made up)."""
import pytest

from moe_gemm_token_b200 import build as libbuild
from moe_gemm_token_b200 import metis

BAD, UNSUPPORTED, OK = metis.METIS_ERR_INVALID_ARG, metis.METIS_ERR_UNSUPPORTED, metis.METIS_OK
P = 0x10000        # aligned to everything that is asked for
BIG = 1 << 40      # more workspace than anything needs


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return metis.load()


def message(lib):
    return lib.metis_last_error().decode()


def w8a16(lib, T=4, k=2, E=8, H=64, I=32, act=0, ws=P, size=BIG, **ptr):
    p = dict(x=P, ids=P, tw=P, wu=P, su=P, wd=P, sd=P, y=P)
    p.update(ptr)
    return lib.metis_moe_w8a16(p["x"], p["ids"], p["tw"], T, k, E, H, I, p["wu"], p["su"], p["wd"], p["sd"], act,
                               p["y"], ws, size, None)


def w4a16(lib, T=4, k=2, E=8, H=256, I=128, act=0, ws=P, size=BIG, **ptr):
    p = dict(x=P, ids=P, tw=P, wu=P, su=P, gu=P, wd=P, sd=P, gd=P, y=P)
    p.update(ptr)
    return lib.metis_moe_nvfp4_w4a16(p["x"], p["ids"], p["tw"], T, k, E, H, I, p["wu"], p["su"], p["gu"], p["wd"],
                                     p["sd"], p["gd"], act, p["y"], ws, size, None)


LAYERS = [(w8a16, metis.METIS_OP_MOE_W8A16, 64, 32, 16), (w4a16, metis.METIS_OP_MOE_NVFP4_W4A16, 256, 128, 128)]


@pytest.mark.parametrize("call,op,H,I,step", LAYERS, ids=["fp8", "nvfp4"])
def test_routed_layers_refuse(lib, call, op, H, I, step):
    for bad in (dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(E=1025), dict(H=H + step // 2), dict(H=0), dict(H=8192 + step),
                dict(I=I + step // 2), dict(I=0), dict(I=8192 + step)):
        assert call(lib, **bad) == BAD, bad
        assert "multiples of" in message(lib)
    assert call(lib, act=1) == UNSUPPORTED
    assert call(lib, T=129) == UNSUPPORTED and "few tokens" in message(lib)
    assert call(lib, T=128, k=9, E=16) == UNSUPPORTED
    assert call(lib, T=1 << 40, k=1) == UNSUPPORTED
    need = metis.metis_workspace_size(op, 4, I, H, 2, 8)
    assert need > 0 and need % 256 == 0
    for ws, size in ((None, BIG), (P, need - 1), (P + 128, need)):
        assert call(lib, ws=ws, size=size) == BAD and str(need) in message(lib)
    for name in ("x", "ids", "tw", "wu", "su", "wd", "sd", "y"):
        assert call(lib, **{name: None}) == BAD and "null" in message(lib)
    for name in ("x", "wu", "wd", "y"):
        assert call(lib, **{name: P + 8}) == BAD and "aligned" in message(lib)
    for name in ("ids", "tw", "su", "sd"):
        assert call(lib, **{name: P + 2}) == BAD and "aligned" in message(lib)
    # no tokens: nothing to do, whatever the pointers
    assert call(lib, T=0, x=None, y=None, ws=None, size=0) == OK and message(lib) == ""


def test_workspace_of_the_routed_layers(lib):
    for op in (metis.METIS_OP_MOE_W8A16, metis.METIS_OP_MOE_NVFP4_W4A16):
        # h [S, I] and o [S, H] in FP32, each rounded up to 256 bytes
        assert metis.metis_workspace_size(op, 3, 1040, 528, 5, 8) == (4 * 15 * 1040 + 255) // 256 * 256 + \
            (4 * 15 * 528 + 255) // 256 * 256
        assert metis.metis_workspace_size(op, 3, 1040, 528, 0, 8) == 0
        assert metis.metis_workspace_size(op, -1, 1040, 528, 5, 8) == 0


def test_nvfp4_product_refuses(lib):
    def call(M=4, N=256, K=128, ws=None, size=0, x=P, qb=P, sfb=P, gb=P, y=P):
        return lib.metis_nvfp4_w4a16_gemm(x, qb, sfb, gb, y, M, N, K, ws, size, None)

    for bad in (dict(M=-1), dict(M=1 << 31), dict(N=64), dict(N=200), dict(N=(1 << 20) + 128), dict(K=32), dict(K=96),
                dict(K=65536 + 64)):
        assert call(**bad) == BAD, bad
    for name in ("x", "qb", "sfb", "gb", "y"):
        assert call(**{name: None}) == BAD and "null" in message(lib)
    for name in ("x", "qb", "sfb", "y"):
        assert call(**{name: P + 8}) == BAD and "aligned" in message(lib)
    assert call(gb=P + 2) == BAD
    assert call(M=0, x=None, y=None) == OK
    op = metis.METIS_OP_NVFP4_W4A16
    assert metis.metis_workspace_size(op, 3000, 256, 128) == 0
    need = metis.metis_workspace_size(op, 3001, 256, 128)
    assert need == 2 * 256 * 128 + 4 * 256
    for ws, size in ((None, BIG), (P, need - 1), (P + 16, need)):
        assert call(M=3001, ws=ws, size=size) == BAD and str(need) in message(lib)


def test_mxfp4_quantizer_refuses(lib):
    A, F = metis.METIS_A_BF16, metis.METIS_A_F32

    def call(kind=A, R=4, K=128, ldx=None, layout=0, x=P, q=P, sf=P):
        return lib.metis_quant_mxfp4(x, kind, R, K, K if ldx is None else ldx, q, sf, layout, None)

    for bad in (dict(kind=0), dict(kind=3), dict(R=-1), dict(R=1 << 31), dict(K=0), dict(K=48), dict(K=65536 + 32),
                dict(layout=2), dict(layout=1, K=96), dict(ldx=120), dict(x=None), dict(q=None), dict(sf=None),
                dict(x=P + 8), dict(q=P + 8), dict(layout=1, sf=P + 2), dict(ldx=132), dict(kind=F, ldx=130)):
        assert call(**bad) == BAD, bad
        assert message(lib)
    assert call(R=0, x=None, q=None, sf=None) == OK


def test_mxfp4_reader_refuses(lib):
    def call(R=4, K=128, layout=0, q=P, sf=P, y=P):
        return lib.metis_dequant_mxfp4(q, sf, layout, R, K, y, None)

    for bad in (dict(R=-1), dict(K=48), dict(layout=7), dict(layout=1, K=160), dict(q=None), dict(sf=None), dict(y=None),
                dict(q=P + 8), dict(y=P + 8), dict(layout=1, sf=P + 1)):
        assert call(**bad) == BAD, bad
    assert call(R=0, q=None, sf=None, y=None) == OK


def test_mxfp4_product_refuses(lib):
    def call(M=4, N=256, K=256, qa=P, sa=P, qb=P, sb=P, y=P):
        return lib.metis_mxfp4_gemm(qa, sa, qb, sb, y, M, N, K, None)

    for bad in (dict(M=-1), dict(M=(1 << 30) + 1), dict(N=64), dict(N=192), dict(N=(1 << 20) + 128), dict(K=64), dict(K=192),
                dict(K=65536 + 128)):
        assert call(**bad) == BAD, bad
    for name in ("qa", "sa", "qb", "sb", "y"):
        assert call(**{name: None}) == BAD and "null" in message(lib)
        assert call(**{name: P + 8}) == BAD and "aligned" in message(lib)
    assert call(M=0, qa=None, y=None) == OK


def test_well_formed_calls_fail_loudly_without_a_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert w8a16(lib) == metis.METIS_ERR_CUDA and message(lib)
    assert w4a16(lib) == metis.METIS_ERR_CUDA
    assert lib.metis_nvfp4_w4a16_gemm(P, P, P, P, P, 4, 256, 128, None, 0, None) == metis.METIS_ERR_CUDA
    assert lib.metis_quant_mxfp4(P, metis.METIS_A_BF16, 4, 128, 128, P, P, 0, None) == metis.METIS_ERR_CUDA
    assert lib.metis_dequant_mxfp4(P, P, 0, 4, 128, P, None) == metis.METIS_ERR_CUDA
    assert lib.metis_mxfp4_gemm(P, P, P, P, P, 4, 256, 256, None) == metis.METIS_ERR_CUDA
