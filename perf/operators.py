"""Measured cases of the default-maths operators for few tokens and of the MXFP4 operators.

Operators (``kind`` of a case) and what they compute:

``moe_fp8``    routed experts with E4M3 weights [E, I, H] / [E, H, I] and one FP32 scale per
               output channel, default maths, up to 128 tokens:
               y[t] = sum_j topk_w[t, j] * W_down[e] (W_up[e] x[t]),  e = topk_ids[t, j].
``moe_nvfp4``  the same with NVFP4 experts: E2M1 codes, an E4M3 scale per 16 inputs in the tensor
               cores' tiled order, an FP32 scale per expert.
``w4a16``      y = x W^T with NVFP4 weights and BF16 activations, one token to a long prompt.
``mx_quant``   MXFP4 quantisation of rows (E2M1 codes, a power-of-two scale per 32 elements) and
               reading the values back as BF16.
``mx_gemm``    product of two MXFP4 matrices, BF16 out.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one stream's decode step through a routed layer (the repository's routed workload's sizes)
        dict(name="moe_fp8_1tok", kind="moe_fp8", T=1, H=2048, I=1024, E=64, topk=8),
        # 32 streams decoding together: nearly every expert is read, a few rows each
        dict(name="moe_fp8_32tok", kind="moe_fp8", T=32, H=2048, I=1024, E=64, topk=8),
        # odd sizes: neither projection a multiple of 32 or 128 elements, few experts
        dict(name="moe_fp8_5tok_odd", kind="moe_fp8", T=5, H=1040, I=528, E=24, topk=3),
        # one stream, 4-bit experts
        dict(name="moe_nvfp4_1tok", kind="moe_nvfp4", T=1, H=2048, I=1024, E=64, topk=8),
        # 64 streams, latent width 1024, many small experts, top-4
        dict(name="moe_nvfp4_64tok", kind="moe_nvfp4", T=64, H=1024, I=512, E=128, topk=4),
        # one stream's decode step through a 4-bit projection (the repository's decode sizes)
        dict(name="w4a16_1x14336x4096", kind="w4a16", M=1, N=14336, K=4096),
        # an odd number of streams
        dict(name="w4a16_37x6144x2048", kind="w4a16", M=37, N=6144, K=2048),
        # a whole prompt
        dict(name="w4a16_4096x6144x2048", kind="w4a16", M=4096, N=6144, K=2048),
        # a few decoded rows, where launches count
        dict(name="mx_quant_7x2048_f32", kind="mx_quant", R=7, K=2048, f32=True),
        # a large activation or weight matrix
        dict(name="mx_quant_8192x8192", kind="mx_quant", R=8192, K=8192, f32=False),
        # 16 streams
        dict(name="mx_gemm_16x6144x2048", kind="mx_gemm", M=16, N=6144, K=2048),
        # the large square product
        dict(name="mx_gemm_8192x8192x8192", kind="mx_gemm", M=8192, N=8192, K=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("moe_fp8", "moe_nvfp4", "w4a16", "mx_quant", "mx_gemm"))
    if kind in ("moe_fp8", "moe_nvfp4"):
        step = 16 if kind == "moe_fp8" else 128
        H = step * max(1, _log(rng, 512, 4096) // step)
        I = step * max(1, _log(rng, 256, 2048) // step)
        E = max(4, min(_log(rng, 8, 192), (1 << 28) // (2 * H * I)))
        topk = rng.randint(1, min(8, E))
        return dict(kind=kind, T=_log(rng, 1, 96), H=H, I=I, E=E, topk=topk)
    if kind == "w4a16":
        N = 128 * max(1, _log(rng, 256, 14336) // 128)
        K = 64 * max(1, _log(rng, 256, 8192) // 64)
        M = _log(rng, 1, 4096)
        while M * N * K > 4096 * 6144 * 2048:
            M = max(1, M // 2)
        return dict(kind=kind, M=M, N=N, K=K)
    if kind == "mx_quant":
        K = 32 * max(1, _log(rng, 64, 8192) // 32)
        return dict(kind=kind, R=_log(rng, 1, 8192), K=K, f32=rng.random() < 0.4)
    N = 128 * max(1, _log(rng, 256, 8192) // 128)
    K = 128 * max(1, _log(rng, 256, 8192) // 128)
    return dict(kind=kind, M=_log(rng, 1, 8192), N=N, K=K)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _fp8_weights(g, E, N, K):
    """N(0, 0.02) weights rounded to E4M3 per output channel: codes [E, N, K], scales [E, N]."""
    w = torch.randn(E, N, K, generator=g, device="cuda") * 0.02
    s = w.abs().amax(dim=2) / 448.0
    return (w / s.unsqueeze(2)).to(torch.float8_e4m3fn), s


def _nvfp4_weights(g, E, N, K):
    """Codes [E, N, K/2], E4M3 block scales between 2^-3 and 2^2 in the tiled order, a scale per expert."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(32, 73, (E * N // 128, K // 64, 512), generator=g, device="cuda", dtype=torch.uint8)
    return q, sf, torch.rand(E, generator=g, device="cuda") * 0.004 + 0.002


def _mxfp4(g, R, K):
    """Codes [R padded to 128 rows, K/2] and E8M0 scales between 2^-6 and 2^-1 in the tiled order."""
    Rp = (R + 127) // 128 * 128
    q = torch.randint(0, 256, (Rp, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    return q, torch.randint(121, 127, (Rp // 128, K // 128, 512), generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    k = c["kind"]
    if k in ("moe_fp8", "moe_nvfp4"):
        T, H, I, E, n = c["T"], c["H"], c["I"], c["E"], c["topk"]
        c["x"] = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        top = torch.randn(T, E, generator=g, device="cuda").softmax(dim=1).topk(n, dim=1)
        c["ids"] = top.indices.to(torch.int32)
        c["tw"] = top.values / top.values.sum(dim=1, keepdim=True)
        make = _fp8_weights if k == "moe_fp8" else _nvfp4_weights
        c["up"], c["down"] = make(g, E, I, H), make(g, E, H, I)
        c["y"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    elif k == "w4a16":
        c["x"] = torch.randn(c["M"], c["K"], generator=g, device="cuda").bfloat16()
        c["w"] = _nvfp4_weights(g, 1, c["N"], c["K"])
        c["y"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device="cuda")
    elif k == "mx_quant":
        R, K = c["R"], c["K"]
        x = torch.randn(R, K, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device="cuda").float())
        c["x"] = x if c["f32"] else x.bfloat16()
        c["q"] = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda")
        c["sf"] = torch.empty(R, K // 32, dtype=torch.uint8, device="cuda")
        c["y"] = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    else:
        c["a"], c["b"] = _mxfp4(g, c["M"], c["K"]), _mxfp4(g, c["N"], c["K"])
        c["y"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device="cuda")
    return c


# ------------------------------------------------------------------ the framework's calls

def _workspace(s, metis, op, m, n, k, topk=0, experts=0):
    """The workspace that a program keeps for a layer, made on first use."""
    if "ws" not in s:
        size = metis.metis_workspace_size(op, m, n, k, topk, experts)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return s["ws"]


def _run_own(s):
    from moe_gemm_token_b200 import metis

    k, y = s["kind"], s["y"]
    if k == "moe_fp8":
        ws = _workspace(s, metis, metis.METIS_OP_MOE_W8A16, s["T"], s["I"], s["H"], s["topk"], s["E"])
        metis.metis_moe_w8a16(s["x"], s["ids"], s["tw"], *s["up"], *s["down"], y, ws)
    elif k == "moe_nvfp4":
        ws = _workspace(s, metis, metis.METIS_OP_MOE_NVFP4_W4A16, s["T"], s["I"], s["H"], s["topk"], s["E"])
        metis.metis_moe_nvfp4_w4a16(s["x"], s["ids"], s["tw"], *s["up"], *s["down"], y, ws)
    elif k == "w4a16":
        ws = _workspace(s, metis, metis.METIS_OP_NVFP4_W4A16, s["M"], s["N"], s["K"])
        metis.metis_nvfp4_w4a16_gemm(s["x"], s["w"][0][0], s["w"][1], s["w"][2], y, ws)
    elif k == "mx_quant":
        metis.metis_quant_mxfp4(s["x"], s["q"], s["sf"])
        metis.metis_dequant_mxfp4(s["q"], s["sf"], y)
    else:
        metis.metis_mxfp4_gemm(*s["a"], s["b"][0][:s["N"]], s["b"][1], y)
    return y


# ------------------------------------------------------------------ the plain form

def _e2m1(q):
    """Packed codes [..., K/2] -> values [..., K] (low nibble first), FP32."""
    lut = torch.tensor(E2M1, device=q.device)
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(*q.shape[:-1], 2 * q.shape[-1])
    return lut[v.int()]


def _untile(sf, per_row):
    """Tiled scales [rows / 128, chunks, 512] -> [rows, 4 * chunks] bytes, row 32 q + l of an atom at byte 16 l + 4 q."""
    a, c, _ = sf.shape
    return sf.view(a, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(a * 128, 4 * c)[:, :per_row]


def _nvfp4_values(q, sf, g):
    """NVFP4 weights [E, N, K/2] as FP32 [E, N, K]."""
    E, N, K = q.shape[0], q.shape[1], 2 * q.shape[2]
    s = _untile(sf, K // 16).contiguous().view(torch.float8_e4m3fn).float().view(E, N, K // 16, 1)
    v = _e2m1(q).view(E, N, K // 16, 16) * s
    return v.view(E, N, K) * g.view(E, 1, 1)


def _moe(s, w_up, w_down, pick):
    """Few slots: each slot with its own expert's weights; else every expert with every token."""
    T, k = s["ids"].shape
    ids = s["ids"].long()
    x = s["x"].float()
    if pick:
        h = torch.bmm(w_up, x.repeat_interleave(k, dim=0).unsqueeze(2))
        o = torch.bmm(w_down, h).view(T, k, -1)
    else:
        h = torch.matmul(x, w_up.transpose(1, 2))                     # [E, T, I]
        full = torch.bmm(h, w_down.transpose(1, 2))                   # [E, T, H]
        o = full[ids, torch.arange(T, device=ids.device).unsqueeze(1)]
    return (o * s["tw"].unsqueeze(2)).sum(dim=1).bfloat16()


def _run_plain(s):
    k = s["kind"]
    if k in ("moe_fp8", "moe_nvfp4"):
        pick = s["T"] * s["topk"] <= s["E"]
        rows = s["ids"].reshape(-1).long() if pick else torch.arange(s["E"], device="cuda")
        if k == "moe_fp8":
            up, down = (w.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * sc[rows].unsqueeze(2)
                        for w, sc in (s["up"], s["down"]))
        else:
            up, down = (_nvfp4_values(q[rows], sf.view(s["E"], -1, *sf.shape[1:])[rows].flatten(0, 1), g[rows])
                        for q, sf, g in (s["up"], s["down"]))
        return _moe(s, up, down, pick)
    if k == "w4a16":
        return torch.matmul(s["x"].float(), _nvfp4_values(*s["w"])[0].t()).bfloat16()
    if k == "mx_quant":
        x = s["x"].float().view(s["R"], -1, 32)
        amax = x.abs().amax(dim=2, keepdim=True)
        # floor(log2(amax)) - 2, the exponent that brings the block's largest element into [4, 8)
        e = (torch.frexp(amax).exponent - 3).clamp(-127, 125)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        m = torch.ldexp(x.abs(), -e)
        # nearest E2M1 value, ties to the even code
        i = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int() +
             (m >= 3.5).int() + (m > 5.0).int())
        v = torch.tensor(E2M1[:8], device="cuda")[i]
        return torch.ldexp(torch.copysign(v, x), e).view(s["R"], s["K"]).bfloat16()
    a, b = (_e2m1(q).view(q.shape[0], -1, 32) * torch.exp2(_untile(sf, s["K"] // 32).float() - 127.0).unsqueeze(2)
            for q, sf in (s["a"], s["b"]))
    return torch.matmul(a.view(-1, s["K"])[:s["M"]], b.view(-1, s["K"])[:s["N"]].t()).bfloat16()


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ 64 bits

def _decode64(byte):
    """E2M1 nibble pairs -> float64 from the format's bit fields."""
    n = torch.stack((byte.int() & 15, byte.int() >> 4), dim=-1).flatten(-2)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    return torch.where(n >= 8, -mag, mag)


def _e4m3_64(byte):
    b = byte.int()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(b >= 128, -mag, mag)


def _tile_row(sf, r, n, per):
    """Scale bytes of rows r (a tensor of row numbers), `per` of them each, from the tiled order."""
    c = torch.arange(n, device=sf.device)
    at = ((r // 128).unsqueeze(1) * sf.shape[1] + c // per) * 512 + (16 * (r % 32) + 4 * (r % 128 // 32)).unsqueeze(1)
    return sf.reshape(-1)[at + c % per]


def _nv64(q, sf, g, e):
    N, K = q.shape[1], 2 * q.shape[2]
    r = torch.arange(e * N, (e + 1) * N, device=q.device)
    s = _e4m3_64(_tile_row(sf, r, K // 16, 4))
    return _decode64(q[e]) * s.repeat_interleave(16, dim=1) * g[e].double()


def exact(case, seed):
    s = prepare(case, seed)
    k = s["kind"]
    if k in ("moe_fp8", "moe_nvfp4"):
        y = torch.zeros(s["T"], s["H"], dtype=torch.float64, device="cuda")
        for e in s["ids"].unique().tolist():
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            if k == "moe_fp8":
                up, down = (_e4m3_64(w[e].view(torch.uint8)) * sc[e].double().unsqueeze(1) for w, sc in (s["up"], s["down"]))
            else:
                up, down = (_nv64(*w, e) for w in (s["up"], s["down"]))
            o = (s["x"][t].double() @ up.t()) @ down.t()
            y.index_add_(0, t, o * s["tw"][t, j].double().unsqueeze(1))
        return y
    if k == "w4a16":
        return s["x"].double() @ _nv64(*s["w"], 0).t()
    if k == "mx_quant":
        x = s["x"].double().view(s["R"], -1, 32)
        grid = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")
        amax = x.abs().amax(dim=2, keepdim=True)
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140))) - 2
        e = torch.where(torch.exp2(e + 2) > amax, e - 1, e)          # a logarithm that was rounded up
        e = torch.where(torch.exp2(e + 3) <= amax, e + 1, e)         # or down
        e = e.clamp(-127, 125)
        m = x.abs() * torch.exp2(-e)
        hi = torch.searchsorted(grid, m.clamp(max=6.0).contiguous()).clamp(1, 7)
        up, lo = grid[hi] - m.clamp(max=6.0), m.clamp(max=6.0) - grid[hi - 1]
        i = torch.where((up < lo) | ((up == lo) & (hi % 2 == 0)), hi, hi - 1)
        return (grid[i] * torch.sign(x) * torch.exp2(e)).view(s["R"], s["K"])
    a, b = (_decode64(q) * torch.exp2(_tile_row(sf, torch.arange(q.shape[0], device="cuda"), s["K"] // 32, 4).double()
                                      - 127).repeat_interleave(32, dim=1) for q, sf in (s["a"], s["b"]))
    return a[:s["M"]] @ b[:s["N"]].t()


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    k = case["kind"]
    if k in ("moe_fp8", "moe_nvfp4"):
        T, H, I, E, n = (case[v] for v in ("T", "H", "I", "E", "topk"))
        read = E * (1.0 - (1.0 - n / E) ** T)                        # experts that some token chose (uniform choice)
        w = 2 * H * I + 4 * (H + I) if k == "moe_fp8" else 2 * H * I * 9 / 16 + 8
        return {"bytes": read * w + 4 * T * H + 8 * T * n, "flops": 4.0 * T * n * H * I}
    if k == "w4a16":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K * 9 / 16 + 2 * M * (N + K), "flops": 2.0 * M * N * K}
    if k == "mx_quant":
        # codes and scales written and read again, the values written
        el = case["R"] * case["K"]
        return {"bytes": el * ((4 if case["f32"] else 2) + 2 * 17 / 32 + 2), "flops": 4.0 * el}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": (M + N) * K * 17 / 32 + 2 * M * N, "flops": 2.0 * M * N * K}
