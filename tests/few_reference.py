"""Plain 64-bit forms of the few-token default-maths operators and of MXFP4,
and the error bounds that the tests hold the kernels to.

A BF16 result is off by at most half a step, 2^-8 of its value. A 16-bit
rounding of h (FP16) adds at most 2^-11 of each h. A sum of n products in
FP32 is off by at most n 2^-23 of the sum of their magnitudes (each addition
by at most one unit of 2^-23: the tensor cores may truncate), and scaling it
by a few more units. The bounds below add these up over the two projections.
"""
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e2m1(packed):
    """Packed codes [..., K/2] -> float64 [..., K], low nibble first."""
    n = torch.stack((packed.int() & 15, packed.int() >> 4), dim=-1).flatten(-2)
    v = torch.tensor(E2M1, dtype=torch.float64, device=packed.device)[n & 7]
    return torch.where(n >= 8, -v, v)


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def untile(sf, rows, per_row):
    """Tiled scales -> [rows, per_row] bytes: atom (r / 128, b / 4), byte 16 (r % 32) + 4 (r % 128 / 32) + b % 4."""
    atoms = (per_row + 3) // 4
    r = torch.arange(rows, device=sf.device).unsqueeze(1)
    b = torch.arange(per_row, device=sf.device).unsqueeze(0)
    at = ((r // 128) * atoms + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    return sf.reshape(-1)[at]


def nvfp4_values(q, sf, g):
    """[E, N, K/2] codes, tiled scales, [E] global scales -> float64 [E, N, K]."""
    E, N, K = q.shape[0], q.shape[1], 2 * q.shape[2]
    s = e4m3(untile(sf, E * N, K // 16).contiguous()).repeat_interleave(16, dim=1).view(E, N, K)
    return e2m1(q) * s * g.double().view(E, 1, 1)


def fp8_values(q, s):
    return e4m3(q) * s.double().unsqueeze(-1)


def moe(x, ids, tw, w_up, w_down):
    """(y64, bound): the routed layer on float64 weights [E, I, H], [E, H, I]."""
    T, H = x.shape
    E, I = w_up.shape[:2]
    x, tw = x.double(), tw.double()
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        h = x[t] @ w_up[e].t()
        w = tw[t, j].unsqueeze(1)
        habs = x[t].abs() @ w_up[e].abs().t()
        # h: the FP32 sum, the 16-bit rounding, and what x and h lose far below their row's largest
        small = x[t].abs().amax(dim=1, keepdim=True) * 2.0 ** -39 * w_up[e].abs().sum(dim=1)
        dh = (H + 8) * 2.0 ** -23 * habs + 2.0 ** -11 * h.abs() + small + 2.0 ** -39 * h.abs().amax(dim=1, keepdim=True)
        wa = w_down[e].abs().t()
        y.index_add_(0, t, (h @ w_down[e].t()) * w)
        bound.index_add_(0, t, (dh @ wa + (I + 8) * 2.0 ** -23 * ((h.abs() + dh) @ wa)) * w.abs())
    return y, bound * 1.01 + 2.0 ** -8 * (y.abs() + bound) + 1e-30


def product(x, w):
    """(y64, bound) of y = bf16(x w^T) with exact 16-bit operands and FP32 sums."""
    x = x.double()
    y = x @ w.t()
    b = (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())
    b = b + x.abs().amax(dim=1, keepdim=True) * 2.0 ** -39 * w.abs().sum(dim=1)
    return y, b + 2.0 ** -8 * (y.abs() + b) + 1e-30


def mxfp4_quant(x):
    """(values, scale codes, E2M1 codes) of rows x [R, K] by the definition, block by block in float64."""
    R, K = x.shape
    xb = x.double().view(R, K // 32, 32)
    amax = xb.abs().amax(dim=2)
    m, e = torch.frexp(amax)                       # amax = m 2^e with m in [0.5, 1)
    c = torch.where(amax > 0, (e - 1 - 2).clamp(-127, 125) + 127, torch.zeros_like(e))
    v = xb.abs() * torch.exp2(127.0 - c.double()).unsqueeze(2)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    d = (v.unsqueeze(-1) - grid).abs()
    best = d.amin(dim=-1, keepdim=True)
    # the nearest value; of two equally near the one with the even code
    code = torch.where(d == best, torch.arange(8, device=x.device) + 100 * (torch.arange(8, device=x.device) % 2),
                       10000).amin(dim=-1) % 100
    values = torch.copysign(grid[code] * torch.exp2(c.double() - 127.0).unsqueeze(2), xb)
    code = code + 8 * torch.signbit(xb).long()
    return values.view(R, K), c.to(torch.uint8), code.view(R, K).to(torch.uint8)


def e8m0(codes):
    v = torch.exp2(codes.double() - 127.0)
    return torch.where(codes == 255, torch.full_like(v, float("nan")), v)


def assert_within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} outside; first at {i}: got {float(got[i])}, "
                             f"exact {float(ref[i])}, bound {float(bound[i])}")
