"""64-bit references of the 8-bit linear operators, and bounds derived from how the
kernels round."""
import torch

EPS32 = 2.0 ** -24


def e4m3_values(q):
    return q.view(torch.float8_e4m3fn).double()


def e8m0_values(s):
    v = torch.exp2(s.view(torch.uint8).double() - 127)
    return torch.where(s.view(torch.uint8) == 255, torch.full_like(v, float("nan")), v)


def x_block(q, S):
    return e4m3_values(q) * S.double().repeat_interleave(128, -1)[..., :q.shape[-1]]


def w_block(q, S):
    n, k = q.shape[-2:]
    s = S.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return e4m3_values(q) * s


def mx(q, s):
    return e4m3_values(q) * e8m0_values(s).repeat_interleave(32, -1)[..., :q.shape[-1]]


def product(x, w):
    """(x w^T, sum of the products' magnitudes, sum over runs of 8 k of the largest
    magnitude) in 64 bits; x [m, k], w [n, k]."""
    k = x.shape[1]
    pad = -k % 8
    x = torch.nn.functional.pad(x, (0, pad))
    w = torch.nn.functional.pad(w, (0, pad))
    total = x.abs() @ w.abs().t().contiguous()
    largest = torch.zeros_like(total)
    for i in range(0, x.shape[1], 8):
        p = x[:, None, i:i + 8].abs() * w[None, :, i:i + 8].abs()
        largest += p.amax(-1)
    return x @ w.t().contiguous(), total, largest


def bound(y, total, largest, k, f32):
    """How far a product may be off.  Sums: at most k / 16 + 64 additions in a row,
    each off by less than 2^-23 of what has been added up in magnitude (the matrix
    cores cut).  bf16 results: the 8-bit matrix instruction also cuts each of 8
    neighbouring products below 2^-13 of the largest, and the result is rounded once,
    by at most half a step of 2^-7."""
    off = (k / 16 + 64) * 2.0 ** -23 * total
    return off if f32 else off + 8 * 2.0 ** -13 * largest + 2.0 ** -8 * y.abs() * (1 + 2.0 ** -8)


def check(out, x, w, f32=None):
    f32 = out.dtype == torch.float32 if f32 is None else f32
    y, total, largest = product(x, w)
    off = (out.double() - y).abs()
    lim = bound(y, total, largest, x.shape[1], f32)
    assert torch.isfinite(out).all()
    assert (off <= lim).all(), f"off by up to {(off / lim.clamp(min=1e-300)).max().item():.3g} of what is allowed"
    return off


def codes(g, *shape):
    """Random finite codes of every size."""
    q = torch.randint(0, 256, shape, generator=g, device=g.device, dtype=torch.uint8)
    return torch.where((q & 127) == 127, q - 9, q)


def block_operands(g, m, n, k, lead=()):
    S = torch.exp2(torch.randint(-12, 3, (m, -(-k // 128)), generator=g, device=g.device).float())
    S = S * (1 + torch.rand(S.shape, generator=g, device=g.device))
    wS = torch.exp2(torch.randint(-12, 3, (*lead, -(-n // 128), -(-k // 128)), generator=g, device=g.device).float())
    wS = wS * (1 + torch.rand(wS.shape, generator=g, device=g.device))
    return codes(g, m, k), S, codes(g, *lead, n, k), wS


def mx_operands(g, m, n, k, lead=()):
    def scales(*shape):
        return torch.randint(110, 132, shape, generator=g, device=g.device, dtype=torch.uint8)
    return codes(g, m, k), scales(m, -(-k // 32)), codes(g, *lead, n, k), scales(*lead, n, -(-k // 32))


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def norm(x, residual, weight, eps):
    """h (64 bits, rounded to bf16), r, y of the norm."""
    h = x.double() if residual is None else (x.double() + residual.double()).bfloat16().double()
    r = 1 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, r[:, 0], h * r * weight.double()


def norm_backward(dy, h, weight, r, dh):
    u = h.double() * r.double()[:, None]
    g = dy.double() * weight.double()
    dx = r.double()[:, None] * (g - u * (g * u).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy.double() * u).sum(0)
