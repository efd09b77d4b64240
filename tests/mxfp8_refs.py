"""float64 forms of the experts' MXFP8 products and of the norm, with the bounds
that the fp32 results are held to.

Products. A product of two E4M3 values and two powers of two is exact; the tensor
core adds K of them in fp32 in an order of its own: at most K u sum |a b| with
u = 2^-22 (four times the unit of rounding to nearest, so that truncating
accumulation is covered too). A bf16 result adds half a step, 2^-8 of its value;
an fp32 one is the sum itself.

SwiGLU. With sums off by dg and du: |silu'| < 1.1, so the result moves by at most
1.1 dg (|u| + du) + |silu(g)| du. Its own arithmetic: e^(-|g|/2) is off by 2 ulps
(2^-22), its square by 2^-21 + 2^-24, which the divisor 1 + t^2 passes on at most
halved; the two products with it by 2^-22 + 2^-24 each, the division by 2 ulps,
the last product by 2^-24: below 2^-20 together.

Norm's gradient. xh = h rstd and g w are rounded once (2^-24), the sum over a row
is 16 chained terms of a thread, two trees over 32 lanes and the division by N:
below 32 2^-24 of the sum of magnitudes. dweight: a chain over a CTA's rows, a
chain over an eighth of the CTAs, eight shares."""
import numpy as np
import torch

U = 2.0 ** -22
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def e4m3(q):
    """float64 values of E4M3 codes, from their bit fields."""
    n = q.to(torch.int32)
    field, man = (n >> 3) & 15, (n & 7).double()
    v = torch.where(field == 0, torch.ldexp(man, torch.full_like(field, -9)), torch.ldexp(1.0 + man / 8.0, field - 7))
    v = torch.where((n & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(n >= 128, -v, v)


def values(q, scale):
    """float64 values of codes [..., K] with E8M0 bytes [..., K/32]."""
    return torch.ldexp(e4m3(q).unflatten(-1, (-1, 32)), (scale.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def untile(flat, M, S):
    """The compact [M, S] scale bytes of an array in 128x4 tiles, entry by entry."""
    r, c = torch.arange(M, device=flat.device)[:, None], torch.arange(S, device=flat.device)[None, :]
    at = (r // 128 * -(-S // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    return flat[at]


def padded(off):
    """First rows of the experts when each is padded to a multiple of 128."""
    at = [0]
    for a, b in zip(off[:-1], off[1:]):
        at.append(at[-1] + -(-(b - a) // 128) * 128)
    return at


def grouped(a, b, off):
    """(sums, sums of magnitudes) [M, N] of rows a [M, K] with their expert's b [E, N, K]; NaN in rows of no expert."""
    y = torch.full((a.shape[0], b.shape[1]), float("nan"), dtype=torch.float64, device=a.device)
    m = y.clone()
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        y[s], m[s] = a[s] @ b[e].t(), a[s].abs() @ b[e].abs().t()
    return y, m


def silu(g):
    return g * torch.sigmoid(g)


def swiglu(y, m, K):
    """(result, bound before the last rounding) of silu(gate) up from sums and magnitudes."""
    H = y.shape[1] // 2
    g, u = y[:, :H], y[:, H:]
    dg, du = K * U * m[:, :H], K * U * m[:, H:]
    r = silu(g) * u
    return r, 1.1 * dg * (u.abs() + du) + silu(g).abs() * du + 2.0 ** -20 * r.abs()


def check(got, want, bound, what):
    """|got - want| <= bound, plus the rounding to got's type where that is narrower than the fp32 sums."""
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} for {tuple(want.shape)}"
    g = got.double()
    tol = bound + 2.0 ** -149
    if got.dtype != torch.float32:
        tol = tol + HALF_STEP[got.dtype] * (want.abs() + bound)
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first "
                           f"{bad.nonzero()[:4].tolist()}: {g[bad][:4].tolist()} for {want[bad][:4].tolist()}")


def norm(x, residual, weight, eps):
    """The norm's steps in numpy, one IEEE operation at a time: (h in x's dtype, rstd, y) as torch CPU tensors."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = h.double().numpy()
    mean = np.square(d).sum(axis=1) / d.shape[1]
    rstd = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
    y = (h.float().numpy() * rstd[:, None]) * weight.float().numpy()[None, :]
    assert y.dtype == np.float32
    return h, torch.from_numpy(rstd), torch.from_numpy(y)


def norm_gradient(g, h, w, rstd, grad_hidden=None):
    """float64 (dx, dweight) and the bounds of each, for float64 inputs [M, N], [N] and [M]."""
    N = h.shape[1]
    xh = h * rstd[:, None]
    gw = g * w
    mean = (gw * xh).mean(1, keepdim=True)
    mags = (gw * xh).abs().mean(1, keepdim=True)
    d = gw - xh * mean
    dx = rstd[:, None] * d
    bound = rstd[:, None] * (2.0 ** -22 * (gw.abs() + (xh * mean).abs()) + xh.abs() * 34 * 2.0 ** -24 * mags)
    if grad_hidden is not None:
        dx = dx + grad_hidden
    bound = bound + 2.0 ** -24 * dx.abs()
    chain = h.shape[0] / min(h.shape[0], 148) + 148 + 16
    return dx, bound, (g * xh).sum(0), (chain + 2) * 2.0 ** -24 * (g * xh).abs().sum(0)
