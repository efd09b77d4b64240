"""SwiGLU of the experts' MXFP8 products at the ends of its range: infinite and NaN
sums, gates so far below zero that e^(g/2) leaves fp32's normal range, ups that
bring their silu back.

Every sum here has one term that is not zero, so gate and up are known numbers and
the bound is that of SwiGLU's own arithmetic, in units of 2^-24. With t = e^(-|g|/2):
the approximate power is off by 4 (2 ulps), the correction of its argument adds a
rounding, and t enters twice: 10, which the divisor 1 + t^2 halves where it is near 2
itself. The divisor is rounded once (1), its reciprocal is off by an ulp (1 where the
divisor is near 1, 2 at most), and there are four products (4): below 16, 2^-20. Below
fp32's normal range half a step is absolute, and there are at most two such
roundings: 2^-149."""
import itertools
import math

import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
H, K = 128, 64
INF = float("inf")


def code(v):
    """(E4M3 code of v 2^-e, E8M0 byte of 2^e) of a value with at most four significant bits; NaN is a code."""
    if v != v:
        return 0x7F, 127
    sign, v = (0x80 if v < 0 else 0), abs(v)
    if v == 0:
        return sign, 127
    man, e = math.frexp(v)
    assert man * 16 == int(man * 16) and -127 <= e - 1 <= 127, v
    return sign | 7 << 3 | int(man * 16) - 8, e - 1 + 127


def e4m3(v):
    """The code of a value that is an E4M3 number."""
    c, byte = code(v)
    return c + 8 * (byte - 127)


def weight(gates, ups):
    """Codes and scales of the weight [1, 2H, K] whose sums with a row of two ones (columns 0 and 32) are
    gates and ups. For an infinity 448 2^127, which leaves fp32 with rows above one."""
    q = torch.zeros(1, 2 * H, K, dtype=torch.uint8)
    s = torch.full((1, 2 * H, K // 32), 127, dtype=torch.uint8)
    for half, col, values in ((0, 0, gates), (1, 32, ups)):
        for i, v in enumerate(values):
            c, b = (0x7E if v > 0 else 0xFE, 254) if abs(v) == INF else code(v)
            q[0, half * H + i, col], s[0, half * H + i, col // 32] = c, b
    return q.cuda(), s.cuda()


def run(gates, ups, rows, out=FP32, row_byte=127):
    """(SwiGLU's result, gate and up sums of the plain product, float64) for a batch of equal rows."""
    qw, sw = weight(gates, ups)
    zw = mxq.swizzle_scales(sw.view(2 * H, K // 32))
    qx = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    qx[:, 0] = qx[:, 32] = 0x38                                    # 1.0
    sx = torch.full((rows, K // 32), row_byte, dtype=torch.uint8, device="cuda")
    zx = mxq.swizzle_scales(sx)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, [0, rows], out, swiglu=True, error_flag=flag)
    d = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, [0, rows], FP32, error_flag=flag).double()
    assert int(flag) == 0
    return y, d[:, :H], d[:, H:]


def check(y, g, u):
    want = R.silu(g) * u
    fp32 = want.float().double()                                   # (its infinities: values beyond the type)
    odd = ~torch.isfinite(fp32)
    got = y.double()
    same = torch.isnan(want) & torch.isnan(got) | (got == fp32)
    half = 0.0 if y.dtype == FP32 else 2.0 ** -8
    tol = (2.0 ** -20 + half) * want.abs() + 2.0 ** -149 + (2.0 ** -134 if half else 0.0)   # bf16: half a step of its subnormals
    bad = torch.where(odd, ~same, ~((got - want).abs() <= tol))
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()}", g[bad][:4].tolist(), u[bad][:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist())


def table(gates, ups):
    """Every pair, H at a time."""
    pairs = list(itertools.product(gates, ups))
    for i in range(0, len(pairs), H):
        part = pairs[i:i + H]
        part += [(1.0, 1.0)] * (H - len(part))
        yield [p[0] for p in part], [p[1] for p in part]


FINITE = [0.0, 0.5, -1.0, -11.0, -88.0, -104.0, -120.0, -128.0, -144.0, -160.0, -176.0, -192.0, -208.0, -256.0, -448.0,
          -2.0 ** 12, -2.0 ** 60, 128.0, 208.0, 2.0 ** 60, 2.0 ** 126]
UPS = [1.0, -2.0 ** -40, 2.0 ** 64, -1.5 * 2.0 ** 100, 2.0 ** 126, 1.875 * 2.0 ** 127, 0.0]


# few rows, more than a chunk of 16 columns a warp, and the form for many rows
@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("out", [FP32, BF16])
def test_far_gates_keep_what_the_up_brings_back(rows, out):
    for gates, ups in table(FINITE, UPS):
        y, g, u = run(gates, ups, rows, out)
        assert torch.equal(g[0].cpu(), torch.tensor(gates, dtype=torch.float64))
        assert torch.equal(u[0].cpu(), torch.tensor(ups, dtype=torch.float64))
        check(y, g, u)


def test_far_gates_between_the_codes():
    """Gates in steps of a half from -160 to -223.5, of terms that are E4M3 numbers, with an up near fp32's largest value."""
    gates = [-(160.0 + 0.5 * i) for i in range(H)]
    qw = torch.zeros(1, 2 * H, K, dtype=torch.uint8)
    sw = torch.full((1, 2 * H, K // 32), 127, dtype=torch.uint8)
    for i, v in enumerate(gates):
        left = -v
        for c, part in enumerate((128.0, 64.0, 32.0, 16.0, 8.0, 4.0, 2.0, 1.0, 0.5)):
            if left >= part:
                qw[0, i, c], left = e4m3(-part), left - part
        assert left == 0
    qw[0, H:, 32], sw[0, H:, 1] = code(1.875 * 2.0 ** 127)
    qx = torch.zeros(3, K, dtype=torch.uint8, device="cuda")
    qx[:, :9] = qx[:, 32] = e4m3(1.0)
    qw, zw = qw.cuda(), mxq.swizzle_scales(sw.view(2 * H, 2).cuda())
    zx = mxq.swizzle_scales(torch.full((3, K // 32), 127, dtype=torch.uint8, device="cuda"))
    d = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, [0, 3], FP32).double()
    assert torch.equal(d[0, :H].cpu(), torch.tensor(gates, dtype=torch.float64))
    check(mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, [0, 3], FP32, swiglu=True), d[:, :H], d[:, H:])


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("out", [FP32, BF16])
def test_infinite_and_nan_sums(rows, out):
    """Sums beyond fp32 are infinities: silu(inf) up is an infinity of up's sign, silu(-inf) up is the formula's NaN."""
    special = [INF, -INF, float("nan"), 0.0, 2.0, -2.0, -144.0, -448.0]
    for gates, ups in table(special, special):
        # rows of 2^100: an infinity's weight leaves fp32 with them, the others' are scaled back
        y, g, u = run(*([v if not math.isfinite(v) else v * 2.0 ** -100 for v in half] for half in (gates, ups)), rows, out, row_byte=227)
        for sums, values in ((g, torch.tensor(gates)), (u, torch.tensor(ups))):
            assert torch.equal(torch.isnan(sums[0]).cpu(), torch.isnan(values))
            assert torch.equal(sums[0].float().cpu().nan_to_num(7.0, INF, -INF), values.nan_to_num(7.0, INF, -INF))
        check(y, g, u)


def test_an_infinite_input():
    """An infinity is quantized to the largest code and scale; the product of two is an infinity again, and nothing of it
    reaches another expert's rows."""
    E, M, N, Kx = 2, 90, 256, 96
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, Kx, generator=gen, device="cuda").to(BF16)
    w = torch.randn(E, N, Kx, generator=gen, device="cuda").to(BF16)
    w[1, :, :3] = w[1, :, 4:] = 0                                  # one term a sum of expert 1
    x[50, 3] = w[1, 5, 3] = INF
    w[1, 133, 3] = -INF
    off = torch.tensor([0, 40, M], device="cuda")
    q, s, z = mxq.mxfp8_quantize_grouped(x, row_offsets=off, swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)
    d = mxq.mxfp8_gemm_grouped(q, z, qw, zw, off, FP32)
    assert d[50, 5] == INF and d[50, 133] == -INF
    want, mags = R.grouped(R.values(q, s), R.values(qw, sw), [0, 40, M])
    R.check(d[:40], want[:40], Kx * R.U * mags[:40], "expert 0")
    y = mxq.mxfp8_gemm_grouped(q, z, qw, zw, off, FP32, swiglu=True)
    want, bound = R.swiglu(want[:40], mags[:40], Kx)
    R.check(y[:40], want, bound, "expert 0, SwiGLU")
    d = d[40:].double()
    check(y[40:], d[:, :N // 2], d[:, N // 2:])
    assert y[50, 5] == -INF
