"""Products with 4-bit weights (mxfp4_matvec, nvfp4_matvec) and the experts'
products, against float64 sums of the decoded weights. Tolerances count the
roundings (fp4_refs.bound)."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq
import fp4_refs as R
from gpu_util import host

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(rng, M, K, dtype, spread=1.0):
    return cuda((rng.standard_normal((M, K)) * spread).astype(np.float32)).to(dtype)


def run(fmt, x, p, s, g=None, dtype=FP32):
    if fmt == "mxfp4":
        return mxq.mxfp4_matvec(x, p, s, dtype=dtype)
    return mxq.nvfp4_matvec(x, p, s, g, dtype=dtype)


def scalar(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


SIZES = [(1, 1, 32), (1, 16, 32), (2, 5, 64), (3, 17, 96), (7, 64, 256), (8, 128, 256), (9, 129, 288),
         (1, 4096, 4096), (5, 1003, 1056), (11, 250, 2080), (16, 131, 512), (17, 200, 544), (32, 96, 1024),
         (33, 130, 800), (70, 40, 320), (2, 40, 65568), (20, 24, 20000 // 32 * 32)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd,yd", [(BF16, BF16), (BF16, FP32), (FP32, FP32), (FP32, BF16)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(fmt, xd, yd, M, N, K):
    rng = np.random.default_rng(M * 1000 + N + K)
    p, s = R.weight(rng, fmt, N, K)
    x = rows(rng, M, K, xd)
    g = 0.037
    y = run(fmt, x, cuda(p), cuda(s), scalar(g), yd)
    exact, size = R.product(R.f64(x), R.decode(p, s, fmt))
    if fmt == "nvfp4":
        g = float(np.float32(g))
        exact, size = exact * g, size * g
    R.check(y, exact, size, K, f"{fmt} {M}x{N}x{K}")


@pytest.mark.parametrize("xd", [BF16, FP32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 3, 48), (4, 130, 272), (9, 33, 1040), (19, 70, 4112)])
def test_nvfp4_rows_that_end_inside_a_group(xd, M, N, K):
    rng = np.random.default_rng(K + M)
    p, s = R.weight(rng, "nvfp4", N, K)
    x = rows(rng, M, K, xd)
    y = run("nvfp4", x, cuda(p), cuda(s), scalar(1.0))
    R.check(y, *R.product(R.f64(x), R.decode(p, s, "nvfp4")), K, f"nvfp4 {M}x{N}x{K}")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_strides_leading_dimensions_and_unaligned_scales(fmt):
    rng = np.random.default_rng(5)
    N, K = 77, 416
    p, s = R.weight(rng, fmt, N, K)
    w = R.decode(p, s, fmt)
    buf = torch.empty(s.size + 1, dtype=torch.uint8, device="cuda")
    buf[1:] = cuda(s).flatten()
    sd = buf[1:].view(s.shape)                                  # an odd address
    base = rows(rng, 6, 512, BF16)
    x = base[:, :K]                                             # row stride 512
    R.check(run(fmt, x, cuda(p), sd, scalar(1.0)), *R.product(R.f64(x), w), K, "strided rows")
    x3 = rows(rng, 6, K, FP32).view(2, 3, K)
    y = run(fmt, x3, cuda(p), sd, scalar(1.0))
    assert y.shape == (2, 3, N)
    R.check(y.view(6, N), *R.product(R.f64(x3).reshape(6, K), w), K, "three dimensions")
    one = rows(rng, 1, K, BF16)[0]
    assert run(fmt, one, cuda(p), sd, scalar(1.0)).shape == (N,)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
def test_every_code_and_scale(fmt, xd):
    """Every pair of codes with every scale byte: MXFP4's ends of the range
    (0, 254) and NaN (255), NVFP4's subnormals, signs and NaN codes."""
    K = 256
    p = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :K // 2]
    p = np.roll(p, 1, axis=1)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // (32 if fmt == "mxfp4" else 16), 1)
    rng = np.random.default_rng(3)
    x = rows(rng, 3, K, xd)
    y = run(fmt, x, cuda(p), cuda(s), scalar(1.0))
    exact, size = R.product(R.f64(x), R.decode(p, s, fmt))
    # past fp32's largest value the sum of 32 is infinite where it rounds there
    over = np.abs(exact) > np.finfo(np.float32).max
    exact = np.where(over, np.sign(exact) * np.inf, exact)
    near = np.abs(size) > np.finfo(np.float32).max / 4          # partial sums may overflow first
    got = y.clone()
    keep = torch.from_numpy(~near).cuda()
    R.check(torch.where(keep, got, 0), np.where(near, 0, exact), np.where(near, 0, size), K, f"{fmt} scales")
    if fmt == "mxfp4":
        assert torch.isnan(y[:, 255]).all()
        # scale 2^-127: subnormal results. Each group's sum is rounded to a
        # multiple of 2^-149 once for each piece of x (one of bf16, three of
        # fp32), off by 2^-150 at most; the additions of such multiples are exact
        tiny = R.f64(y[:, 0])
        assert np.all(np.abs(tiny - exact[:, 0]) <= (K // 32) * (1 if xd == BF16 else 3) * 2.0 ** -150)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
def test_wide_range_inside_a_group(fmt, xd):
    """Elements 2^40 to 2^200 below their group's largest, which meets zero
    weights: what remains of the product is theirs alone, to full precision."""
    rng = np.random.default_rng(8)
    M, N, K = 4, 40, 320
    p, s = R.weight(rng, fmt, N, K, spread=1)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, 0::32] *= np.float32(2.0 ** 90)
    x[:, 1::32] *= np.float32(2.0 ** 50)
    x[1, 3::32] *= np.float32(2.0 ** -60)
    x[2] = np.ldexp(rng.standard_normal(K), rng.integers(-100, 20, K)).astype(np.float32)
    codes = np.stack([p & 15, p >> 4], -1).reshape(N, K)
    codes[:, 0::32] = 0
    codes[:, 1::32] = 8                                         # -0
    codes[5:, 2::32] = 0
    p = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    xt = cuda(x).to(xd)
    y = run(fmt, xt, cuda(p), cuda(s), scalar(1.0))
    exact, size = R.product(R.f64(xt), R.decode(p, s, fmt))
    R.check(y, exact, size, K, "wide range")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
def test_ends_of_the_range_of_x(fmt, xd):
    """Subnormal rows, rows near the type's largest value, rows that hold both,
    and zeros: scales of the pieces at both ends."""
    rng = np.random.default_rng(12)
    N, K = 24, 288
    p, s = R.weight(rng, fmt, N, K, spread=1)
    big = float(torch.finfo(xd).max)
    x = np.zeros((6, K))
    x[0] = rng.integers(-127, 128, K) * 2.0 ** -133             # bf16 subnormals
    x[1] = rng.uniform(-1, 1, K) * big
    x[2] = np.where(rng.random(K) < 0.5, rng.uniform(-1, 1, K) * big, rng.integers(-127, 128, K) * 2.0 ** -133)
    x[3] = -0.0
    x[4, 7] = 2.0 ** -126
    x[5, ::32] = big
    xt = torch.from_numpy(x.astype(np.float32)).to(xd).cuda()
    assert torch.isfinite(xt).all()
    for m in (6, 1):                                            # both forms of the product
        y = run(fmt, xt[:m] if m == 6 else xt[:1], cuda(p), cuda(s), scalar(2.0 ** -20))
        w = R.decode(p, s, fmt) * (2.0 ** -20 if fmt == "nvfp4" else 1)
        exact, size = R.product(R.f64(xt)[:m], w)
        top = float(np.finfo(np.float32).max)
        safe = size * 64 < top                                  # no partial sum overflows
        keep = torch.from_numpy(safe).cuda()
        R.check(torch.where(keep, y, 0), np.where(safe, exact, 0), np.where(safe, size, 0), K, "range")
        assert not y[3:4].any()


def test_many_rows():
    rng = np.random.default_rng(13)
    N, K, M = 40, 512, 1000
    p, s = R.weight(rng, "mxfp4", N, K)
    x = rows(rng, M, K, BF16)
    R.check(mxq.mxfp4_matvec(x, cuda(p), cuda(s), dtype=FP32), *R.product(R.f64(x), R.decode(p, s, "mxfp4")), K, "many rows")


def test_fp32_rows_keep_their_bits():
    """x of 24 bits against one non-zero weight, a power of two: the product
    itself needs no rounding. It is the sum of the pieces of x, three a pass;
    with 2^60 between a group's elements two passes cover all bits (a piece
    takes 11 bits, and what a pass leaves is scaled up anew), so five additions
    join six terms. Each is off by 2^-24 of a partial sum, none of which exceeds
    the product by more than the first piece's rounding, 2^-11."""
    rng = np.random.default_rng(9)
    K, N = 96, 16
    x = cuda(np.ldexp(1 + rng.random((5, K)), rng.integers(-30, 30, (5, K))).astype(np.float32))
    codes = np.zeros((N, K), np.uint8)
    at = rng.integers(0, K, N)
    codes[np.arange(N), at] = rng.choice([2, 4, 6, 10, 12], N)  # powers of two: the product does not round
    p = codes[:, 0::2] | (codes[:, 1::2] << 4)
    s = np.full((N, K // 32), 127, np.uint8)
    y = mxq.mxfp4_matvec(x, cuda(p), cuda(s), dtype=FP32)
    exact = R.product(R.f64(x), R.decode(p, s, "mxfp4"))[0]
    assert np.all(np.abs(R.f64(y) - exact) <= 5 * 2.0 ** -24 * (1 + 2.0 ** -11) * np.abs(exact))
    # where the element is its group's largest, one pass holds all of it in
    # order, and nothing rounds
    top = np.abs(R.f64(x)).reshape(5, -1, 32).max(-1)[:, at // 32]
    assert np.array_equal(R.f64(y)[np.abs(R.f64(x))[:, at] == top], exact[np.abs(R.f64(x))[:, at] == top])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
def test_infinities_and_nan_in_x(fmt, xd):
    rng = np.random.default_rng(10)
    M, N, K = 6, 50, 192
    p, s = R.weight(rng, fmt, N, K)
    x = R.f64(rows(rng, M, K, xd))
    x[0, 5] = np.inf
    x[1, 70] = -np.inf
    x[2, 100] = np.nan
    x[3, 8], x[3, 40] = np.inf, -np.inf
    xt = torch.from_numpy(x).to(xd).cuda()
    y = run(fmt, xt, cuda(p), cuda(s), scalar(1.0))
    w = R.decode(p, s, fmt)
    exact, size = R.product(R.f64(xt), w)
    R.check(y, exact, size, K, "non-finite x")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_empty_sizes(fmt):
    p = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 2 if fmt == "mxfp4" else 4, dtype=torch.uint8, device="cuda")
    x = torch.ones(3, 64, dtype=BF16, device="cuda")
    assert run(fmt, x[:0], p, s, scalar(1.0)).shape == (0, 8)
    assert run(fmt, x, p[:0], s[:0], scalar(1.0)).shape == (3, 0)
    y = run(fmt, x[:, :0], p[:, :0], s[:, :0], scalar(1.0))
    assert y.shape == (3, 8) and not y.any()


def test_same_bits_every_time_and_on_other_streams():
    rng = np.random.default_rng(11)
    p, s = R.weight(rng, "mxfp4", 1024, 2048)
    x = rows(rng, 4, 2048, BF16)
    pd, sd = cuda(p), cuda(s)
    want = mxq.mxfp4_matvec(x, pd, sd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(mxq.mxfp4_matvec(x, pd, sd))
    torch.cuda.synchronize()
    assert all(torch.equal(want, y) for y in got)


# ------------------------------------------------------------------ experts

def grouped_exact(x, w, off, src, gs=None, swiglu=False):
    """Row by row: (exact, bound) of the fp32 sums, after SwiGLU where asked."""
    N, K = w.shape[1:]
    Rn = len(src)
    exact, size = np.zeros((Rn, N)), np.zeros((Rn, N))
    for e in range(w.shape[0]):
        for r in range(off[e], off[e + 1]):
            row = x[src[r]] if 0 <= src[r] < x.shape[0] else np.zeros(K)
            exact[r], size[r] = R.product(row, w[e])
            if gs is not None:
                f = np.where(np.arange(N) < N // 2, gs[e, 0], gs[e, -1])
                exact[r] *= f
                size[r] *= np.abs(f)
    return exact, size


def silu_mul(exact, size, K):
    """(value, error bound) of silu(gate) * up from the sums' bounds: the
    derivative of silu is below 1.1, and four more roundings of the result."""
    h = exact.shape[1] // 2
    tol = R.bound(exact, size, K, False)
    gate, up = exact[:, :h], exact[:, h:]
    act = gate / (1 + np.exp(-gate))
    err = 1.1 * tol[:, :h] * (np.abs(up) + tol[:, h:]) + (np.abs(act) + 1.1 * tol[:, :h]) * tol[:, h:]
    return act * up, err + 8 * 2.0 ** -24 * np.abs(act * up) + 2.0 ** -140


def check_err(got, exact, err, what):
    g = R.f64(got)
    if got.dtype == BF16:
        err = err + 2.0 ** -8 * (np.abs(exact) + err)
    bad = ~(np.abs(g - exact) <= err)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, first {np.argwhere(bad)[:4].tolist()}"


CASES = [  # E, N, K, rows of the experts
    (1, 16, 32, [3]),
    (4, 40, 64, [0, 1, 0, 2]),
    (5, 130, 288, [9, 0, 17, 1, 8]),
    (3, 258, 1056, [40, 33, 1]),
    (70, 32, 96, [1, 0, 2] * 23 + [5]),
    (300, 16, 64, [0] * 120 + [1, 4, 0, 2] + [0] * 170 + [3] * 6),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd,yd", [(BF16, BF16), (FP32, FP32)])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("E,N,K,counts", CASES)
def test_grouped(fmt, xd, yd, swiglu, halves, E, N, K, counts):
    if halves and fmt == "mxfp4":
        pytest.skip("MXFP4 has no global scales")
    rng = np.random.default_rng(E * 7 + N)
    p, s = R.weight(rng, fmt, E, N, K)
    w = R.decode(p, s, fmt)
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    x = rows(rng, M, K, xd, 0.2)
    gs = rng.uniform(0.01, 0.03, (E, 2 if halves else 1)).astype(np.float32)
    offs = cuda(off)
    if fmt == "mxfp4":
        y = mxq.mxfp4_matvec_grouped(x, cuda(p), cuda(s), offs, swiglu=swiglu, dtype=yd)
    else:
        y = mxq.nvfp4_matvec_grouped(x, cuda(p), cuda(s), cuda(gs if halves else gs[:, 0]), offs, swiglu=swiglu, dtype=yd)
    exact, size = grouped_exact(R.f64(x), w, off, np.arange(M), gs.astype(np.float64) if fmt == "nvfp4" else None)
    if swiglu:
        check_err(y, *silu_mul(exact, size, K), f"{fmt} swiglu")
    else:
        R.check(y, exact, size, K, f"{fmt} grouped")


@pytest.mark.parametrize("top_k", [1, 2, 5])
def test_gather_through_order(top_k):
    rng = np.random.default_rng(top_k)
    E, N, K, T = 6, 48, 160, 11
    p, s = R.weight(rng, "mxfp4", E, N, K)
    ids = np.stack([rng.permutation(E)[:top_k] for _ in range(T)])
    off, order, _ = R.dispatch(ids, E)
    x = rows(rng, T, K, BF16)
    y = mxq.mxfp4_matvec_grouped(x, cuda(p), cuda(s), cuda(off), order=cuda(order.astype(np.int32)), top_k=top_k, dtype=FP32)
    exact, size = grouped_exact(R.f64(x), R.decode(p, s, "mxfp4"), off, order // top_k)
    R.check(y, exact, size, K, "gathered")


def test_order_that_leads_outside_counts_as_zeros():
    rng = np.random.default_rng(20)
    p, s = R.weight(rng, "mxfp4", 2, 32, 64)
    x = rows(rng, 3, 64, BF16)
    order = np.array([0, -1, 3, 2 ** 31 - 1, -2 ** 31, 2], np.int32)
    y = mxq.mxfp4_matvec_grouped(x, cuda(p), cuda(s), [0, 3, 6], order=cuda(order), dtype=FP32)
    src = np.where((order >= 0) & (order < 3), order, -1)
    exact, size = grouped_exact(R.f64(x), R.decode(p, s, "mxfp4"), [0, 3, 6], src)
    R.check(y, exact, size, 64, "outside")
    assert not y[1].any() and not y[2:5].any()


def _canary(t):
    return bool((host(t).view(np.uint8) == 0xA5).all())


@pytest.mark.parametrize("off", [[0, 2, 2, 5], [3, 3, 5, 7], [0, 0, 0, 0], [9, 9, 9, 9]])
def test_rows_of_no_expert_stay_as_they_were(off):
    """The guarded allocator fills outputs with a canary byte."""
    rng = np.random.default_rng(21)
    E, N, K, M = 3, 32, 64, 9
    p, s = R.weight(rng, "mxfp4", E, N, K)
    x = rows(rng, M, K, BF16)
    y = mxq.mxfp4_matvec_grouped(x, cuda(p), cuda(s), torch.tensor(off).cuda(), dtype=FP32)
    exact, size = grouped_exact(R.f64(x), R.decode(p, s, "mxfp4"), off, np.arange(M))
    lo, hi = off[0], off[-1]
    if hi > lo:
        R.check(y[lo:hi], exact[lo:hi], size[lo:hi], K, "rows of experts")
    assert _canary(y[:lo]) and _canary(y[hi:])


@pytest.mark.parametrize("off", [[0, 7, 3, 9], [-5, 4, 400, 9], [9, 0, 9, 0], [2 ** 62, -2 ** 62, 2 ** 62, 1]])
def test_bad_offsets_stay_inside(off):
    """Offsets that break the rules are clamped: no write leaves the output
    (its guard bands are checked when the test ends)."""
    rng = np.random.default_rng(22)
    p, s = R.weight(rng, "nvfp4", 3, 40, 96)
    x = rows(rng, 9, 96, BF16)
    mxq.nvfp4_matvec_grouped(x, cuda(p), cuda(s), torch.ones(3, device="cuda"), torch.tensor(off).cuda())
    torch.cuda.synchronize()


def test_experts_without_rows_are_not_read():
    """NaN scales in the experts that nobody chose change nothing."""
    rng = np.random.default_rng(23)
    E, N, K = 4, 64, 128
    p, s = R.weight(rng, "mxfp4", E, N, K)
    s[1] = s[3] = 255
    x = rows(rng, 5, K, BF16)
    y = mxq.mxfp4_matvec_grouped(x, cuda(p), cuda(s), [0, 2, 2, 5, 5], dtype=FP32)
    exact, size = grouped_exact(R.f64(x), R.decode(p, np.where(s == 255, 0, s), "mxfp4"), [0, 2, 2, 5, 5], np.arange(5))
    R.check(y, exact, size, K, "others")


@pytest.mark.parametrize("N", [64, 37])
@pytest.mark.parametrize("yd", [BF16, FP32])
def test_combine(N, yd):
    rng = np.random.default_rng(24)
    Rn, T, k = 20, 7, 3
    r = cuda(rng.standard_normal((Rn, N)).astype(np.float32))
    pos = rng.integers(-1, Rn, (T, k)).astype(np.int32)
    pos[2] = -1
    pos[3] = 5                                                  # the same row three times
    pos[4, 0] = Rn
    wt = rng.standard_normal((T, k)).astype(np.float32)
    wt[2] = np.nan                                              # dropped: its weight does not matter
    y = mxq.moe_combine(r, cuda(pos), cuda(wt), dtype=yd)
    ok = (pos >= 0) & (pos < Rn)
    terms = np.where(ok[..., None], R.f64(r)[np.where(ok, pos, 0)] * np.where(ok, wt, 0)[..., None].astype(np.float64), 0)
    exact = terms.sum(1)
    check_err(y, exact, k * 2.0 ** -24 * np.abs(terms).sum(1) + 1e-40, "combine")
    assert not y[2].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", [1, 13])
def test_a_layer_of_experts(fmt, T):
    """Router, dispatch, gate/up product with SwiGLU, down product added up
    into the tokens: as a decoder runs them, against the same in float64."""
    rng = np.random.default_rng(T)
    E, k, D, H = 12, 4, 256, 192                               # model and expert widths
    p1, s1 = R.weight(rng, fmt, E, 2 * H, D)
    p2, s2 = R.weight(rng, fmt, E, D, H)
    x = rows(rng, T, D, BF16, 0.3)
    logits = cuda(rng.standard_normal((T, E)).astype(np.float32))
    bias = cuda((0.1 * rng.standard_normal(E)).astype(np.float32))
    gs1, gs2 = np.full((E, 2), 0.02, np.float32), np.full(E, 0.02, np.float32)

    def layer(x, logits):
        weights, experts = mxq.moe_route(logits, k, scoring="sigmoid", bias=bias, groups=4, top_groups=2)
        off, order, pos = mxq.moe_dispatch(experts, E)
        if fmt == "mxfp4":
            h = mxq.mxfp4_matvec_grouped(x, P1, S1, off, order=order, top_k=k, swiglu=True, dtype=FP32)
            y = mxq.mxfp4_matvec_grouped(h, P2, S2, off, combine=(pos, weights), dtype=FP32)
        else:
            h = mxq.nvfp4_matvec_grouped(x, P1, S1, G1, off, order=order, top_k=k, swiglu=True, dtype=FP32)
            y = mxq.nvfp4_matvec_grouped(h, P2, S2, G2, off, combine=(pos, weights), dtype=FP32)
        return y, weights, experts, h, off

    P1, S1, P2, S2, G1, G2 = cuda(p1), cuda(s1), cuda(p2), cuda(s2), cuda(gs1), cuda(gs2)
    y, weights, experts, h, off = layer(x, logits)

    wt, ids = R.route(R.f64(logits), k, "sigmoid", R.f64(bias), 4, 2)
    assert np.array_equal(experts.cpu().numpy(), ids)
    offs, order, pos = R.dispatch(ids, E)
    assert np.array_equal(off.cpu().numpy(), offs)
    e1, z1 = grouped_exact(R.f64(x), R.decode(p1, s1, fmt), offs, order // k, gs1.astype(np.float64) if fmt == "nvfp4" else None)
    check_err(h, *silu_mul(e1, z1, D), "gate and up")
    # the second product from the first's own fp32 rows
    e2, z2 = grouped_exact(R.f64(h), R.decode(p2, s2, fmt), offs, np.arange(T * k), gs2[:, None].astype(np.float64) if fmt == "nvfp4" else None)
    wd = R.f64(weights)
    exact = (e2[pos] * wd[..., None]).sum(1)
    err = ((R.bound(e2, z2, H, False)[pos] + (k + 1) * 2.0 ** -24 * np.abs(e2[pos])) * np.abs(wd)[..., None]).sum(1)
    check_err(y, exact, err, "down and combine")

    # captured once, replayed on other inputs; another graph of the same calls beside it
    xs, ls = x.clone(), logits.clone()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer(xs, ls))
        graphs.append(gr)
    x2 = rows(rng, T, D, BF16, 0.3)
    l2 = cuda(rng.standard_normal((T, E)).astype(np.float32))
    want2 = [t.clone() for t in layer(x2, l2)]
    xs.copy_(x2)
    ls.copy_(l2)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want2):
            assert torch.equal(a, b)
    xs.copy_(x)
    ls.copy_(logits)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1][0], y)


def test_quantizers_output_is_what_the_product_takes():
    """mxfp4_quantize and nvfp4_quantize_experts feed the products; the router's
    dispatch feeds the grouped quantizer."""
    rng = np.random.default_rng(30)
    w = rows(rng, 3 * 64, 256, BF16, 0.05).view(3, 64, 256)
    x = rows(rng, 7, 256, BF16)
    q, s = mxq.mxfp4_quantize(w[0])
    y = mxq.mxfp4_matvec(x, q, s, dtype=FP32)
    exact, size = R.product(R.f64(x), R.f64(mxq.mxfp4_dequantize(q, s, FP32)))
    R.check(y, exact, size, 256, "quantized")
    pk, bs, gs = mxq.nvfp4_quantize_experts(w, per_half=True)
    experts = cuda(rng.integers(0, 3, (7, 1)).astype(np.int32))
    off, order, pos = mxq.moe_dispatch(experts, 3)
    y = mxq.nvfp4_matvec_grouped(x, pk, bs, gs, off, order=order, top_k=1, dtype=FP32)
    exact, size = grouped_exact(R.f64(x), R.decode(pk.cpu().numpy(), bs.cpu().numpy(), "nvfp4"), off.tolist(), order.cpu().numpy(), R.f64(gs))
    R.check(y, exact, size, 256, "quantized experts")
    xq, xs, xz = mxq.mxfp8_quantize_grouped(x[order.long()], row_offsets=off, swizzled=True)
    want = mxq.mxfp8_quantize_grouped(x[order.long()], row_offsets=off.tolist(), swizzled=True)
    assert torch.equal(xq, want[0]) and torch.equal(xs, want[1])


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A stack of experts of more than 4 GiB: the last expert's weight lies
    behind 2^32 bytes of codes."""
    E, N, K = 9, 65536, 16384
    packed = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    assert packed.numel() > 2 ** 32
    rng = np.random.default_rng(31)
    p, s = R.weight(rng, "mxfp4", 64, K)
    packed[E - 1, N - 64:] = cuda(p)
    scale[E - 1, N - 64:] = cuda(s)
    x = rows(rng, 2, K, BF16)
    y = mxq.mxfp4_matvec_grouped(x, packed, scale, [0] * E + [2], dtype=FP32)
    R.check(y[:, N - 64:], *R.product(R.f64(x), R.decode(p, s, "mxfp4")), K, "last rows")
    assert not y[:, :N - 64].any()


def test_calls_from_two_threads():
    import threading
    rng = np.random.default_rng(34)
    p, s = R.weight(rng, "nvfp4", 256, 512)
    x = rows(rng, 6, 512, FP32)
    pd, sd, g = cuda(p), cuda(s), scalar(0.5)
    want = mxq.nvfp4_matvec(x, pd, sd, g, dtype=FP32)
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got[i].append(mxq.nvfp4_matvec(x, pd, sd, g, dtype=FP32))
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(want, y) for l in got for y in l)


def test_refusals():
    x = torch.zeros(2, 64, dtype=BF16, device="cuda")
    p = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    s16 = torch.zeros(8, 4, dtype=torch.uint8, device="cuda")
    one = torch.ones((), device="cuda")
    off = torch.tensor([0, 2], device="cuda")
    order = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: mxq.mxfp4_matvec(x.half(), p, s),
        lambda: mxq.mxfp4_matvec(x, p, s, dtype=torch.float16),
        lambda: mxq.mxfp4_matvec(x[:, :32], p, s),
        lambda: mxq.mxfp4_matvec(x, p, s16),
        lambda: mxq.mxfp4_matvec(x, p.view(torch.int8), s),
        lambda: mxq.mxfp4_matvec(x, p.t(), s),
        lambda: mxq.mxfp4_matvec(x.cpu(), p, s),
        lambda: mxq.mxfp4_matvec(x[:1].expand(2, 64), p, s),
        lambda: mxq.mxfp4_matvec(x, p.cpu(), s),
        lambda: mxq.mxfp4_matvec(torch.zeros(2, 128, dtype=BF16, device="cuda")[:, ::2], p, s),
        lambda: mxq.mxfp4_matvec(torch.zeros(130, dtype=BF16, device="cuda")[1:129].view(2, 64), p, s),
        lambda: mxq.nvfp4_matvec(x, p, s16, torch.ones(2, device="cuda")),
        lambda: mxq.nvfp4_matvec(x, p, s16, one.double()),
        lambda: mxq.mxfp4_matvec_grouped(x, p, s, off),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], off.int()),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], [0, 3]),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], [2, 1]),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], off, top_k=2),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], off, order=order.long()),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], off, order=order, top_k=0),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None, :7], s[None, :7], off, swiglu=True),
        lambda: mxq.nvfp4_matvec_grouped(x, p[None], s16[None], torch.ones(3, device="cuda"), off),
        lambda: mxq.nvfp4_matvec_grouped(x, p[None, :7], s16[None, :7], torch.ones(2, device="cuda"), off),
        lambda: mxq.mxfp4_matvec_grouped(x, p[None], s[None], off, combine=(order, torch.ones(3, device="cuda"))),
        lambda: mxq.moe_combine(torch.zeros(2, 8, device="cuda", dtype=BF16), order, torch.ones(2, device="cuda")),
        lambda: mxq.moe_combine(torch.zeros(2, 8, device="cuda"), order, torch.ones(2, device="cuda").double()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mxq.MxqError)):
            f()
            print("not refused:", i)


def test_another_device():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    rng = np.random.default_rng(33)
    p, s = R.weight(rng, "mxfp4", 64, 128)
    x = rows(rng, 2, 128, BF16).to("cuda:1")
    y = mxq.mxfp4_matvec(x, cuda(p).to("cuda:1"), cuda(s).to("cuda:1"), dtype=FP32)
    R.check(y, *R.product(R.f64(x), R.decode(p, s, "mxfp4")), 128, "cuda:1")
