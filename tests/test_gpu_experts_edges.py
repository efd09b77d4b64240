"""Products with 4-bit weights, the weighted sum and the router at the ends of
their ranges. Tolerances of products count the roundings (fp4_refs.bound)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq
import fp4_refs as R
from test_gpu_fp4_matvec import check_err, cuda, grouped_exact, rows, silu_mul

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


# --------------------------------------------------- NVFP4's global scales

# a global scale and the size of the rows that it meets, so that the sums stay
# within fp32's range (or below its normal range, where the bound counts
# roundings to multiples of 2^-149)
GLOBALS = [(1.37 * 2.0 ** 110, 2.0 ** -8), (1.91 * 2.0 ** 115, 2.0 ** -14), (1.37 * 2.0 ** 127, 2.0 ** -30),
           (1.99 * 2.0 ** 91, 1.0), (1.01 * 2.0 ** 92, 1.0), (-1.5 * 2.0 ** 100, 1.0),
           (1.37 * 2.0 ** -120, 1.0), (1.37 * 2.0 ** -120, 2.0 ** 100), (1.0 * 2.0 ** -92, 1.0), (1.99 * 2.0 ** -93, 1.0),
           (1.9 * 2.0 ** -126, 2.0 ** 60), (5 * 2.0 ** -140, 2.0 ** 90), (2.0 ** -149, 2.0 ** 105), (0.0, 1.0)]


@pytest.mark.parametrize("xd", [BF16, FP32])
@pytest.mark.parametrize("M,N,K", [(1, 24, 544), (2, 24, 2080), (3, 20, 272), (6, 130, 1056), (20, 40, 288)])
def test_global_scales_of_any_size(xd, M, N, K):
    """Weights near fp32's largest value have global scales up to 2^117, and a
    caller may give any fp32: where the result is in range, so is each step."""
    rng = np.random.default_rng(M * 100 + K)
    p, s = R.weight(rng, "nvfp4", N, K)
    w = R.decode(p, s, "nvfp4")
    base = R.f64(rows(rng, M, K, xd))
    for g, size in GLOBALS:
        g = float(np.float32(g))
        x = torch.from_numpy(base * size).to(xd).cuda()
        y = mxq.nvfp4_matvec(x, cuda(p), cuda(s), torch.tensor(g, dtype=FP32, device="cuda"), dtype=FP32)
        exact, mag = R.product(R.f64(x), w)
        assert mag.max() * abs(g) * 64 < np.finfo(np.float32).max
        R.check(y, exact * g, mag * abs(g), K, f"global scale {g}")


@pytest.mark.parametrize("xd", [BF16, FP32])
@pytest.mark.parametrize("M", [2, 9])
def test_global_scales_of_any_size_in_further_passes(xd, M):
    """Rows that span more than one pass takes, with global scales at both ends."""
    rng = np.random.default_rng(M)
    N, K = 40, 320
    p, s = R.weight(rng, "nvfp4", N, K)
    w = R.decode(p, s, "nvfp4")
    x = rng.standard_normal((M, K))
    x[:, 1::3] *= 2.0 ** -45
    x[:, 2::3] *= 2.0 ** -90
    codes = np.stack([p & 15, p >> 4], -1).reshape(N, K)
    codes[:N // 2, 0::3] = 0                                  # what is left is the small elements' alone
    codes[:N // 4, 1::3] = 0
    p = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    w = R.decode(p, s, "nvfp4")
    for g, size in ((1.3 * 2.0 ** 108, 2.0 ** -6), (1.3 * 2.0 ** -125, 2.0 ** 110)):
        g = float(np.float32(g))
        xt = torch.from_numpy(x * size).to(xd).cuda()
        y = mxq.nvfp4_matvec(xt, cuda(p), cuda(s), torch.tensor(g, dtype=FP32, device="cuda"), dtype=FP32)
        exact, mag = R.product(R.f64(xt), w)
        R.check(y, exact * g, mag * abs(g), K, f"global scale {g}")


@pytest.mark.parametrize("counts", [[1, 0, 1], [9, 0, 4]])
def test_global_scales_of_halves_at_both_ends(counts):
    rng = np.random.default_rng(sum(counts))
    E, N, K = 3, 136, 288
    p, s = R.weight(rng, "nvfp4", E, N, K)
    w = R.decode(p, s, "nvfp4")
    off = np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1])
    x = rows(rng, M, K, BF16, 0.1)
    gs = np.array([[1.7 * 2.0 ** -100, 1.3 * 2.0 ** 105]] * E, np.float32)
    exact, size = grouped_exact(R.f64(x), w, off, np.arange(M), gs.astype(np.float64))
    y = mxq.nvfp4_matvec_grouped(x, cuda(p), cuda(s), cuda(gs), cuda(off), dtype=FP32)
    R.check(y, exact, size, K, "halves")
    h = mxq.nvfp4_matvec_grouped(x, cuda(p), cuda(s), cuda(gs), cuda(off), swiglu=True, dtype=FP32)
    check_err(h, *silu_mul(exact, size, K), "halves, swiglu")


def test_a_quantized_weight_near_the_largest_value():
    """nvfp4_quantize of weights up to 2^127 leaves a global scale of 2^115: the
    product with ordinary rows is that of the dequantized weight."""
    rng = np.random.default_rng(40)
    w = torch.from_numpy(rng.uniform(-1, 1, (48, 256)) * 2.0 ** 127).to(BF16).cuda()
    p, s, g = mxq.nvfp4_quantize(w)
    x = rows(rng, 3, 256, BF16, 2.0 ** -12)
    exact, size = R.product(R.f64(x), R.decode(p.cpu().numpy(), s.cpu().numpy(), "nvfp4"))
    R.check(mxq.nvfp4_matvec(x, p, s, g, dtype=FP32), exact * float(g), size * float(g), 256, "large weights")


# ------------------------------------------------------------------ SwiGLU

@pytest.mark.parametrize("xd", [BF16, FP32])
def test_swiglu_of_gates_far_below_zero(xd):
    """silu(z) is a normal fp32 number down to z = -90, and times a large up
    projection far below that. Gate and up are one product each here, so both
    are exact: what rounds is the exponential (two units in the last place,
    2^-22), the sum, the quotient and the two products (2^-24 each)."""
    z = np.concatenate([[0.0, 1.0, -1.0, -20.0, -60.0], -np.arange(72.0, 176.0, 1.0 if xd == BF16 else 0.59375)])
    up = 1.5 * 2.0 ** 100
    T, H, K = len(z), 8, 32
    codes = np.zeros((1, 2 * H, K), np.uint8)
    codes[0, :H, 0] = 2                                       # 1 x the gate's element
    codes[0, H:, 1] = 2
    p = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    s = np.full((1, 2 * H, 1), 127, np.uint8)
    x = np.zeros((T, K))
    x[:, 0], x[:, 1] = z, up
    xt = torch.from_numpy(x).to(xd).cuda()
    z = R.f64(xt)[:, :1]
    y = R.f64(mxq.mxfp4_matvec_grouped(xt, cuda(p), cuda(s), [0, T], swiglu=True, dtype=FP32))
    want = np.broadcast_to(z / (1 + np.exp(-z)) * up, (T, H))
    assert np.abs(want[np.abs(z[:, 0] + 90) < 1]).min() > 1e-8
    assert np.all(np.abs(y - want) <= 9 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149)


# ------------------------------------------------------------ lengths of zero

@pytest.fixture
def plain_allocator():
    """torch's own allocation, under which an empty tensor has no address."""
    prev = mxq.set_output_allocator(None)
    yield
    mxq.set_output_allocator(prev)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_layer_of_no_tokens(fmt, plain_allocator):
    E, k, D, H = 4, 2, 64, 32
    rng = np.random.default_rng(41)
    p1, s1 = (cuda(a) for a in R.weight(rng, fmt, E, 2 * H, D))
    p2, s2 = (cuda(a) for a in R.weight(rng, fmt, E, D, H))
    g = () if fmt == "mxfp4" else (torch.ones(E, device="cuda"),)
    f = mxq.mxfp4_matvec_grouped if fmt == "mxfp4" else mxq.nvfp4_matvec_grouped
    x = torch.empty(0, D, dtype=BF16, device="cuda")
    weights, experts = mxq.moe_route(torch.empty(0, E, device="cuda"), k)
    off, order, pos = mxq.moe_dispatch(experts, E)
    assert off.tolist() == [0] * (E + 1) and order.numel() == 0
    h = f(x, p1, s1, *g, off, order=order, top_k=k, swiglu=True)
    assert h.shape == (0, H)
    y = f(h, p2, s2, *g, off, combine=(pos, weights))
    assert y.shape == (0, D)


@pytest.mark.parametrize("shape", [(5, 0), (0,), (2, 3, 0)])
@pytest.mark.parametrize("yd", [BF16, FP32])
def test_combine_of_no_choices_is_zero(shape, yd):
    """An empty sum (the guarded allocator fills outputs with a canary byte)."""
    y = mxq.moe_combine(torch.ones(4, 12, device="cuda"), torch.empty(shape, dtype=torch.int32, device="cuda"),
                        torch.empty(shape, device="cuda"), dtype=yd)
    assert y.shape == (*shape[:-1], 12) and not y.any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
def test_no_columns_in_contiguous_rows(fmt, xd):
    p = torch.empty(8, 0, dtype=torch.uint8, device="cuda")
    x = torch.empty(3, 0, dtype=xd, device="cuda")
    args = () if fmt == "mxfp4" else (torch.ones((), device="cuda"),)
    f = mxq.mxfp4_matvec if fmt == "mxfp4" else mxq.nvfp4_matvec
    y = f(x, p, p, *args, dtype=FP32)
    assert y.shape == (3, 8) and not y.any()


def test_a_column_as_one_row_is_refused():
    base = torch.zeros(64, 32, device="cuda")
    p, s = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    for call in (lambda: mxq.mxfp4_matvec(base[:, 1], p, s), lambda: mxq.moe_route(base[:, 1], 2),
                 lambda: mxq.mxfp8_quantize(base[:, 1]), lambda: mxq.mxfp4_quantize(base.to(BF16)[:, 0])):
        with pytest.raises(ValueError, match="contiguous"):
            call()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [BF16, FP32])
@pytest.mark.parametrize("M", [1, 4, 8, 30])
def test_sums_of_one_sign(fmt, xd, M):
    """What the tensor cores cut off of a sum goes one way: nothing cancels."""
    rng = np.random.default_rng(M)
    for K in (256, 4096):
        p, s = R.weight(rng, fmt, 96, K)
        p &= 0x77                                             # no signs
        x = torch.from_numpy(np.abs(rng.standard_normal((M, K)))).to(xd).cuda()
        args = () if fmt == "mxfp4" else (torch.ones((), device="cuda"),)
        f = mxq.mxfp4_matvec if fmt == "mxfp4" else mxq.nvfp4_matvec
        R.check(f(x, cuda(p), cuda(s), *args, dtype=FP32), *R.product(R.f64(x), R.decode(p, s, fmt)), K, f"{fmt} one sign")


# ------------------------------------------------------------ first calls

FIRST_CALLS = """
import sys
import torch
import nvfp4_block_scaled_sm_b200 as mxq

torch.manual_seed(0)
E, k, D, H, T = 8, 2, 256, 64, {T}
x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
logits, bias = torch.randn(T, E, device="cuda"), torch.randn(E, device="cuda") * 0.1
p1 = torch.randint(0, 256, (E, 2 * H, D // 2), dtype=torch.uint8, device="cuda")
s1 = torch.randint(118, 124, (E, 2 * H, D // 32), dtype=torch.uint8, device="cuda")
p2 = torch.randint(0, 256, (E, D, H // 2), dtype=torch.uint8, device="cuda")
s2 = torch.randint(40, 90, (E, D, H // 16), dtype=torch.uint8, device="cuda")
g2 = torch.full((E,), 0.01, device="cuda")


def layer():
    w, e = mxq.moe_route(logits, k, scoring="sigmoid", bias=bias)
    off, order, pos = mxq.moe_dispatch(e, E)
    h = mxq.mxfp4_matvec_grouped(x, p1, s1, off, order=order, top_k=k, swiglu=True)
    y = mxq.nvfp4_matvec_grouped(h, p2, s2, g2, off, combine=(pos, w))
    return y, mxq.moe_route_backward(w, logits, e, scoring="sigmoid"), mxq.mxfp4_matvec(x, p1[0], s1[0])


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = layer()
graph.replay()
torch.cuda.synchronize()
captured = [t.clone() for t in captured]
for a, b in zip(captured, layer()):
    assert torch.equal(a, b)
print("first calls ok")
"""


@pytest.mark.parametrize("T", [3, 3000])
def test_first_calls_of_a_process_inside_a_capture(T):
    """Nothing that a first call sets up (limits of shared memory, queries of
    the device) needs an eager call before."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(mxq.__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(T=T)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls ok" in r.stdout, r.stderr[-2000:]
