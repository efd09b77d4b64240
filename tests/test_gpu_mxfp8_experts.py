"""The experts' MXFP8 products and the columnwise quantizers of their gradients
against float64 and the oracle; the bounds are derived in mxfp8_refs.py."""
import numpy as np
import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq
import oracle
import workloads as W
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def offsets(seed, E, M, empty=0.2, unused=0):
    rng = np.random.default_rng(seed)
    share = rng.exponential(size=E) * (rng.random(E) >= empty)
    share[rng.integers(E)] += 0.1
    cut = np.rint(np.cumsum(share) / share.sum() * (M - unused)).astype(np.int64)
    return [0] + [int(v) for v in cut]


def normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def on_device(off):
    return torch.tensor(off, dtype=torch.int64, device="cuda")


def product(x, w, off, **call):
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    qx, sx, zx = mxq.mxfp8_quantize_grouped(x, row_offsets=on_device(off[:-1] + [x.shape[0]]), swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, on_device(off), error_flag=flag, **call)
    assert int(flag) == 0, "a wait in the kernel gave up"
    return y, R.values(qx, sx), R.values(qw, sw)


# E, M, N, K: one expert, odd sizes, tails of N and K, many experts with few rows, pairs of CTAs and single ones
SHAPES = [(1, 1, 16, 32), (1, 300, 272, 160), (3, 5, 48, 96), (5, 777, 208, 320), (2, 600, 528, 1024), (4, 1200, 256, 224),
          (64, 64, 400, 256), (40, 333, 1040, 512), (100, 3000, 128, 128), (8, 2048, 768, 2048), (1024, 1100, 32, 64), (33, 20000, 144, 96)]


@pytest.mark.parametrize("E,M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows(E, M, N, K, dtype):
    off = offsets(E + M, E, M)
    y, a, b = product(normal(M, M, K), normal(N, E, N, K, scale=0.1), off, dtype=dtype)
    want, mags = R.grouped(a, b, off)
    R.check(y, want, K * R.U * mags, f"rows {E} {M} {N} {K}")


@pytest.mark.parametrize("E,M,N,K", [(3, 500, 272, 256), (6, 40, 144, 160), (2, 900, 512, 96)])
def test_power_of_two_operands_are_exact(E, M, N, K):
    """Every partial sum is an fp32 number: whatever reads a wrong row, scale or piece of K shows."""
    x = dev(W.gemm_pow2_operand(1, M, K))
    w = torch.stack([dev(W.gemm_pow2_operand(10 + e, N, K)) for e in range(E)])
    off = offsets(M, E, M)
    y, a, b = product(x, w, off, dtype=FP32)
    assert torch.equal(y.double(), R.grouped(a, b, off)[0])


@pytest.mark.parametrize("E,M,H,K", [(1, 3, 128, 64), (5, 777, 384, 288), (64, 100, 256, 128), (4, 3000, 640, 512), (8, 8, 1024, 256)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_swiglu(E, M, H, K, dtype):
    off = offsets(E * M, E, M)
    y, a, b = product(normal(M, M, K), normal(H, E, 2 * H, K, scale=0.3), off, dtype=dtype, swiglu=True)
    assert y.shape == (M, H)
    want, bound = R.swiglu(*R.grouped(a, b, off), K)
    R.check(y, want, bound, f"swiglu {E} {M} {H} {K}")


def test_swiglu_far_gates():
    """Gates from -200 to 200 with ups that bring small values back: one exact product a sum, so no bound of sums enters."""
    H, K = 128, 32
    gates = torch.linspace(-200, 200, H, device="cuda").to(BF16)
    x = torch.zeros(4, K, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, torch.tensor([1.0, 2.0 ** 30, 2.0 ** 60, -2.0 ** 90], device="cuda")
    w = torch.zeros(1, 2 * H, K, dtype=BF16, device="cuda")
    w[0, :H, 0], w[0, H:, 1] = gates, 1.0
    # (x's second value needs a scale of its own: every row is one group)
    x0 = x.clone(); x0[:, 1] = 0
    qx = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    qx[:, 0] = qx[:, 32] = 0x38                                    # 1.0
    sx = torch.full((4, 2), 127, dtype=torch.uint8, device="cuda")
    sx[:, 1] = torch.tensor([127, 157, 187, 217], dtype=torch.uint8, device="cuda")
    w2 = torch.zeros(1, 2 * H, 64, dtype=BF16, device="cuda")
    w2[0, :H, 0], w2[0, H:, 32] = gates, 1.0
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w2, swizzled=True)
    y = mxq.mxfp8_gemm_grouped(qx, mxq.swizzle_scales(sx), qw, zw, [0, 4], FP32, swiglu=True)
    d = R.values(qx, sx) @ R.values(qw, sw)[0].t()
    g, u = d[:, :H], d[:, H:]
    want = R.silu(g) * u
    # below fp32's normal range a step is absolute; sigmoid in float64 reaches e^-200
    bad = (y.double() - want).abs() > 2.0 ** -20 * want.abs() + 2.0 ** -149
    assert not bad.any(), (g[bad][:4], y[bad][:4], want[bad][:4])


def test_rows_of_no_expert_are_left(guard_bands):
    """Rows behind the last offset, and empty experts, on the guarded allocator's canary bytes."""
    off = [0, 0, 130, 130, 131, 400, 400]
    y, a, b = product(normal(1, 520, 96), normal(2, 6, 64, 96), off, dtype=FP32)
    want, mags = R.grouped(a[:400], b, off)
    R.check(y[:400], want, 96 * R.U * mags, "rows of experts")
    assert bool((y[400:].contiguous().view(torch.uint8) == guard_bands.CANARY).all())


def test_offsets_out_of_order_are_clamped():
    """A sequence that falls or leaves the rows acts as its running maximum within them; nothing outside is written."""
    E, M, N, K = 5, 300, 64, 64
    qx, sx, zx = mxq.mxfp8_quantize_grouped(normal(1, M, K), row_offsets=on_device([0, 100, 100, 250, 300, 300]), swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(normal(2, E, N, K), swizzled=True)
    bad = torch.tensor([7, 100, -50, 250, 1 << 40, 12], dtype=torch.int64, device="cuda")
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, bad, FP32)
    assert torch.equal(y, mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, [0, 100, 100, 250, 300, 300], FP32))


def test_no_sum_writes_zeros():
    off = on_device([0, 2, 5])
    qa, qb = torch.empty(5, 0, dtype=torch.uint8, device="cuda"), torch.empty(2, 16, 0, dtype=torch.uint8, device="cuda")
    s = torch.empty(0, dtype=torch.uint8, device="cuda")
    y = mxq.mxfp8_gemm_grouped(qa, s, qb, s, off)
    assert y.shape == (5, 16) and not y.any()
    none = torch.empty(0, 32, dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, 16, 32, dtype=torch.uint8, device="cuda")
    assert mxq.mxfp8_gemm_grouped(none, s, w, torch.zeros(1024, dtype=torch.uint8, device="cuda"), on_device([0, 0, 0])).shape == (0, 16)
    d = mxq.mxfp8_gemm_grouped_wgrad(torch.empty(48, 0, dtype=torch.uint8, device="cuda"), s,
                                     torch.empty(32, 0, dtype=torch.uint8, device="cuda"), s, on_device([0, 0]), FP32)
    assert d.shape == (1, 48, 32) and not d.any()


# ------------------------------------------------------- transposes

def columns(x, off):
    """[P', N]: the experts' rows, each padded with zeros to a multiple of 128, and zeros up to the bound."""
    E, at = len(off) - 1, R.padded(off)
    out = torch.zeros((x.shape[0] + 127 * E) // 128 * 128, x.shape[1], dtype=x.dtype, device=x.device)
    for e in range(E):
        out[at[e]:at[e] + off[e + 1] - off[e]] = x[off[e]:off[e + 1]]
    return out


def to_oracle(x):
    return host(x) if x.dtype == BF16 else x.cpu().numpy()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E,M,N,unused", [(1, 1, 16, 0), (1, 128, 128, 0), (5, 777, 208, 0), (3, 300, 80, 41), (64, 64, 48, 0), (9, 2000, 336, 0),
                                          (1024, 500, 32, 0), (2, 0, 64, 0), (7, 5000, 64, 5000)])
def test_ragged_columns(E, M, N, unused, dtype):
    off = offsets(E + M, E, M, unused=unused)
    x = normal(M + 1, M, N, dtype=dtype)
    q, z = mxq.mxfp8_quantize_columnwise_grouped(x, row_offsets=on_device(off))
    want_q, want_s = oracle.mxfp8_quantize(np.ascontiguousarray(to_oracle(columns(x, off)).T))
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(z.cpu().numpy(), oracle.swizzle_scales(want_s))


def test_ragged_columns_of_strided_rows():
    base = normal(3, 200, 96)
    off = [0, 50, 50, 190]
    a = mxq.mxfp8_quantize_columnwise_grouped(base[:, 16:64], row_offsets=off)
    b = mxq.mxfp8_quantize_columnwise_grouped(base[:, 16:64].contiguous(), row_offsets=on_device(off))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E,M,N", [(1, 32, 16), (3, 160, 208), (2, 512, 128), (5, 96, 80), (2, 2048, 64)])
def test_stacked_columns(E, M, N, dtype):
    x = normal(M, E, M, N, dtype=dtype)
    q, z = mxq.mxfp8_quantize_columnwise_grouped(x)
    tiles = []
    for e in range(E):
        want_q, want_s = oracle.mxfp8_quantize(np.ascontiguousarray(to_oracle(x[e]).T))
        assert np.array_equal(q[e].cpu().numpy(), want_q)
        tiles.append(oracle.swizzle_scales(want_s))
    assert np.array_equal(z.cpu().numpy(), np.concatenate(tiles))


# ------------------------------------------------- weights' gradients

@pytest.mark.parametrize("E,M,Na,Nb", [(1, 1, 16, 16), (5, 777, 208, 336), (3, 300, 80, 48), (4, 2000, 512, 272), (64, 64, 160, 144),
                                       (2, 5000, 256, 1024), (1024, 500, 16, 32), (6, 900, 288, 128)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_wgrad(E, M, Na, Nb, dtype):
    off = offsets(M, E, M)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = on_device(off)
    qa, za = mxq.mxfp8_quantize_columnwise_grouped(normal(1, M, Na), row_offsets=d)
    qb, zb = mxq.mxfp8_quantize_columnwise_grouped(normal(2, M, Nb), row_offsets=d)
    y = mxq.mxfp8_gemm_grouped_wgrad(qa, za, qb, zb, d, dtype, error_flag=flag)
    assert int(flag) == 0, "a wait in the kernel gave up"
    P = qa.shape[1]
    a, b = R.values(qa, R.untile(za, Na, P // 32)), R.values(qb, R.untile(zb, Nb, P // 32))
    at = R.padded(off)
    for e in range(E):
        s, n = slice(at[e], at[e + 1]), off[e + 1] - off[e]
        R.check(y[e], a[:, s] @ b[:, s].t(), n * R.U * (a[:, s].abs() @ b[:, s].abs().t()), f"wgrad {e} of {E}")
        if n == 0:
            assert not y[e].any()


# --------------------------------------------------------- a layer

def test_a_layer_and_its_gradients():
    """Norm, router, dispatch, both products and the way back, each against
    float64 on the operands that it was given; eager, and captured with other
    data replayed into the graph."""
    T, D, H, E, k = 300, 256, 384, 6, 2
    x, res = normal(1, T, D), normal(2, T, D)
    w, router = normal(3, D, scale=0.2) + 1, normal(4, E, D, scale=0.3)
    up, down = normal(5, E, 2 * H, D, scale=0.1), normal(6, E, D, H, scale=0.1)
    qu, su, zu = mxq.mxfp8_quantize_grouped(up, swizzled=True)
    qd, sd, zd = mxq.mxfp8_quantize_grouped(down, swizzled=True)
    qdt, zdt = mxq.mxfp8_quantize_columnwise_grouped(down)
    grad = normal(7, T, D, scale=0.1)

    def layer():
        n = mxq.mxfp8_rmsnorm(x, w, residual=res, normed=True)
        weights, experts = mxq.moe_route(n.normed.float() @ router.float().t(), k)
        off, order, pos = mxq.moe_dispatch(experts, E)
        rows = n.normed[order.long() // k]
        qx, sx, zx = mxq.mxfp8_quantize_grouped(rows, row_offsets=off, swizzled=True)
        h = mxq.mxfp8_gemm_grouped(qx, zx, qu, zu, off, swiglu=True)
        qh, sh, zh = mxq.mxfp8_quantize_grouped(h, row_offsets=off, swizzled=True)
        y = mxq.moe_combine(mxq.mxfp8_gemm_grouped(qh, zh, qd, zd, off, FP32), pos, weights)
        # back through the second product: its rows' gradient and its weights'
        gy = (grad.float()[order.long() // k] * weights.reshape(-1)[order.long()].unsqueeze(1)).to(BF16)
        qg, sg, zg = mxq.mxfp8_quantize_grouped(gy, row_offsets=off, swizzled=True)
        gh = mxq.mxfp8_gemm_grouped(qg, zg, qdt, zdt, off)
        a, za = mxq.mxfp8_quantize_columnwise_grouped(gy, row_offsets=off)
        b, zb = mxq.mxfp8_quantize_columnwise_grouped(h, row_offsets=off)
        gw = mxq.mxfp8_gemm_grouped_wgrad(a, za, b, zb, off, FP32)
        gx, gn = mxq.rmsnorm_backward(grad, n.hidden, w, n.rstd, grad_hidden=grad)
        return dict(n=n, off=off, qx=qx, sx=sx, h=h, qh=qh, sh=sh, y=y, pos=pos, weights=weights, qg=qg, sg=sg, gh=gh, gy=gy, gw=gw,
                    gx=gx, gn=gn, a=a, za=za, b=b, zb=zb)

    def check(r):
        off = r["off"].tolist()
        want, bound = R.swiglu(*R.grouped(R.values(r["qx"], r["sx"]), R.values(qu, su), off), D)
        R.check(r["h"], want, bound, "up")
        rows, mags = R.grouped(R.values(r["qh"], r["sh"]), R.values(qd, sd), off)
        wt = r["weights"].double().unsqueeze(-1)
        at = r["pos"].long()
        R.check(r["y"], (rows[at] * wt).sum(1), ((H * R.U + 2.0 ** -22) * mags[at] * wt).sum(1), "down")
        dt = R.values(qdt, torch.stack([R.untile(zdt.view(E, -1)[e], H, D // 32) for e in range(E)]))
        want, mags = R.grouped(R.values(r["qg"], r["sg"]), dt, off)
        R.check(r["gh"], want, D * R.U * mags, "rows' gradient")
        P = r["a"].shape[1]
        a, b = R.values(r["a"], R.untile(r["za"], D, P // 32)), R.values(r["b"], R.untile(r["zb"], H, P // 32))
        start = R.padded(off)
        for e in range(E):
            s = slice(start[e], start[e + 1])
            R.check(r["gw"][e], a[:, s] @ b[:, s].t(), (off[e + 1] - off[e]) * R.U * (a[:, s].abs() @ b[:, s].abs().t()), "weights' gradient")
        # and the operands are within a quantizer's step of what they stand for: E4M3 half a step 2^-4 of a value, at the least
        # half a step 2^-10 of the group's scale
        gold = torch.stack([r["gy"][off[e]:off[e + 1]].double().t() @ r["h"][off[e]:off[e + 1]].double() for e in range(E)])
        assert float((r["gw"].double() - gold).norm() / gold.norm()) < 2 * 0.125
        want, bound, want_w, bound_w = R.norm_gradient(grad.double(), r["n"].hidden.double(), w.double(), r["n"].rstd.double(), grad.double())
        R.check(r["gx"], want, bound, "norm's rows")
        R.check(r["gn"], want_w, bound_w, "norm's weight")

    check(layer())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    prev = mxq.set_output_allocator(None)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = layer()
        for seed in (20, 30):
            x.copy_(normal(seed, T, D))
            res.copy_(normal(seed + 1, T, D))
            grad.copy_(normal(seed + 2, T, D, scale=0.1))
            graph.replay()
            torch.cuda.synchronize()
            check(captured)
            eager = layer()
            for name in ("h", "y", "gh", "gw", "gx", "gn"):
                assert torch.equal(eager[name], captured[name]), name
    finally:
        mxq.set_output_allocator(prev)


def test_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    q, w = u8(4, 64), u8(2, 32, 64)
    sa, sb, off = u8(1024), u8(1024), on_device([0, 1, 4])
    mxq.mxfp8_gemm_grouped(q, sa, w, sb, off)
    for call, kind in (
            (lambda: mxq.mxfp8_gemm_grouped(q.cpu(), sa, w, sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q.view(torch.int8), sa, w, sb, off), TypeError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w[0], sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, u8(2, 32, 32), sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(u8(4, 48), sa, u8(2, 32, 48), sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, u8(2, 24, 64), sb, off), mxq.MxqError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, off, swiglu=True), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa[:256], w, sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb[:512], off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, [0, 1, 5]), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, [1, 1, 4]), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa[:512], w, sb, [0, 1, 4]), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, off.int()), TypeError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, off[:2]), TypeError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, off, torch.float16), TypeError),
            (lambda: mxq.mxfp8_gemm_grouped(q, sa, w, sb, off, error_flag=off), TypeError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(q), TypeError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(q.float()), ValueError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(torch.zeros(2, 40, 32, device="cuda")), ValueError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(q.float(), row_offsets=[0]), ValueError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(torch.zeros(4, 24, device="cuda"), row_offsets=[0, 4]), ValueError),
            (lambda: mxq.mxfp8_quantize_columnwise_grouped(q.float(), row_offsets=[0, 5]), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped_wgrad(u8(16, 128), sa, u8(16, 256), sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped_wgrad(u8(16, 64), sa, u8(16, 64), sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped_wgrad(u8(16, 128), sa, u8(24, 128), sb, off), ValueError),
            (lambda: mxq.mxfp8_gemm_grouped_wgrad(u8(16, 128), sa[:256], u8(16, 128), sb, off), ValueError)):
        with pytest.raises(kind):
            call()
