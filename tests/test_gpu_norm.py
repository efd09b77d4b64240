"""The norm with an MXFP8 output, bit for bit against its steps in numpy and the
oracle's quantizer, and its gradient against float64 and against differences."""
import numpy as np
import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq
import oracle

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def rows(seed, M, N, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * torch.exp(torch.randn(M, 1, generator=g)) * scale
    x[:, torch.rand(N, generator=g) < 0.01] *= 30.0
    return x.to(dtype)


def weights(seed, N, dtype):
    return (1.0 + 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(seed))).to(dtype)


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    if a.dtype.is_floating_point:
        kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
        nan = torch.isnan(a) & torch.isnan(b)
        return torch.equal(torch.where(nan, 0, a.view(kind)), torch.where(nan, 0, b.view(kind)))
    return torch.equal(a, b)


def check_norm(x, residual, w, eps=1e-6, **call):
    h, rstd, y = R.norm(x.reshape(-1, x.shape[-1]), None if residual is None else residual.reshape(-1, x.shape[-1]), w, eps)
    r = mxq.mxfp8_rmsnorm(x.cuda(), w.cuda(), eps=eps, residual=None if residual is None else residual.cuda(), **call)
    q, s = oracle.mxfp8_quantize(y.numpy())
    assert same_bits(r.hidden.view_as(h), h)
    assert same_bits(r.rstd.reshape(-1), rstd)
    assert np.array_equal(r.qweight.cpu().numpy().reshape(q.shape), q)
    assert np.array_equal(r.scale.cpu().numpy().reshape(s.shape), s)
    assert (r.scale_swizzled is not None) == bool(call.get("swizzled"))
    if r.scale_swizzled is not None:
        assert np.array_equal(r.scale_swizzled.cpu().numpy(), oracle.swizzle_scales(s))
    if call.get("normed"):
        assert same_bits(r.normed.view_as(y), y.to(x.dtype))
    return r


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("wd", [BF16, FP32])
@pytest.mark.parametrize("M,N", [(1, 32), (5, 96), (3, 512), (130, 1056), (7, 2048), (2, 2080), (4, 4096), (129, 7168),
                                 (1, 16384), (3, 32768), (2, 32800), (1, 65536)])
def test_bits(M, N, dtype, wd):
    x, w = rows(M + N, M, N, dtype), weights(N, N, wd)
    check_norm(x, None, w, swizzled=True, normed=True)
    check_norm(x, rows(M + N + 1, M, N, dtype, 2.0), w, swizzled=N % 64 == 0)


def test_strides_and_leading_dimensions():
    base = rows(1, 12, 200, BF16)
    x = base[:, 8:136]                                    # row stride 200, 16-byte but not 32-byte aligned
    w = weights(2, 128, BF16)
    h, rstd, y = R.norm(x, base[:, 64:192], w, 1e-6)
    d = base.cuda()
    r = mxq.mxfp8_rmsnorm(d[:, 8:136], w.cuda(), residual=d[:, 64:192], swizzled=True, normed=True)
    q, s = oracle.mxfp8_quantize(y.numpy())
    assert np.array_equal(r.qweight.cpu().numpy(), q) and np.array_equal(r.scale.cpu().numpy(), s)
    assert same_bits(r.hidden, h) and same_bits(r.normed, y.to(BF16))
    x3 = rows(3, 12, 96, FP32).view(2, 6, 96)
    r = check_norm(x3, None, weights(4, 96, FP32), normed=True)
    assert r.qweight.shape == (2, 6, 96) and r.scale.shape == (2, 6, 3) and r.rstd.shape == (2, 6)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_values_at_the_ends(dtype):
    """Squares beyond fp32's range, zeros, infinities and NaN in a row."""
    x = rows(5, 9, 128, dtype)
    x[0] = 0.0
    x[1] = 1e30
    x[2] = -1e-30
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    x[5] = torch.finfo(dtype).max
    x[6] = 2.0 ** -133 if dtype == BF16 else 2.0 ** -149
    x[7, 40:] = 0.0
    for eps in (1e-6, 0.0):
        with np.errstate(all="ignore"):
            check_norm(x, None, weights(6, 128, dtype), eps=eps, swizzled=True, normed=True)


def test_empty_rows_and_columns():
    w = weights(1, 64, BF16).cuda()
    r = mxq.mxfp8_rmsnorm(torch.empty(0, 64, dtype=BF16, device="cuda"), w, swizzled=True)
    assert r.qweight.shape == (0, 64) and r.scale_swizzled.numel() == 0
    dx, dw = mxq.rmsnorm_backward(torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 64, dtype=BF16, device="cuda"),
                                  w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 96), (400, 136), (61, 1056), (300, 2048), (500, 4096), (150, 4104), (333, 7168),
                                 (301, 8192), (300, 9216), (5, 16384), (9, 16392), (160, 20480)])
def test_gradient(M, N, dtype):
    for wd, with_hidden in ((dtype, True), (FP32, False)):
        g, h, w = rows(M, M, N, dtype, 0.1), rows(N, M, N, dtype), weights(7, N, wd)
        gh = rows(M + N, M, N, dtype, 0.1) if with_hidden else None
        rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
        dx, dw = mxq.rmsnorm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda(), grad_hidden=None if gh is None else gh.cuda())
        want, bound, want_w, bound_w = R.norm_gradient(g.double(), h.double(), w.double(), rstd.double(), None if gh is None else gh.double())
        R.check(dx.cpu(), want, bound, f"dx {M}x{N}")
        R.check(dw.cpu(), want_w, bound_w, f"dweight {M}x{N}")
        again = mxq.rmsnorm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda(), grad_hidden=None if gh is None else gh.cuda())
        assert same_bits(dx, again[0]) and same_bits(dw, again[1])


# few rows are summed over by a cluster: both sides of its limits (64 rows, 2^18 elements, rows of 16384)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,N", [(2, 8), (16, 16384), (17, 16384), (15, 16392), (33, 1000), (64, 4096), (65, 4096), (64, 4104)])
def test_gradient_of_few_rows(M, N, dtype):
    g, h, gh, w = rows(M, M, N, dtype, 0.1).cuda(), rows(N, M, N, dtype).cuda(), rows(M + N, M, N, dtype, 0.1).cuda(), weights(7, N, dtype).cuda()
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dx, dw = mxq.rmsnorm_backward(g, h, w, rstd, grad_hidden=gh)
    want, bound, want_w, bound_w = R.norm_gradient(*(t.cpu().double() for t in (g, h, w, rstd, gh)))
    R.check(dx.cpu(), want, bound, f"dx {M}x{N}")
    R.check(dw.cpu(), want_w, bound_w, f"dweight {M}x{N}")
    # captured, and dx in place of grad
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    n = mxq.lib.mxq_rmsnorm_backward_workspace_bytes(M, N)
    work, out, out_w = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), g.clone(), torch.empty_like(dw)
    with torch.cuda.graph(graph, stream=side):
        a = mxq.rmsnorm_backward(g, h, w, rstd, grad_hidden=gh)
        st = mxq.lib.mxq_rmsnorm_backward(out.data_ptr(), 0 if dtype == BF16 else 1, M, N, N, h.data_ptr(), N, w.data_ptr(),
                                          0 if dtype == BF16 else 1, rstd.data_ptr(), gh.data_ptr(), N, out.data_ptr(), out_w.data_ptr(),
                                          work.data_ptr() if n else None, n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    graph.replay()
    torch.cuda.synchronize()
    for x, y in ((a[0], dx), (a[1], dw), (out, dx), (out_w, dw)):
        assert same_bits(x, y)


def test_gradient_against_differences():
    """Central differences of sum(g y) in float64: off by the third derivative's h^2 term, below 1e-7 here."""
    M, N, step = 3, 64, 1e-4
    gen = torch.Generator().manual_seed(3)
    g, h, w = (torch.randn(*s, generator=gen) for s in ((M, N), (M, N), (N,)))

    def loss(h, w):
        y = h * (1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)) * w
        return (g.double() * y).sum()

    r = mxq.mxfp8_rmsnorm(h.cuda(), w.cuda())
    dx, dw = (t.cpu().double() for t in mxq.rmsnorm_backward(g.cuda(), r.hidden, w.cuda(), r.rstd))
    _, bound, _, bound_w = R.norm_gradient(g.double(), h.double(), w.double(), r.rstd.cpu().double())
    for i in range(M):
        for j in range(0, N, 7):
            d = torch.zeros(M, N, dtype=torch.float64)
            d[i, j] = step
            diff = float((loss(h.double() + d, w.double()) - loss(h.double() - d, w.double())) / (2 * step))
            assert abs(diff - float(dx[i, j])) <= float(bound[i, j]) + 2e-6
    for j in range(0, N, 5):
        d = torch.zeros(N, dtype=torch.float64)
        d[j] = step
        diff = float((loss(h.double(), w.double() + d) - loss(h.double(), w.double() - d)) / (2 * step))
        assert abs(diff - float(dw[j])) <= float(bound_w[j]) + 2e-6


def test_strided_gradients():
    base = rows(1, 40, 400, BF16).cuda()
    g, h, gh = base[:, :96], base[:, 96:192], base[:, 200:296]
    w = weights(1, 96, BF16).cuda()
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    a = mxq.rmsnorm_backward(g, h, w, rstd, grad_hidden=gh)
    b = mxq.rmsnorm_backward(g.contiguous(), h.contiguous(), w, rstd, grad_hidden=gh.contiguous())
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    rstd = torch.ones(4, device="cuda")
    for call, kind in (
            (lambda: mxq.mxfp8_rmsnorm(x.cpu(), w), ValueError), (lambda: mxq.mxfp8_rmsnorm(x, w.cpu()), ValueError),
            (lambda: mxq.mxfp8_rmsnorm(x.half(), w), TypeError), (lambda: mxq.mxfp8_rmsnorm(x, w.half()), TypeError),
            (lambda: mxq.mxfp8_rmsnorm(x, w[:32]), ValueError), (lambda: mxq.mxfp8_rmsnorm(x[:, :40], w[:40]), ValueError),
            (lambda: mxq.mxfp8_rmsnorm(x, w, residual=x[:2]), ValueError),
            (lambda: mxq.mxfp8_rmsnorm(x, w, residual=x.float()), ValueError),
            (lambda: mxq.mxfp8_rmsnorm(x, w, eps=-1.0), mxq.MxqError), (lambda: mxq.mxfp8_rmsnorm(x, w, eps=float("nan")), mxq.MxqError),
            (lambda: mxq.mxfp8_rmsnorm(x.t(), w[:4]), ValueError),
            (lambda: mxq.rmsnorm_backward(x, x, w, rstd[:2]), TypeError), (lambda: mxq.rmsnorm_backward(x[:2], x, w, rstd), ValueError),
            (lambda: mxq.rmsnorm_backward(x.float(), x, w, rstd), ValueError),
            (lambda: mxq.rmsnorm_backward(x, x, w, rstd, grad_hidden=x[:, :32]), ValueError),
            (lambda: mxq.rmsnorm_backward(x[:, :12], x[:, :12], w[:12], rstd), ValueError)):
        with pytest.raises(kind):
            call()
