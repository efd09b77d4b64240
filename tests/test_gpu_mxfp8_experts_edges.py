"""The experts' MXFP8 products, their transposes and the norm where they are
used with other things: streams, graphs, first calls of a process, buffers that
a caller shares between arguments, and more than 2^31 elements."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def on_device(*off):
    return torch.tensor(off, dtype=torch.int64, device="cuda")


FIRST_CALLS = """
import torch
import nvfp4_block_scaled_sm_b200 as mxq

torch.manual_seed(0)
E, M, N, K = 5, {M}, 512, 256
x, r = (torch.randn(M, K, device="cuda").to(torch.bfloat16) for _ in range(2))
w, n = torch.randn(E, N, K, device="cuda").to(torch.bfloat16), torch.ones(K, device="cuda")
cut = torch.tensor([0, M // 3, M // 3, M // 2, M - 1, M], device="cuda")
qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)      # (a stack's offsets come from the host)


def layer():
    a = mxq.mxfp8_rmsnorm(x, n, residual=r, swizzled=True, normed=True)
    q, s, z = mxq.mxfp8_quantize_grouped(a.normed, row_offsets=cut, swizzled=True)
    h = mxq.mxfp8_gemm_grouped(q, z, qw, zw, cut, swiglu=True)
    y = mxq.mxfp8_gemm_grouped(q, z, qw, zw, cut, torch.float32)
    qt, zt = mxq.mxfp8_quantize_columnwise_grouped(a.normed, row_offsets=cut)
    ht, hz = mxq.mxfp8_quantize_columnwise_grouped(h, row_offsets=cut)
    wt = mxq.mxfp8_quantize_columnwise_grouped(w)
    return (*a, h, y, qt, zt, ht, hz, *wt, mxq.mxfp8_gemm_grouped_wgrad(ht, hz, qt, zt, cut),
            *mxq.rmsnorm_backward(r, a.hidden, n, a.rstd, grad_hidden=x))


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = layer()
graph.replay()
torch.cuda.synchronize()
captured = [t.clone() for t in captured]
for a, b in zip(captured, layer()):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
print("first calls ok")
"""


# SwiGLU's weight scales go through groups of eight K blocks, two at a time: one block, ends of and
# inside a group, more groups than are held; one tile and several for a pair of CTAs
@pytest.mark.parametrize("K", [32, 1024, 1056, 2048, 2176, 4000])
@pytest.mark.parametrize("E,M,H", [(3, 700, 256), (2, 9000, 640), (9, 9, 128)])
def test_swiglu_over_k(E, M, H, K):
    cut = torch.linspace(0, M, E + 1).long()
    off = on_device(*cut.tolist())
    qx, sx, zx = mxq.mxfp8_quantize_grouped(normal(K, M, K), row_offsets=off, swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(normal(H, E, 2 * H, K, scale=0.05), swizzled=True)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, off, FP32, swiglu=True, error_flag=flag)
    want, bound = R.swiglu(*R.grouped(R.values(qx, sx), R.values(qw, sw), cut.tolist()), K)
    R.check(y, want, bound, f"swiglu {E} {M} {H} {K}")
    assert int(flag) == 0


@pytest.mark.parametrize("swiglu", [False, True])
def test_a_sum_of_nothing(swiglu):
    """K = 0: the experts' rows are zeros, rows of no expert are left."""
    M, N, E = 3000, 512, 4
    none = lambda *shape: torch.empty(*shape, dtype=torch.uint8, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.full((M, N // 2 if swiglu else N), 7.0, dtype=BF16, device="cuda")
    off = on_device(0, 5, 5, 1700, 2990)
    st = mxq.lib.mxfp8_gemm_grouped(None, None, 0, None, None, E, off.data_ptr(), M, N, 0, int(swiglu), d.data_ptr(), 0,
                                    flag.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert not d[:2990].any() and (d[2990:] == 7).all() and int(flag) == 0
    y = mxq.mxfp8_gemm_grouped(none(M, 0), none(0), none(E, N, 0), none(0), off, swiglu=swiglu)
    assert not y[:2990].any()


@pytest.mark.parametrize("M", [7, 1500])
def test_first_calls_of_a_process_inside_a_capture(M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(mxq.__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(M=M)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls ok" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once():
    """Calls share nothing: results on two busy streams are those of one."""
    E, M, N, K = 6, 900, 768, 640
    off = on_device(0, 100, 430, 430, 700, 880, 900)
    w = mxq.mxfp8_quantize_grouped(normal(1, E, N, K, scale=0.1), swizzled=True)
    weight = normal(2, K) + 1

    def work(seed):
        n = mxq.mxfp8_rmsnorm(normal(seed, M, K), weight, normed=True)
        q, s, z = mxq.mxfp8_quantize_grouped(n.normed, row_offsets=off, swizzled=True)
        y = mxq.mxfp8_gemm_grouped(q, z, w[0], w[2], off, swiglu=True)
        t, tz = mxq.mxfp8_quantize_columnwise_grouped(y, row_offsets=off)
        return [n.rstd, y, t, tz, mxq.mxfp8_gemm_grouped_wgrad(t, tz, t, tz, off),
                *mxq.rmsnorm_backward(n.normed, n.hidden, weight, n.rstd)]

    want = {s: work(s) for s in (1, 2)}
    torch.cuda.synchronize()
    streams = {s: torch.cuda.Stream() for s in (1, 2)}
    got = {1: [], 2: []}
    for _ in range(4):
        for s, st in streams.items():
            with torch.cuda.stream(st):
                got[s].append(work(s))
    torch.cuda.synchronize()
    for s in (1, 2):
        for run in got[s]:
            for a, b in zip(run, want[s]):
                assert torch.equal(a, b)


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N", [96, 7168, 40960])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_hidden_in_place_of_an_input(dtype, N, into):
    """The C entry allows hidden to be x or residual itself."""
    M, code = 5, 0 if dtype == BF16 else 1
    x, r, w = normal(1, M, N, dtype=dtype), normal(2, M, N, dtype=dtype), normal(3, N)
    want = mxq.mxfp8_rmsnorm(x, w, residual=r)
    q, s = torch.empty_like(want.qweight), torch.empty_like(want.scale)
    rstd = torch.empty_like(want.rstd)
    hidden = x if into == "x" else r
    st = torch.cuda.current_stream().cuda_stream
    assert mxq.lib.mxfp8_rmsnorm(ptr(x), code, M, N, N, ptr(r), N, ptr(w), 0, 1e-6, ptr(hidden), ptr(q), ptr(s), None, None, ptr(rstd), st) == 0
    for a, b in ((hidden, want.hidden), (q, want.qweight), (s, want.scale), (rstd, want.rstd)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N", [96, 7168, 20480])
@pytest.mark.parametrize("into", ["grad", "grad_hidden"])
def test_gradient_in_place_of_an_input(dtype, N, into):
    M, code = 300, 0 if dtype == BF16 else 1
    g, h, gh = (normal(i, M, N, dtype=dtype) for i in (1, 2, 3))
    w = normal(4, N)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    want, want_w = mxq.rmsnorm_backward(g, h, w, rstd, grad_hidden=gh)
    out, dw = g if into == "grad" else gh, torch.empty_like(w)
    n = mxq.lib.mxq_rmsnorm_backward_workspace_bytes(M, N)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert mxq.lib.mxq_rmsnorm_backward(ptr(g), code, M, N, N, ptr(h), N, ptr(w), 0, ptr(rstd), ptr(gh), N, ptr(out), ptr(dw), ptr(work), n, st) == 0
    assert torch.equal(out, want) and torch.equal(dw, want_w)


def test_without_a_weight_gradient_no_workspace_is_touched():
    M, N = 40, 256
    g, h, w = normal(1, M, N), normal(2, M, N), normal(3, N)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    dx, st = torch.empty_like(h), torch.cuda.current_stream().cuda_stream
    assert mxq.lib.mxq_rmsnorm_backward(ptr(g), 0, M, N, N, ptr(h), N, ptr(w), 0, ptr(rstd), None, 0, ptr(dx), None, None, 0, st) == 0
    assert torch.equal(dx, mxq.rmsnorm_backward(g, h, w, rstd)[0])


def test_nan_and_infinities_stay_in_their_rows_and_columns():
    """A NaN code in one row, and one in another expert's weight, reach only what the formula gives them."""
    E, M, N, K = 3, 300, 144, 160
    x, w = normal(1, M, K), normal(2, E, N, K)
    off = [0, 100, 101, 300]
    x[100, 3] = float("nan")                                     # the only row of expert 1, inside the others' tiles
    w[1, 5] = float("nan")
    q, s, z = mxq.mxfp8_quantize_grouped(x, row_offsets=on_device(*off), swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)
    y = mxq.mxfp8_gemm_grouped(q, z, qw, zw, on_device(*off), FP32)
    want, mags = R.grouped(R.values(q, s), R.values(qw, sw), off)
    assert bool(torch.isnan(y[100]).all()) and not torch.isnan(y[:100]).any() and not torch.isnan(y[101:]).any()
    R.check(y[:100], want[:100], K * R.U * mags[:100], "expert 0")
    R.check(y[101:], want[101:], K * R.U * mags[101:], "expert 2")


@pytest.mark.parametrize("tail", [32, 64, 96])
def test_what_lies_behind_k_is_not_read(tail):
    """K ends inside a block of 128: the next row's codes (here NaN) are not part of the sum."""
    K = 128 + tail
    x = normal(1, 40, K)
    w = normal(2, 2, 64, K)
    off = on_device(0, 17, 40)
    q, s, z = mxq.mxfp8_quantize_grouped(x, row_offsets=off, swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)
    q[18:] = 0x7F
    qw[1, 1:] = 0x7F
    y = mxq.mxfp8_gemm_grouped(q, z, qw, zw, off, FP32)
    assert not torch.isnan(y[:17]).any() and not torch.isnan(y[17, 0])
    want, mags = R.grouped(R.values(q, s)[:17], R.values(qw, sw)[:1], [0, 17])
    R.check(y[:17], want, K * R.U * mags, "expert 0")


# ------------------------------------------------- beyond 2^31 elements

@pytest.fixture
def plain_allocator():
    prev = mxq.set_output_allocator(None)
    yield
    mxq.set_output_allocator(prev)
    torch.cuda.empty_cache()


@pytest.mark.slow
def test_large_norm(plain_allocator):
    M, N = 300_001, 7168                                         # 2.15e9 elements
    x, w = torch.empty(M, N, dtype=BF16, device="cuda"), normal(1, N)
    for i in range(0, M, 50_000):
        x[i:i + 50_000] = normal(i, min(50_000, M - i), N)
    r = mxq.mxfp8_rmsnorm(x, w, residual=x, swizzled=True)
    dx, _ = mxq.rmsnorm_backward(x, r.hidden, w, r.rstd)
    for rows in (slice(0, 300), slice(299_700, M)):
        part = mxq.mxfp8_rmsnorm(x[rows], w, residual=x[rows])
        for a, b in ((r.qweight, part.qweight), (r.scale, part.scale), (r.hidden, part.hidden), (r.rstd, part.rstd)):
            assert torch.equal(a[rows], b)
        assert torch.equal(dx[rows], mxq.rmsnorm_backward(x[rows], part.hidden, w, part.rstd)[0])
        assert torch.equal(R.untile(r.scale_swizzled, M, N // 32)[rows], part.scale)


@pytest.mark.slow
def test_large_transpose_and_products(plain_allocator):
    M, N = 70_000, 32_768                                        # 2.3e9 elements
    off = on_device(0, 1000, 1000, 69_990, M)
    x = torch.empty(M, N, dtype=BF16, device="cuda")
    for i in range(0, M, 10_000):
        x[i:i + 10_000] = normal(i, min(10_000, M - i), N)
    q, z = mxq.mxfp8_quantize_columnwise_grouped(x, row_offsets=off)
    P = q.shape[1]
    start = R.padded(off.tolist())
    for c in (slice(0, 64), slice(N - 64, N)):
        for e, (a, b) in enumerate(((0, 1000), (1000, 1000), (1000, 69_990), (69_990, M))):
            if b > a:
                want, ws = mxq.mxfp8_quantize_columnwise(x[a:b, c].contiguous())
                assert torch.equal(q[c, start[e]:start[e] + b - a], want)
    assert not q[:, start[-1]:].any()
    # an output of 2.3e9 elements: rows of 32 values against a weight of one block
    qx, sx, zx = mxq.mxfp8_quantize_grouped(x[:, :32].contiguous(), row_offsets=off, swizzled=True)
    del x, q, z
    qw, sw, zw = mxq.mxfp8_quantize_grouped(normal(5, 4, N, 32), swizzled=True)
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, off)
    a, b = R.values(qx, sx), R.values(qw, sw)
    for e, rows in ((0, slice(900, 1000)), (2, slice(69_900, 69_990)), (3, slice(69_990, M))):
        want, mags = R.grouped(a[rows], b[e:e + 1], [0, rows.stop - rows.start])
        R.check(y[rows], want, 32 * R.U * mags, "large")
