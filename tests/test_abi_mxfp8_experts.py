"""Host checks of the C entry points of the experts' MXFP8 products, their
transposes and the norm: each bad argument gives its documented status before
anything is enqueued. Runs only without a GPU: the addresses are fake."""
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, CUDA, ARG = range(8)
A = 0x10000

if torch.cuda.is_available():
    pytest.skip("host-validation tests with fake addresses run without a GPU only", allow_module_level=True)


def edit(args, **changes):
    return tuple(dict(args, **changes).values())


def test_gemm_grouped():
    f = mxq.lib.mxfp8_gemm_grouped
    base = dict(qa=A, sa=A, sab=2048, qb=A, sb=A, E=3, off=A, M=4, N=256, K=64, sw=0, d=A, out=0, err=None, stream=None)
    assert f(*edit(base)) == CUDA                   # the checks pass; no driver here
    assert f(*edit(base, out=2)) == DTYPE
    assert f(*edit(base, sw=2)) == ARG
    for bad in (dict(E=0), dict(E=1025), dict(M=-1), dict(N=-16), dict(K=-32), dict(K=48), dict(N=24), dict(sw=1, N=128), dict(sab=-1),
                dict(sab=0), dict(sab=600), dict(M=600), dict(M=1 << 31), dict(N=1 << 31), dict(K=(1 << 26) + 32), dict(N=1 << 30),
                dict(N=(1 << 29), K=1 << 20),
                dict(K=1 << 31)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for p in ("qa", "sa", "qb", "sb", "d", "off"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 4})) == ALIGN
    assert f(*edit(base, M=0, qa=None, d=None, off=None)) == OK
    assert f(*edit(base, N=0, qb=None, d=None)) == OK
    assert f(*edit(base, K=0, qa=None, qb=None, sa=None, sb=None, sab=0)) == CUDA


def test_wgrad():
    f = mxq.lib.mxfp8_gemm_grouped_wgrad
    base = dict(qa=A, sa=A, qb=A, sb=A, E=3, off=A, P=384, Na=16, Nb=32, d=A, out=1, err=None, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, out=-1)) == DTYPE
    for bad in (dict(E=0), dict(E=1025), dict(P=64), dict(P=-128), dict(Na=-1), dict(Nb=8), dict(Nb=-16), dict(P=(1 << 26) + 128), dict(Na=1 << 31),
                dict(Nb=1 << 31), dict(Na=1 << 30, Nb=1 << 30), dict(Na=1 << 30, P=1 << 20)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for p in ("qa", "sa", "qb", "sb", "d", "off"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 4})) == ALIGN
    assert f(*edit(base, Na=0, d=None)) == OK
    assert f(*edit(base, P=0, qa=None, qb=None, sa=None, sb=None)) == CUDA


def test_columnwise():
    f = mxq.lib.mxfp8_quantize_columnwise_grouped
    base = dict(x=A, dt=0, E=3, off=A, M=40, N=32, ld=32, q=A, s=A, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=2)) == DTYPE
    for bad in (dict(E=0), dict(E=1025), dict(M=-1), dict(N=24), dict(N=-16), dict(ld=16), dict(M=1 << 31), dict(N=1 << 31, ld=1 << 31),
                dict(M=1 << 30, N=1 << 30, ld=1 << 30), dict(ld=1 << 60)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for p in ("x", "off", "q", "s"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 4})) == ALIGN
    assert f(*edit(base, ld=36)) == ALIGN
    assert f(*edit(base, E=1, M=0, x=None, off=None, q=None, s=None)) == OK
    assert f(*edit(base, M=0, x=None)) == CUDA      # columns of no row are written
    f = mxq.lib.mxfp8_quantize_columnwise_stacked
    base = dict(x=A, dt=0, E=3, R=64, N=32, q=A, s=A, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=2)) == DTYPE
    for bad in (dict(E=0), dict(E=1025), dict(R=48), dict(R=-32), dict(N=24), dict(R=1 << 31), dict(N=1 << 31), dict(R=1 << 30, N=1 << 30)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for p in ("x", "q", "s"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 8})) == ALIGN
    assert f(*edit(base, R=0, x=None, q=None)) == OK


def test_norm():
    f = mxq.lib.mxfp8_rmsnorm
    base = dict(x=A, dt=0, M=4, N=64, ld=64, res=A, ldr=64, w=A, wdt=1, eps=1e-6, h=A, q=A, s=A, swz=A, y=A, rstd=A, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=2)) == DTYPE
    assert f(*edit(base, wdt=-1)) == DTYPE
    for bad in (dict(M=-1), dict(N=48), dict(N=-32), dict(ld=32), dict(ldr=32), dict(M=1 << 31), dict(N=1 << 30, ld=1 << 30, ldr=1 << 30)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(h=None), dict(res=None)):
        assert f(*edit(base, **bad)) == ARG, bad
    for p in ("x", "w", "q", "s", "rstd"):
        assert f(*edit(base, **{p: None})) == NULL
    for p in ("x", "w", "q", "h", "y", "res", "swz"):
        assert f(*edit(base, **{p: A + 8})) == ALIGN
    assert f(*edit(base, rstd=A + 2)) == ALIGN
    assert f(*edit(base, ld=68)) == ALIGN
    assert f(*edit(base, s=A + 1, swz=None, y=None)) == CUDA
    assert f(*edit(base, M=0, x=None)) == OK


def test_norm_backward():
    f = mxq.lib.mxq_rmsnorm_backward
    n = mxq.lib.mxq_rmsnorm_backward_workspace_bytes(400, 64)
    assert n == 400 * 64 * 4
    base = dict(g=A, dt=0, M=400, N=64, ldg=64, h=A, ldh=64, w=A, wdt=1, rstd=A, gh=A, ldgh=64, dx=A, dw=A, ws=A, wsb=n, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=2)) == DTYPE
    assert f(*edit(base, wdt=2)) == DTYPE
    for bad in (dict(M=-1), dict(N=12), dict(N=-8), dict(ldg=32), dict(ldh=32), dict(ldgh=32), dict(M=1 << 31)):
        assert f(*edit(base, **bad)) == SHAPE, bad
    for p in ("g", "h", "w", "rstd", "dx"):
        assert f(*edit(base, **{p: None})) == NULL
    for p in ("g", "h", "w", "gh", "dx", "ws"):
        assert f(*edit(base, **{p: A + 8})) == ALIGN
    for bad in (dict(ldg=68), dict(ldh=68), dict(ldgh=68), dict(rstd=A + 2), dict(dw=A + 2)):
        assert f(*edit(base, **bad)) == ALIGN, bad
    assert f(*edit(base, ws=None)) == WORKSPACE
    assert f(*edit(base, wsb=n - 1)) == WORKSPACE
    assert f(*edit(base, dw=None, ws=None, wsb=0, gh=None, ldgh=0)) == CUDA
    assert f(*edit(base, M=0, dw=None)) == OK
    assert mxq.lib.mxq_rmsnorm_backward_workspace_bytes(64, 64) == 0 < mxq.lib.mxq_rmsnorm_backward_workspace_bytes(65, 64)
    assert mxq.lib.mxq_rmsnorm_backward_workspace_bytes(17, 16384) == 17 * 16384 * 4
    assert f(*edit(base, M=64, ws=None, wsb=0)) == CUDA


def test_sizes():
    assert mxq.lib.mxq_grouped_padded_rows(3, 10) == 384
    assert mxq.lib.mxq_grouped_padded_rows(1, 1) == 128
    assert mxq.lib.mxq_grouped_padded_rows(1, 0) == 0
    assert mxq.lib.mxq_grouped_padded_rows(-1, 5) == -1
    assert mxq.lib.mxq_rmsnorm_backward_workspace_bytes(0, 64) == 0


def test_sizes_in_python_are_the_librarys():
    for M in (0, 1, 127, 128, 129, 5000):
        for S in (0, 1, 3, 4, 5, 224):
            assert mxq._tile_bytes(M, S) == mxq.lib.mxq_swizzled_scale_bytes(M, S)
        for E in (1, 3, 1024):
            assert (M + 127 * E) // 128 * 128 == mxq.lib.mxq_grouped_padded_rows(E, M)
