"""Host checks of the 4-bit products' and the routing's C entry points: each
bad argument gives its documented status before anything is enqueued. Runs only
without a GPU, like test_abi.py: the addresses are fake."""
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, CUDA, ARG = range(8)
A = 0x10000

if torch.cuda.is_available():
    pytest.skip("host-validation tests with fake addresses run without a GPU only", allow_module_level=True)


def edit(args, **changes):
    args = dict(args, **changes)
    return tuple(args.values())


MV = dict(x=A, dt=0, M=2, K=64, ld=64, p=A, s=A, N=8, y=A, out=0, stream=None)
NV = dict(x=A, dt=0, M=2, K=64, ld=64, p=A, s=A, g=A, N=8, y=A, out=0, stream=None)
MG = dict(x=A, dt=0, xr=4, K=64, ld=64, p=A, s=A, E=3, N=8, off=A, R=4, order=None, k=1, sw=0, y=A, out=0, stream=None)
NG = dict(x=A, dt=0, xr=4, K=64, ld=64, p=A, s=A, g=A, per=1, E=3, N=8, off=A, R=4, order=None, k=1, sw=0, y=A, out=0, stream=None)


@pytest.mark.parametrize("fn,base,block", [("mxfp4_matvec", MV, 32), ("nvfp4_matvec", NV, 16),
                                           ("mxfp4_matvec_grouped", MG, 32), ("nvfp4_matvec_grouped", NG, 16)])
def test_products(fn, base, block):
    f = getattr(mxq.lib, fn)
    rows = "M" if "M" in base else "R"
    assert f(*edit(base)) == CUDA                   # the checks pass, the launch fails here
    assert f(*edit(base, dt=2)) == DTYPE
    assert f(*edit(base, out=-1)) == DTYPE
    assert f(*edit(base, K=block // 2)) == SHAPE
    assert f(*edit(base, K=-block)) == SHAPE
    assert f(*edit(base, N=-1)) == SHAPE
    assert f(*edit(base, ld=32)) == SHAPE
    assert f(*edit(base, N=1 << 31)) == SHAPE
    assert f(*edit(base, K=1 << 32, ld=1 << 32)) == SHAPE
    for p in ("x", "p", "s", "y") + (("g",) if "g" in base else ()):
        assert f(*edit(base, **{p: None})) == NULL
    for p in ("x", "p", "y"):
        assert f(*edit(base, **{p: A + 8})) == ALIGN
    assert f(*edit(base, ld=68)) == ALIGN
    assert f(*edit(base, s=A + 1)) == CUDA          # scales have no alignment
    assert f(*edit(base, N=0, y=None)) == OK
    empty = {rows: 0, "x": None, "y": None, "p": None, "s": None}
    if rows == "R":
        empty.update(xr=0, off=None)
    assert f(*edit(base, **empty)) == OK
    assert f(*edit(base, **{rows: -1, **({"xr": -1} if rows == "R" else {})})) == SHAPE
    if "g" in base:
        assert f(*edit(base, g=A + 2)) == ALIGN


@pytest.mark.parametrize("fn,base", [("mxfp4_matvec_grouped", MG), ("nvfp4_matvec_grouped", NG)])
def test_grouped(fn, base):
    f = getattr(mxq.lib, fn)
    assert f(*edit(base, E=0)) == SHAPE
    assert f(*edit(base, E=1025)) == SHAPE
    assert f(*edit(base, off=None)) == NULL
    assert f(*edit(base, off=A + 4)) == ALIGN
    assert f(*edit(base, R=5)) == ARG               # without an order x has the R rows
    assert f(*edit(base, k=2)) == ARG
    assert f(*edit(base, order=A, k=0)) == ARG
    assert f(*edit(base, order=A + 2, k=2)) == ALIGN
    assert f(*edit(base, order=A, k=2, R=9)) == CUDA
    assert f(*edit(base, sw=2)) == ARG
    assert f(*edit(base, sw=1, N=7)) == SHAPE
    assert f(*edit(base, sw=1)) == CUDA
    if "per" in base:
        assert f(*edit(base, per=3)) == ARG
        assert f(*edit(base, per=2, N=7)) == SHAPE
        assert f(*edit(base, per=2)) == CUDA


def test_combine():
    f = mxq.lib.moe_combine
    base = dict(rows=A, R=4, N=8, pos=A, w=A, T=2, k=2, y=A, out=0, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, out=5)) == DTYPE
    for n in ("R", "N", "T", "k"):
        assert f(*edit(base, **{n: -1})) == SHAPE
    for p in ("rows", "pos", "w", "y"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 2})) == ALIGN
    assert f(*edit(base, T=0, y=None)) == OK
    assert f(*edit(base, T=1 << 30, N=1 << 20)) == SHAPE


def test_route():
    f = mxq.lib.moe_route
    base = dict(l=A, dt=1, T=4, E=16, ld=16, sc=0, b=None, g=1, tg=1, k=2, rn=1, scale=1.0, w=A, e=A, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=3)) == DTYPE
    for n, v in (("T", -1), ("E", 0), ("E", 1025), ("ld", 15), ("k", 0), ("k", 17), ("g", 0), ("g", 3), ("g", 33), ("tg", 0), ("tg", 2)):
        assert f(*edit(base, **{n: v})) == SHAPE, (n, v)
    assert f(*edit(base, E=64, ld=64, k=33)) == SHAPE
    assert f(*edit(base, g=8, tg=2, k=5)) == SHAPE
    assert f(*edit(base, sc=2)) == ARG
    assert f(*edit(base, rn=2)) == ARG
    for p in ("l", "w", "e"):
        assert f(*edit(base, **{p: None})) == NULL
    for p in ("l", "w", "e", "b"):
        assert f(*edit(base, **{p: A + 2})) == ALIGN
    assert f(*edit(base, dt=0, l=A + 2)) == CUDA
    assert f(*edit(base, T=0, l=None, w=None, e=None)) == OK


def test_route_backward():
    f = mxq.lib.moe_route_backward
    base = dict(gw=A, l=A, dt=1, T=4, E=16, ld=16, e=A, sc=0, k=2, rn=1, scale=1.0, gl=A, stream=None)
    assert f(*edit(base)) == CUDA
    assert f(*edit(base, dt=3)) == DTYPE
    for n, v in (("T", -1), ("E", 0), ("E", 1025), ("ld", 15), ("k", 0), ("k", 17)):
        assert f(*edit(base, **{n: v})) == SHAPE
    assert f(*edit(base, sc=-1)) == ARG
    for p in ("gw", "l", "e", "gl"):
        assert f(*edit(base, **{p: None})) == NULL
        assert f(*edit(base, **{p: A + 2})) == ALIGN
    assert f(*edit(base, T=0, gw=None, l=None, e=None, gl=None)) == OK


def test_dispatch():
    f = mxq.lib.moe_dispatch
    base = dict(e=A, P=10, E=4, off=A, order=A, pos=A, ws=None, n=0, stream=None)
    assert f(*edit(base)) == CUDA
    for n, v in (("P", -1), ("P", 1 << 31), ("E", 0), ("E", 1025)):
        assert f(*edit(base, **{n: v})) == SHAPE
    for p in ("e", "off", "order", "pos"):
        assert f(*edit(base, **{p: None})) == NULL
    for p, d in (("e", 2), ("off", 4), ("order", 1), ("pos", 2)):
        assert f(*edit(base, **{p: A + d})) == ALIGN
    assert f(*edit(base, P=0, e=None, order=None, pos=None)) == CUDA      # row_offsets are written
    need = mxq.lib.mxq_moe_dispatch_workspace_bytes
    assert need(4096, 64) == 0 and need(-1, 4) == 0 and need(9999, 0) == 0
    assert need(4097, 64) == 2 * 65 * 4 and need(131072, 256) == 32 * 257 * 4
    assert need(2 ** 31 - 1, 1024) <= 128 * 1025 * 4
    big = dict(base, P=5000, ws=A, n=need(5000, 4))
    assert f(*edit(big)) == CUDA
    assert f(*edit(big, ws=None)) == WORKSPACE
    assert f(*edit(big, n=big["n"] - 1)) == WORKSPACE
    assert f(*edit(big, ws=A + 2)) == ALIGN


def test_python_refuses_host_tensors():
    u8 = torch.zeros(8, 32, dtype=torch.uint8)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: mxq.mxfp4_matvec(x, u8, u8[:, :2]), lambda: mxq.moe_route(x, 2),
                 lambda: mxq.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), 4),
                 lambda: mxq.moe_combine(x.float(), torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1))):
        with pytest.raises(ValueError):
            call()


def test_python_refuses_counts_beyond_32_bits():
    logits, pairs = torch.zeros(2, 64), torch.zeros(4, 2, dtype=torch.int32)
    big = 2 ** 32 + 1                 # cut off to 1 without the check
    for what, call in (("top_k", lambda: mxq.moe_route(logits, big)),
                       ("groups", lambda: mxq.moe_route(logits, 2, groups=big)),
                       ("top_groups", lambda: mxq.moe_route(logits, 2, groups=4, top_groups=big)),
                       ("E", lambda: mxq.moe_dispatch(pairs, big))):
        with pytest.raises(ValueError, match=f"^{what} must fit"):
            call()
