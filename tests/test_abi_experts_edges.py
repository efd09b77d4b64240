"""Host checks of the 4-bit products' and the routing's entry points at sizes
of zero and at counts beyond their types. Runs only without a GPU, like
test_abi.py: the addresses are fake."""
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, CUDA, ARG = range(8)
A = 0x10000

if torch.cuda.is_available():
    pytest.skip("host-validation tests with fake addresses run without a GPU only", allow_module_level=True)


def test_a_global_scale_is_asked_for_without_columns_too():
    """K == 0: the products write zeros, and the kernel still reads the scale."""
    one = lambda g: mxq.lib.nvfp4_matvec(None, 0, 2, 0, 0, None, None, g, 8, A, 0, None)
    stack = lambda g: mxq.lib.nvfp4_matvec_grouped(None, 0, 4, 0, 0, None, None, g, 1, 3, 8, A, 4, None, 1, 0, A, 0, None)
    for f in (one, stack):
        assert f(None) == NULL
        assert f(A) == CUDA                         # the checks pass, the launch fails here
    assert mxq.lib.nvfp4_matvec(None, 0, 0, 0, 0, None, None, None, 8, None, 0, None) == OK


def test_python_refuses_counts_of_the_products_beyond_32_bits():
    """Cut off to 1, 2^32 + 1 would be taken as another count."""
    big = 2 ** 32 + 1
    x, off, order = torch.zeros(2, 64), [0, 2], torch.zeros(2, dtype=torch.int32)
    w, s = torch.zeros(1, 8, 32, dtype=torch.uint8), torch.zeros(1, 8, 4, dtype=torch.uint8)
    for call in (lambda: mxq.mxfp4_matvec_grouped(x, w, s[..., :2].contiguous(), off, order=order, top_k=big),
                 lambda: mxq.nvfp4_matvec_grouped(x, w, s, torch.ones(1), off, order=order, top_k=big)):
        with pytest.raises(ValueError, match="^top_k must fit"):
            call()


def test_python_refuses_sizes_beyond_32_bits(monkeypatch):
    """Sizes that come with a tensor (none of these holds any memory)."""
    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    big = 2 ** 32 + 1
    meta = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="meta")
    with pytest.raises(ValueError, match="^E must fit"):
        mxq.moe_route(meta(1, big), 1)
    with pytest.raises(ValueError, match="^E must fit"):
        mxq.moe_route_backward(meta(1, 1), meta(1, big), meta(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="^E must fit"):
        u8 = torch.uint8
        mxq.mxfp4_matvec_grouped(meta(1, 32), meta(big, 8, 16, dtype=u8), meta(big, 8, 1, dtype=u8), [0, 1])


def test_an_order_of_no_rows_may_be_null():
    """A batch without tokens: an empty array need not have an address."""
    f, g = mxq.lib.mxfp4_matvec_grouped, mxq.lib.nvfp4_matvec_grouped
    assert f(None, 0, 0, 64, 64, A, A, 3, 8, A, 0, None, 8, 0, None, 0, None) == OK
    assert g(None, 0, 0, 64, 64, A, A, A, 1, 3, 8, A, 0, None, 8, 1, None, 0, None) == OK
    assert f(None, 0, 5, 64, 64, A, A, 3, 8, A, 0, None, 2, 0, None, 0, None) == OK
    assert f(A, 0, 0, 64, 64, A, A, 3, 8, A, 4, None, 8, 0, A, 0, None) == ARG


def test_combine_of_no_choices_asks_for_every_token(monkeypatch):
    """The output's rows are the library's to write (zeros), not left as allocated."""
    calls = []
    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_int32", lambda t, index, what: t)
    monkeypatch.setattr(mxq, "_launch", lambda fn, index, *args: calls.append(args))
    for shape, T in (((5, 0), 5), ((2, 3, 0), 6), ((0,), 1), ((0, 2), 0), ((4, 2), 4)):
        y = mxq.moe_combine(torch.ones(4, 12), torch.empty(shape, dtype=torch.int32), torch.empty(shape))
        assert y.shape == (*shape[:-1], 12) and calls[-1][5:7] == (T, shape[-1])


def test_rows_without_columns_need_no_alignment():
    """The row stride of a contiguous [M, 0] tensor is 1."""
    for x, ld in ((None, 1), (A + 2, 3)):
        assert mxq.lib.mxfp4_matvec(x, 0, 3, 0, ld, None, None, 8, A, 0, None) == CUDA
        assert mxq.lib.nvfp4_matvec(x, 1, 3, 0, ld, None, None, A, 8, A, 0, None) == CUDA
    assert mxq.lib.mxfp4_matvec(None, 0, 3, 0, 1, None, None, 8, A + 8, 0, None) == ALIGN
    assert mxq.lib.mxfp4_matvec(A + 2, 0, 3, 32, 40, A, A, 8, A, 0, None) == ALIGN


def test_one_row_with_a_stride_is_refused():
    """A column of a matrix is one row whose elements lie apart."""
    base = torch.zeros(8, 4)
    for x in (base[:, 1], base[0, ::2], base[:, 1:2], base.t(), base.t()[None]):
        if x.dim() == 2 and x.shape[-1] == 1:
            assert mxq._rows_view(x) == (8, 1, 4)
            continue
        with pytest.raises(ValueError, match="contiguous"):
            mxq._rows_view(x)
    assert mxq._rows_view(base[3]) == (1, 4, 4) and mxq._rows_view(base[:1, 0]) == (1, 1, 1)


def test_refused_counts_allocate_no_outputs_of_their_size(monkeypatch):
    """The library refuses the count; an output of that size may not fit."""
    sizes = []

    def allocate(shape, dtype, device):
        sizes.append(torch.Size(shape).numel())
        return torch.empty(min(sizes[-1], 4096), dtype=dtype)[:sizes[-1]].view(shape)

    def launch(fn, index, *args):
        mxq._check(fn, getattr(mxq.lib, fn)(*args, None))

    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_int32", lambda t, index, what: t)
    monkeypatch.setattr(mxq, "_launch", launch)
    prev = mxq.set_output_allocator(allocate)
    try:
        for call in (lambda: mxq.moe_route(torch.zeros(4, 64), 2 ** 31 - 1), lambda: mxq.moe_route(torch.zeros(4, 64), 33),
                     lambda: mxq.moe_route(torch.zeros(4, 64), -1), lambda: mxq.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), 2 ** 31 - 1),
                     lambda: mxq.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), 1025),
                     lambda: mxq.moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), -1)):
            with pytest.raises(mxq.MxqError, match="status 2"):
                call()
    finally:
        mxq.set_output_allocator(prev)
    assert max(sizes) <= 1025


def test_global_scales_in_another_order_are_refused(monkeypatch):
    """[2, E] holds the values of [E, 2] in another order: read as they lie, an
    expert would get another's scales."""
    calls = []
    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_launch", lambda fn, index, *args: calls.append(args))
    x, E = torch.zeros(3, 64, dtype=torch.bfloat16), 3
    w, s = torch.zeros(E, 8, 32, dtype=torch.uint8), torch.zeros(E, 8, 4, dtype=torch.uint8)
    for shape in ((2, E), (1, 2, E), (2 * E, 1)):
        with pytest.raises(ValueError, match=r"must be \[E, 2\]"):
            mxq.nvfp4_matvec_grouped(x, w, s, torch.ones(shape), [0, 1, 2, 3])
    assert not calls
    for shape, per in (((E,), 1), ((E, 1), 1), ((E, 2), 2), ((2 * E,), 2)):
        mxq.nvfp4_matvec_grouped(x, w, s, torch.ones(shape), [0, 1, 2, 3])
        assert calls[-1][8] == per


def test_a_stack_of_no_experts_is_refused_by_the_library(monkeypatch):
    monkeypatch.setattr(mxq, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(mxq, "_launch", lambda fn, index, *args: mxq._check(fn, getattr(mxq.lib, fn)(*args, None)))
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    w, s = torch.zeros(0, 8, 32, dtype=torch.uint8), torch.zeros(0, 8, 4, dtype=torch.uint8)
    with pytest.raises(mxq.MxqError, match="status 2"):
        mxq.nvfp4_matvec_grouped(x, w, s, torch.ones(0), [0])
    with pytest.raises(mxq.MxqError, match="status 2"):
        mxq.mxfp4_matvec_grouped(x, w, s[..., :2].contiguous(), [0])
