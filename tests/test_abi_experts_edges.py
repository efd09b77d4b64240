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
