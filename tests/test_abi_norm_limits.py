"""Which calls of the norm's gradient need a workspace, as include/mxq.h states it:
none for few rows, M <= 64, N <= 16384 and M N <= 2^18. Runs only without a GPU:
the addresses are fake."""
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, CUDA, ARG = range(8)
A = 0x10000

if torch.cuda.is_available():
    pytest.skip("host-validation tests with fake addresses run without a GPU only", allow_module_level=True)


def call(M, N, work, nbytes, dweight=A):
    return mxq.lib.mxq_rmsnorm_backward(A, 0, M, N, N, A, N, A, 0, A, None, 0, A, dweight, work, nbytes, None)


@pytest.mark.parametrize("M,N", [(1, 8), (1, 16384), (16, 16384), (64, 4096), (15, 16384), (32, 8192), (64, 8),
                                 (17, 16384), (15, 16392), (1, 16392), (64, 4104), (65, 8), (65, 4096), (1, 65536)])
def test_workspace(M, N):
    few = M <= 64 and N <= 16384 and M * N <= 1 << 18
    need = mxq.lib.mxq_rmsnorm_backward_workspace_bytes(M, N)
    assert (need == 0) == few
    if need:
        assert call(M, N, None, 0) == call(M, N, A, need - 1) == WORKSPACE
    assert call(M, N, A if need else None, need) == CUDA               # the checks pass; no driver here
    assert call(M, N, None, 0, dweight=None) == CUDA                  # without dweight none is needed


def test_rows_of_nothing():
    assert mxq.lib.mxq_rmsnorm_backward_workspace_bytes(0, 64) == mxq.lib.mxq_rmsnorm_backward_workspace_bytes(5, 0) == 0
    assert mxq.lib.mxfp8_rmsnorm(None, 0, 5, 0, 0, None, 0, None, 0, 1e-6, None, None, None, None, None, None, None) == OK
    assert call(5, 0, None, 0) == OK
