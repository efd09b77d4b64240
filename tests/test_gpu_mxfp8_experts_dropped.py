"""The experts' MXFP8 products with rows behind the last offset (dropped pairs), and
scales for the experts' rows only: nothing is refused, the experts' rows are those
of the call with all scales, the others are left."""
import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,off", [(1000, [0, 800]), (1000, [0, 0, 130, 640]), (64, [0, 3, 3, 10]), (300, [0, 1]), (700, [0, 128, 256]),
                                   (9000, [0, 2000, 6000])])
def test_scales_of_the_experts_rows_only(M, off, swiglu, guard_bands):
    E, N, K = len(off) - 1, 512, 416
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * 0.1).to(BF16)
    device = torch.tensor(off, device="cuda")
    q, s = mxq.mxfp8_quantize(x)
    tiles = torch.cat([mxq.swizzle_scales(s[a:b].contiguous()) for a, b in zip(off[:-1], off[1:]) if b > a])
    qw, sw, zw = mxq.mxfp8_quantize_grouped(w, swizzled=True)
    want, bound = R.grouped(R.values(q, s), R.values(qw, sw), off)
    bound = K * R.U * bound
    if swiglu:
        want, bound = R.swiglu(want, bound / (K * R.U), K)
    for offsets in (device, off, device.cpu()):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = mxq.mxfp8_gemm_grouped(q, tiles, qw, zw, offsets, FP32, swiglu=swiglu, error_flag=flag)
        n = off[-1]
        R.check(y[:n], want[:n], bound[:n], "experts' rows")
        assert int(flag) == 0 and bool((y[n:].contiguous().view(torch.uint8) == guard_bands.CANARY).all())
