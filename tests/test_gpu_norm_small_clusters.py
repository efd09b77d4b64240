"""The norm's gradient of few rows where the device holds no cluster of 16 CTAs at
once (a part of its multiprocessors only, say): smaller clusters, down to one CTA,
from the same entry point, against float64."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))
PACKAGE = os.path.dirname(os.path.abspath(mxq.__file__))


@pytest.fixture(scope="module")
def limited(tmp_path_factory):
    """The library of tests/c/small_clusters.cu (the rest from libmxq.so)."""
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp_path_factory.mktemp("clusters") / "small.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-ftz=false", "-prec-div=true",
                    "-prec-sqrt=true", "-fmad=false", "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(PACKAGE, "..", "include"),
                    "-I", os.path.join(PACKAGE, "csrc"), os.path.join(HERE, "c", "small_clusters.cu"), mxq.library_path,
                    "-Xlinker", "-rpath", "-Xlinker", PACKAGE, "-o", out], check=True)
    return out


def rows(seed, M, N, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("most", [16, 8, 5, 2, 1])
def test_gradient(limited, tmp_path, most):
    path = str(tmp_path / f"most{most}.so")
    shutil.copy(limited, path)                                     # (the answer is kept per process and library)
    lib = ctypes.CDLL(path)
    lib.set_largest_cluster(most)
    f = lib.mxq_rmsnorm_backward
    f.argtypes, f.restype = mxq.lib.mxq_rmsnorm_backward.argtypes, ctypes.c_int
    for M, N, dtype, with_hidden in ((1, 8, FP32, False), (3, 1056, BF16, True), (16, 16384, BF16, True), (16, 16384, FP32, False),
                                     (61, 1056, FP32, True), (64, 4096, BF16, False), (33, 5000, FP32, False)):
        g, h, w = rows(M, M, N, dtype, 0.1), rows(N, M, N, dtype), rows(7, 1, N, dtype)[0]
        gh = rows(M + N, M, N, dtype, 0.1) if with_hidden else None
        rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
        dx, dw = torch.empty_like(h), torch.empty_like(w)
        code = 0 if dtype == BF16 else 1
        st = f(g.data_ptr(), code, M, N, N, h.data_ptr(), N, w.data_ptr(), code, rstd.data_ptr(), None if gh is None else gh.data_ptr(),
               N, dx.data_ptr(), dw.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0, (most, M, N)
        want, bound, want_w, bound_w = R.norm_gradient(*(t.double() for t in (g, h, w, rstd)), None if gh is None else gh.double())
        R.check(dx, want, bound, f"dx {M}x{N} in clusters of {most}")
        R.check(dw, want_w, bound_w, f"dweight {M}x{N} in clusters of {most}")
        if most == 16:
            a = mxq.rmsnorm_backward(g, h, w, rstd, grad_hidden=gh)
            assert torch.equal(a[0], dx) and torch.equal(a[1], dw)
