"""The experts' MXFP8 kernels where a CTA has more than one turn: rings of stages
that go round several times, accumulators that are handed back and filled again,
tiles whose sums differ in length or are empty, walks over rows, columns and
experts of the transposes. The bounds are derived in mxfp8_refs.py."""
import numpy as np
import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq
import oracle
from gpu_util import host, oracle_map

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def on_device(off):
    return torch.tensor(off, dtype=torch.int64, device="cuda")


def spread(seed, E, M, empty):
    """Offsets of M rows over E experts, a share of them empty."""
    rng = np.random.default_rng(seed)
    share = rng.exponential(size=E) * (rng.random(E) >= empty)
    share[rng.integers(E)] += 0.1
    cut = np.rint(np.cumsum(share) / share.sum() * M).astype(np.int64)
    return [0] + [int(v) for v in cut]


def rows(off, M, N, K, dtype=FP32, swiglu=False, seed=0):
    E = len(off) - 1
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = on_device(off)
    qx, sx, zx = mxq.mxfp8_quantize_grouped(normal(seed + M, M, K), row_offsets=d, swizzled=True)
    qw, sw, zw = mxq.mxfp8_quantize_grouped(normal(seed + N, E, N, K, scale=0.1), swizzled=True)
    y = mxq.mxfp8_gemm_grouped(qx, zx, qw, zw, d, dtype, swiglu=swiglu, error_flag=flag)
    assert int(flag) == 0, "a wait in the kernel gave up"
    want, mags = R.grouped(R.values(qx, sx), R.values(qw, sw), off)
    bound = K * R.U * mags
    if swiglu:
        want, bound = R.swiglu(want, mags, K)
    R.check(y, want, bound, f"rows {E} {M} {N} {K}")


# at most 64 rows: a ring of ten stages that three warps fill in turn (nine with SwiGLU). K at ten blocks, just past
# them and over several laps; with one tile a pair of CTAs, and with several
@pytest.mark.parametrize("K", [1152, 1280, 1408, 2560, 4000, 7168])
@pytest.mark.parametrize("off,N", [([0, 8], 528), ([0, 33, 33, 64], 272), ([0, 5, 6, 10, 11, 64], 4112)])
def test_few_rows_over_long_sums(off, N, K):
    rows(off, off[-1], N, K)


# 320 tiles for some 74 pairs, sums of one to four blocks and of eleven: the block that a loading warp has in turn goes on
# from tile to tile at every remainder of three
@pytest.mark.parametrize("K", [32, 128, 160, 288, 416, 1408])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_few_rows_over_many_tiles(K, dtype):
    rows(list(range(65)), 64, 1040, K, dtype)
    rows(spread(K, 64, 60, 0.5), 60, 1040, K, dtype, seed=1)


@pytest.mark.parametrize("n", [1, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("swiglu", [False, True])
def test_few_rows_of_one_expert(n, swiglu):
    """Tiles of every number of columns that the form for few rows has, beside an empty expert and the rest."""
    rows([0, 0, n, 64], 64, 768, 1536, swiglu=swiglu)
    rows([0, n], n, 768, 1536, BF16, swiglu=swiglu)


@pytest.mark.parametrize("K", [96, 1280, 2304])
def test_few_rows_swiglu_over_many_tiles(K):
    rows(spread(K, 40, 64, 0.3), 64, 2048, K, swiglu=True)


@pytest.mark.parametrize("K,swiglu", [(96, False), (896, False), (1664, False), (224, True), (1280, True)])
def test_many_rows_over_many_tiles(K, swiglu):
    rows(spread(K, 30, 7000, 0.2), 7000, 1024, K, BF16, swiglu=swiglu)


# ------------------------------------------------- weights' gradients

# several hundred tiles of 256 x 256 for some 74 pairs, with experts of no rows, of one block and of many between them;
# single CTAs (a side of at most 128) likewise
@pytest.mark.parametrize("E,M,Na,Nb", [(40, 6000, 528, 528), (300, 900, 272, 272), (25, 20000, 528, 1040), (64, 3000, 528, 128),
                                       (200, 700, 128, 272)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_weight_gradients_over_many_tiles(E, M, Na, Nb, dtype):
    off = spread(E, E, M, 0.3)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = on_device(off)
    qa, za = mxq.mxfp8_quantize_columnwise_grouped(normal(1, M, Na), row_offsets=d)
    qb, zb = mxq.mxfp8_quantize_columnwise_grouped(normal(2, M, Nb), row_offsets=d)
    y = mxq.mxfp8_gemm_grouped_wgrad(qa, za, qb, zb, d, dtype, error_flag=flag)
    assert int(flag) == 0, "a wait in the kernel gave up"
    P, at = qa.shape[1], R.padded(off)
    a, b = R.values(qa, R.untile(za, Na, P // 32)), R.values(qb, R.untile(zb, Nb, P // 32))
    for e in range(E):
        s, n = slice(at[e], at[e + 1]), off[e + 1] - off[e]
        R.check(y[e], a[:, s] @ b[:, s].t(), n * R.U * (a[:, s].abs() @ b[:, s].abs().t()), f"expert {e} of {E}")


# --------------------------------------------------------- transposes

def columns(x, off):
    """[P, N]: the experts' rows, each padded with zeros to a multiple of 128, and zeros up to the bound."""
    E, at = len(off) - 1, R.padded(off)
    out = torch.zeros((x.shape[0] + 127 * E) // 128 * 128, x.shape[1], dtype=x.dtype, device=x.device)
    for e in range(E):
        out[at[e]:at[e] + off[e + 1] - off[e]] = x[off[e]:off[e + 1]]
    return out


def transposed(x):
    """The oracle's codes and compact scales of the transpose, columns of x shared out over the host's threads."""
    a = host(x.t().contiguous()) if x.dtype == BF16 else x.t().contiguous().cpu().numpy()
    parts = oracle_map(oracle.mxfp8_quantize, np.array_split(a, 16))
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])


# 810 and 1539 tiles for at most 296 CTAs, in a number of column tiles that divides no grid; experts of one tile, so that
# a CTA's next one is many experts on
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E,M,N", [(9, 1120, 1200), (700, 32, 144), (33, 160, 1040)])
def test_stacked_columns_over_many_tiles(E, M, N, dtype):
    x = normal(M, E, M, N, dtype=dtype)
    q, z = mxq.mxfp8_quantize_columnwise_grouped(x)
    q, z = q.cpu().numpy(), z.view(E, -1).cpu().numpy()
    for e in range(E):
        want_q, want_s = transposed(x[e])
        assert np.array_equal(q[e], want_q), e
        assert np.array_equal(z[e], oracle.swizzle_scales(want_s)), e


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E,M,N,empty", [(7, 9000, 1200, 0.2), (600, 2000, 400, 0.4), (1, 5000, 1040, 0.0), (1000, 300, 144, 0.8)])
def test_ragged_columns_over_many_tiles(E, M, N, empty, dtype):
    off = spread(E + M, E, M, empty)
    x = normal(M, M, N, dtype=dtype)
    q, z = mxq.mxfp8_quantize_columnwise_grouped(x, row_offsets=on_device(off))
    want_q, want_s = transposed(columns(x, off))
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(z.cpu().numpy(), oracle.swizzle_scales(want_s))
