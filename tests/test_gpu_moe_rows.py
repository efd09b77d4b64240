"""The router's weights and gradients in rows of masks, infinities and values
far out, each row held to its own bound: rows of other sizes do not widen it."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq
import fp4_refs as R
from test_gpu_fp4_matvec import cuda
from test_gpu_moe import gradient64

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


def scores64(l, scoring):
    """p in float64, NaN as -inf; sigmoids without a loss at either end."""
    l = np.where(np.isnan(l), -np.inf, l)
    if scoring == "softmax":
        return R.scores(l, "softmax")
    with np.errstate(over="ignore", invalid="ignore"):
        e = np.exp(-np.abs(l))
    return np.where(l < 0, e, 1.0) / (1 + e)


def reach(l):
    """How far below its row's largest value a logit can lie and still count:
    e^-104 is below half of fp32's smallest number."""
    l = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(over="ignore", invalid="ignore"):
        top = np.nanmax(np.where(np.isnan(l), -1e300, l), axis=1, keepdims=True)
        d = np.where(np.isnan(l), 0.0, np.minimum(top - l, 104.0))
    return d.max(1, keepdims=True)


def weight_bound(l, scoring, E, k, renormalize):
    """Relative error of a row's weights, in fp32. An exponential is off by two
    units in the last place, 2^-22, and by the rounding of its argument, 2^-24
    of the distance to the row's largest logit; a sum of n terms adds n - 1
    roundings at most. Softmax: numerator, sum (whose terms err as much), the
    quotient, the scale. Sigmoid: exponential, sum, quotient; renormalized with
    a second exponential and product, a sum of k, a quotient; the scale."""
    d = reach(l)
    if scoring == "softmax":
        return UNIT * (2 * (4 + d) + (k if renormalize else E / 32 + 5) + 3)
    one = 4 + d * (1 if renormalize else 0) + 6
    return UNIT * (2 * one + k + 3 if renormalize else 4 + 3)


def masked_logits():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((12, 40)).astype(np.float32)
    l[0] = -np.inf                                  # nothing left
    l[1, 5:] = -np.inf                              # fewer than top_k
    l[2, [3, 30]] = np.inf
    l[3, ::2] = np.nan
    l[4] = np.nan
    l[5] = np.finfo(np.float32).min                 # masks of the type's lowest value
    l[5, 7] = 1
    l[6] = -200 - np.arange(40)                     # sigmoids below fp32's range
    l[7] = np.float32(3e38) * np.sign(l[7])
    l[8] = np.finfo(np.float32).min
    l[9] = -86 - 0.5 * np.arange(40)                # sigmoids at the end of fp32's range
    l[10, 6:] = np.finfo(np.float32).min
    l[11] = 80 + np.arange(40)
    return l


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("k", [1, 3, 8])
@pytest.mark.parametrize("scale", [1.0, 2.5, 2.0 ** 60])
def test_weights_of_rows_of_masks(scoring, renormalize, k, scale):
    """Each row against its own bound, which rows of other sizes do not widen.
    Below fp32's normal range p rounds to multiples of 2^-149 (an exponential
    by two of them)."""
    l = masked_logits()
    w, e = mxq.moe_route(cuda(l), k, scoring=scoring, renormalize=renormalize, scale=scale)
    l64 = l.astype(np.float64)
    want, ids = R.route(l64, k, scoring, renormalize=renormalize, scale=scale)
    assert np.array_equal(e.cpu().numpy(), ids)
    if not renormalize:
        want = scale * np.take_along_axis(scores64(l64, scoring), ids, 1)
    chosen = np.take_along_axis(l64, ids, 1) if renormalize else l64
    tol = weight_bound(chosen, scoring, 40, k, renormalize) * np.abs(want) + scale * 3 * 2.0 ** -149
    off = np.abs(R.f64(w) - want)
    assert np.all(off <= tol), (np.argwhere(off > tol)[:5].tolist(), off[off > tol][:5], tol[off > tol][:5])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 60])
def test_gradient_of_rows_of_masks(scoring, renormalize, scale):
    """dl = p (d - mean): each of p and the mean err as a weight does, twice a
    weight's bound and k + 4 more roundings of the terms' magnitudes; an
    infinite logit's 1 - p is 0. Below fp32's range each of the k + 1 terms
    rounds p by three multiples of 2^-149."""
    l = masked_logits()
    k = 6
    rng = np.random.default_rng(5)
    g = rng.standard_normal((12, k)).astype(np.float32)
    ids = np.tile(np.arange(k), (12, 1))
    ids[2] = [3, 30, 0, 1, 2, 5]
    ids[5] = [7, 0, 1, 2, 3, 4]
    ids[7] = np.arange(20, 26)
    ids[9] = np.arange(6, 12)
    ids[11] = np.arange(34, 40)
    out = mxq.moe_route_backward(cuda(g), cuda(l), cuda(ids.astype(np.int32)), scoring=scoring, renormalize=renormalize, scale=scale)
    l64 = l.astype(np.float64)
    want, size = gradient64(l64, ids, g.astype(np.float64), scoring, renormalize, scale)
    if scoring == "sigmoid" and not renormalize:
        want, size = np.zeros_like(want), np.zeros_like(size)
        p = scores64(l64, "sigmoid")
        q = scores64(np.where(np.isnan(l64), np.inf, -l64), "sigmoid")
        for j in range(k):
            r = np.arange(12)
            want[r, ids[:, j]] += g[:, j].astype(np.float64) * scale * p[r, ids[:, j]] * q[r, ids[:, j]]
        size = np.abs(want)
    chosen = np.take_along_axis(l64, ids, 1) if renormalize else l64
    rel = 2 * weight_bound(chosen, scoring, 40, k, renormalize) + (k + 4) * UNIT
    tol = rel * size + 3 * 2.0 ** -149 * (k + 1) * scale * np.abs(g).max()
    off = np.abs(R.f64(out) - want)
    assert np.all(off <= tol), (np.argwhere(off > tol)[:5].tolist(), off[off > tol][:5], tol[off > tol][:5])
