"""Plain 64-bit forms of the 4-bit products and of the routing, for the tests.

None of it uses the library or the oracle: codes are decoded from tables and
bit fields, sums are float64 numpy."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values() -> np.ndarray:
    b = np.arange(256)
    exp, man = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * 2.0 ** (exp - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def decode(packed: np.ndarray, scale: np.ndarray, fmt: str) -> np.ndarray:
    """float64 weight [..., K] without NVFP4's global scale."""
    c = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    w = E2M1[c]
    if fmt == "mxfp4":
        s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
        return w * np.repeat(s, 32, axis=-1)
    return w * np.repeat(e4m3_values()[scale], 16, axis=-1)


def weight(rng, fmt: str, *shape, spread: int = 4):
    """(packed, scale) of random codes [*shape[:-1], K/2] with scales of a few
    powers of two around 2^-5 (MXFP4) or positive block scales (NVFP4)."""
    *lead, K = shape
    packed = rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scale = (122 + rng.integers(-spread, spread + 1, (*lead, K // 32))).astype(np.uint8)
    else:
        scale = rng.integers(0x18, 0x78, (*lead, K // 16)).astype(np.uint8)
    return packed, scale


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def product(x: np.ndarray, w: np.ndarray):
    """(x w^T, sum |x| |w|) in float64."""
    with np.errstate(invalid="ignore", over="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def bound(exact, size, K: int, bf16: bool):
    """Tolerance of a product of K terms with sum of magnitudes `size`. The
    products are exact. A group of 32 is summed by the tensor core (at most 32
    additions, each taken as off by 2^-22, four times the unit roundoff, for
    truncating hardware), scaled by two roundings and added to one of K / 32
    partial sums in fp32 (2^-24 each), which at most 8 more additions join;
    bf16 outputs round once more by half a step, 2^-8 of the value. NVFP4's
    general form sums 256 products in a chain of 16 MMAs instead: an MMA that
    cuts off the sum of its 16 products and the accumulator once is off by
    2^-23 of it, taken as 2^-21, which makes the same 32 2^-22 (sums of one
    sign, where each cut goes the same way, are off by 40 2^-24 at most in
    measurement). Below fp32's normal range a rounding is off by 2^-150
    instead: one for each block of 16 at most (three where x has three pieces),
    besides the 8 + 2."""
    acc = (32 * 2.0 ** -22 + (K / 32 + 10) * 2.0 ** -24) * size + (3 * K / 16 + 10) * 2.0 ** -150
    return acc + (2.0 ** -8 * (np.abs(exact) + acc) + 2.0 ** -134 if bf16 else 0)


def check(got: torch.Tensor, exact, size, K: int, what: str, extra=0.0):
    g = f64(got)
    assert g.shape == exact.shape, f"{what}: shape {g.shape} != {exact.shape}"
    fine = np.isfinite(exact)
    assert np.array_equal(np.isnan(g), np.isnan(exact)), f"{what}: NaNs differ"
    assert np.array_equal(g[~fine & ~np.isnan(exact)], exact[~fine & ~np.isnan(exact)]), f"{what}: infinities differ"
    tol = np.where(fine, bound(np.where(fine, exact, 0), np.where(fine, size, 0), K, got.dtype == torch.bfloat16), 0) + extra
    off = np.where(fine, np.abs(np.where(fine, g, 0) - np.where(fine, exact, 0)), 0)
    bad = off > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first "
                           f"{np.argwhere(bad)[:4].tolist()}, {off[bad][:4]} > {np.broadcast_to(tol, off.shape)[bad][:4]}")


# ------------------------------------------------------------------ routing

def scores(l: np.ndarray, scoring: str) -> np.ndarray:
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.where(l == top, 1.0, np.exp(l - top))
        e = np.where(np.isneginf(l), 0.0, e)
        s = e.sum(1, keepdims=True)
        return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route(l, top_k, scoring, bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    T, E = l.shape
    l = np.where(np.isnan(l), -np.inf, l) + 0.0
    p = scores(l, scoring)
    with np.errstate(invalid="ignore"):
        key = p if bias is None else p + bias.astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    kept = np.ones((T, E), bool)
    if groups > 1:
        size = E // groups
        two = -np.sort(-key.reshape(T, groups, size), axis=2)[:, :, :2]
        with np.errstate(invalid="ignore"):
            two = two.sum(2)
        two = np.where(np.isnan(two), -np.inf, two)
        best = np.argsort(-two, axis=1, kind="stable")[:, :top_groups]
        g = np.zeros((T, groups), bool)
        np.put_along_axis(g, best, True, 1)
        kept = np.repeat(g, size, axis=1)
    order = l if bias is None else key           # without a bias the logits decide
    ids = np.empty((T, top_k), np.int64)
    for t in range(T):
        cand = np.flatnonzero(kept[t])
        ids[t] = cand[np.argsort(-order[t, cand], kind="stable")[:top_k]]
    return route_weights(l, p, ids, scoring, renormalize, scale), ids


def route_weights(l, p, ids, scoring, renormalize, scale):
    if not renormalize:
        return scale * np.take_along_axis(p, ids, 1)
    lj = np.take_along_axis(l, ids, 1)
    if scoring == "softmax":
        q = scores(lj, "softmax")
    else:
        with np.errstate(over="ignore", invalid="ignore"):
            top = np.minimum(lj.max(1, keepdims=True), 0)
            q = np.where(np.isneginf(lj), 0, np.exp(np.where(np.isneginf(lj), 0, np.minimum(lj, 700) - top)) / (1 + np.exp(np.minimum(lj, 700))))
            q = np.where(lj > 30, 1 / (1 + np.exp(-lj)), q)
    s = q.sum(1, keepdims=True)
    return scale * np.divide(q, s, out=np.zeros_like(q), where=s > 0)


def dispatch(ids: np.ndarray, E: int):
    flat = ids.reshape(-1)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    place = np.empty(flat.size, np.int64)
    place[order] = np.arange(flat.size)
    place[key == E] = -1
    return offsets, order, place.reshape(ids.shape)
