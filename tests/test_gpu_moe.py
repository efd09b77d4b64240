"""Routing to experts (moe_route and its gradient) and the sort of the pairs
by expert (moe_dispatch), against float64 and numpy's stable sort."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_sm_b200 as mxq
import fp4_refs as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def tolerance(l, E):
    """Relative error of a weight, in fp32: an exponential is off by two units
    in the last place and by the rounding of its argument (2^-24 of at most
    twice the largest finite logit), the sum of E terms by E / 32 + 5
    additions, and there are a quotient, a second exponential (sigmoid), a
    second sum and the scale."""
    finite = np.abs(l[np.isfinite(l)])
    reach = 2 * (finite.max() if finite.size else 0)
    return 2.0 ** -24 * (2 * (4 + reach) + 2 * (E / 32 + 5) + 6)


def check_route(logits, top_k, **kw):
    bias = kw.get("bias")
    weights, experts = mxq.moe_route(logits, top_k, **kw)
    l = R.f64(logits)
    kw64 = dict(kw, bias=None if bias is None else R.f64(bias))
    scoring = kw64.pop("scoring", "softmax")
    want, ids = R.route(l, top_k, scoring, **kw64)
    got = experts.cpu().numpy()
    bad = np.argwhere((got != ids).any(1)).flatten()
    assert bad.size == 0, f"{bad.size} tokens chosen otherwise, first {bad[:4]}: {got[bad[:2]].tolist()} for {ids[bad[:2]].tolist()}"
    w = R.f64(weights)
    assert weights.dtype == FP32 and experts.dtype == torch.int32
    assert np.all(np.abs(w - want) <= tolerance(l, l.shape[1]) * np.abs(want) + 1e-37), np.abs(w - want).max()
    return weights, experts


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 32, 32), (5, 33, 4), (70, 64, 6), (33, 100, 8), (64, 128, 1),
                                   (200, 256, 8), (7, 300, 10), (9, 512, 16), (6, 1000, 32), (4, 1024, 8)])
def test_route(scoring, renormalize, dtype, T, E, k):
    rng = np.random.default_rng(T + E)
    logits = cuda((2 * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    check_route(logits, k, scoring=scoring, renormalize=renormalize, scale=1.5)
    bias = cuda((0.2 * rng.standard_normal(E)).astype(np.float32))
    check_route(logits, k, scoring=scoring, renormalize=renormalize, bias=bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 2, 1, 3), (8, 8, 3, 3), (64, 8, 4, 8), (256, 8, 4, 8), (160, 8, 3, 6),
                                                   (96, 3, 2, 5), (90, 6, 2, 7), (512, 32, 5, 8), (1024, 4, 1, 4), (256, 8, 8, 8), (31, 31, 4, 4)])
def test_groups(scoring, dtype, with_bias, E, groups, top_groups, k):
    rng = np.random.default_rng(E + groups)
    logits = cuda((1.5 * rng.standard_normal((150, E))).astype(np.float32)).to(dtype)
    bias = cuda((0.1 * rng.standard_normal(E)).astype(np.float32)) if with_bias else None
    check_route(logits, k, scoring=scoring, bias=bias, groups=groups, top_groups=top_groups, renormalize=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_exact_ties_go_to_the_lowest_index(scoring, dtype):
    rng = np.random.default_rng(1)
    few = rng.choice([-1.0, 0.0, 0.5, -0.0], (40, 64)).astype(np.float32)
    few[0] = 0
    few[1] = -3
    for bias in (None, torch.zeros(64, device="cuda"), cuda(rng.choice([0.0, 0.25], 64).astype(np.float32))):
        check_route(cuda(few).to(dtype), 8, scoring=scoring, bias=bias)
        check_route(cuda(few).to(dtype), 8, scoring=scoring, bias=bias, groups=8, top_groups=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 1), (64, 4), (300, 1), (256, 8)])
def test_scores_closer_than_fp32_tells_apart(scoring, E, groups):
    """A bias that brings all sums p + bias of the first token to within an
    fp32 rounding of one value: their order is that of the exact sums."""
    rng = np.random.default_rng(2)
    l = rng.standard_normal((8, E)).astype(np.float32)
    p = R.scores(l.astype(np.float64), scoring)
    bias = (0.75 - p[0]).astype(np.float32)
    l[1:] = l[0] + np.where(rng.random((7, E)) < 0.1, 1e-6, 0).astype(np.float32)
    exact = p[0] + bias.astype(np.float64)
    assert np.ptp(exact) < 2.0 ** -23 and np.unique(exact).size > E // 2
    check_route(cuda(l), 8, scoring=scoring, bias=cuda(bias), groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_rows_with_infinities_and_nan(scoring, renormalize):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((9, 40)).astype(np.float32)
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
    w, e = check_route(cuda(l), 8, scoring=scoring, renormalize=renormalize)
    assert torch.isfinite(w).all()
    assert not w[0].any() and e[0].tolist() == list(range(8))
    bias = rng.standard_normal(40).astype(np.float32)
    bias[4], bias[6], bias[9] = -np.inf, np.inf, np.nan
    check_route(cuda(l), 8, scoring=scoring, renormalize=renormalize, bias=cuda(bias))
    check_route(cuda(l), 4, scoring=scoring, renormalize=renormalize, bias=cuda(bias), groups=5, top_groups=2)


def test_strides_alignment_and_dimensions():
    rng = np.random.default_rng(4)
    base = cuda(rng.standard_normal((12, 80)).astype(np.float32))
    check_route(base[:, :64], 6)
    check_route(base[:, 3:67], 6, scoring="sigmoid")
    check_route(base.to(BF16)[:, 1:65], 6)
    w, e = mxq.moe_route(base.view(3, 4, 80), 5)
    w2, e2 = mxq.moe_route(base, 5)
    assert w.shape == (3, 4, 5) and torch.equal(w.view(12, 5), w2) and torch.equal(e.view(12, 5), e2)
    w1, e1 = mxq.moe_route(base[7], 5)
    assert w1.shape == (5,) and torch.equal(w1, w2[7])
    w0, e0 = mxq.moe_route(base[:0], 5)
    assert w0.shape == (0, 5) and e0.shape == (0, 5)


# ---------------------------------------------------------------- gradient

def gradient64(l, ids, g, scoring, renormalize, scale):
    """(gradient, sum of the magnitudes of its terms) in float64."""
    T, E = l.shape
    k = ids.shape[1]
    ok = (ids >= 0) & (ids < E)
    safe = np.where(ok, ids, 0)
    p = R.scores(l, scoring)
    q = np.where(ok, np.take_along_axis(p, safe, 1), 0)
    gg = np.where(ok, g, 0) * scale
    other = np.where(ok, np.take_along_axis(R.scores(-l, "sigmoid"), safe, 1), 0)
    d, size = np.zeros((T, E)), np.zeros((T, E))

    def add(v, mag):
        for j in range(k):
            r = np.flatnonzero(ok[:, j])
            np.add.at(d, (r, safe[r, j]), v[r, j])
            np.add.at(size, (r, safe[r, j]), mag[r, j])

    if renormalize:
        lj = np.where(ok, np.take_along_axis(np.where(np.isnan(l), -np.inf, l), safe, 1), -np.inf)
        w = R.route_weights(lj, R.scores(lj, scoring), np.tile(np.arange(k), (T, 1)), scoring, True, 1.0)
        mean, amean = (gg * w).sum(1, keepdims=True), (np.abs(gg) * w).sum(1, keepdims=True)
        f = other if scoring == "sigmoid" else 1.0
        add(w * (gg - mean) * f, w * (np.abs(gg) + amean) * f)
        return d, size
    if scoring == "sigmoid":
        add(gg * q * other, np.abs(gg) * q * other)
        return d, size
    add(gg, np.abs(gg))
    mean, amean = (gg * q).sum(1, keepdims=True), (np.abs(gg) * q).sum(1, keepdims=True)
    return p * (d - mean), p * (size + amean)


def check_gradient(logits, ids, g, **kw):
    out = mxq.moe_route_backward(cuda(g), logits, cuda(ids.astype(np.int32)), **kw)
    assert out.dtype == logits.dtype and out.shape == logits.shape
    l = R.f64(logits)
    want, size = gradient64(l, ids, g.astype(np.float64), kw.get("scoring", "softmax"), kw.get("renormalize", True), kw.get("scale", 1.0))
    tol = 2 * tolerance(l, l.shape[1]) * size + 1e-37
    if logits.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    bad = ~(np.abs(R.f64(out) - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} outside, first {np.argwhere(bad)[:3].tolist()}"
    return out


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (2, 32, 32), (65, 64, 6), (9, 100, 5), (40, 256, 8), (5, 300, 9), (6, 1000, 16), (4, 1024, 32)])
def test_gradient(scoring, renormalize, dtype, T, E, k):
    rng = np.random.default_rng(T * E)
    logits = cuda((1.5 * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    check_gradient(logits, ids, rng.standard_normal((T, k)).astype(np.float32), scoring=scoring, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_left_out_and_repeated_experts(scoring, renormalize):
    rng = np.random.default_rng(6)
    T, E, k = 20, 48, 6
    logits = cuda(rng.standard_normal((T, E)).astype(np.float32))
    ids = rng.integers(-2, E + 2, (T, k))
    ids[0] = -1
    ids[1] = 7
    ids[2] = [2 ** 31 - 1, -2 ** 31, 0, 47, 48, 1]
    out = check_gradient(logits, ids, rng.standard_normal((T, k)).astype(np.float32), scoring=scoring, renormalize=renormalize)
    assert not out[0].any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(scoring, renormalize):
    """Central differences of the weights in float64, the chosen experts held."""
    rng = np.random.default_rng(7)
    T, E, k, h = 4, 12, 3, 1e-5
    l = rng.standard_normal((T, E)).astype(np.float32)
    w, experts = mxq.moe_route(cuda(l), k, scoring=scoring, renormalize=renormalize)
    ids = experts.cpu().numpy().astype(np.int64)
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = R.f64(mxq.moe_route_backward(cuda(g), cuda(l), experts, scoring=scoring, renormalize=renormalize))
    for e in range(E):
        f = []
        for sign in (1, -1):
            z = l.astype(np.float64)
            z[:, e] += sign * h
            f.append((R.route_weights(z, R.scores(z, scoring), ids, scoring, renormalize, 1.0) * g).sum(1))
        # the difference's own error: h^2 of a third derivative below 6 |g|, and the roundings over h
        assert np.all(np.abs((f[0] - f[1]) / (2 * h) - got[:, e]) <= 1e-6)


def test_gradient_of_masked_rows_is_finite():
    l = np.zeros((4, 32), np.float32)
    l[0] = -np.inf
    l[1, 4:] = -np.inf
    l[2, 3] = np.inf
    l[3, ::2] = np.nan
    ids = np.tile(np.arange(6), (4, 1))
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            out = mxq.moe_route_backward(torch.ones(4, 6, device="cuda"), cuda(l), cuda(ids.astype(np.int32)), scoring=scoring, renormalize=renormalize)
            assert torch.isfinite(out).all()
            assert not out[0].any()


def test_gradient_strides():
    rng = np.random.default_rng(8)
    base = cuda(rng.standard_normal((6, 80)).astype(np.float32))
    ids = np.stack([rng.permutation(64)[:4] for _ in range(6)])
    g = rng.standard_normal((6, 4)).astype(np.float32)
    check_gradient(base[:, 8:72], ids, g)
    check_gradient(base[:, 3:67], ids, g, scoring="sigmoid")
    check_gradient(base.to(BF16)[:, 5:69], ids, g, renormalize=False)
    wide = torch.zeros(6, 8, device="cuda")
    wide[:, ::2] = cuda(g)
    out = mxq.moe_route_backward(wide[:, ::2], base, cuda(ids.astype(np.int32)))
    assert torch.equal(out, mxq.moe_route_backward(cuda(g), base, cuda(ids.astype(np.int32))))


# ---------------------------------------------------------------- dispatch

def check_dispatch(ids, E):
    off, order, pos = mxq.moe_dispatch(cuda(ids.astype(np.int32)), E)
    woff, worder, wpos = R.dispatch(ids, E)
    assert off.dtype == torch.int64 and order.dtype == pos.dtype == torch.int32
    assert np.array_equal(off.cpu().numpy(), woff), "row offsets"
    assert np.array_equal(order.cpu().numpy(), worder), "order"
    assert np.array_equal(pos.cpu().numpy(), wpos), "positions"


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (31, 1, 7), (33, 3, 1024), (64, 8, 64), (512, 8, 256), (513, 8, 255),
                                   (3000, 8, 128), (512, 8, 1024), (4097, 1, 1024), (16384, 8, 256), (131072, 8, 64), (30011, 7, 1000), (200003, 1, 31)])
@pytest.mark.parametrize("kind", ["random", "dropped", "skewed"])
def test_dispatch(T, k, E, kind):
    rng = np.random.default_rng(T + k)
    ids = rng.integers(0, E, (T, k))
    if kind == "dropped":
        ids = rng.integers(-3, E + 3, (T, k))
    if kind == "skewed":
        ids = np.minimum(rng.geometric(0.4, (T, k)) - 1, E - 1)
    check_dispatch(ids, E)


def test_dispatch_edges():
    check_dispatch(np.full((700, 4), 5), 9)                    # one expert takes all
    check_dispatch(np.full((700, 4), -1), 9)                   # all dropped
    check_dispatch(np.array([[2 ** 31 - 1, -2 ** 31, 0, 8, 9]]), 9)
    check_dispatch(np.zeros((0, 4), np.int64), 9)
    check_dispatch(np.arange(5000)[:, None] % 1024, 1024)


def test_dispatch_on_two_streams_at_once():
    rng = np.random.default_rng(9)
    ids = [rng.integers(0, 64, (20000, 4)) for _ in range(4)]
    dev = [cuda(i.astype(np.int32)) for i in ids]
    torch.cuda.synchronize()
    got = []
    for d in dev:
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got.append(mxq.moe_dispatch(d, 64))
    torch.cuda.synchronize()
    for i, g in zip(ids, got):
        for a, b in zip(g, R.dispatch(i, 64)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_refusals():
    l = torch.zeros(4, 16, device="cuda")
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    g = torch.zeros(4, 2, device="cuda")
    bad = [
        lambda: mxq.moe_route(l.half(), 2),
        lambda: mxq.moe_route(l.cpu(), 2),
        lambda: mxq.moe_route(l, 0),
        lambda: mxq.moe_route(l, 17),
        lambda: mxq.moe_route(torch.zeros(4, 64, device="cuda"), 33),
        lambda: mxq.moe_route(torch.zeros(4, 1025, device="cuda"), 2),
        lambda: mxq.moe_route(l.t(), 2),
        lambda: mxq.moe_route(l, 2, scoring="tanh"),
        lambda: mxq.moe_route(l, 2, bias=torch.zeros(15, device="cuda")),
        lambda: mxq.moe_route(l, 2, bias=torch.zeros(16, device="cuda", dtype=BF16)),
        lambda: mxq.moe_route(l, 2, bias=torch.zeros(16)),
        lambda: mxq.moe_route(l, 2, groups=3),
        lambda: mxq.moe_route(l, 2, groups=4, top_groups=5),
        lambda: mxq.moe_route(l, 5, groups=4, top_groups=1),
        lambda: mxq.moe_route(l, 2, groups=0),
        lambda: mxq.moe_route_backward(g, l, e.long()),
        lambda: mxq.moe_route_backward(g.to(BF16), l, e),
        lambda: mxq.moe_route_backward(g[:3], l, e[:3]),
        lambda: mxq.moe_route_backward(g[:, :1], l, e),
        lambda: mxq.moe_dispatch(e.long(), 4),
        lambda: mxq.moe_dispatch(e.cpu(), 4),
        lambda: mxq.moe_dispatch(e, 0),
        lambda: mxq.moe_dispatch(e, 1025),
    ]
    for f in bad:
        with pytest.raises((ValueError, TypeError, mxq.MxqError)):
            f()
