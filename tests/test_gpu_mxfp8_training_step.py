"""A training step of a layer of experts in MXFP8 as one chain: every gradient is
computed from what came back from the one behind it, down to the norm's input, the
norm's weight, the router's and both weights of the experts.

Each product is held to float64 on the operands that it was given, with the bounds
of mxfp8_refs.py. The chain as a whole is held to autograd of the layer in float64
without quantization: the gradients' differences are below half of their norm.
Rounding to E4M3 takes at most 2^-4 / sqrt 3 of an operand's norm (half a step of
2^-3 a value, evenly spread), the clamp at 448 a little more of a group's largest
value: s = 2^-4 together. Errors added up as if they pointed the same way:
  gate and up     2 s each (rows, weight)
  silu(gate) up   1.3 * 2 s + 2 s = 4.6 s   (|g silu' / silu| < 1.3)
  down's weight   4.6 s + s (its rows quantized) + s (the gradient's) = 6.6 s
  routing         4.6 s + 2 s of the second product = 6.6 s
  d(gate), d(up)  2 s + 2 s + 1.7 s = 5.7 s  (|silu''| < 1/2 against silu' of 0.6)
  up's weight, and the rows' gradient         5.7 s + 2 s = 7.7 s = 0.48.
Gradients of another layer, of other rows or in another order are off by 1 or more."""
import pytest
import torch

import mxfp8_refs as R
import nvfp4_block_scaled_sm_b200 as mxq

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
T, D, H, E, TOP = 500, 256, 384, 6, 2


def normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


class Layer:
    def __init__(self):
        self.w, self.router = normal(3, D, scale=0.2) + 1, normal(4, E, D, scale=0.1)
        self.up, self.down = normal(5, E, 2 * H, D, scale=0.07), normal(6, E, D, H, scale=0.07)
        self.x, self.residual, self.grad = normal(1, T, D), normal(2, T, D), normal(7, T, D)
        # (a stack's offsets come from the host, which a capture does not allow: the weights' codes are kept)
        self.qup, self.qdown = (mxq.mxfp8_quantize_grouped(v, swizzled=True) for v in (self.up, self.down))

    def step(self):
        """The forward pass and every gradient of sum(grad * (hidden + y)), by the library and a few lines of torch."""
        r = {}
        rowwise = lambda v: mxq.mxfp8_quantize_grouped(v, row_offsets=off, swizzled=True)
        columnwise = lambda v: mxq.mxfp8_quantize_columnwise_grouped(v, row_offsets=off)
        (qu, su, zu), (qd, sd, zd) = self.qup, self.qdown
        n = mxq.mxfp8_rmsnorm(self.x, self.w, residual=self.residual, normed=True)
        logits = n.normed.float() @ self.router.float().t()
        weights, experts = mxq.moe_route(logits, TOP)
        off, order, pos = mxq.moe_dispatch(experts, E)
        token = order.long() // TOP
        rows = n.normed[token]
        qx, sx, zx = rowwise(rows)
        h = mxq.mxfp8_gemm_grouped(qx, zx, qu, zu, off, swiglu=True)
        qh, sh, zh = rowwise(h)
        out = mxq.mxfp8_gemm_grouped(qh, zh, qd, zd, off, FP32)
        r["y"] = mxq.moe_combine(out, pos, weights)
        # back: the second product, with the routing weights
        g = self.grad.float()
        grad_weights = torch.einsum("td,tkd->tk", g, out[pos.long()])
        gy = (g[token] * weights.reshape(-1)[order.long()].unsqueeze(1)).to(BF16)
        dt, dz = mxq.mxfp8_quantize_columnwise_grouped(self.down)
        qg, sg, zg = rowwise(gy)
        gh = mxq.mxfp8_gemm_grouped(qg, zg, dt, dz, off, FP32)
        a, b = columnwise(gy), columnwise(h)
        r["down"] = mxq.mxfp8_gemm_grouped_wgrad(*a, *b, off, FP32)
        # SwiGLU: its factors are not kept, the product forms them again
        gu = mxq.mxfp8_gemm_grouped(qx, zx, qu, zu, off, FP32)
        gate, up = gu[:, :H], gu[:, H:]
        s = torch.sigmoid(gate)
        gg = torch.cat((gh * up * s * (1 + gate * (1 - s)), gh * gate * s), 1).to(BF16)
        # the first product, and the rows back to their tokens
        ut, uz = mxq.mxfp8_quantize_columnwise_grouped(self.up)
        qq, sq, zq = rowwise(gg)
        grows = mxq.mxfp8_gemm_grouped(qq, zq, ut, uz, off, FP32)
        c, d = columnwise(gg), columnwise(rows)
        r["up"] = mxq.mxfp8_gemm_grouped_wgrad(*c, *d, off, FP32)
        gl = mxq.moe_route_backward(grad_weights, logits, experts)
        r["router"] = gl.t() @ n.normed.float()
        gn = mxq.moe_combine(grows, pos, torch.ones_like(weights), FP32) + gl @ self.router.float()
        gn = gn.to(BF16)
        r["x"], r["w"] = mxq.rmsnorm_backward(gn, n.hidden, self.w, n.rstd, grad_hidden=self.grad)
        r["pieces"] = dict(n=n, experts=experts, off=off, qx=qx, sx=sx, qu=qu, su=su, h=h, gu=gu, qg=qg, sg=sg, dt=dt, dz=dz, gh=gh, a=a, b=b,
                           qq=qq, sq=sq, ut=ut, uz=uz, grows=grows, c=c, d=d, gn=gn)
        return r

    def exact(self, experts):
        """Autograd of the layer in float64, without quantization, for the experts that were chosen."""
        hidden = (self.x.float() + self.residual.float()).to(BF16).double().requires_grad_()
        leaves = [t.double().requires_grad_() for t in (self.w, self.router, self.up, self.down)]
        w, router, up, down = leaves
        normed = hidden * torch.rsqrt(hidden.square().mean(1, keepdim=True) + 1e-6) * w
        p = torch.softmax(normed @ router.t(), 1).gather(1, experts.long())
        p = p / p.sum(1, keepdim=True)
        y = torch.zeros_like(hidden)
        for e in range(E):
            t, j = (experts == e).nonzero(as_tuple=True)
            gu = normed[t] @ up[e].t()
            y = y.index_add(0, t, (R.silu(gu[:, :H]) * gu[:, H:]) @ down[e].t() * p[t, j].unsqueeze(1))
        (self.grad.double() * (hidden + y)).sum().backward()
        return dict(y=y.detach(), x=hidden.grad, **{k: v.grad for k, v in zip(("w", "router", "up", "down"), leaves)})


def check_pieces(layer, r):
    p = r["pieces"]
    off = p["off"].tolist()
    x, u = R.values(p["qx"], p["sx"]), R.values(p["qu"], p["su"])
    y, mags = R.grouped(x, u, off)
    R.check(p["gu"], y, D * R.U * mags, "gate and up")
    want, bound = R.swiglu(y, mags, D)
    R.check(p["h"], want, bound, "SwiGLU")
    tiles = lambda z, M, S: torch.stack([R.untile(z.view(E, -1)[e], M, S) for e in range(E)])
    for q, s, t, z, rows, cols, got, what in ((p["qg"], p["sg"], p["dt"], p["dz"], H, D, p["gh"], "gradient of SwiGLU's output"),
                                              (p["qq"], p["sq"], p["ut"], p["uz"], D, 2 * H, p["grows"], "rows' gradient")):
        y, mags = R.grouped(R.values(q, s), R.values(t, tiles(z, rows, cols // 32)), off)
        R.check(got, y, cols * R.U * mags, what)
    at = R.padded(off)
    for (qa, za), (qb, zb), got, what in ((p["a"], p["b"], r["down"], "down's weight"), (p["c"], p["d"], r["up"], "up's weight")):
        P = qa.shape[1]
        a, b = R.values(qa, R.untile(za, qa.shape[0], P // 32)), R.values(qb, R.untile(zb, qb.shape[0], P // 32))
        for e in range(E):
            s = slice(at[e], at[e + 1])
            R.check(got[e], a[:, s] @ b[:, s].t(), (off[e + 1] - off[e]) * R.U * (a[:, s].abs() @ b[:, s].abs().t()), what)
    n = p["n"]
    want, bound, want_w, bound_w = R.norm_gradient(p["gn"].double(), n.hidden.double(), layer.w.double(), n.rstd.double(), layer.grad.double())
    R.check(r["x"], want, bound, "norm's rows")
    R.check(r["w"], want_w, bound_w, "norm's weight")


def check_chain(layer, r):
    want = layer.exact(r["pieces"]["experts"])
    through = dict(r, x=r["x"].double() - layer.grad.double())             # (the residual stream's own gradient is exact)
    want["x"] = want["x"] - layer.grad.double()
    for name in ("y", "x", "w", "router", "up", "down"):
        off = float((through[name].double() - want[name]).norm() / want[name].norm())
        assert off < 0.5, f"{name}: off by {off:.3f} of its norm"


def test_a_training_step():
    layer = Layer()
    r = layer.step()
    check_pieces(layer, r)
    check_chain(layer, r)


def test_a_captured_training_step():
    """The whole step in one graph, replayed with other data."""
    layer = Layer()
    prev = mxq.set_output_allocator(None)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = layer.step()
        for seed in (11, 21):
            for i, t in enumerate((layer.x, layer.residual, layer.grad)):
                t.copy_(normal(seed + i, T, D))
            graph.replay()
            torch.cuda.synchronize()
            check_pieces(layer, r)
            check_chain(layer, r)
            eager = layer.step()
            for name in ("y", "x", "w", "up", "down"):
                assert torch.equal(eager[name], r[name]), name
    finally:
        mxq.set_output_allocator(prev)
