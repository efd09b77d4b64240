"""Workloads of the decode-time operators: products with 4-bit weights, the
experts' products and the routing that feeds them.

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU
from a seed, ``run`` makes one call and returns its outputs. With ``own``
false, ``run`` computes the operators in elementary torch operations in 32 or
64 bits; with ``own`` true it calls the library. ``exact`` gives the outputs in
64 bits from the operators' definitions, and ``work`` the bytes and
operations that one call cannot do without.

Operators (``case["op"]``):

``matvec``   y = x W^T for a few rows x and a weight W held as MXFP4 or NVFP4.
``grouped``  the same for experts' weights: row r of the sorted rows is
             multiplied by its expert's weight. Form ``up`` gathers the tokens'
             rows and ends in SwiGLU, ``down`` adds each token's rows up with
             the router's weights, ``plain`` does neither.
``route``    the router: scores, an optional bias and groups, the best experts
             and their weights.
``route_backward``  the gradient of the logits from the weights' gradient.
``dispatch`` the (token, choice) pairs sorted by expert: row offsets, the order
             and its inverse.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a 4096x4096 linear layer: the smallest product, where latency counts
        dict(name="matvec mxfp4 1x4096x4096", op="matvec", fmt="mxfp4", M=1, N=4096, K=4096, x="bf16", y="bf16"),
        # eight sequences decoded together through a square 8192 layer
        dict(name="matvec nvfp4 8x8192x8192", op="matvec", fmt="nvfp4", M=8, N=8192, K=8192, x="bf16", y="bf16"),
        # logits of a speculated run of 5 tokens over a ragged vocabulary, in full precision
        dict(name="matvec mxfp4 fp32 5x100003x4096", op="matvec", fmt="mxfp4", M=5, N=100003, K=4096, x="fp32", y="fp32"),
        # one token's eight experts of 64, gate and up halves of 1024 rows: decoding a single sequence
        dict(name="experts up mxfp4 1 token", op="grouped", form="up", fmt="mxfp4", T=1, top_k=8, E=64, N=2048, K=7168, x="bf16", y="bf16"),
        # a batch of 64 sequences decoded together: nearly every expert has a few rows
        dict(name="experts up mxfp4 64 tokens", op="grouped", form="up", fmt="mxfp4", T=64, top_k=8, E=64, N=2048, K=7168, x="bf16", y="bf16"),
        # the way back of the same batch, with one scale per half of an expert, added up into the tokens
        dict(name="experts down nvfp4 64 tokens", op="grouped", form="down", fmt="nvfp4", T=64, top_k=8, E=64, N=7168, K=2048, x="bf16", y="bf16", halves=True),
        # a small odd layer in full precision: 7 tokens, 5 experts, sizes off every tile
        dict(name="experts fp32 odd", op="grouped", form="plain", fmt="nvfp4", T=7, top_k=2, E=5, N=1003, K=1040, x="fp32", y="fp32", halves=False),
        # one token's router: softmax over 64 experts
        dict(name="route softmax 1x64", op="route", T=1, E=64, top_k=8, x="bf16", scoring="softmax", bias=False, groups=1, top_groups=1, renormalize=True, scale=1.0),
        # a training batch's router: sigmoid scores, a bias for balance, four of eight groups
        dict(name="route sigmoid 16384x256", op="route", T=16384, E=256, top_k=8, x="fp32", scoring="sigmoid", bias=True, groups=8, top_groups=4, renormalize=True, scale=2.5),
        # its backward pass, with softmax scores that are not renormalized (every logit has a gradient)
        dict(name="route backward 16384x256", op="route_backward", T=16384, E=256, top_k=8, x="fp32", scoring="softmax", renormalize=False, scale=1.0),
        # sorting a decode batch's pairs by expert
        dict(name="dispatch 64x8 of 64", op="dispatch", T=64, top_k=8, E=64, dropped=0.0),
        # sorting a training batch's pairs, a part of them for experts of other ranks
        dict(name="dispatch 16384x8 of 256", op="dispatch", T=16384, top_k=8, E=256, dropped=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "grouped", "grouped", "route", "route_backward", "dispatch"])
    if op == "matvec":
        fmt = rng.choice(["mxfp4", "nvfp4"])
        unit = 32 if fmt == "mxfp4" else 16
        K = unit * _log(rng, 2, 8192 // unit)
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 32), N=_log(rng, 16, 32000), K=K,
                    x=rng.choice(["bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]))
    if op == "grouped":
        fmt = rng.choice(["mxfp4", "nvfp4"])
        unit = 32 if fmt == "mxfp4" else 16
        E = _log(rng, 2, 64)
        N = 2 * _log(rng, 8, 2048)
        K = unit * _log(rng, 2, min(7168, (1 << 29) // (E * N)) // unit)
        return dict(op=op, form=rng.choice(["up", "down", "plain"]), fmt=fmt, T=_log(rng, 1, 64), top_k=rng.randint(1, min(8, E)),
                    E=E, N=N, K=K, x=rng.choice(["bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]), halves=rng.random() < 0.5)
    if op == "dispatch":
        E = _log(rng, 2, 512)
        return dict(op=op, T=_log(rng, 1, 16384), top_k=rng.randint(1, min(8, E)), E=E, dropped=rng.choice([0.0, 0.0, 0.5]))
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * _log(rng, 4, 512 // groups)
    T = _log(rng, 1, 8192)
    scoring = rng.choice(["softmax", "sigmoid"])
    if op == "route_backward":
        top_k = rng.randint(1, min(16, E))
        return dict(op=op, T=T, E=E, top_k=top_k, x=rng.choice(["bf16", "fp32"]), scoring=scoring,
                    renormalize=top_k > 1 and rng.random() < 0.5,      # one renormalized weight is constant: no gradient
                    scale=rng.choice([1.0, 2.5]))
    top_groups = rng.randint(1, groups)
    return dict(op=op, T=T, E=E, top_k=rng.randint(1, min(16, E // groups * top_groups)), x=rng.choice(["bf16", "fp32"]), scoring=scoring,
                bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))


# ------------------------------------------------------------------ inputs

def _codes(u):
    """E2M1 codes, two per byte, of values in units of their scale."""
    mag = torch.bucketize(u.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=u.device), out_int32=True)
    code = (mag + 8 * (u < 0)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _weight(g, fmt, E, N, K, halves, dev):
    """E weights of N rows as a quantizer leaves them: N(0, std) with a std of each expert's own."""
    packed = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
    scale = torch.empty(E, N, K // (32 if fmt == "mxfp4" else 16), dtype=torch.uint8, device=dev)
    g_scale = torch.empty(E, 2, dtype=torch.float32, device=dev)
    std = 0.01 + 0.04 * torch.rand(E, generator=g, device=dev)
    step = max(1, (1 << 28) // K)                # rows at a time
    for e in range(E):
        top = std[e] * 6.0                        # the largest magnitude that a half holds
        g_scale[e, 0], g_scale[e, 1] = top / 2688.0, top * (0.75 if halves else 1.0) / 2688.0
        for n0 in range(0, N, step):
            w = torch.randn(min(step, N - n0), K, generator=g, device=dev) * std[e]
            rows = slice(n0, n0 + w.shape[0])
            if fmt == "mxfp4":
                b = w.view(w.shape[0], -1, 32)
                byte = torch.floor(torch.log2(b.abs().amax(-1).clamp_min(1e-30))) - 2 + 127
                packed[e, rows] = _codes((b * torch.exp2(127 - byte).unsqueeze(-1)).view_as(w))
                scale[e, rows] = byte.to(torch.uint8)
            else:
                b = w.view(w.shape[0], -1, 16)
                half = (torch.arange(n0, n0 + w.shape[0], device=dev) >= N // 2).long()
                gs = g_scale[e][half].unsqueeze(-1)
                s = (b.abs().amax(-1) / (6.0 * gs)).clamp(max=448.0).to(torch.float8_e4m3fn)
                packed[e, rows] = _codes((b / (s.float() * gs).clamp_min(1e-30).unsqueeze(-1)).view_as(w))
                scale[e, rows] = s.view(torch.uint8)
    return packed, scale, (g_scale if halves else g_scale[:, 0].contiguous())


def _experts(g, T, top_k, E, dev):
    """Distinct experts of each token, some more often chosen than others."""
    liking = torch.randn(E, generator=g, device=dev) * 0.5
    return torch.sort(torch.randn(T, E, generator=g, device=dev) + liking, dim=1, descending=True, stable=True)[1][:, :top_k].to(torch.int32)


def _sorted_pairs(ids, E):
    """(row offsets, order, positions) of the pairs sorted by expert; ids outside [0, E) come last and have position -1."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(key, stable=True)[1]
    count = (key.unsqueeze(1) == torch.arange(E, device=ids.device)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(count, 0)])
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    place = torch.where(key == E, -1, place)
    return offsets, order.to(torch.int32), place.to(torch.int32).view_as(ids)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    c = dict(case)
    op = c["op"]
    s = {"case": c}
    if op == "matvec":
        p, b, gs = _weight(g, c["fmt"], 1, c["N"], c["K"], False, dev)
        s.update(packed=p[0], scale=b[0], g=gs[0].clone())
        s["x"] = torch.randn(c["M"], c["K"], generator=g, device=dev).to(DTYPES[c["x"]])
        return s
    if op == "grouped":
        T, k, E = c["T"], c["top_k"], c["E"]
        s["packed"], s["scale"], s["g"] = _weight(g, c["fmt"], E, c["N"], c["K"], bool(c.get("halves")), dev)
        ids = _experts(g, T, k, E, dev)
        s["offsets"], s["order"], s["positions"] = _sorted_pairs(ids, E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())     # the plan of the padded plain form
        rows = T if c["form"] == "up" else T * k
        s["x"] = torch.randn(rows, c["K"], generator=g, device=dev).to(DTYPES[c["x"]])
        w = torch.rand(T, k, generator=g, device=dev) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        return s
    if op == "dispatch":
        ids = _experts(g, c["T"], c["top_k"], c["E"], dev)
        gone = torch.rand(c["T"], c["top_k"], generator=g, device=dev) < c["dropped"]
        s["experts"] = torch.where(gone, -1, ids).to(torch.int32).contiguous()
        return s
    s["logits"] = (torch.randn(c["T"], c["E"], generator=g, device=dev) * 1.5).to(DTYPES[c["x"]])
    if op == "route":
        s["bias"] = torch.randn(c["E"], generator=g, device=dev) * 0.1 if c["bias"] else None
    else:
        s["experts"] = _experts(g, c["T"], c["top_k"], c["E"], dev)
        s["grad"] = torch.randn(c["T"], c["top_k"], generator=g, device=dev)
    return s


# ------------------------------------------------------------ plain forms

def _decode_fp4(packed):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    pair = torch.stack([packed & 15, packed >> 4], dim=-1)
    return table[pair.flatten(-2).int()]


def _plain_weight(s, which=slice(None)):
    """The weight (of the experts `which`) in 32 bits without NVFP4's global scale, which is applied to the product."""
    w, scale = _decode_fp4(s["packed"][which]), s["scale"][which]
    if s["case"]["fmt"] == "mxfp4":
        return w * torch.exp2(scale.float() - 127.0).repeat_interleave(32, dim=-1)
    return w * scale.view(torch.float8_e4m3fn).float().repeat_interleave(16, dim=-1)


def _plain_matvec(s):
    y = s["x"].float() @ _plain_weight(s).t()
    if s["case"]["fmt"] == "nvfp4":
        y = y * s["g"]
    return y.to(DTYPES[s["case"]["y"]])


def _plain_grouped(s):
    c = s["case"]
    x = s["x"].float()
    if c["form"] == "up":
        x = x[s["order"].long() // c["top_k"]]
    off, R = s["offsets"], x.shape[0]
    at = torch.arange(R, device=x.device)
    e = torch.searchsorted(off[1:], at, right=True)
    if R <= c["E"]:                # fewer rows than experts: each row with a copy of its expert's weight
        y = torch.bmm(_plain_weight(s, e), x.unsqueeze(2)).squeeze(2)
    else:                          # the rows of each expert, padded to the longest
        row = off[:-1, None] + torch.arange(s["most"], device=x.device)
        there = row < off[1:, None]
        padded = x[row.clamp(max=R - 1)] * there.unsqueeze(-1)
        y = torch.bmm(padded, _plain_weight(s).transpose(1, 2))[e, at - off[e]]
    if c["fmt"] == "nvfp4":
        gs = s["g"][e]
        if c.get("halves"):
            gs = gs[:, (torch.arange(c["N"], device=x.device) >= c["N"] // 2).long()]
        else:
            gs = gs.unsqueeze(-1)
        y = y * gs
    if c["form"] == "up":
        gate, up = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    if c["form"] == "down":
        y = (y[s["positions"].long()] * s["weights"].unsqueeze(-1)).sum(1)
    return y.to(DTYPES[c["y"]])


def _scores(logits, scoring):
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    """In 64 bits: neighbours in the order of the scores are closer than 32 bits tell apart."""
    c = s["case"]
    p = _scores(s["logits"].double(), c["scoring"])
    key = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        by = key.view(c["T"], c["groups"], -1)
        two = torch.sort(by, dim=2, descending=True)[0][:, :, :2].sum(2)
        kept = torch.sort(two, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        best = (kept.unsqueeze(1) == torch.arange(c["groups"], device=p.device).view(1, -1, 1)).any(2)
        key = torch.where(best.unsqueeze(2), by, -math.inf).reshape(c["T"], c["E"])
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = torch.gather(p, 1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return (w * c["scale"]).float(), ids.to(torch.int32)


def _plain_route_backward(s):
    c = s["case"]
    p = _scores(s["logits"].float(), c["scoring"])
    ids = s["experts"].long()
    q = torch.gather(p, 1, ids)
    g = s["grad"] * c["scale"]
    if c["renormalize"]:
        total = q.sum(1, keepdim=True)
        g = (g - (g * q).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter(1, ids, g)
    if c["scoring"] == "sigmoid":
        d = dp * p * (1.0 - p)
    else:
        d = p * (dp - (dp * p).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import nvfp4_block_scaled_sm_b200 as mxq
        if op == "matvec":
            if c["fmt"] == "mxfp4":
                return mxq.mxfp4_matvec(s["x"], s["packed"], s["scale"], dtype=DTYPES[c["y"]])
            return mxq.nvfp4_matvec(s["x"], s["packed"], s["scale"], s["g"], dtype=DTYPES[c["y"]])
        if op == "grouped":
            more = {"dtype": DTYPES[c["y"]]}
            if c["form"] == "up":
                more.update(order=s["order"], top_k=c["top_k"], swiglu=True)
            if c["form"] == "down":
                more.update(combine=(s["positions"], s["weights"]))
            if c["fmt"] == "mxfp4":
                return mxq.mxfp4_matvec_grouped(s["x"], s["packed"], s["scale"], s["offsets"], **more)
            return mxq.nvfp4_matvec_grouped(s["x"], s["packed"], s["scale"], s["g"], s["offsets"], **more)
        if op == "route":
            return mxq.moe_route(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], renormalize=c["renormalize"], scale=c["scale"])
        if op == "route_backward":
            return mxq.moe_route_backward(s["grad"], s["logits"], s["experts"], scoring=c["scoring"],
                                          renormalize=c["renormalize"], scale=c["scale"])
        return mxq.moe_dispatch(s["experts"], c["E"])
    if op == "matvec":
        return _plain_matvec(s)
    if op == "grouped":
        return _plain_grouped(s)
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        return _plain_route_backward(s)
    return _sorted_pairs(s["experts"], c["E"])


# ------------------------------------------------------------------- work

def _weight_bytes(fmt, N, K):
    return N * (K // 2 + (K // 32 if fmt == "mxfp4" else K // 16))


def work(case):
    c = case
    size = {"bf16": 2, "fp32": 4}
    op = c["op"]
    if op == "matvec":
        return {"bytes": _weight_bytes(c["fmt"], c["N"], c["K"]) + c["M"] * (c["K"] * size[c["x"]] + c["N"] * size[c["y"]]),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    if op == "grouped":
        T, k, E, N, K = c["T"], c["top_k"], c["E"], c["N"], c["K"]
        active = E * (1.0 - (1.0 - k / E) ** T)          # experts that some token chose, on average
        rows_in = T if c["form"] == "up" else T * k
        out = {"up": T * k * N // 2, "down": T * N, "plain": T * k * N}[c["form"]]
        return {"bytes": active * _weight_bytes(c["fmt"], N, K) + rows_in * K * size[c["x"]] + out * size[c["y"]],
                "flops": 2 * T * k * N * K}
    if op == "dispatch":
        return {"bytes": 4 * c["T"] * c["top_k"] * 3 + 8 * (c["E"] + 1), "flops": 4 * c["T"] * c["top_k"]}
    read = c["T"] * c["E"] * size[c["x"]]
    if op == "route":
        return {"bytes": read + c["T"] * c["top_k"] * 8 + (4 * c["E"] if c["bias"] else 0), "flops": 10 * c["T"] * c["E"]}
    return {"bytes": 2 * read + c["T"] * c["top_k"] * 8, "flops": 10 * c["T"] * c["E"]}


# ------------------------------------------------------------------ exact

def _exact_weight(packed, scale, fmt):
    """float64 weight from its bit fields: sign, two exponent bits and one of mantissa; E8M0 or E4M3 scales."""
    n = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).to(torch.int32)
    field, man = (n >> 1) & 3, (n & 1).double()
    w = torch.where(field == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, field - 1))
    w = torch.where(n >= 8, -w, w)
    b = scale.to(torch.int32)
    if fmt == "mxfp4":
        return torch.ldexp(w.unflatten(-1, (-1, 32)), (b - 127).unsqueeze(-1)).flatten(-2)
    exp, man = (b >> 3) & 15, (b & 7).double()
    v = torch.where(exp == 0, torch.ldexp(man, torch.full_like(exp, -9)), torch.ldexp(1.0 + man / 8.0, exp - 7))
    v = torch.where(b >= 128, -v, v)
    return (w.unflatten(-1, (-1, 16)) * v.unsqueeze(-1)).flatten(-2)


def _exact_product(x, packed, scale, fmt):
    step = max(1, (1 << 28) // max(1, packed.shape[1] * 2))
    return torch.cat([x @ _exact_weight(packed[i:i + step], scale[i:i + step], fmt).t()
                      for i in range(0, packed.shape[0], step)], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "matvec":
        y = _exact_product(s["x"].double(), s["packed"], s["scale"], c["fmt"])
        return y * s["g"].double() if c["fmt"] == "nvfp4" else y
    if op == "grouped":
        off = s["offsets"].tolist()
        x = s["x"].double()
        if c["form"] == "up":
            x = x[s["order"].long() // c["top_k"]]
        y = torch.zeros(x.shape[0], c["N"], dtype=torch.float64, device=x.device)
        for e in range(c["E"]):
            if off[e + 1] > off[e]:
                part = _exact_product(x[off[e]:off[e + 1]], s["packed"][e], s["scale"][e], c["fmt"])
                if c["fmt"] == "nvfp4":
                    gs = s["g"][e].double().reshape(-1)
                    part[:, :c["N"] // 2] *= gs[0]
                    part[:, c["N"] // 2:] *= gs[-1]
                y[off[e]:off[e + 1]] = part
        if c["form"] == "up":
            gate, up = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
            return gate * torch.sigmoid(gate) * up
        if c["form"] == "down":
            token = s["order"].long() // c["top_k"]
            weight = s["weights"].double().reshape(-1)[s["order"].long()]
            return torch.zeros(c["T"], c["N"], dtype=torch.float64, device=y.device).index_add_(0, token, y * weight.unsqueeze(1))
        return y
    if op == "dispatch":
        ids = s["experts"].cpu().reshape(-1).tolist()
        order = sorted(range(len(ids)), key=lambda p: (ids[p] if 0 <= ids[p] < c["E"] else c["E"], p))
        place = [-1] * len(ids)
        offsets = [0] * (c["E"] + 1)
        for r, p in enumerate(order):
            if 0 <= ids[p] < c["E"]:
                place[p] = r
                offsets[ids[p] + 1] += 1
        for e in range(c["E"]):
            offsets[e + 1] += offsets[e]
        return (torch.tensor(offsets), torch.tensor(order, dtype=torch.int32),
                torch.tensor(place, dtype=torch.int32).view(c["T"], c["top_k"]))
    z = s["logits"].double()
    p = torch.sigmoid(z) if c["scoring"] == "sigmoid" else torch.softmax(z, dim=1)
    if op == "route":
        key = p if s["bias"] is None else p + s["bias"].double()
        if c["groups"] > 1:
            size = c["E"] // c["groups"]
            first = key.view(-1, c["groups"], size).topk(min(2, size), dim=2)[0].sum(2)
            last = torch.sort(-first, dim=1, stable=True)[1][:, c["top_groups"]:]        # the groups left out
            out = torch.zeros_like(first, dtype=torch.bool).scatter_(1, last, True)
            key = key.masked_fill(out.repeat_interleave(size, dim=1), -math.inf)
        ids = torch.sort(-key, dim=1, stable=True)[1][:, :c["top_k"]]
        w = p.gather(1, ids)
        if c["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return w * c["scale"], ids.to(torch.int32)
    ids = s["experts"].long()
    chosen = p.gather(1, ids)
    grad = s["grad"].double() * c["scale"]
    if c["renormalize"]:
        share = chosen / chosen.sum(1, keepdim=True)
        grad = (grad - (grad * share).sum(1, keepdim=True)) / chosen.sum(1, keepdim=True)
    chain = torch.zeros_like(p).scatter_(1, ids, grad)
    if c["scoring"] == "sigmoid":
        return chain * p * torch.sigmoid(-z)
    return p * chain - p * (p * chain).sum(1, keepdim=True)
