"""Workloads of the 8-bit layers of experts: the norm that ends in MXFP8, the
experts' MXFP8 products and what their training needs.

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU
from a seed, ``run`` makes one call and returns its outputs. With ``own``
false, ``run`` computes the operators in elementary torch operations in 32 or
64 bits; with ``own`` true it calls the library. ``exact`` gives the outputs in
64 bits from the operators' definitions, and ``work`` the bytes and
operations that one call cannot do without.

Operators (``case["op"]``):

``norm``      root-mean-square norm of x, or of x + residual, quantized to
              MXFP8: codes, scales (compact and, where asked for, in 128x4
              tiles), the sum that goes on, 1/rms of each row.
``norm_backward``  its gradient: of the rows and of the norm's weight.
``experts``   the experts' products: row r of the sorted rows times its
              expert's weight, both in MXFP8; optionally ending in SwiGLU.
``transpose`` MXFP8 of the transposed rows of each expert, in groups of 32 of
              its own rows; of sorted rows (each expert padded to 128) or of a
              stack of weights.
``wgrad``     each expert's product over its rows: the weights' gradients.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token between two layers while decoding: the smallest call, where latency counts
        dict(name="norm 1x4096 residual", op="norm", M=1, N=4096, x="bf16", w="bf16", residual=True, swizzled=True, normed=False),
        # a training batch's rows between two layers
        dict(name="norm 16384x7168 residual", op="norm", M=16384, N=7168, x="bf16", w="bf16", residual=True, swizzled=True, normed=False),
        # an odd batch in full precision, no residual, the normed rows kept for the router
        dict(name="norm fp32 333x1056", op="norm", M=333, N=1056, x="fp32", w="fp32", residual=False, swizzled=False, normed=True),
        # the training batch's backward pass, with the gradient of the residual stream
        dict(name="norm backward 16384x7168", op="norm_backward", M=16384, N=7168, x="bf16", w="bf16", grad_hidden=True),
        # an odd one in full precision
        dict(name="norm backward fp32 61x1056", op="norm_backward", M=61, N=1056, x="fp32", w="fp32", grad_hidden=False),
        # decoding one sequence: eight rows for eight experts of 64, gate and up halves of 2048
        dict(name="experts up 1 token", op="experts", R=8, E=64, N=4096, K=7168, swiglu=True, y="bf16", dropped=0),
        # the way back of 64 sequences decoded together: a few rows for nearly every expert
        dict(name="experts down 64 tokens", op="experts", R=512, E=64, N=7168, K=2048, swiglu=False, y="bf16", dropped=0),
        # a prompt or a training batch of 4096 tokens, eight experts each
        dict(name="experts up 4096 tokens", op="experts", R=32768, E=64, N=4096, K=7168, swiglu=True, y="bf16", dropped=0),
        # the rows of that batch, transposed for the weights' gradients
        dict(name="transpose 32768x7168 of 64", op="transpose", stacked=False, E=64, M=32768, N=7168, x="bf16"),
        # weights of 8 experts, transposed for the rows' gradients
        dict(name="transpose 8 x 2048x7168", op="transpose", stacked=True, E=8, M=2048, N=7168, x="bf16"),
        # the gradients of 8 experts' weights from 8192 rows
        dict(name="wgrad 8 x 2048x7168 of 8192", op="wgrad", E=8, R=8192, Na=2048, Nb=7168, y="bf16"),
        # a small odd layer in full precision, where some experts have few rows or none
        dict(name="wgrad fp32 777 rows of 5", op="wgrad", E=5, R=777, Na=208, Nb=336, y="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "experts", "experts", "transpose", "wgrad"])
    if op in ("norm", "norm_backward"):
        N = 32 * _log(rng, 1, 512)
        M = _log(rng, 1, min(32768, 16384 * 7168 // N))
        c = dict(op=op, M=M, N=N, x=rng.choice(["bf16", "bf16", "fp32"]), w=rng.choice(["bf16", "fp32"]))
        if op == "norm":
            c.update(residual=rng.random() < 0.5, swizzled=rng.random() < 0.5, normed=rng.random() < 0.3)
        else:
            c.update(grad_hidden=rng.random() < 0.5)
        return c
    E = _log(rng, 1, 64)
    if op == "experts":
        swiglu = rng.random() < 0.4
        N = 256 * _log(rng, 1, 16) if swiglu else 16 * _log(rng, 1, 448)
        K = 32 * _log(rng, 1, min(224, (1 << 30) // (E * N * 32)))
        return dict(op=op, R=_log(rng, 1, 8192), E=E, N=N, K=K, swiglu=swiglu, y=rng.choice(["bf16", "fp32"]), dropped=rng.choice([0, 0, 1]))
    if op == "transpose":
        stacked = rng.random() < 0.4
        N = 16 * _log(rng, 1, 448)
        M = 32 * _log(rng, 1, min(256, (1 << 27) // (E * N * 32))) if stacked else _log(rng, 1, 16384)
        return dict(op=op, stacked=stacked, E=E, M=M, N=N, x=rng.choice(["bf16", "bf16", "fp32"]))
    Na = 16 * _log(rng, 1, 256)
    Nb = 16 * _log(rng, 1, min(448, (1 << 27) // (E * Na * 16)))
    return dict(op=op, E=E, R=_log(rng, 1, 8192), Na=Na, Nb=Nb, y=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs

def _mx_groups(v):
    """MXFP8 of groups of 32 along the last axis: E4M3 codes (as float8) and E8M0 bytes, from the library's rule."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    byte = torch.where(amax == 0, 127, (torch.frexp(amax)[1] - 1 - 8 + 127).clamp(0, 254)).to(torch.int32)
    scaled = b * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)          # times 2^(127 - byte)
    return scaled.clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _tiles(scale):
    """[..., M, S] scale bytes in 128x4 tiles, padded with zeros: flat."""
    M, S = scale.shape[-2:]
    Mp, Sp = -(-M // 128) * 128, -(-S // 4) * 4
    full = torch.zeros(*scale.shape[:-2], Mp, Sp, dtype=torch.uint8, device=scale.device)
    full[..., :M, :S] = scale
    return full.view(-1, Mp // 128, 4, 32, Sp // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)


def _untiled(flat, L, M, S):
    """The [L, M, S] scale bytes of L arrays in 128x4 tiles."""
    Mp, Sp = -(-M // 128) * 128, -(-S // 4) * 4
    return flat.view(L, Mp // 128, Sp // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(L, Mp, Sp)[:, :M, :S]


def _counts(g, E, R, dropped, dev):
    """Rising offsets of E experts in R rows, some experts with more rows than others, some with none; a part of the rows may belong to none."""
    share = torch.exp(0.7 * torch.randn(E, generator=g, device=dev))
    share[1:] *= torch.rand(E - 1, generator=g, device=dev) > 0.1
    if R <= E:                                     # few rows: each for an expert of its own
        own_row = torch.randperm(E, generator=g, device=dev)[:R]
        n = torch.zeros(E, dtype=torch.int64, device=dev).scatter_(0, own_row, 1)
        return torch.cat([n.new_zeros(1), n.cumsum(0)])
    edge = share.cumsum(0) / share.sum().clamp_min(1e-9)
    R = R - R // 5 if dropped else R
    return torch.cat([edge.new_zeros(1), edge]).mul(R).round().clamp(max=R).to(torch.int64)


def _padded(off):
    """Where each expert's rows begin when every expert is padded to a multiple of 128."""
    n = off[1:] - off[:-1]
    return torch.cat([off.new_zeros(1), ((n + 127) // 128 * 128).cumsum(0)])


def _ragged_tiles(byte, off):
    """[R, S] scale bytes of sorted rows with each expert in tiles of its own."""
    start = _padded(off)
    full = torch.zeros(int(start[-1]), byte.shape[1], dtype=torch.uint8, device=byte.device)
    r = torch.arange(int(off[-1]), device=byte.device)
    e = torch.searchsorted(off[1:], r, right=True)
    full[start[e] + r - off[e]] = byte[:r.numel()]
    return _tiles(full)


def _columns(x, off):
    """The rows [R, N] transposed, each expert padded with zeros to a multiple of 128, and zeros up to what that can come to: [N, P]."""
    start = _padded(off)
    P = (x.shape[0] + 127 * (off.numel() - 1)) // 128 * 128
    out = torch.zeros(P, x.shape[1], dtype=x.dtype, device=x.device)
    r = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(off[1:], r, right=True)
    out[start[e] + r - off[e]] = x[:r.numel()]
    return out.t().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    c = dict(case)
    s = {"case": c}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] in ("norm", "norm_backward"):
        M, N = c["M"], c["N"]
        t = DTYPES[c["x"]]
        spread = torch.exp(0.5 * normal(M, 1))                 # rows of their own size, a few large columns
        columns = 1.0 + 15.0 * (torch.rand(N, generator=g, device=dev) < 0.004)
        s["x"] = (normal(M, N) * spread * columns).to(t)
        s["weight"] = (1.0 + 0.2 * normal(N)).to(DTYPES[c["w"]])
        if c["op"] == "norm":
            s["residual"] = (normal(M, N) * 2.0).to(t) if c["residual"] else None
        else:
            s["grad"] = (normal(M, N) * 0.01).to(t)
            s["grad_hidden"] = (normal(M, N) * 0.01).to(t) if c["grad_hidden"] else None
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + 1e-6).float()
        return s
    E = c["E"]
    if c["op"] == "experts":
        R, N, K = c["R"], c["N"], c["K"]
        s["offsets"] = _counts(g, E, R, c["dropped"], dev)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())     # the plan of the padded plain form
        s["rows"] = int(s["offsets"][-1])
        q, b = _mx_groups(normal(R, K).to(torch.bfloat16).float())
        s["q"], s["scale"] = q.view(torch.uint8), _ragged_tiles(b, s["offsets"])
        s["w"] = torch.empty(E, N, K, dtype=torch.uint8, device=dev)
        parts = []
        std = 0.01 + 0.04 * torch.rand(E, generator=g, device=dev)
        for e in range(E):
            q, b = _mx_groups((normal(N, K) * std[e]).to(torch.bfloat16).float())
            s["w"][e] = q.view(torch.uint8)
            parts.append(_tiles(b))
        s["w_scale"] = torch.cat(parts)
        return s
    if c["op"] == "transpose":
        if c["stacked"]:
            s["x"] = (normal(E, c["M"], c["N"]) * 0.02).to(DTYPES[c["x"]])
        else:
            s["x"] = (normal(c["M"], c["N"]) * torch.exp(0.5 * normal(c["M"], 1))).to(DTYPES[c["x"]])
            s["offsets"] = _counts(g, E, c["M"], 0, dev)
        return s
    s["offsets"] = _counts(g, E, c["R"], 0, dev)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    for name, n in (("a", c["Na"]), ("b", c["Nb"])):
        v = (normal(c["R"], n) * torch.exp(0.5 * normal(c["R"], 1))).to(torch.bfloat16).float()
        q, b = _mx_groups(_columns(v, s["offsets"]))
        s[name], s[name + "_scale"] = q.view(torch.uint8), _tiles(b)
    return s


# ------------------------------------------------------------ plain forms

def _values(q, byte):
    """fp32 values of E4M3 codes [..., K] with E8M0 bytes [..., K / 32]."""
    return (q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * torch.exp2(byte.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _plain_norm(s):
    c = s["case"]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    mean = h.double().square().sum(1, keepdim=True) / c["N"]
    rstd = (1.0 / torch.sqrt(mean + 1e-6)).float()
    y = h.float() * rstd * s["weight"].float()
    q, b = _mx_groups(y)
    return _norm_outputs(c, q, b, _tiles(b) if c["swizzled"] else None, h, rstd.squeeze(1), y.to(h.dtype))


def _norm_outputs(c, q, b, tiles, h, rstd, y):
    out = {"codes": q.view(torch.float8_e4m3fn), "scale": b.view(torch.float8_e8m0fnu), "rstd": rstd}
    if c["swizzled"]:
        out["scale_tiles"] = tiles
    if c["residual"]:
        out["hidden"] = h
    if c["normed"]:
        out["normed"] = y
    return out


def _plain_norm_backward(s):
    h, g, rstd = s["x"].float(), s["grad"].float(), s["rstd"].unsqueeze(1)
    gw = g * s["weight"].float()
    dx = rstd * (gw - h * (rstd * rstd * (gw * h).mean(1, keepdim=True)))
    if s["grad_hidden"] is not None:
        dx = dx + s["grad_hidden"].float()
    dw = (g * h * rstd).sum(0)
    return dx.to(s["x"].dtype), dw.to(s["weight"].dtype)


def _plain_experts(s):
    c = s["case"]
    E, N, K, R = c["E"], c["N"], c["K"], s["rows"]
    off = s["offsets"]
    start = _padded(off)
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off[1:], r, right=True)
    byte = _untiled(s["scale"], 1, s["scale"].numel() // (-(-K // 128) * 4), K // 32)[0][start[e] + r - off[e]]
    x = _values(s["q"][:R], byte)
    w_byte = _untiled(s["w_scale"], E, N, K // 32)
    if R <= E:                     # few rows: each with a copy of its expert's weight
        y = torch.bmm(_values(s["w"][e], w_byte[e]), x.unsqueeze(2)).squeeze(2)
    else:                          # the rows of each expert, padded to the longest
        row = off[:-1, None] + torch.arange(s["most"], device=x.device)
        there = row < off[1:, None]
        padded = x[row.clamp(max=R - 1)] * there.unsqueeze(-1)
        y = torch.bmm(padded, _values(s["w"], w_byte).transpose(1, 2))[e, r - off[e]]
    if c["swiglu"]:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(DTYPES[c["y"]])


def _plain_transpose(s):
    v = s["x"].float()
    v = v.transpose(1, 2) if s["case"]["stacked"] else _columns(v, s["offsets"])
    q, b = _mx_groups(v)
    return q, _tiles(b)


def _plain_wgrad(s):
    c = s["case"]
    off = s["offsets"]
    start = _padded(off)
    col = start[:-1, None] + torch.arange(s["most"], device=off.device)
    there = (col < (start[:-1] + off[1:] - off[:-1])[:, None]).unsqueeze(0)

    def side(q, tiles):
        v = _values(q, _untiled(tiles, 1, q.shape[0], q.shape[1] // 32)[0])
        return (v[:, col.clamp(max=q.shape[1] - 1)] * there).transpose(0, 1)

    return torch.bmm(side(s["a"], s["a_scale"]), side(s["b"], s["b_scale"]).transpose(1, 2)).to(DTYPES[c["y"]])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import nvfp4_block_scaled_sm_b200 as mxq
        if op == "norm":
            r = mxq.mxfp8_rmsnorm(s["x"], s["weight"], eps=1e-6, residual=s["residual"], swizzled=c["swizzled"], normed=c["normed"])
            return _norm_outputs(c, r.qweight, r.scale, r.scale_swizzled, r.hidden, r.rstd, r.normed)
        if op == "norm_backward":
            return mxq.rmsnorm_backward(s["grad"], s["x"], s["weight"], s["rstd"], grad_hidden=s["grad_hidden"])
        if op == "experts":
            y = mxq.mxfp8_gemm_grouped(s["q"], s["scale"], s["w"], s["w_scale"], s["offsets"], DTYPES[c["y"]], swiglu=c["swiglu"])
            return y[:s["rows"]]                   # rows of no expert are left as they were
        if op == "transpose":
            if c["stacked"]:
                q, tiles = mxq.mxfp8_quantize_columnwise_grouped(s["x"])
                return mxq.as_float8_e4m3(q), tiles
            q, tiles = mxq.mxfp8_quantize_columnwise_grouped(s["x"], row_offsets=s["offsets"])
            return mxq.as_float8_e4m3(q), tiles
        return mxq.mxfp8_gemm_grouped_wgrad(s["a"], s["a_scale"], s["b"], s["b_scale"], s["offsets"], DTYPES[c["y"]])
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    if op == "experts":
        return _plain_experts(s)
    if op == "transpose":
        return _plain_transpose(s)
    return _plain_wgrad(s)


# ------------------------------------------------------------------- work

def work(case):
    c = case
    size = {"bf16": 2, "fp32": 4}
    op = c["op"]
    mx = 33 / 32                                    # bytes of a value in MXFP8
    if op == "norm":
        M, N, x = c["M"], c["N"], size[c["x"]]
        tiles = -(-M // 128) * 128 * -(-N // 128) * 4 if c["swizzled"] else 0
        return {"bytes": M * N * (x * (1 + 2 * c["residual"] + c["normed"]) + mx) + N * size[c["w"]] + tiles + 4 * M, "flops": 6 * M * N}
    if op == "norm_backward":
        M, N, x = c["M"], c["N"], size[c["x"]]
        return {"bytes": M * N * x * (3 + c["grad_hidden"]) + 2 * N * size[c["w"]] + 4 * M, "flops": 12 * M * N}
    if op == "experts":
        R, E, N, K = c["R"] - (c["R"] // 5 if c["dropped"] and c["R"] > c["E"] else 0), c["E"], c["N"], c["K"]
        active = min(E, R) if R <= E else 0.9 * E if E > 1 else 1
        return {"bytes": (active * N + R) * K * mx + R * N // (2 if c["swiglu"] else 1) * size[c["y"]], "flops": 2 * R * N * K}
    if op == "transpose":
        n = c["M"] * c["N"] * (c["E"] if c["stacked"] else 1)
        return {"bytes": n * (size[c["x"]] + mx), "flops": 2 * n}
    return {"bytes": c["R"] * (c["Na"] + c["Nb"]) * mx + c["E"] * c["Na"] * c["Nb"] * size[c["y"]], "flops": 2 * c["R"] * c["Na"] * c["Nb"]}


# ------------------------------------------------------------------ exact

def _exact_values(q, byte):
    """float64 values from the bit fields of E4M3 codes [N, K] and E8M0 bytes [N, K / 32]."""
    n = q.to(torch.int32)
    field, man = (n >> 3) & 15, (n & 7).double()
    v = torch.where(field == 0, torch.ldexp(man, torch.full_like(field, -9)), torch.ldexp(1.0 + man / 8.0, field - 7))
    v = torch.where(n >= 128, -v, v)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (byte.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _exact_byte(flat, rows, S):
    """Scale bytes of the given padded rows, entry by entry from where each lies in its tile."""
    j = torch.arange(S, device=flat.device)
    tile = (rows // 128)[:, None] * -(-S // 4) + j // 4
    return flat[tile * 512 + (rows % 32)[:, None] * 16 + (rows % 128 // 32)[:, None] * 4 + j % 4]


def _exact_quantized(v):
    """MXFP8 of float64 values in groups of 32: codes as float64 in units of their scale, and bytes."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    byte = torch.where(amax == 0, 127.0, torch.floor(torch.log2(amax.clamp_min(1e-300))) + 119).clamp(0, 254)
    u = b * torch.exp2(127 - byte)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)      # three bits behind the leading one
    return (torch.round(u / step) * step).clamp(-448, 448).flatten(-2), byte.squeeze(-1)


def exact(case, seed):
    c = case
    op = c["op"]
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()     # rounded before it is normed
        rstd = (h.square().mean(1) + 1e-6).rsqrt()
        y = h * rstd.unsqueeze(1) * s["weight"].double()
        q, byte = _exact_quantized(y)
        out = {"codes": q, "scale": torch.exp2(byte - 127), "rstd": rstd}
        if c["swizzled"]:
            out["scale_tiles"] = None
        if c["residual"]:
            out["hidden"] = h
        if c["normed"]:
            out["normed"] = y
        return out
    if op == "norm_backward":
        h, g, w = s["x"].double(), s["grad"].double(), s["weight"].double()
        unit = h * s["rstd"].double().unsqueeze(1)
        gw = g * w
        dx = (gw - unit * (gw * unit).sum(1, keepdim=True) / c["N"]) * s["rstd"].double().unsqueeze(1)
        if c["grad_hidden"]:
            dx += s["grad_hidden"].double()
        return dx, (g * unit).sum(0)
    if op == "transpose":
        if c["stacked"]:
            return _exact_quantized(s["x"].double().transpose(1, 2))[0], None
        off, parts = s["offsets"].tolist(), []
        for e in range(c["E"]):
            rows = s["x"][off[e]:off[e + 1]].double().t()
            parts.append(torch.nn.functional.pad(rows, (0, -rows.shape[1] % 128)))
        x = torch.cat(parts, dim=1)
        rest = (c["M"] + 127 * c["E"]) // 128 * 128 - x.shape[1]       # zeros up to what the padding can come to
        return _exact_quantized(torch.nn.functional.pad(x, (0, rest)))[0], None
    off = s["offsets"].tolist()
    if op == "wgrad":
        out, at = [], 0
        for e in range(c["E"]):
            n = off[e + 1] - off[e]
            p = -(-n // 128) * 128
            sides = []
            for name, rows in (("a", c["Na"]), ("b", c["Nb"])):
                byte = _exact_byte(s[name + "_scale"], torch.arange(rows, device="cuda"), s[name].shape[1] // 32)
                sides.append(_exact_values(s[name][:, at:at + p], byte[:, at // 32:(at + p) // 32]))
            out.append(sides[0] @ sides[1].t())
            at += p
        return torch.stack(out)
    y, at, per = [], 0, -(-c["N"] // 128) * 512 * -(-c["K"] // 128)
    for e in range(c["E"]):
        n = off[e + 1] - off[e]
        if n == 0:
            continue
        a = _exact_values(s["q"][off[e]:off[e + 1]], _exact_byte(s["scale"], at + torch.arange(n, device="cuda"), c["K"] // 32))
        b = _exact_values(s["w"][e], _exact_byte(s["w_scale"][e * per:(e + 1) * per], torch.arange(c["N"], device="cuda"), c["K"] // 32))
        y.append(a @ b.t())
        at += -(-n // 128) * 128
    y = torch.cat(y)
    if c["swiglu"]:
        gate, up = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = gate * torch.sigmoid(gate) * up
    return y
