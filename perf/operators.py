"""Timed passes of the operators around and inside a W8A8 state-space block: the RMS norm with an
int8 output, the W8A8 linear layer, and the int8 recurrent state of the decode update.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, 64 where a
rounding decision or a long sum needs them) or, where ``own`` is true, through the library. The
int8 codes are whole numbers that the operators' definition fixes bit for bit, so they are returned
as they are, beside the scales that give the values they stand for.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
LO, HI = 2.0 ** -100, 2.0 ** 100  # range of a valid scale

# Sizes are those of a Mamba2-8B-shaped block (model width 4096, 128 heads of 64, state 128, 8
# groups, in-projection 4096 -> 18560, out-projection 8192 -> 4096) and generic odd ones.


def listed():
    f = dict(op="norm", xt="f16", rt="f32", gate=False, groups=1, static=False)
    g = dict(op="gemm", yt="f16", bias=False, pad=0, per_row=True)
    u = dict(op="update", heads=128, hdim=64, n=128, groups=8)
    return [
        # pre-norm of one decoded token: latency of one call
        dict(f, name="norm-1-token", m=1, d=4096),
        # pre-norm of a decode batch, fp32 residual stream
        dict(f, name="norm-256-tokens", m=256, d=4096),
        # pre-norm of a prefill of 4 x 4096 tokens
        dict(f, name="norm-16384-tokens", m=16384, d=4096),
        # gated norm before the out-projection, the gate a slice of the in-projection's output
        dict(f, name="gated-norm-16384-tokens", m=16384, d=8192, rt="none", gate=True, groups=8),
        # odd width, fp32 stream, static scale for a layer with one activation scale
        dict(f, name="norm-odd-static", m=1111, d=1543, xt="f32", static=True),
        # in-projection of one decoded token: bound by the weights
        dict(g, name="gemm-1-token", m=1, n=18560, k=4096),
        # out-projection of a decode batch
        dict(g, name="gemm-256-tokens-out", m=256, n=4096, k=8192, yt="f32"),
        # in-projection of a prefill
        dict(g, name="gemm-16384-tokens", m=16384, n=18560, k=4096),
        # ragged sizes with a bias, rows of a wider buffer
        dict(g, name="gemm-ragged", m=777, n=1001, k=1500, yt="f32", bias=True, pad=52),
        # decode update of a few sequences
        dict(u, name="update-2-sequences", b=2),
        # decode update of a large batch
        dict(u, name="update-256-sequences", b=256),
        # a prefill's final states written to the cache and read back
        dict(op="store", name="state-store-32-sequences", rows=32 * 128 * 64, n=128, ht="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "update", "store"])
    if op == "norm":
        groups = rng.choice([1, 1, 2, 8])
        d = _log(rng, 64, 8192 // groups) * groups if rng.random() < 0.5 else 64 * groups * rng.randint(1, 128 // groups)
        gate = rng.random() < 0.4
        return dict(op=op, m=_log(rng, 1, 16384), d=min(d, 8192), groups=groups, gate=gate,
                    xt=rng.choice(["f16", "f32"]), rt="none" if gate else rng.choice(["f16", "f32", "none"]),
                    static=rng.random() < 0.25)
    if op == "gemm":
        odd = rng.random() < 0.4
        n, k = _log(rng, 64, 18560), _log(rng, 64, 8192)
        if not odd:
            n, k = 64 * max(1, n // 64), 64 * max(1, k // 64)
        m = _log(rng, 1, 16384)
        while m * n * k > 16384 * 18560 * 4096:
            m //= 2
        return dict(op=op, m=m, n=n, k=k, yt=rng.choice(["f16", "f32"]), bias=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 16, 5]), per_row=rng.random() < 0.8)
    if op == "update":
        groups = rng.choice([1, 2, 4, 8])
        return dict(op=op, b=_log(rng, 1, 256), heads=groups * rng.randint(1, 128 // groups),
                    hdim=rng.choice([32, 48, 64, 64, 80]) if rng.random() < 0.5 else 64,
                    n=rng.choice([16, 32, 64, 128, 128]), groups=groups)
    return dict(op=op, rows=_log(rng, 100, 32 * 128 * 64), n=rng.choice([16, 64, 100, 128, 128]),
                ht=rng.choice(["f32", "f16"]))


# ------------------------------------------------------------------------------------------------
# Inputs

DT = {"f16": torch.float16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    c = dict(case)
    s = {"case": c}
    if c["op"] == "norm":
        m, d = c["m"], c["d"]
        # activations with a few channels far above the others, as trained models have
        ch = torch.exp(0.5 * randn(d)) * torch.where(rand(d) < 0.004, 20.0, 1.0)
        s["x"] = (randn(m, d) * ch).to(DT[c["xt"]])
        s["weight"] = 1.0 + 0.2 * randn(d)
        s["residual"] = None if c["rt"] == "none" else (2.0 * randn(m, d)).to(DT[c["rt"]])
        s["residual_out"] = None if c["rt"] == "none" else empty((m, d), DT[c["rt"]])
        # the gate is the first columns of the in-projection's rows
        s["gate"] = randn(m, d + d + 64).to(torch.float16)[:, :d] if c["gate"] else None
        s["eps"] = 1e-5
        s["q"] = empty((m, d), torch.int8)
        s["scales"] = torch.full((1,), 0.03, device=DEV) if c["static"] else empty((m,), torch.float32)
    elif c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        codes = lambda r, cols: (randn(r, cols) * 32.0).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
        s["a"] = codes(m, k + c["pad"])[:, :k]
        s["a_scales"] = 0.03 * torch.exp(0.3 * randn(m if c["per_row"] else 1))
        s["w"] = codes(n, k)
        s["w_scales"] = torch.exp(0.3 * randn(n)) / (32.0 * math.sqrt(k))
        s["bias"] = 0.1 * randn(n) if c["bias"] else None
        s["y"] = empty((m, n), DT[c["yt"]])
    elif c["op"] == "update":
        b, nh, p, n, gr = c["b"], c["heads"], c["hdim"], c["n"], c["groups"]
        s["x"], s["B"], s["C"] = randn(b, nh, p), randn(b, gr, n), randn(b, gr, n)
        s["x_group_of"] = torch.arange(nh * p, device=DEV).remainder(4).to(torch.uint8)
        s["x_scales"] = torch.tensor([0.02, 0.025, 0.03, 0.035], device=DEV)
        s["B_scales"] = 0.02 + 0.01 * rand(gr * n // 16)
        s["C_scales"] = 0.02 + 0.01 * rand(gr * n // 16)
        s["delta"] = torch.nn.functional.softplus(0.5 * randn(b, nh) - 2.0)
        s["A"] = -torch.exp(2.0 * rand(nh))
        s["D"] = randn(nh)
        # a cache as the update leaves it: rows of codes up to +-127, each with its scale
        h = randn(b * nh * p, n)
        h = h * (127.0 / h.abs().amax(1, keepdim=True))
        s["codes"] = h.round_().to(torch.int8).view(b, nh, p, n)
        s["scales"] = 0.002 * torch.exp(0.5 * randn(b, nh, p))
        s["codes_out"] = empty((b, nh, p, n), torch.int8)
        s["scales_out"] = empty((b, nh, p), torch.float32)
        s["y"] = empty((b, nh, p), torch.float32)
    else:
        rows, n = c["rows"], c["n"]
        s["h"] = (0.2 * randn(rows, n) * torch.exp(randn(rows, 1))).to(DT[c["ht"]])
        s["codes"] = empty((rows, n), torch.int8)
        s["scales"] = empty((rows,), torch.float32)
        s["back"] = empty((rows, n), torch.float32)
    return s


# ------------------------------------------------------------------------------------------------
# Plain forms

def _scale_of(v, dims):
    """The scale of the largest finite |v| over dims: absmax / 127 within the valid range, 1 for 0."""
    a = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(dims)
    return torch.where(a == 0, 1.0, (a / 127.0).clamp(LO, HI))


def _quant(v, s):
    """clamp(RNE(v / s), -128, 127) of fp32 values: the fp64 quotient of two fp32 numbers rounds to
    a half-integer only where it is one. NaN is 0, and so is what has no valid scale."""
    q = torch.round(v.double() / s.double()).clamp(-128, 127)
    return torch.where(torch.isnan(v) | ~((s >= LO) & (s <= HI)), 0.0, q).to(torch.int8)


def _plain_norm(s):
    c = s["case"]
    m, d, gr = c["m"], c["d"], c["groups"]
    t = s["x"].float()
    res = None
    if s["residual"] is not None:
        res = (t + s["residual"].float()).to(s["residual"].dtype)
        t = res.float()
    if s["gate"] is not None:
        z = s["gate"].double()
        t = t * (z / (1.0 + torch.exp(-z))).float()
    ms = t.double().square().view(m, gr, d // gr).sum(2) / (d // gr)
    r = (1.0 / torch.sqrt(ms + float(np.float32(s["eps"])))).float()
    v = (t.view(m, gr, d // gr) * r[:, :, None]).view(m, d) * s["weight"]
    sc = s["scales"] if c["static"] else _scale_of(v, 1)
    return {"q": _quant(v, sc[:, None]), "scales": sc, "residual": res}


def _plain_gemm(s):
    y = torch.matmul(s["a"].float(), s["w"].float().t())
    y = y * (s["a_scales"][:, None] * s["w_scales"][None, :])
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(DT[s["case"]["yt"]])}


def _plain_update(s):
    c = s["case"]
    b, nh, p, n, gr = c["b"], c["heads"], c["hdim"], c["n"], c["groups"]
    sx = s["x_scales"][s["x_group_of"].long()].view(nh, p)
    xh = _quant(s["x"], sx).float() * sx
    sb, sc = (s[k].repeat_interleave(16).view(gr, n) for k in ("B_scales", "C_scales"))
    Bh = (_quant(s["B"], sb).float() * sb).repeat_interleave(nh // gr, 1)  # [b, nh, n]
    Ch = (_quant(s["C"], sc).float() * sc).repeat_interleave(nh // gr, 1)
    dA = torch.exp((s["delta"] * s["A"]).double()).float()
    keep = dA[:, :, None] * s["scales"]  # [b, nh, p]
    add = (s["delta"][:, :, None] * xh)[..., None] * Bh[:, :, None, :]
    # one rounding of the fused product and sum
    h = (keep.double()[..., None] * s["codes"].double() + add.double()).float()
    y = (h.double() * Ch.double()[:, :, None, :]).sum(3) + (s["D"][None, :, None] * xh).double()
    sn = _scale_of(h, 3)
    return {"y": y.float(), "codes": _quant(h, sn[..., None]), "scales": sn}


def _plain_store(s):
    h = s["h"].float()
    sc = _scale_of(h, 1)
    q = _quant(h, sc[:, None])
    return {"codes": q, "scales": sc, "values": q.float() * sc[:, None]}


PLAIN = {"norm": _plain_norm, "gemm": _plain_gemm, "update": _plain_update, "store": _plain_store}


# ------------------------------------------------------------------------------------------------
# The library's calls. The argument blocks are built at a state's first pass and kept, as the layer
# objects of a program keep them.

def _own_norm(s):
    import quantized_state_space_amd as qs
    c = s["case"]
    if "args" not in s:
        s["args"] = qs.rmsnorm_args(s["x"], s["q"], s["scales"], weight=s["weight"], eps=s["eps"],
                                    residual=s["residual"], residual_out=s["residual_out"],
                                    gate=s["gate"], norm_groups=c["groups"],
                                    compute_scales=not c["static"])
    qs.qssm_rmsnorm_i8(s["args"])
    return {"q": s["q"], "scales": s["scales"], "residual": s["residual_out"]}


def _own_gemm(s):
    import quantized_state_space_amd as qs
    if "args" not in s:
        s["args"] = qs.gemm_w8a8_args(s["a"], s["a_scales"], s["w"], s["w_scales"], s["y"],
                                      bias=s["bias"])
    qs.qssm_gemm_w8a8(s["args"])
    return {"y": s["y"]}


def _own_update(s):
    import quantized_state_space_amd as qs
    if "args" not in s:
        s["args"] = qs.update_args(s["x"], s["x_group_of"], s["x_scales"], s["B"], s["C"],
                                   s["B_scales"], s["C_scales"], 16, s["delta"], s["A"],
                                   s["codes_out"], s["y"], Dskip=s["D"])
    # the previous state stays as it was, as a program keeps it that may take a token back
    qs.qssm_state_update_i8(s["args"], s["scales_out"], state_in=s["codes"], scales_in=s["scales"])
    return {"y": s["y"], "codes": s["codes_out"], "scales": s["scales_out"]}


def _own_store(s):
    import quantized_state_space_amd as qs
    qs.qssm_state_quant(s["h"], s["codes"], s["scales"])
    qs.qssm_state_dequant(s["codes"], s["scales"], s["back"])
    return {"codes": s["codes"], "scales": s["scales"], "values": s["back"]}


OWN = {"norm": _own_norm, "gemm": _own_gemm, "update": _own_update, "store": _own_store}


def run(state):
    if own:
        return OWN[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# Least work, and the values in 64 bits

SIZE = {"f16": 2, "f32": 4, "none": 0}


def work(case):
    c = case
    if c["op"] == "norm":
        e = c["m"] * c["d"]
        per = SIZE[c["xt"]] + 2 * SIZE[c["rt"]] + (2 if c["gate"] else 0) + 1
        return {"bytes": e * per + 4 * c["d"] + (4 if c["static"] else 4 * c["m"]), "flops": 7 * e}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        b = m * k + n * k + SIZE[c["yt"]] * m * n + 4 * (m if c["per_row"] else 1) + 4 * n * (2 if c["bias"] else 1)
        return {"bytes": b, "flops": 2 * m * n * k}
    if c["op"] == "update":
        rows = c["b"] * c["heads"] * c["hdim"]
        b = rows * (2 * c["n"] + 16) + 8 * c["b"] * c["groups"] * c["n"] + 4 * c["b"] * c["heads"]
        return {"bytes": b, "flops": 8 * rows * c["n"]}
    e = c["rows"] * c["n"]
    return {"bytes": e * (SIZE[c["ht"]] + 1 + 1 + 4) + 8 * c["rows"], "flops": 4 * e}


def exact(case, seed):
    """The floating outputs in 64 bits. Codes have no such value: their definition rounds to 32
    bits on the way, and they are compared as whole numbers."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        t = s["x"].double()
        res = None
        if s["residual"] is not None:
            t = t + s["residual"].double()
            res = t
            if c["rt"] == "f16":  # the norm is of the stream as it is stored
                t = t.half().double()
        if s["gate"] is not None:
            t = t * s["gate"].double() * torch.sigmoid(s["gate"].double())
        t = t.reshape(c["m"], c["groups"], -1)
        t = t * (t.pow(2).mean(2, keepdim=True) + s["eps"]).rsqrt()
        v = t.reshape(c["m"], c["d"]) * s["weight"].double()
        return {"q": None, "scales": s["scales"].double() if c["static"] else v.abs().amax(1) / 127.0,
                "residual": res}
    if c["op"] == "gemm":
        # sums of 1024 products of 8-bit codes are whole numbers up to 2^24: exact in 32 bits
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device=DEV)
        for k in range(0, c["k"], 1024):
            y += s["a"][:, k:k + 1024].float() @ s["w"][:, k:k + 1024].float().t()
        y *= s["a_scales"].double()[:, None]
        y *= s["w_scales"].double()
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if c["op"] == "update":
        nh, p, n, gr = c["heads"], c["hdim"], c["n"], c["groups"]

        def value(v, sc):  # the 8-bit value of an input, decided in 64 bits
            return (v.double() / sc.double()).round().clamp(-128, 127) * sc.double()

        of = torch.arange(gr * n, device=DEV) // 16
        xh = value(s["x"].reshape(c["b"], -1), s["x_scales"][s["x_group_of"].long()]).view(c["b"], nh, p)
        Bh = value(s["B"].reshape(c["b"], -1), s["B_scales"][of]).view(c["b"], gr, 1, 1, n)
        Ch = value(s["C"].reshape(c["b"], -1), s["C_scales"][of]).view(c["b"], gr, 1, 1, n)
        dt = s["delta"].double()
        h = s["codes"].double() * s["scales"].double()[..., None]
        h *= torch.exp(dt * s["A"].double())[:, :, None, None]
        h = h.view(c["b"], gr, nh // gr, p, n)
        h += (dt[:, :, None] * xh).view(c["b"], gr, nh // gr, p, 1) * Bh
        y = (h * Ch).sum(4).view(c["b"], nh, p)
        y = y + s["D"].double()[None, :, None] * xh
        return {"y": y, "codes": None, "scales": h.abs().amax(4).view(c["b"], nh, p) / 127.0}
    h = s["h"].double()
    sc = h.abs().amax(1) / 127.0
    s32 = sc.float().double()
    return {"codes": None, "scales": sc,
            "values": torch.round(h / s32[:, None]) * s32[:, None]}
