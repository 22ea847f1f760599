"""The operators around the expert layer, as cases that can be timed and compared.

Three operators of one MoE block:

* add_rmsnorm: the residual's addition, the RMS norm and the MXFP8 operand of the next product
  (e4m3 codes, one E8M0 scale per 32 elements), and its backward pass;
* moe_route: the top-k choice of experts with its weights from the gate's logits, and its
  backward pass;
* moe_decode: a whole expert layer (FC1, SwiGLU, FC2, weighted combine) for a few tokens, with
  BF16, MXFP8 or MXFP4 weights.

`run` with own = False is the plain form: elementary torch operations in 32 bits, rounded once
at the end.  With own = True it makes the calls of this package that a user makes.  `exact` is
the same from the definitions in 64 bits, written on its own.

Codes and scales are returned as the floating types whose bytes they are (float8_e4m3fn and
float8_e8m0fnu): the values that they stand for.
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"
MASK = float("-inf")


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # the norm before the experts of a decode step: four sequences, latency counts
        {"name": "norm_fwd_4x4096", "op": "norm_fwd", "rows": 4, "cols": 4096, "residual": True},
        # the same norm over a training micro-batch of the hidden-4096 layers
        {"name": "norm_fwd_16384x4096", "op": "norm_fwd", "rows": 16384, "cols": 4096, "residual": True},
        # its backward pass in the hidden-2880 layer
        {"name": "norm_bwd_8192x2880", "op": "norm_bwd", "rows": 8192, "cols": 2880, "residual": True},
        # a short, narrow batch without a residual gradient: few rows to share out, odd sizes
        {"name": "norm_bwd_333x1056", "op": "norm_bwd", "rows": 333, "cols": 1056, "residual": False},
        # the gate of a decode step: sigmoid scores with a balancing bias and three blocked experts
        {"name": "route_fwd_33x256", "op": "route_fwd", "tokens": 33, "experts": 256, "k": 6, "dtype": "f32",
         "score": "sigmoid", "renormalize": True, "scale": 2.5, "bias": True, "blocked": 3},
        # the gate of a training batch, bf16 logits as a bf16 gate product gives them (many ties)
        {"name": "route_fwd_16384x256", "op": "route_fwd", "tokens": 16384, "experts": 256, "k": 8, "dtype": "bf16",
         "score": "softmax", "renormalize": True, "scale": 1.0, "bias": False, "blocked": 0},
        # the gate's backward pass, softmax over all experts (every logit gets a gradient), two blocked
        {"name": "route_bwd_8191x32", "op": "route_bwd", "tokens": 8191, "experts": 32, "k": 4, "dtype": "f32",
         "score": "softmax", "renormalize": False, "scale": 1.0, "bias": True, "blocked": 2},
        # one token through the 256-expert layer in BF16: pure weight streaming, six experts
        {"name": "decode_bf16_t1", "op": "decode", "fmt": "bf16", "tokens": 1, "k": 6, "experts": 256, "hidden": 4096,
         "inter": 2048, "zipf": 0.0, "blocked": 0, "limit": 0.0},
        # a decode batch through the hidden-2880 layer (sizes off the tiles, two experts blocked, clamped SwiGLU)
        {"name": "decode_bf16_t32", "op": "decode", "fmt": "bf16", "tokens": 32, "k": 4, "experts": 32,
         "hidden": 2880, "inter": 2880, "zipf": 0.0, "blocked": 2, "limit": 7.0},
        # a small batch in MXFP8
        {"name": "decode_mxfp8_t8", "op": "decode", "fmt": "e4m3", "tokens": 8, "k": 6, "experts": 256,
         "hidden": 4096, "inter": 2048, "zipf": 0.0, "blocked": 0, "limit": 0.0},
        # one token in MXFP4: the least to read, so that launches and joins show
        {"name": "decode_mxfp4_t1", "op": "decode", "fmt": "e2m1", "tokens": 1, "k": 8, "experts": 256,
         "hidden": 4096, "inter": 2048, "zipf": 0.0, "blocked": 0, "limit": 0.0},
        # a skewed batch in MXFP4: a few experts with most of the tokens, many with one
        {"name": "decode_mxfp4_t64_zipf", "op": "decode", "fmt": "e2m1", "tokens": 64, "k": 8, "experts": 256,
         "hidden": 4096, "inter": 2048, "zipf": 1.2, "blocked": 0, "limit": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(n):
    """The odd number at or below n: of the units of a size, so that it ends inside the kernels' tiles."""
    return (n - 1) | 1


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "route_fwd", "route_bwd", "decode", "decode"])
    if op.startswith("norm"):
        cols = 32 * _odd(_log_int(rng, 2, 256))
        rows = _log_int(rng, 1, min(16384, 16384 * 4096 // cols))
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.75}
    if op.startswith("route"):
        experts = _log_int(rng, 8, 1024)
        tokens = _log_int(rng, 1, min(16384, 16384 * 256 // experts))
        return {"op": op, "tokens": tokens, "experts": experts, "k": rng.randint(1, min(16, experts)),
                "dtype": rng.choice(["f32", "bf16"]), "score": rng.choice(["softmax", "sigmoid"]),
                "renormalize": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "bias": rng.random() < 0.5,
                "blocked": rng.choice([0, 0, experts // 8])}
    fmt = rng.choice(["bf16", "e4m3", "e2m1"])
    unit = 8 if fmt == "bf16" else 128
    hidden = unit * _odd(_log_int(rng, 256 // unit, 4096 // unit))
    inter = unit * _odd(_log_int(rng, 256 // unit, 4096 // unit))
    # at most the weights of the largest listed layer
    experts = _log_int(rng, 8, min(512, 256 * 4096 * 2048 // (hidden * inter)))
    k = rng.randint(1, 8)
    # no more (token, choice) entries, and no more weight bytes, than the largest listed cases have
    size = {"bf16": 2.0, "e4m3": 1.04, "e2m1": 0.54}[fmt]
    most = 64 * 8 * 4096 * 2048 // (hidden * inter)
    if min(most, experts) * 3 * hidden * inter * size > 2e9:
        most = int(2e9 / (3 * hidden * inter * size))
    most = max(1, min(128, most // k))
    return {"op": op, "fmt": fmt, "tokens": _log_int(rng, 1, most), "k": k, "experts": experts, "hidden": hidden,
            "inter": inter, "zipf": rng.choice([0.0, 1.2]), "blocked": rng.choice([0, min(2, experts - k)]),
            "limit": rng.choice([0.0, 0.0, 7.0])}


# ---------------------------------------------------------------------------- inputs

def _generator(case, seed):
    # the case itself goes into the seed, so that two cases of one seed differ
    mix = zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode())
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + mix) % (1 << 62))
    return g


def _ids(case, seed):
    """Distinct expert ids [tokens, k] of a token, by Gumbel keys; the last `blocked` experts get none."""
    rng = np.random.default_rng([int(seed) % (1 << 31), case["tokens"], case["experts"], case["k"]])
    p = -case["zipf"] * np.log(np.arange(1, case["experts"] + 1))
    if case["zipf"]:
        p = rng.permutation(p)
    keys = p[None, :] - np.log(-np.log(rng.random((case["tokens"], case["experts"]))))
    if case["blocked"]:
        keys[:, -case["blocked"]:] = -np.inf
    return np.argsort(-keys, axis=1, kind="stable")[:, :case["k"]].astype(np.int32)


_QMAX = {"e4m3": 448.0, "e2m1": 6.0}
_EMAX = {"e4m3": 8, "e2m1": 2}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx(v, fmt):
    """Blocks of 32 of the last axis -> (values of the element type before rounding, saturated, exponents)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - _EMAX[fmt]).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    q = torch.ldexp(b, -e).clamp(-_QMAX[fmt], _QMAX[fmt])
    return q, e.squeeze(-1)


def _round_e2m1(q):
    """Round to nearest, ties to even, on the e2m1 grid."""
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return torch.round(a / step) * step * torch.where(q < 0, -1.0, 1.0).to(a.dtype)


def _codes(q, fmt):
    """Element values on their grid or off it -> the bytes that hold them, [..., C] or packed [..., C/2]."""
    q = q.reshape(*q.shape[:-2], -1)
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8)
    r = _round_e2m1(q.float())
    a = r.abs()
    n = (torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)) + 8 * (r < 0)).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _blocked(s):
    """Row-major scale bytes [R, C/32], R and C multiples of 128 -> the 512-byte atoms of the weight operand."""
    r, c = s.shape
    return s.view(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(r, c).contiguous()


def _mx_weights(rows, cols, std, fmt, gen):
    """Codes and blocked scales of a normal weight matrix, made in pieces."""
    w = cols if fmt == "e4m3" else cols // 2
    codes = torch.empty((rows, w), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    step = 128 * max(1, (1 << 28) // (128 * cols))
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q, e = _mx(torch.randn((n, cols), generator=gen, device=DEV) * std, fmt)
        codes[r:r + n] = _codes(q, fmt)
        scales[r:r + n] = _blocked((e + 127).to(torch.uint8))
    return codes, scales


def _logits(case, gen):
    t, e = case["tokens"], case["experts"]
    x = torch.randn((t, e), generator=gen, device=DEV) * 1.5
    if case["blocked"]:
        x[:, -case["blocked"]:] = MASK
    x = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    bias = torch.randn((e,), generator=gen, device=DEV) * 0.1 if case["bias"] else None
    return x, bias


def prepare(case, seed):
    gen = _generator(case, seed)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op.startswith("norm"):
        r, c = case["rows"], case["cols"]
        # activations with a few large channels, as residual streams have
        big = 1 + 20 * (torch.rand((c,), generator=gen, device=DEV) < 0.01)
        s["eps"] = 1e-6
        s["gamma"] = (1 + 0.2 * rnd(c)).bfloat16()
        if op == "norm_fwd":
            s["x"] = rnd(r, c).bfloat16()
            s["residual"] = (rnd(r, c) * big).bfloat16() if case["residual"] else None
        else:
            h = (rnd(r, c) * big).bfloat16()
            s["h"], s["dy"] = h, (rnd(r, c) * 0.01).bfloat16()
            s["dh"] = (rnd(r, c) * 0.01).bfloat16() if case["residual"] else None
            s["rstd"] = torch.rsqrt(h.float().square().mean(-1) + s["eps"])
            s["scratch"] = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    elif op.startswith("route"):
        s["logits"], s["bias"] = _logits(case, gen)
        if op == "route_bwd":
            key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
            s["ids"] = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :case["k"]].int().contiguous()
            s["dw"] = rnd(case["tokens"], case["k"])
    else:
        t, k, e, hd, it, fmt = (case[n] for n in ("tokens", "k", "experts", "hidden", "inter", "fmt"))
        s["ids"] = torch.from_numpy(_ids(case, seed)).to(DEV)
        w = torch.rand((t, k), generator=gen, device=DEV) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        x = rnd(t, hd)
        if fmt == "bf16":
            s["x"] = x.bfloat16()
            s["w1"] = torch.randn((e, 2 * it, hd), generator=gen, device=DEV, dtype=torch.bfloat16).mul_(0.02)
            s["w2"] = torch.randn((e, hd, it), generator=gen, device=DEV, dtype=torch.bfloat16).mul_(0.02)
        else:
            q, ex = _mx(x, fmt)
            s["xq"] = (_codes(q, fmt), (ex + 127).to(torch.uint8))
            s["w1q"] = _mx_weights(e * 2 * it, hd, 0.02, fmt, gen)
            s["w2q"] = _mx_weights(e * hd, it, 0.02, fmt, gen)
        s["scratch"] = torch.zeros(128 << 20, dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((t, hd), dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------- the package's calls

def _own(s):
    import precision_grouped_gemm_gb300 as pgg
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        h, y, codes, scales, rstd = pgg.add_rmsnorm(s["x"], s["residual"], s["gamma"], s["eps"], fmt="e4m3")
        return {"h": h, "y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu),
                "rstd": rstd}
    if op == "norm_bwd":
        dx, dgamma = pgg.add_rmsnorm_bwd(s["dy"], s["dh"], s["h"], s["gamma"], s["rstd"], ws=s["scratch"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "route_fwd":
        ids, w = pgg.moe_route(s["logits"], c["k"], bias=s["bias"], score=c["score"], renormalize=c["renormalize"],
                               scale=c["scale"])
        return {"ids": ids, "w": w}
    if op == "route_bwd":
        return {"dlogits": pgg.moe_route_bwd(s["logits"], s["ids"], s["dw"], bias=s["bias"], score=c["score"],
                                             renormalize=c["renormalize"], scale=c["scale"])}
    if c["fmt"] == "bf16":
        return pgg.moe_decode(s["x"], s["ids"], s["w"], s["w1"], s["w2"], out=s["out"], swiglu_limit=c["limit"],
                              ws=s["scratch"])
    return pgg.mx_moe_decode(c["fmt"], *s["xq"], s["ids"], s["w"], *s["w1q"], *s["w2q"], out=s["out"],
                             swiglu_limit=c["limit"], ws=s["scratch"])


# ---------------------------------------------------------------------------- the plain forms

def _norm_fwd(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + s["eps"])
    y = v * rstd * s["gamma"].float()
    q, e = _mx(y, "e4m3")
    return {"h": v.bfloat16(), "y": y.bfloat16(), "codes": _codes(q, "e4m3").view(torch.float8_e4m3fn),
            "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), "rstd": rstd.squeeze(-1)}


def _norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["h"].float() * rstd
    u = dy * s["gamma"].float()
    dx = rstd * (u - xh * (u * xh).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.bfloat16(), "dgamma": (dy * xh).sum(0)}


def _keys(s):
    x = s["logits"].float()
    key = x if s["bias"] is None else x + s["bias"]
    return x, key, key == MASK


def _route_fwd(s):
    c = s["case"]
    x, key, masked = _keys(s)
    bad = torch.isnan(key).any(1, keepdim=True)
    key = torch.where(torch.isnan(key), MASK, key)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["k"]]
    x = torch.where(masked, MASK, x)
    if c["score"] == "softmax":
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(m == MASK, 0.0, m))
        total = p.sum(1, keepdim=True)
    else:
        p = torch.where(masked, 0.0, torch.sigmoid(x))
        total = 1.0
    w = p.gather(1, ids)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
    w = torch.where(w == 0, 0.0, c["scale"] * w / total)
    return {"ids": ids.int(), "w": torch.where(bad, float("nan"), w)}


def _route_bwd(s):
    c = s["case"]
    x, key, masked = _keys(s)
    ids = s["ids"].long()
    x = torch.where(masked, MASK, x)
    dw = s["dw"] * c["scale"]
    if c["score"] == "softmax" and not c["renormalize"]:
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(m == MASK, 0.0, m))
        p = torch.where(p == 0, 0.0, p / p.sum(1, keepdim=True))
        full = torch.zeros_like(p).scatter_add(1, ids, dw)
        d = p * (full - (dw * p.gather(1, ids)).sum(1, keepdim=True))
    else:
        xs = x.gather(1, ids)
        if c["score"] == "softmax":
            m = xs.amax(1, keepdim=True)
            a = torch.exp(xs - torch.where(m == MASK, 0.0, m))
            slope = 1.0
        else:
            a = torch.sigmoid(xs)
            slope = torch.sigmoid(-xs)
        if c["renormalize"]:
            a = torch.where(a == 0, 0.0, a / a.sum(1, keepdim=True))
            dw = dw - (dw * a).sum(1, keepdim=True)
        d = torch.zeros_like(x).scatter_add(1, ids, a * slope * dw)
    d = torch.where(torch.isnan(key).any(1, keepdim=True), float("nan"), d)
    return {"dlogits": d.to(s["logits"].dtype)}


def _unblocked(s, rows):
    """The atoms of whole experts [n, rows * C/32] -> row-major scale bytes [n, rows, C/32]."""
    n = s.shape[0]
    c = s.shape[1] // rows
    return s.view(n, rows // 128, c // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, rows, c)


def _values(codes, scales, fmt):
    """MX codes [..., C or C/2] and row-major scale bytes [..., C/32] -> 32-bit values [..., C]."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=DEV)
        n = torch.stack((codes & 15, codes >> 4), -1).flatten().int()
        v = lut.index_select(0, n).view(*codes.shape[:-1], -1)
    b = v.view(*v.shape[:-1], -1, 32)
    return b.mul_(torch.exp2(scales.float() - 127).unsqueeze(-1)).view_as(v)


def _weights(w, fmt, experts, rows, pick):
    """Rows of the picked experts as 32-bit values [n, rows, cols]."""
    if fmt == "bf16":
        return w[pick].float()
    codes, scales = w
    return _values(codes.view(experts, rows, -1)[pick], _unblocked(scales.view(experts, -1)[pick], rows), fmt)


def _decode(s):
    c = s["case"]
    t, k, e, hd, it, fmt, limit = (c[n] for n in ("tokens", "k", "experts", "hidden", "inter", "fmt", "limit"))
    x = s["x"].float() if fmt == "bf16" else _values(*s["xq"], fmt)
    w1, w2 = (s["w1"], s["w2"]) if fmt == "bf16" else (s["w1q"], s["w2q"])
    ids = s["ids"].long().flatten()
    xe = x.repeat_interleave(k, 0)
    ys = []
    # every (token, choice) entry with its own expert's weights; in pieces that hold about 2^30 of them
    n = max(1, (1 << 30) // (2 * it * hd))
    for a in range(0, t * k, n):
        pick = ids[a:a + n]
        g = torch.bmm(_weights(w1, fmt, e, 2 * it, pick), xe[a:a + n, :, None]).squeeze(-1)
        gate, up = g[:, :it], g[:, it:]
        if limit:
            gate, up = gate.clamp(max=limit), up.clamp(-limit, limit)
        act = gate / (1 + torch.exp(-gate)) * up
        if fmt != "bf16":  # the second product's operand is in the same format
            q, ex = _mx(act, fmt)
            q = q.to(torch.float8_e4m3fn).float() if fmt == "e4m3" else _round_e2m1(q)
            act = torch.ldexp(q, ex.unsqueeze(-1)).reshape(act.shape)
        ys.append(torch.bmm(_weights(w2, fmt, e, hd, pick), act[:, :, None]).squeeze(-1))
    y = torch.cat(ys).view(t, k, hd)
    return (y * s["w"][:, :, None]).sum(1).bfloat16()


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "route_fwd": _route_fwd, "route_bwd": _route_bwd,
            "decode": _decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def _distinct(case):
    """Experts that a batch touches, over a few draws of its routing."""
    return float(np.mean([np.unique(_ids(case, q)).size for q in range(8)]))


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, c, r = case["rows"] * case["cols"], case["cols"], case["rows"]
        if op == "norm_fwd":  # x, residual; h, y, codes, scales, rstd
            return {"bytes": n * (2 + 2 * case["residual"] + 4 + 1 + 1 / 32) + 2 * c + 4 * r, "flops": 8 * n}
        return {"bytes": n * (6 + 2 * case["residual"]) + 6 * c + 4 * r, "flops": 10 * n}
    if op.startswith("route"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": t * e * size * (2 if op == "route_bwd" else 1) + 8 * t * k + 4 * e * case["bias"],
                "flops": 4 * t * e}
    t, k, hd, it = case["tokens"], case["k"], case["hidden"], case["inter"]
    per = {"bf16": 2.0, "e4m3": 1 + 1 / 32, "e2m1": 0.5 + 1 / 32}[case["fmt"]]
    return {"bytes": _distinct(case) * 3 * hd * it * per + t * hd * (per + 2) + 8 * t * k,
            "flops": 6 * t * k * hd * it}


# ---------------------------------------------------------------------------- from the definitions, in 64 bits

def _mx64(v, fmt):
    """Blocks of 32 in 64 bits -> (element values on the type's grid, powers of two)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    # log2 may land on the wrong side of a whole number: put it right by comparison
    power = power - (torch.exp2(power) > amax).double() * (amax > 0) + (torch.exp2(power + 1) <= amax).double()
    power = torch.where(amax > 0, power - _EMAX[fmt], torch.full_like(power, -127.0)).clamp(-127, 127)
    z = b / torch.exp2(power)
    a = z.abs().clamp(max=_QMAX[fmt])
    lowest, bits = (-6, 3) if fmt == "e4m3" else (0, 1)  # least normal exponent, mantissa bits
    binade = torch.floor(torch.log2(a.clamp(min=2.0 ** (lowest - bits - 2)))).clamp(min=lowest)
    binade = binade - (torch.exp2(binade) > a).double() * (binade > lowest) + (torch.exp2(binade + 1) <= a).double()
    step = torch.exp2(binade - bits)
    return torch.sign(z) * torch.round(a / step) * step, power.squeeze(-1)


def _values64(codes, scales, fmt):
    grid = []
    for n in range(256 if fmt == "e4m3" else 16):
        if fmt == "e4m3":
            sign, ex, man = n >> 7, (n >> 3) & 15, n & 7
            v = man / 8 * 2.0 ** -6 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        else:
            sign, ex, man = n >> 3, (n >> 1) & 3, n & 1
            v = man / 2 if ex == 0 else (1 + man / 2) * 2.0 ** (ex - 1)
        grid.append(-v if sign else v)
    grid = torch.tensor(grid, dtype=torch.float64, device=codes.device)
    n = codes.long()
    if fmt == "e2m1":
        n = torch.stack((n % 16, n // 16), -1).flatten(-2)
    return grid[n] * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _rows64(atoms, r0, rows, cols):
    """Row-major scale bytes of weight rows [r0, r0 + rows), read one by one from the blocked atoms."""
    r = torch.arange(r0, r0 + rows, device=atoms.device)[:, None]
    j = torch.arange(cols // 32, device=atoms.device)[None, :]
    at = (r // 128 * (cols // 128) + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4
    return atoms.flatten()[at]


def _exact_decode(s):
    c = s["case"]
    e, hd, it, fmt, limit = (c[n] for n in ("experts", "hidden", "inter", "fmt", "limit"))
    x = s["x"].double() if fmt == "bf16" else _values64(*s["xq"], fmt)
    out = torch.zeros((c["tokens"], hd), dtype=torch.float64, device=DEV)
    for ex in range(e):
        tok, choice = torch.nonzero(s["ids"] == ex, as_tuple=True)
        if not tok.numel():
            continue
        if fmt == "bf16":
            w1, w2 = s["w1"][ex].double(), s["w2"][ex].double()
        else:
            (c1, s1), (c2, s2) = s["w1q"], s["w2q"]
            w1 = _values64(c1[ex * 2 * it:(ex + 1) * 2 * it], _rows64(s1, ex * 2 * it, 2 * it, hd), fmt)
            w2 = _values64(c2[ex * hd:(ex + 1) * hd], _rows64(s2, ex * hd, hd, it), fmt)
        hid = x[tok] @ w1.T
        gate, up = hid[:, :it], hid[:, it:]
        if limit:
            gate, up = torch.clamp(gate, max=limit), torch.clamp(up, -limit, limit)
        act = gate * torch.sigmoid(gate) * up
        if fmt != "bf16":
            v, power = _mx64(act, fmt)
            act = (v * torch.exp2(power)[..., None]).reshape(act.shape)
        out.index_add_(0, tok, s["w"].double()[tok, choice][:, None] * (act @ w2.T))
    return out


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    key32 = s["logits"].float()  # the choice is by the 32-bit sums: a definition, not a rounding
    key32 = (key32 if s["bias"] is None else key32 + s["bias"]).cpu().numpy()
    masked = np.isneginf(key32)
    t, k = x.shape[0], c["k"]
    rows = np.arange(t)[:, None]
    ids = np.argsort(-key32, axis=1, kind="stable")[:, :k] if c["op"] == "route_fwd" else s["ids"].cpu().numpy()
    chosen = np.zeros_like(masked)
    chosen[rows, ids] = True
    over = (chosen if c["renormalize"] else np.ones_like(chosen)) & ~masked
    if c["score"] == "softmax":
        top = np.max(np.where(masked, -np.inf, x), axis=1, keepdims=True)
        score = np.where(masked, 0, np.exp(np.where(masked, 0, x) - np.where(np.isfinite(top), top, 0)))
        slope = np.ones_like(score)
    else:
        score = np.where(masked, 0, 1 / (1 + np.exp(-np.where(masked, 0, x))))
        slope = 1 - score
    shared = c["score"] == "softmax" or c["renormalize"]
    total = np.sum(score * over, axis=1, keepdims=True) if shared else np.ones((t, 1))
    part = np.divide(score, total, out=np.zeros_like(score), where=total > 0) * over
    if c["op"] == "route_fwd":
        return {"ids": ids.astype(np.int32), "w": c["scale"] * (part * chosen)[rows, ids]}
    dw = np.zeros_like(part)
    dw[rows, ids] = s["dw"].double().cpu().numpy() * c["scale"]
    if shared:
        dw = dw - np.sum(dw * part * chosen, axis=1, keepdims=True)
    elif not c["renormalize"]:
        dw = dw * chosen
    return {"dlogits": part * slope * dw}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decode":
        return _exact_decode(s)
    if op.startswith("route"):
        return _exact_route(s)
    if op == "norm_fwd":
        v = s["x"].double()
        if s["residual"] is not None:
            v = v + s["residual"].double()
        rstd = 1 / torch.sqrt((v * v).mean(1) + s["eps"])
        y = s["gamma"].double() * (v * rstd[:, None])
        code, power = _mx64(y, "e4m3")
        return {"h": v, "y": y, "codes": code.reshape(y.shape), "scales": torch.exp2(power), "rstd": rstd}
    h, dy, gamma, rstd = (s[n].double() for n in ("h", "dy", "gamma", "rstd"))
    rows = torch.arange(h.shape[0], device=DEV)
    n = h * rstd[rows, None]
    dot = torch.einsum("rc,rc->r", dy * gamma, n) / h.shape[1]
    dx = (dy * gamma - n * dot[:, None]) * rstd[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, n)}
