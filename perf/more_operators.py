"""The products with biases and the joints between blocks, as cases that can be timed and compared.

Four operators around the experts:

* grouped_linear: a matrix product per group of rows (experts, or one dense product) with the bias,
  the activation and the residual's addition in its epilogue;
* grouped_linear_bwd: the gradient before the activation, and the biases' gradient per group;
* block_join: what stands between two blocks -- the norm of a block's output, dropout, its gate,
  the scaled residual's addition, the next block's norm and its MXFP8 operand;
* block_join_bwd: its gradients.

`run` with own = False is the plain form: elementary torch operations in 32 bits, rounded once
at the end.  With own = True it makes the calls of this package that a user makes.  `exact` is
the same from the definitions in 64 bits, written on its own.

Dropout's mask is that of the counter-based generator Philox4x32-10 (Salmon et al., "Parallel random
numbers: as easy as 1, 2, 3"): element i of the row-major tensor takes word i % 4 of the block whose
counter is (i / 4, offset), both 64 bits, under the key seed; it is kept where that word is at least
floor(p 2^32).

Codes and scales are returned as the floating types whose bytes they are (float8_e4m3fn and
float8_e8m0fnu): the values that they stand for.
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decode step through a dense product whose result joins the residual stream
        # (an attention's output, a shared expert's second product): weight streaming, latency counts
        {"name": "linear_dense_1x4096x4096", "op": "linear", "rows": 1, "n": 4096, "k": 4096, "groups": 1, "empty": 0,
         "zipf": 0.0, "act": "none", "bias": True, "residual": True, "out": "bf16", "save_z": False},
        # the gate of a decode batch: few rows, few columns, fp32 logits (ties of bf16 logits would decide the routing)
        {"name": "linear_gate_37x256x4096", "op": "linear", "rows": 37, "n": 256, "k": 4096, "groups": 1, "empty": 0,
         "zipf": 0.0, "act": "none", "bias": True, "residual": False, "out": "f32", "save_z": False},
        # a shared expert's second product over a training batch, added to what the routed experts gave
        {"name": "linear_dense_16384x4096x2048", "op": "linear", "rows": 16384, "n": 4096, "k": 2048, "groups": 1,
         "empty": 0, "zipf": 0.0, "act": "none", "bias": False, "residual": True, "out": "bf16", "save_z": False},
        # the first product of the 32 biased experts of hidden size 2880 (two of them blocked) in training
        {"name": "linear_experts32_gated", "op": "linear", "rows": 32768, "n": 5760, "k": 2880, "groups": 32, "empty": 2,
         "zipf": 0.0, "act": "swiglu", "bias": True, "residual": False, "out": "bf16", "save_z": True},
        # the second product of 256 experts over a ragged batch: some 96 rows each, every weight read once
        {"name": "linear_experts256_fc2", "op": "linear", "rows": 24576, "n": 4096, "k": 2048, "groups": 256, "empty": 0,
         "zipf": 0.0, "act": "none", "bias": True, "residual": False, "out": "bf16", "save_z": False},
        # a decode batch of 32 tokens, four experts each, through the biased experts: 128 rows over 32 experts
        {"name": "linear_experts32_decode", "op": "linear", "rows": 128, "n": 5760, "k": 2880, "groups": 32, "empty": 2,
         "zipf": 0.0, "act": "swiglu", "bias": True, "residual": False, "out": "bf16", "save_z": False},
        # the gradient of the biased experts' activation over the same training batch
        {"name": "linear_bwd_experts32_gated", "op": "linear_bwd", "rows": 32768, "n": 5760, "groups": 32, "empty": 2,
         "zipf": 0.0, "act": "swiglu"},
        # a short ragged batch through an ungated layer: odd sizes, an empty group, few rows to share out
        {"name": "linear_bwd_777x1032_gelu", "op": "linear_bwd", "rows": 777, "n": 1032, "groups": 5, "empty": 1,
         "zipf": 1.0, "act": "gelu"},
        # between two blocks of a decode step: four sequences, latency counts
        {"name": "join_fwd_4x4096", "op": "join_fwd", "rows": 4, "cols": 4096, "post": True, "gate": "token", "p": 0.0,
         "a": 1.0, "c": 0.5, "mx": True},
        # the same over a training micro-batch, with dropout
        {"name": "join_fwd_16384x4096_dropout", "op": "join_fwd", "rows": 16384, "cols": 4096, "post": True,
         "gate": "channel", "p": 0.1, "a": 1.0, "c": 1.0, "mx": False},
        # its backward pass in the hidden-2880 layer
        {"name": "join_bwd_8192x2880_dropout", "op": "join_bwd", "rows": 8192, "cols": 2880, "post": True,
         "gate": "channel", "p": 0.1, "a": 1.0, "c": 1.0},
        # a short, narrow batch with a gate per token and a scaled residual: few rows to share out, odd sizes
        {"name": "join_bwd_333x1056", "op": "join_bwd", "rows": 333, "cols": 1056, "post": True, "gate": "token",
         "p": 0.0, "a": 0.9, "c": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(n):
    """The odd number at or below n: of the units of a size, so that it ends inside the kernels' tiles."""
    return (n - 1) | 1


ACTS = ("none", "silu", "gelu", "swiglu")
# of the generalised SwiGLU g sigmoid(alpha g) (u + offset), clamped at the limit, and of silu
ALPHA, OFFSET, LIMIT = 1.702, 1.0, 7.0


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "join_fwd", "join_bwd"])
    if op.startswith("linear"):
        act = rng.choice(ACTS)
        unit = 16 if act == "swiglu" else 8
        n = unit * _odd(_log_int(rng, 128 // unit, 8192 // unit))
        groups = rng.choice([1, _log_int(rng, 2, 32), _log_int(rng, 32, 256)])
        case = {"op": op, "n": n, "groups": groups, "empty": groups // 8 * rng.randint(0, 1),
                "zipf": rng.choice([0.0, 1.0]), "act": act}
        if op == "linear_bwd":
            # at most the elements of the largest listed gradient
            case["rows"] = _log_int(rng, 1, min(32768, 32768 * 5760 // n))
            return case
        k = case["k"] = 8 * _odd(_log_int(rng, 16, 1024))
        # at most the weights, the operations and the rows of the largest listed layers
        groups = case["groups"] = max(1, min(groups, 256 * 4096 * 2048 // (n * k)))
        case["empty"] = min(case["empty"], groups // 8)
        most = min(32768, 32768 * 5760 * 2880 // (n * k), 32768 * 5760 // n)
        case["rows"] = _log_int(rng, 1, rng.choice([min(256, most), most]))
        case["bias"] = rng.random() < 0.75
        case["residual"] = rng.random() < 0.5
        case["out"] = rng.choice(["bf16", "bf16", "f32"])
        case["save_z"] = act != "none" and rng.random() < 0.5
        return case
    cols = 32 * _odd(_log_int(rng, 2, 256))
    rows = _log_int(rng, 1, min(16384, 16384 * 4096 // cols))
    case = {"op": op, "rows": rows, "cols": cols, "post": rng.random() < 0.75,
            "gate": rng.choice(["none", "token", "channel"]), "p": rng.choice([0.0, 0.0, 0.1, 0.5]),
            "a": rng.choice([1.0, 0.9]), "c": rng.choice([1.0, 0.5])}
    if op == "join_fwd":
        case["mx"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------- inputs

def _generator(case, seed):
    # the case itself goes into the seed, so that two cases of one seed differ
    mix = zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode())
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + mix) % (1 << 62))
    return g


def _lens(case, seed):
    """Rows of each group: a multinomial draw, the last `empty` groups with none."""
    rng = np.random.default_rng([int(seed) % (1 << 31), case["rows"], case["groups"], case["n"]])
    p = 1.0 / np.arange(1, case["groups"] + 1) ** case["zipf"]
    if case["empty"]:
        p[-case["empty"]:] = 0
    return rng.multinomial(case["rows"], p / p.sum())


_EMAX, _QMAX = 8, 448.0


def _mx(v):
    """Blocks of 32 of the last axis -> (e4m3 values before rounding, saturated, exponents)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - _EMAX).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return torch.ldexp(b, -e).clamp(-_QMAX, _QMAX), e.squeeze(-1)


def prepare(case, seed):
    gen = _generator(case, seed)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op.startswith("linear"):
        m, n, g = case["rows"], case["n"], case["groups"]
        lens = _lens(case, seed)
        s["lens_host"] = [int(x) for x in lens]
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        width = n // 2 if case["act"] == "swiglu" else n
        if op == "linear_bwd":
            s["z"] = (1.5 * rnd(m, n)).bfloat16() if case["act"] != "none" else None
            s["dy"] = (rnd(m, width) * 0.01).bfloat16()
            s["scratch"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
        else:
            s["x"] = rnd(m, case["k"]).bfloat16()
            s["w"] = torch.randn((g, n, case["k"]), generator=gen, device=DEV, dtype=torch.bfloat16).mul_(0.02)
            s["bias"] = rnd(g, n).bfloat16() if case["bias"] else None
            out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["residual"] = rnd(m, width).to(out) if case["residual"] else None
        return s
    r, c = case["rows"], case["cols"]
    # activations with a few large channels, as residual streams have
    big = 1 + 20 * (torch.rand((c,), generator=gen, device=DEV) < 0.01)
    s["eps"] = 1e-6
    s["x"] = rnd(r, c).bfloat16()
    s["gamma_post"] = (1 + 0.2 * rnd(c)).bfloat16() if case["post"] else None
    s["gamma"] = (1 + 0.2 * rnd(c)).bfloat16()
    s["gate"] = {"none": None, "token": torch.sigmoid(rnd(r)), "channel": (0.5 + 0.2 * rnd(c)).bfloat16()}[case["gate"]]
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device=DEV) if case["p"] else None
    if op == "join_fwd":
        s["residual"] = (rnd(r, c) * big).bfloat16()
    else:
        s["h"] = (rnd(r, c) * big).bfloat16()
        s["dy"], s["dh"] = (rnd(r, c) * 0.01).bfloat16(), (rnd(r, c) * 0.01).bfloat16()
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + s["eps"])
        s["rstd_post"] = torch.rsqrt(s["x"].float().square().mean(-1) + s["eps"]) if case["post"] else None
        s["scratch"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------- the package's calls

def _own(s):
    import precision_grouped_gemm_gb300 as pgg
    c = s["case"]
    op = c["op"]
    if op.startswith("linear"):
        act = None if c["act"] == "none" else c["act"]
        form = {"act": act}
        if act in ("silu", "swiglu"):
            form["alpha"] = ALPHA
        if act == "swiglu":
            form.update(offset=OFFSET, limit=LIMIT)
        if op == "linear_bwd":
            dz, db = pgg.grouped_linear_bwd(s["dy"], s["z"], s["lens"], ws=s["scratch"], **form)
            return {"dz": dz, "db": db} if act else {"db": db}
        y, z = pgg.grouped_linear(s["x"], s["w"], s["lens"], bias=s["bias"], residual=s["residual"],
                                  save_z=c["save_z"], out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32,
                                  **form)
        return {"y": y, "z": z} if c["save_z"] else {"y": y}
    form = {"gamma_post": s["gamma_post"], "gamma": s["gamma"], "gate": s["gate"], "residual_scale": c["a"],
            "branch_scale": c["c"], "p": c["p"], "rng": s["rng"]}
    if op == "join_fwd":
        h, y, codes, scales, rstd_post, rstd = pgg.block_join(s["x"], s["residual"], eps=s["eps"],
                                                              fmt="e4m3" if c["mx"] else None, **form)
        out = {"h": h, "y": y, "rstd": rstd}
        if c["post"]:
            out["rstd_post"] = rstd_post
        if c["mx"]:
            out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
        return out
    dx, dr, dgp, dg, dgate = pgg.block_join_bwd(s["dy"], s["dh"], s["x"], s["h"], s["rstd_post"], s["rstd"],
                                                ws=s["scratch"], **form)
    return _drop_none({"dx": dx, "dresidual": dr, "dgamma_post": dgp, "dgamma": dg, "dgate": dgate})


def _drop_none(d):
    return {k: v for k, v in d.items() if v is not None}


# ---------------------------------------------------------------------------- the plain forms

def _halves(z):
    g, u = z.chunk(2, -1)
    return g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-ALPHA * z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "swiglu":
        g, u = _halves(z)
        return g / (1 + torch.exp(-ALPHA * g)) * (u + OFFSET)
    return z


def _act_bwd(dy, z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-ALPHA * z))
        return dy * p * (1 + ALPHA * z * (1 - p))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return dy * (cdf + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        gc, uc = _halves(z)
        p = 1 / (1 + torch.exp(-ALPHA * gc))
        dg = torch.where(g > LIMIT, 0.0, dy * (uc + OFFSET) * p * (1 + ALPHA * gc * (1 - p)))
        return torch.cat((dg, torch.where(u.abs() > LIMIT, 0.0, dy * gc * p)), -1)
    return dy


def _linear(s):
    c = s["case"]
    ys, zs, a = [], [], 0
    for e, n in enumerate(s["lens_host"]):
        if n:
            z = s["x"][a:a + n].float() @ s["w"][e].float().T
            if s["bias"] is not None:
                z += s["bias"][e].float()
            y = _act(z, c["act"])
            if s["residual"] is not None:
                y = y + s["residual"][a:a + n].float()
            ys.append(y.to(torch.bfloat16 if c["out"] == "bf16" else torch.float32))
            if c["save_z"]:
                zs.append(z.bfloat16())
            a += n
    return {"y": torch.cat(ys), "z": torch.cat(zs)} if c["save_z"] else {"y": torch.cat(ys)}


def _linear_bwd(s):
    act = s["case"]["act"]
    dzs, a = [], 0
    db = torch.zeros((s["case"]["groups"], s["case"]["n"]), device=DEV)
    for e, n in enumerate(s["lens_host"]):
        if n:
            dz = _act_bwd(s["dy"][a:a + n].float(), None if act == "none" else s["z"][a:a + n].float(), act)
            db[e] = dz.sum(0)
            dzs.append(dz.bfloat16())
            a += n
    return {"db": db} if act == "none" else {"dz": torch.cat(dzs), "db": db}


_LOW = 0xFFFFFFFF


def _mulhilo(a, m):
    """High and low words of the product of 32-bit words a (in int64) with the constant m."""
    lo, hi = a * (m & 0xFFFF), a * (m >> 16)  # 48 bits each
    mid = (lo >> 16) + hi
    return mid >> 16, ((mid << 16) | (lo & 0xFFFF)) & _LOW


def _keep(s, shape):
    """The truth values of dropout's mask."""
    n = shape[0] * shape[1]
    i = torch.arange((n + 3) // 4, device=DEV)
    seed, offset = s["rng"][0], s["rng"][1]
    x = [i & _LOW, i >> 32, (offset & _LOW).expand_as(i), ((offset >> 32) & _LOW).expand_as(i)]
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        h0, l0 = _mulhilo(x[0], 0xD2511F53)
        h1, l1 = _mulhilo(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return (torch.stack(x, 1).flatten()[:n] >= int(s["case"]["p"] * 2 ** 32)).view(shape)


def _branch(s, v, rstd):
    """gate-less branch b from x in 32 bits, and dropout's factors (None without dropout)."""
    t = v if rstd is None else v * rstd[:, None] * s["gamma_post"].float()
    if not s["case"]["p"]:
        return t, None
    f = _keep(s, v.shape).float() / (1 - s["case"]["p"])
    return t * f, f


def _gate(s):
    c, g = s["case"], s["gate"]
    if c["gate"] == "none":
        return c["c"]
    return c["c"] * (g[:, None] if c["gate"] == "token" else g.float())


def _join_fwd(s):
    c = s["case"]
    x = s["x"].float()
    rstd_post = torch.rsqrt(x.square().mean(-1) + s["eps"]) if c["post"] else None
    b, _ = _branch(s, x, rstd_post)
    v = c["a"] * s["residual"].float() + _gate(s) * b
    rstd = torch.rsqrt(v.square().mean(-1) + s["eps"])
    y = v * rstd[:, None] * s["gamma"].float()
    out = {"h": v.bfloat16(), "y": y.bfloat16(), "rstd": rstd}
    if c["post"]:
        out["rstd_post"] = rstd_post
    if c["mx"]:
        q, e = _mx(y)
        out["codes"] = q.reshape(y.shape).to(torch.float8_e4m3fn)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm_bwd(w, xh, rstd):
    return rstd[:, None] * (w - xh * (w * xh).mean(-1, keepdim=True))


def _join_bwd(s):
    c = s["case"]
    dy, x = s["dy"].float(), s["x"].float()
    hh = s["h"].float() * s["rstd"][:, None]
    d = s["dh"].float() + _norm_bwd(dy * s["gamma"].float(), hh, s["rstd"])
    b, f = _branch(s, x, s["rstd_post"])
    out = {"dgamma": (dy * hh).sum(0), "dresidual": (c["a"] * d).bfloat16()}
    if c["gate"] != "none":
        out["dgate"] = c["c"] * (d * b).sum(1 if c["gate"] == "token" else 0)
    dt = d * _gate(s) if f is None else d * _gate(s) * f
    if c["post"]:
        xh = x * s["rstd_post"][:, None]
        out["dgamma_post"] = (dt * xh).sum(0)
        dt = _norm_bwd(dt * s["gamma_post"].float(), xh, s["rstd_post"])
    out["dx"] = dt.bfloat16()
    return out


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "linear_bwd": _linear_bwd, "join_fwd": _join_fwd,
            "join_bwd": _join_bwd}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("linear"):
        m, n, g = case["rows"], case["n"], case["groups"]
        gated = case["act"] == "swiglu"
        width = n // 2 if gated else n
        if op == "linear_bwd":
            if case["act"] == "none":
                return {"bytes": 2 * m * n + 4 * g * n, "flops": m * n}
            return {"bytes": 2 * m * (width + 2 * n) + 4 * g * n, "flops": 12 * m * n}
        # weights of the groups that have rows, over a few draws
        live = float(np.mean([(_lens(case, q) > 0).sum() for q in range(8)]))
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * m * case["k"] + 2 * live * n * (case["k"] + case["bias"])
                + m * width * size * (1 + case["residual"]) + 2 * m * n * case["save_z"],
                "flops": 2 * m * n * case["k"]}
    r, c = case["rows"], case["cols"]
    gate = {"none": 0, "token": 4 * r, "channel": 2 * c}[case["gate"]]
    if op == "join_fwd":  # x, residual; h, y, codes, scales, statistics
        return {"bytes": r * c * (8 + case["mx"] * (1 + 1 / 32)) + gate + 2 * c * (1 + case["post"])
                + 4 * r * (1 + case["post"]), "flops": 16 * r * c}
    # dy, dh, h, x; dx, dresidual; the sums
    return {"bytes": r * c * 12 + gate * (2 if case["gate"] == "token" else 3) + 6 * c * (1 + case["post"])
            + 4 * r * (1 + case["post"]), "flops": 24 * r * c}


# ---------------------------------------------------------------------------- from the definitions, in 64 bits

def _sigmoid64(v):
    return torch.sigmoid(v)


def _phi64(v):
    return torch.special.ndtr(v)


def _exact_linear(s):
    c = s["case"]
    ends = np.concatenate([[0], np.cumsum(s["lens_host"])])
    width = c["n"] // 2 if c["act"] == "swiglu" else c["n"]
    out = torch.empty((c["rows"], width), dtype=torch.float64, device=DEV)
    pre = torch.empty((c["rows"], c["n"]), dtype=torch.float64, device=DEV) if c["save_z"] else None
    for e in range(c["groups"]):
        rows = slice(int(ends[e]), int(ends[e + 1]))
        if rows.start == rows.stop:
            continue
        z = torch.einsum("mk,nk->mn", s["x"][rows].double(), s["w"][e].double())
        if c["bias"]:
            z = z + s["bias"][e].double()
        if c["save_z"]:
            pre[rows] = z
        if c["act"] == "silu":
            z = z * _sigmoid64(ALPHA * z)
        elif c["act"] == "gelu":
            z = z * _phi64(z)
        elif c["act"] == "swiglu":
            g = torch.minimum(z[:, :width], torch.full_like(z[:, :width], LIMIT))
            z = g * _sigmoid64(ALPHA * g) * (OFFSET + torch.clamp(z[:, width:], -LIMIT, LIMIT))
        out[rows] = z + s["residual"][rows].double() if c["residual"] else z
    return {"y": out, "z": pre} if c["save_z"] else {"y": out}


def _exact_linear_bwd(s):
    c = s["case"]
    ends = np.concatenate([[0], np.cumsum(s["lens_host"])])
    db = torch.zeros((c["groups"], c["n"]), dtype=torch.float64, device=DEV)
    full = None if c["act"] == "none" else torch.empty(s["z"].shape, dtype=torch.float64, device=DEV)
    half = c["n"] // 2
    for e in range(c["groups"]):
        rows = slice(int(ends[e]), int(ends[e + 1]))
        d = s["dy"][rows].double()
        if c["act"] != "none":
            z = s["z"][rows].double()
            if c["act"] == "silu":
                q = _sigmoid64(ALPHA * z)
                d = d * (q + ALPHA * z * q * _sigmoid64(-ALPHA * z))
            elif c["act"] == "gelu":
                d = d * (_phi64(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            else:
                g, u = torch.clamp(z[:, :half], max=LIMIT), torch.clamp(z[:, half:], -LIMIT, LIMIT)
                q = _sigmoid64(ALPHA * g)
                dg = d * (u + OFFSET) * (q + ALPHA * g * q * _sigmoid64(-ALPHA * g)) * (z[:, :half] <= LIMIT)
                du = d * g * q * (z[:, half:].abs() <= LIMIT)
                d = torch.hstack((dg, du))
            full[rows] = d
        db[e] = d.sum(0)
    return {"db": db} if c["act"] == "none" else {"dz": full, "db": db}


def _philox64(n, seed, offset):
    """Words of the generator for the first n elements, in numpy's unsigned 64-bit integers."""
    u = np.uint64
    words = np.empty(((n + 3) // 4, 4), dtype=np.uint32)
    step = 1 << 20
    for b in range(0, words.shape[0], step):
        block = np.arange(b, min(b + step, words.shape[0]), dtype=u)
        r = [block & u(_LOW), block >> u(32), np.full_like(block, offset & _LOW),
             np.full_like(block, (offset >> 32) & _LOW)]
        key = [seed & _LOW, (seed >> 32) & _LOW]
        for _ in range(10):
            p0, p1 = r[0] * u(0xD2511F53), r[2] * u(0xCD9E8D57)  # the factors are below 2^32: nothing wraps
            r = [(p1 >> u(32)) ^ r[1] ^ u(key[0]), p1 & u(_LOW), (p0 >> u(32)) ^ r[3] ^ u(key[1]), p0 & u(_LOW)]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        for j in range(4):
            words[b:b + step, j] = r[j]
    return words.reshape(-1)[:n]


def _mask64(s, shape):
    p = s["case"]["p"]
    if not p:
        return torch.ones(shape, dtype=torch.float64, device=DEV)
    seed, offset = (int(v) for v in s["rng"].tolist())
    kept = _philox64(shape[0] * shape[1], seed, offset) >= np.uint32(math.floor(p * 2 ** 32))
    return torch.from_numpy(kept.reshape(shape)).to(DEV).double() / (1 - p)


def _mx64(v):
    """Blocks of 32 in 64 bits -> (e4m3 values on the grid, powers of two)."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    # log2 may land on the wrong side of a whole number: put it right by comparison
    power = power - (torch.exp2(power) > amax).double() * (amax > 0) + (torch.exp2(power + 1) <= amax).double()
    power = torch.where(amax > 0, power - 8, torch.full_like(power, -127.0)).clamp(-127, 127)
    z = b / torch.exp2(power)
    a = z.abs().clamp(max=448.0)
    binade = torch.floor(torch.log2(a.clamp(min=2.0 ** -11))).clamp(min=-6)
    binade = binade - (torch.exp2(binade) > a).double() * (binade > -6) + (torch.exp2(binade + 1) <= a).double()
    step = torch.exp2(binade - 3)
    return (torch.sign(z) * torch.round(a / step) * step).reshape(v.shape), torch.exp2(power).squeeze(-1)


def _exact_join(s):
    c = s["case"]
    x = s["x"].double()
    rows, cols = x.shape
    fwd = c["op"] == "join_fwd"
    if c["post"]:
        r1 = 1 / torch.sqrt((x * x).mean(1) + s["eps"]) if fwd else s["rstd_post"].double()
        n1 = torch.einsum("rc,r->rc", x, r1)
        t = n1 * s["gamma_post"].double()
    else:
        t = x
    mask = _mask64(s, (rows, cols))
    gate = {"none": lambda: torch.ones((), dtype=torch.float64, device=DEV), "token": lambda: s["gate"].double()[:, None],
            "channel": lambda: s["gate"].double()[None, :]}[c["gate"]]()
    if fwd:
        h = c["a"] * s["residual"].double() + c["c"] * gate * mask * t
        r2 = 1 / torch.sqrt((h * h).mean(1) + s["eps"])
        y = torch.einsum("rc,r,c->rc", h, r2, s["gamma"].double())
        out = {"h": h, "y": y, "rstd": r2}
        if c["post"]:
            out["rstd_post"] = r1
        if c["mx"]:
            out["codes"], out["scales"] = _mx64(y)
        return out
    dy, r2 = s["dy"].double(), s["rstd"].double()
    n2 = torch.einsum("rc,r->rc", s["h"].double(), r2)
    u = dy * s["gamma"].double()
    d = s["dh"].double() + (u - n2 * (torch.einsum("rc,rc->r", u, n2) / cols)[:, None]) * r2[:, None]
    out = {"dgamma": torch.einsum("rc,rc->c", dy, n2), "dresidual": c["a"] * d}
    db = c["c"] * d
    if c["gate"] == "token":
        out["dgate"] = torch.einsum("rc,rc,rc->r", db, mask, t)
    elif c["gate"] == "channel":
        out["dgate"] = torch.einsum("rc,rc,rc->c", db, mask, t)
    dt = db * gate * mask
    if c["post"]:
        out["dgamma_post"] = torch.einsum("rc,rc->c", dt, n1)
        w = dt * s["gamma_post"].double()
        dt = (w - n1 * (torch.einsum("rc,rc->r", w, n1) / cols)[:, None]) * r1[:, None]
    out["dx"] = dt
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s)
    return _exact_linear_bwd(s) if case["op"] == "linear_bwd" else _exact_join(s)
