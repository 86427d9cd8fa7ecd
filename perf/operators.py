"""The operators of a transformer's feed-forward sub-block, as cases to time and check.

Three operators, used together in one sub-block of a training step (and, the first
two, for one token at a time when serving):

* the gated linear layer  H = act(X Wg^T + bg) * (X Wu^T + bu), with W = [Wg; Wu]
  stored 2F x K, and its backward pass (dP, dX, dW and the bias gradient);
* the norms before and after a block: XO = X + scale * gate * Norm_post(Z) and
  Y = Norm_pre(XO) in one pass over the rows, and their backward pass;
* the global norm of many gradient tensors, and their clipping.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true:
the framework's kernels.  Sizes are those of the repository's transformer layer
(8192 tokens, 4096 -> 14336), its ragged problem (1000 x 1023 x 777) and its decode
problem (64 tokens), and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
# cost of the largest listed case of each kind: draws stay below
MOST_MKF = 8192 * 4096 * 14336
MOST_MN = 8192 * 4096
MOST_GRAD = 120_000_000


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a served request through the gated layer: latency
        _glu("glu_token", 1, 1024, 4096, "bf16", "silu"),
        # a decode batch of 64 tokens: the weights' 235 MB stream through once
        _glu("glu_decode", 64, 4096, 14336, "fp16", "gelu"),
        # a ragged batch, nothing a multiple of anything, with a bias, as in training
        _glu("glu_ragged", 1000, 777, 1023, "bf16", "gelu", bias=True, save=True),
        # the prompt / training forward of the transformer layer
        _glu("glu_layer", 8192, 4096, 14336, "bf16", "silu", save=True),
        # its backward pass
        _glu("glu_layer_backward", 8192, 4096, 14336, "bf16", "silu", back=True),
        # the ragged batch's backward pass, with the bias gradient
        _glu("glu_ragged_backward", 1000, 777, 1023, "fp16", "gelu", bias=True, back=True),
        # the norms between two blocks for a decode batch of 64 tokens: latency
        _norm("norm_decode", 64, 4096, "bf16", "bf16", post="rms", pre="rms", gate="none"),
        # the same in training: residual stream in bf16, a gate per channel
        _norm("norm_layer", 8192, 4096, "bf16", "bf16", post="rms", pre="rms", gate="channel"),
        # its backward pass
        _norm("norm_layer_backward", 8192, 4096, "bf16", "bf16", post="rms", pre="rms", gate="channel",
              back=True),
        # LayerNorm with a 32-bit stream, an odd width and a gate per sequence, backward
        _norm("norm_odd_backward", 2000, 1023, "fp32", "bf16", post="layer", pre="layer",
              gate="sequence", back=True),
        # the gradients of one layer's feed-forward block in bf16
        _clip("clip_layer", 7, MOST_GRAD, "bf16", 1.0),
        # many small odd tensors in fp32 with a loss scale, as of a small model: latency
        _clip("clip_many", 60, 900_000, "fp32", 1.0 / 1024),
    ]


def _glu(name, m, k, f, dtype, act, bias=False, save=False, back=False):
    return {"name": name, "op": "glu_backward" if back else "glu", "m": m, "k": k, "f": f,
            "dtype": dtype, "act": act, "bias": bias, "save": save}


def _norm(name, m, n, x, z, post, pre, gate, back=False):
    return {"name": name, "op": "norm_backward" if back else "norm", "m": m, "n": n, "x": x, "z": z,
            "post": post, "pre": pre, "gate": gate}


def _clip(name, tensors, total, dtype, inv_scale):
    return {"name": name, "op": "clip", "tensors": tensors, "total": total, "dtype": dtype,
            "inv_scale": inv_scale}


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; half of them odd sizes, half multiples of 64."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = int(v) if v < 64 or rng.random() < 0.5 else int(v / 64) * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_backward", "norm", "norm_backward", "clip"])
    if op in ("glu", "glu_backward"):
        m, k, f = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 64, 16384)
        while m * k * f > MOST_MKF:
            m = max(1, m // 2)
        c = _glu("", m, k, f, rng.choice(["bf16", "fp16"]), rng.choice(["silu", "gelu", "relu", "none"]),
                 bias=rng.random() < 0.4, save=rng.random() < 0.5, back=op == "glu_backward")
    elif op in ("norm", "norm_backward"):
        n, m = _spread(rng, 32, 16384), _spread(rng, 1, 32768)
        while m * n > MOST_MN:
            m = max(1, m // 2)
        x, z = rng.choice([("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("fp32", "fp32")])
        c = _norm("", m, n, x, z, rng.choice(["rms", "layer", "none"]), rng.choice(["rms", "layer"]),
                  rng.choice(["none", "channel", "sequence", "token"]), back=op == "norm_backward")
    else:
        t = _spread(rng, 1, 60)
        c = _clip("", t, max(t, _spread(rng, 1000, MOST_GRAD)), rng.choice(["bf16", "fp16", "fp32"]),
                  rng.choice([1.0, 0.5, 1.0 / 1024]))
    del c["name"]
    return c


# ----------------------------------------------------------------------- inputs

def _gate_rows(c):
    """Rows that share one row of the gate: all of them, one sequence's (a quarter of them), or one."""
    return {"channel": c["m"], "sequence": max(1, (c["m"] + 3) // 4), "token": 1, "none": 1}[c["gate"]]


def _sizes(c):
    """The tensors' sizes of a clipping case: a few large, many small, every one at least 1."""
    t, total = c["tensors"], c["total"]
    w = [1.0 / (1 + (i * 7) % 13) ** 2 for i in range(t)]
    s = sum(w)
    sizes = [max(1, int(total * v / s)) for v in w]
    return [v - 1 if v > 64 and i % 3 == 1 else v for i, v in enumerate(sizes)]


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, scale=1.0, mean=0.0, dtype="fp32"):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(mean).to(DTYPES[dtype])

    s = {"case": c}
    if c["op"] in ("glu", "glu_backward"):
        m, k, f, dt = c["m"], c["k"], c["f"], c["dtype"]
        # activations of unit size and the usual initialisation of the weights
        s["X"] = randn(m, k, dtype=dt)
        s["W"] = randn(2 * f, k, scale=k ** -0.5, dtype=dt)
        s["bias"] = randn(2 * f, scale=0.1) if c["bias"] else None
        if c["op"] == "glu_backward":
            s["P"] = randn(m, 2 * f, dtype=dt)          # what the forward pass saved
            s["dH"] = randn(m, f, scale=0.05, dtype=dt)
    elif c["op"] in ("norm", "norm_backward"):
        m, n, groups = c["m"], c["n"], -(-c["m"] // _gate_rows(c))
        # a residual stream that is larger than a block's output, with channels of unlike size
        size = randn(1, n).abs_().add_(0.5)
        s["X"] = (randn(m, n) * size * 3.0 + 0.2).to(DTYPES[c["x"]])
        s["Z"] = randn(m, n, scale=0.7, mean=0.1, dtype=c["z"])
        s["gate"] = None if c["gate"] == "none" else randn(groups, n, scale=0.3, mean=0.5)
        s["wpost"] = randn(n, scale=0.1, mean=1.0) if c["post"] != "none" else None
        s["bpost"] = randn(n, scale=0.1) if c["post"] == "layer" else None
        s["wpre"] = randn(n, scale=0.1, mean=1.0)
        s["bpre"] = randn(n, scale=0.1) if c["pre"] == "layer" else None
        if c["op"] == "norm_backward":
            s["dY"] = randn(m, n, scale=0.05, dtype=c["z"])
            s["dXO"] = randn(m, n, scale=0.05, dtype=c["x"])
    else:
        sizes = _sizes(c)
        flat = randn(sum(sizes), scale=2e-3 / c["inv_scale"])
        s["grads"] = [t.to(DTYPES[c["dtype"]], copy=True) for t in flat.split(sizes)]
        s["outs"] = [torch.empty_like(t) for t in s["grads"]]   # the optimizer's own buffers
    return s


# -------------------------------------------------------------------- plain form

def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if name == "gelu":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "relu":
        return torch.where(g > 0, g, 0.0 * g), (g > 0).to(g.dtype)
    return g, torch.ones_like(g)


def _plain_glu(s):
    c, f = s["case"], s["case"]["f"]
    dt = DTYPES[c["dtype"]]
    p = s["X"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        p = p + s["bias"]
    h = _act(c["act"], p[:, :f])[0] * p[:, f:]
    return {"H": h.to(dt), "P": p.to(dt)} if c["save"] else {"H": h.to(dt)}


def _plain_glu_backward(s):
    c, f = s["case"], s["case"]["f"]
    dt = DTYPES[c["dtype"]]
    p, dh = s["P"].float(), s["dH"].float()
    a, da = _act(c["act"], p[:, :f])
    dp = torch.cat([dh * p[:, f:] * da, dh * a], dim=1)
    out = {"dP": dp.to(dt), "dX": (dp @ s["W"].float()).to(dt), "dW": (dp.t() @ s["X"].float()).to(dt)}
    if c["bias"]:
        out["dbias"] = dp.sum(dim=0)
    return out


def _norm_of(kind, x):
    """(normalised x, 1 / its size) along the rows; x itself where there is no norm."""
    if kind == "none":
        return x, None
    d = x - x.mean(dim=1, keepdim=True) if kind == "layer" else x
    r = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    return d * r, r


def _norm_back(kind, xhat, r, g):
    """Gradient with respect to the norm's input, from that with respect to xhat."""
    if kind == "none":
        return g
    d = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(dim=1, keepdim=True)
    return d * r


def _rows_gate(s):
    """The gate of each row (1 where there is none), with the residual scale."""
    c = s["case"]
    if s["gate"] is None:
        return torch.full((1, 1), 0.5, device="cuda")
    return 0.5 * s["gate"].repeat_interleave(_gate_rows(c), dim=0)[: c["m"]]


def _affine(x, w, b):
    x = x if w is None else x * w
    return x if b is None else x + b


def _plain_norm(s):
    c = s["case"]
    n = _affine(_norm_of(c["post"], s["Z"].float())[0], s["wpost"], s["bpost"])
    # the stream is held in its own type: the norm that follows sees what was stored
    xo = (s["X"].float() + _rows_gate(s) * n).to(DTYPES[c["x"]])
    y = _affine(_norm_of(c["pre"], xo.float())[0], s["wpre"], s["bpre"])
    return {"XO": xo, "Y": y.to(DTYPES[c["z"]])}


def _plain_norm_backward(s):
    c = s["case"]
    xt, zt = DTYPES[c["x"]], DTYPES[c["z"]]
    xhat, rx = _norm_of(c["pre"], s["X"].float())       # X holds the stream after the block
    zhat, rz = _norm_of(c["post"], s["Z"].float())
    dy, gate = s["dY"].float(), _rows_gate(s)
    dx = s["dXO"].float() + _norm_back(c["pre"], xhat, rx, dy * s["wpre"])
    dn = dx * gate
    dz = _norm_back(c["post"], zhat, rz, dn if s["wpost"] is None else dn * s["wpost"])
    out = {"dX": dx.to(xt), "dZ": dz.to(zt), "dwpre": (dy * xhat).sum(dim=0)}
    if s["bpre"] is not None:
        out["dbpre"] = dy.sum(dim=0)
    if s["wpost"] is not None:
        out["dwpost"] = (dn * zhat).sum(dim=0)
    if s["bpost"] is not None:
        out["dbpost"] = dn.sum(dim=0)
    if s["gate"] is not None:
        rows = _gate_rows(c)
        dg = 0.5 * dx * _affine(zhat, s["wpost"], s["bpost"])
        pad = s["gate"].shape[0] * rows - c["m"]
        dg = torch.cat([dg, dg.new_zeros(pad, c["n"])]) if pad else dg
        out["dgate"] = dg.view(s["gate"].shape[0], rows, c["n"]).sum(dim=1)
    return out


def _plain_clip(s):
    inv = s["case"]["inv_scale"]
    # squares and their long sum in 64 bits
    norm = torch.sqrt(torch.stack([(t.double() * t.double()).sum() for t in s["grads"]]).sum()) * inv
    coef = torch.where(norm > 1.0, 1.0 / norm, torch.ones_like(norm)).float() * inv
    return {"norm": norm.float().view(1), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


# --------------------------------------------------------------- the framework's

_kept = {}


def _gemm():
    """The library and the handle that a program keeps."""
    if not _kept:
        import mixed_precision_dense_sm_gb300 as lib
        _kept["lib"], _kept["g"] = lib, lib.Gemm()
    return _kept["lib"], _kept["g"]


def _kind(k):
    return None if k == "none" else k


def _own_glu(s):
    c = s["case"]
    _, g = _gemm()
    p = torch.empty(c["m"], 2 * c["f"], dtype=s["X"].dtype, device="cuda") if c["save"] else None
    h = g.glu(s["X"], s["W"], act=_kind(c["act"]), bias=s["bias"], P=p)
    return {"H": h, "P": p} if c["save"] else {"H": h}


def _own_glu_backward(s):
    c = s["case"]
    _, g = _gemm()
    out = {"dP": torch.empty_like(s["P"]), "dX": torch.empty_like(s["X"]), "dW": torch.empty_like(s["W"])}
    if c["bias"]:
        out["dbias"] = torch.empty_like(s["bias"])
    g.glu_backward(s["dH"], s["P"], s["X"], s["W"], act=_kind(c["act"]), **out)
    return out


def _own_norm(s):
    c = s["case"]
    lib, _ = _gemm()
    xo, y = lib.norm_block(s["X"], s["Z"], pre=c["pre"], pre_weight=s["wpre"], pre_bias=s["bpre"],
                           post=_kind(c["post"]), post_weight=s["wpost"], post_bias=s["bpost"],
                           gate=s["gate"], gate_rows=_gate_rows(c), scale=0.5, eps=EPS)
    return {"XO": xo, "Y": y}


def _own_norm_backward(s):
    c = s["case"]
    lib, _ = _gemm()
    out = {"dX": torch.empty_like(s["X"]), "dZ": torch.empty_like(s["Z"]), "dwpre": torch.empty_like(s["wpre"])}
    for name, of in (("dbpre", "bpre"), ("dwpost", "wpost"), ("dbpost", "bpost"), ("dgate", "gate")):
        if s[of] is not None:
            out[name] = torch.empty_like(s[of])
    lib.norm_block_backward(s["X"], s["dY"], s["dXO"], s["Z"], pre=c["pre"], pre_weight=s["wpre"],
                            post=_kind(c["post"]), post_weight=s["wpost"], post_bias=s["bpost"],
                            gate=s["gate"], gate_rows=_gate_rows(c), scale=0.5, eps=EPS,
                            dX=out["dX"], dZ=out["dZ"], dgate=out.get("dgate"),
                            dpre_weight=out["dwpre"], dpre_bias=out.get("dbpre"),
                            dpost_weight=out.get("dwpost"), dpost_bias=out.get("dbpost"))
    return out


def _own_clip(s):
    lib, _ = _gemm()
    norm = lib.grad_clip(s["grads"], 1.0, outputs=s["outs"], inv_scale=s["case"]["inv_scale"])
    return {"norm": norm, "grads": s["outs"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"glu": _own_glu, "glu_backward": _own_glu_backward, "norm": _own_norm,
                "norm_backward": _own_norm_backward, "clip": _own_clip}[op](state)
    return {"glu": _plain_glu, "glu_backward": _plain_glu_backward, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward, "clip": _plain_clip}[op](state)


# ------------------------------------------------------------------------- work

def work(case):
    c = case
    e = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "glu":
        m, k, f, b = c["m"], c["k"], c["f"], e[c["dtype"]]
        by = (m * k + 2 * f * k + m * f + (2 * m * f if c["save"] else 0)) * b + (8 * f if c["bias"] else 0)
        return {"bytes": by, "flops": 4 * m * k * f}
    if c["op"] == "glu_backward":
        m, k, f, b = c["m"], c["k"], c["f"], e[c["dtype"]]
        # dH, P, X, W in; dP, dX, dW out
        by = (m * f + 2 * m * f + m * k + 2 * f * k + 2 * m * f + m * k + 2 * f * k) * b
        return {"bytes": by + (8 * f if c["bias"] else 0), "flops": 8 * m * k * f}
    if c["op"] in ("norm", "norm_backward"):
        m, n, x, z = c["m"], c["n"], e[c["x"]], e[c["z"]]
        gate = 0 if c["gate"] == "none" else 4 * n * -(-m // _gate_rows(c))
        vec = 4 * n * (1 + (c["post"] != "none") + (c["post"] == "layer") + (c["pre"] == "layer"))
        if c["op"] == "norm":
            return {"bytes": m * n * (2 * x + 2 * z) + gate + vec, "flops": 16 * m * n}
        return {"bytes": m * n * (3 * x + 3 * z) + 2 * gate + 2 * vec, "flops": 40 * m * n}
    n = sum(_sizes(c))
    return {"bytes": 2 * n * e[c["dtype"]] + 4, "flops": 3 * n}


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if c["op"] in ("glu", "glu_backward"):
        return _exact_glu(c, s)
    if c["op"] in ("norm", "norm_backward"):
        return _exact_norm(c, s)
    inv, g = c["inv_scale"], [t.double() * c["inv_scale"] for t in s["grads"]]
    norm = math.sqrt(math.fsum(float(t.square().sum()) for t in g))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t / max(norm, 1.0) for t in g]}


def _exact_phi(x):
    """The activations' factor act(x) / x and its derivative, in 64 bits."""
    cdf = torch.special.ndtr(x)
    return cdf, torch.exp(-x.square() / 2) * (2 * math.pi) ** -0.5


def _exact_glu(c, s):
    f, w, x = c["f"], s["W"], s["X"]
    if c["op"] == "glu":
        gate, up = torch.einsum("mk,fk->mf", x, w[:f]), torch.einsum("mk,fk->mf", x, w[f:])
        if s["bias"] is not None:
            gate, up = gate + s["bias"][:f], up + s["bias"][f:]
    else:
        gate, up = s["P"][:, :f], s["P"][:, f:]
    if c["act"] == "silu":
        sg = torch.sigmoid(gate)
        a, da = gate * sg, sg + gate * sg * torch.sigmoid(-gate)
    elif c["act"] == "gelu":
        cdf, pdf = _exact_phi(gate)
        a, da = gate * cdf, cdf + gate * pdf
    elif c["act"] == "relu":
        a, da = gate.clamp(min=0), gate.gt(0).double()
    else:
        a, da = gate, torch.ones_like(gate)
    if c["op"] == "glu":
        out = {"H": a * up}
        return {**out, "P": torch.cat([gate, up], 1)} if c["save"] else out
    dg, du = s["dH"] * up * da, s["dH"] * a
    del a, da
    out = {"dP": torch.cat([dg, du], 1),
           "dX": torch.mm(dg, w[:f]).addmm_(du, w[f:]),
           "dW": torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)], 0)}
    if c["bias"]:
        out["dbias"] = torch.cat([dg.sum(0), du.sum(0)])
    return out


def _exact_stats(kind, v):
    """(mean, reciprocal size) of each row."""
    if kind == "none":
        return torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
    if kind == "layer":
        var, mean = torch.var_mean(v, dim=1, correction=0, keepdim=True)
        return mean, (var + EPS).rsqrt()
    return torch.zeros_like(v[:, :1]), (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).rsqrt()


def _exact_jacobian(kind, hat, r, g):
    """g times the Jacobian of the norm: r (I - 1 1^T / n - hat hat^T / n), without the parts the kind lacks."""
    n = hat.shape[1]
    if kind == "none":
        return g
    out = g - torch.einsum("mn,mn->m", g, hat)[:, None] * hat / n
    if kind == "layer":
        out -= g.sum(1, keepdim=True) / n
    return r * out


def _exact_norm(c, s):
    m, n, rows = c["m"], c["n"], _gate_rows(c)
    row = torch.arange(m, device="cuda") // rows
    gate = torch.full((m, n), 0.5, dtype=torch.float64, device="cuda")
    if s["gate"] is not None:
        gate *= s["gate"][row]
    mz, rz = _exact_stats(c["post"], s["Z"])
    zhat = (s["Z"] - mz) * rz
    wpost = s["wpost"] if s["wpost"] is not None else torch.ones(n, dtype=torch.float64, device="cuda")
    bpost = s["bpost"] if s["bpost"] is not None else 0.0
    branch = zhat * wpost + bpost
    if c["op"] == "norm":
        xo = s["X"] + gate * branch
        held = xo.to(DTYPES[c["x"]]).double()
        mx, rx = _exact_stats(c["pre"], held)
        y = (held - mx) * rx * s["wpre"]
        return {"XO": xo, "Y": y if s["bpre"] is None else y + s["bpre"]}
    mx, rx = _exact_stats(c["pre"], s["X"])
    xhat = (s["X"] - mx) * rx
    dx = s["dXO"] + _exact_jacobian(c["pre"], xhat, rx, s["dY"] * s["wpre"])
    dn = gate * dx
    out = {"dX": dx, "dZ": _exact_jacobian(c["post"], zhat, rz, dn * wpost),
           "dwpre": torch.einsum("mn,mn->n", s["dY"], xhat)}
    if s["bpre"] is not None:
        out["dbpre"] = s["dY"].sum(0)
    if s["wpost"] is not None:
        out["dwpost"] = torch.einsum("mn,mn->n", dn, zhat)
    if s["bpost"] is not None:
        out["dbpost"] = dn.sum(0)
    if s["gate"] is not None:
        out["dgate"] = torch.zeros_like(s["gate"]).index_add_(0, row, 0.5 * dx * branch)
    return out
