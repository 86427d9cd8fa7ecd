"""The rows of a feed-forward block with experts, and the update of its weights, as cases to time and check.

Two sets of operators, used in one training step (and, the first set's forward half, for a
few tokens at a time when serving):

* tokens sorted by expert and back: the sort of the T x k chosen experts (``sort``), the
  rows into expert order (``gather``) and back with the router's weights applied
  (``combine``), and the backward passes of the last two;
* ``ortho``: the Newton-Schulz orthogonalisation of a weight matrix's update, of one matrix
  or of a batch of them (the experts').

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true:
the framework's kernels.  Sizes are those of the repository's transformer layer
(8192 tokens, 4096 -> 14336), its ragged problem (1000 x 1023 x 777) and its decode
problem (64 tokens), and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "i32": torch.int32, "i64": torch.int64}
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
# cost of the largest listed case of each kind: draws stay below
MOST_SLOTS = 65536 * 7
MOST_ROWS = 8192 * 9 * 4096
MOST_ORTHO = 4096 * 4096 * 14336
MOST_MATRIX = 4096 * 14336


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # the choices of one token of a served request: latency
        _sort("sort_token", 1, 8, 64, "i64"),
        # those of a prompt or of a training batch of the transformer layer
        _sort("sort_layer", 8192, 8, 128, "i64"),
        # a large padded batch over an odd number of experts; three in ten tokens are padding
        _sort("sort_masked", 65536, 7, 999, "i32", drop=0.3),
        # a decode batch of 64 tokens goes to its experts
        _rows("gather_decode", "gather", 64, 8, 4096, "bf16"),
        # the layer's tokens go to their experts
        _rows("gather_layer", "gather", 8192, 8, 4096, "bf16"),
        # a ragged batch's gradient comes back from them, the weights applied on the way out
        _rows("gather_ragged_backward", "gather_backward", 1000, 3, 1023, "fp16", weight="fp32", drop=0.2),
        # one token comes back
        _rows("combine_token", "combine", 1, 8, 4096, "bf16", weight="fp32"),
        # the layer's tokens come back
        _rows("combine_layer", "combine", 8192, 8, 4096, "bf16", weight="fp32"),
        # its backward pass: the experts' rows and the weights' gradient
        _rows("combine_layer_backward", "combine_backward", 8192, 8, 4096, "bf16", weight="fp32"),
        # the update of one small matrix: latency
        _ortho("ortho_small", 1, 256, 1024, "bf16"),
        # those of sixteen experts' odd, tall matrices, from 32-bit momentum
        _ortho("ortho_experts", 16, 1023, 777, "fp32"),
        # that of the layer's largest matrix
        _ortho("ortho_layer", 1, 4096, 14336, "bf16"),
    ]


def _sort(name, t, k, e, ids, drop=0.0):
    return {"name": name, "op": "sort", "t": t, "k": k, "e": e, "ids": ids, "drop": drop}


def _rows(name, op, t, k, d, dtype, weight="none", drop=0.0):
    return {"name": name, "op": op, "t": t, "k": k, "e": 64, "d": d, "dtype": dtype, "weight": weight,
            "drop": drop}


def _ortho(name, batch, rows, cols, dtype):
    return {"name": name, "op": "ortho", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; half of them odd sizes, half multiples of 64."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    v = int(v) if v < 64 or rng.random() < 0.5 else int(v / 64) * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["sort", "gather", "gather_backward", "combine", "combine_backward", "ortho", "ortho"])
    drop = rng.choice([0.0, 0.0, 0.1, 0.6])
    if op == "sort":
        e = _spread(rng, 1, 1024)
        k = min(e, rng.randint(1, 8))
        t = min(_spread(rng, 1, 65536), MOST_SLOTS // k)
        c = _sort("", t, k, e, rng.choice(["i32", "i64"]), drop)
    elif op == "ortho":
        rows, cols, batch = _spread(rng, 16, 14336), _spread(rng, 16, 14336), _spread(rng, 1, 32)
        while batch > 1 and (batch * rows * cols * min(rows, cols) > MOST_ORTHO or batch * rows * cols > MOST_MATRIX):
            batch //= 2
        while rows * cols * min(rows, cols) > MOST_ORTHO or rows * cols > MOST_MATRIX:
            rows, cols = (rows * 3 // 4, cols) if rows > cols else (rows, cols * 3 // 4)
        c = _ortho("", batch, rows, cols, rng.choice(["bf16", "fp16", "fp32"]))
    else:
        d, t, k = _spread(rng, 16, 16384), _spread(rng, 1, 65536), rng.randint(1, 8)
        dt = rng.choice(["bf16", "fp16", "fp32"])
        while t * (k + 1) * d * (2 if dt == "fp32" else 1) > MOST_ROWS:
            t = max(1, t // 2)
        c = _rows("", op, t, k, d, dt, rng.choice(["none", "fp32", dt]), drop)
    del c["name"]
    return c


# ----------------------------------------------------------------------- inputs

def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype="fp32"):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).to(DTYPES[dtype])

    s = {"case": c}
    if c["op"] == "ortho":
        b, r, n = c["batch"], c["rows"], c["cols"]
        # an update as training has it: a few strong directions over noise
        low = max(1, min(r, n) // 32)
        g = torch.baddbmm(randn(b, r, n), randn(b, r, low), randn(b, low, n), alpha=low ** -0.5)
        s["G"] = g.mul_(1e-3).to(DTYPES[c["dtype"]])
        return s
    t, k, e = c["t"], c["k"], c["e"]
    # logits with favoured experts; the choices of a token differ, and padding tokens have none
    logits = randn(t, e).add_(randn(1, e, scale=0.7))
    top, ids = logits.topk(k, dim=1)
    del logits
    padding = torch.rand(t, generator=gen, device="cuda") < c["drop"]
    ids = torch.where(padding[:, None], -1, ids)
    if c["op"] == "sort":
        s["ids"] = ids.to(DTYPES[c["ids"]])
        return s
    s["pos"], offsets, _ = _plain_sort(ids, e)
    if c["weight"] != "none":
        s["weight"] = torch.softmax(top, dim=1).to(DTYPES[c["weight"]])
    else:
        s["weight"] = None
    d, dt = c["d"], c["dtype"]
    if c["op"] in ("gather", "combine_backward"):
        s["X"] = randn(t, d, dtype=dt)               # X, or dY
        # the experts' rows, kept by the program; what lies behind the last expert's is not touched
        s["out"] = torch.zeros(t * k, d, dtype=DTYPES[dt], device="cuda")
    if c["op"] != "gather":
        s["Xs"] = randn(t * k, d, dtype=dt)          # dXs, or Ys
    if c["op"] == "gather_backward":
        s["X"] = randn(t, d, dtype=dt)
    return s


# -------------------------------------------------------------------- plain form

def _plain_sort(ids, e):
    """(pos, offsets, order): the row of each choice, the experts' first rows, the choice of each row."""
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < e), key, e)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(e + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:e].cumsum(0)])
    row = torch.arange(key.numel(), device=ids.device)
    pos = torch.empty_like(row).scatter_(0, order, row)
    pos = torch.where(key < e, pos, -1).view(ids.shape)
    order = torch.where(row < offsets[e], order, -1)
    return pos.int(), offsets.int(), order.int()


def _plain_out(s):
    """Rows of X, weighted, to their places among the experts' rows."""
    k = s["case"]["k"]
    pos, x = s["pos"].reshape(-1).long(), s["X"].float()
    x = x.repeat_interleave(k, dim=0)
    if s["weight"] is not None:
        x = x * s["weight"].float().reshape(-1, 1)
    on = pos >= 0
    return torch.zeros_like(s["out"]).index_copy_(0, pos[on], x[on].to(s["out"].dtype))


def _plain_in(s):
    """The weighted sum of each token's rows among the experts'."""
    c = s["case"]
    acc = torch.zeros(c["t"], c["d"], device="cuda")
    for j in range(c["k"]):
        p = s["pos"][:, j].long()
        row = s["Xs"][p.clamp(min=0)].float()
        if s["weight"] is not None:
            row = row * s["weight"][:, j : j + 1].float()
        acc += torch.where((p >= 0)[:, None], row, 0.0)
    return acc.to(s["Xs"].dtype)


def _plain_dots(s):
    """The weights' gradient: each token's row times each of its rows among the experts'."""
    x, dots = s["X"].float(), []
    for j in range(s["case"]["k"]):
        p = s["pos"][:, j].long()
        d = (x * s["Xs"][p.clamp(min=0)].float()).sum(dim=1)
        dots.append(torch.where(p >= 0, d, 0.0))
    return torch.stack(dots, dim=1).to(s["weight"].dtype)


def _plain_ortho(s):
    c = s["case"]
    a, b, q = COEFFICIENTS
    x = s["G"].float()
    if c["rows"] > c["cols"]:
        x = x.mT
    # the long sum of squares in 64 bits
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt().float()
    x = x / (norm + EPS)
    for _ in range(STEPS):
        g = x @ x.mT
        x = a * x + (b * g + q * (g @ g)) @ x
    if c["rows"] > c["cols"]:
        x = x.mT
    return x.to(torch.bfloat16).contiguous()


def _plain(s):
    op = s["case"]["op"]
    if op == "sort":
        pos, offsets, order = _plain_sort(s["ids"], s["case"]["e"])
        return {"pos": pos, "offsets": offsets, "order": order}
    if op == "ortho":
        return {"O": _plain_ortho(s)}
    out = {"rows": _plain_out(s)} if op in ("gather", "combine_backward") else {"tokens": _plain_in(s)}
    if op.endswith("backward") and s["weight"] is not None:
        out["dweight"] = _plain_dots(s)
    return out


# --------------------------------------------------------------- the framework's

_kept = {}


def _gemm():
    """The library and the handle that a program keeps."""
    if not _kept:
        import mixed_precision_dense_sm_gb300 as lib
        _kept["lib"], _kept["g"] = lib, lib.Gemm()
    return _kept["lib"], _kept["g"]


def _own(s):
    lib, g = _gemm()
    op, w = s["case"]["op"], s.get("weight")
    if op == "sort":
        pos, offsets, order = lib.expert_sort(s["ids"], s["case"]["e"])
        return {"pos": pos, "offsets": offsets, "order": order}
    if op == "ortho":
        return {"O": g.orthogonalize(s["G"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}
    if op == "gather":
        return {"rows": lib.expert_gather(s["X"], s["pos"], w, Xs=s["out"])}
    if op == "combine":
        return {"tokens": lib.expert_combine(s["Xs"], s["pos"], w)}
    dw = None if w is None else torch.empty_like(w)
    if op == "gather_backward":
        dx = torch.empty_like(s["X"])
        lib.expert_gather_backward(s["Xs"], s["pos"], w, s["X"], dX=dx, dweight=dw)
        out = {"tokens": dx}
    else:
        lib.expert_combine_backward(s["X"], s["pos"], w, s["Xs"], dYs=s["out"], dweight=dw)
        out = {"rows": s["out"]}
    if dw is not None:
        out["dweight"] = dw
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------- work

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "i32": 4, "i64": 8, "none": 0}
    if c["op"] == "sort":
        n = c["t"] * c["k"]
        return {"bytes": n * (size[c["ids"]] + 8) + 4 * (c["e"] + 1), "flops": n}
    if c["op"] == "ortho":
        b, n, m = c["batch"], min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # of the two symmetric products only half the elements are needed
        return {"bytes": b * n * m * (size[c["dtype"]] + 2), "flops": STEPS * b * (3 * n * n * m + n * n * n)}
    t, d, es = c["t"], c["d"], size[c["dtype"]]
    n = t * c["k"] * (1 - c["drop"])                       # rows among the experts', on average
    by = (t + n) * d * es + t * c["k"] * (4 + size[c["weight"]])
    flops = n * d * (0 if c["weight"] == "none" else 2)
    if c["op"].endswith("backward") and c["weight"] != "none":
        other = t if c["op"] == "gather_backward" else n   # the rows that only the dots need
        by, flops = by + other * d * es + t * c["k"] * size[c["weight"]], 2 * flops
    return {"bytes": int(by), "flops": int(flops)}


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    if c["op"] == "sort":
        return _exact_sort(c, s["ids"])
    if c["op"] == "ortho":
        return {"O": _exact_ortho(c, s["G"].double())}
    t, k, d = c["t"], c["k"], c["d"]
    weight = torch.ones(t, k, device="cuda").double() if s["weight"] is None else s["weight"].double()
    token, choice = torch.nonzero(s["pos"] >= 0, as_tuple=True)
    place, w = s["pos"][token, choice].long(), weight[token, choice]
    if c["op"] in ("gather", "combine_backward"):
        rows = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
        rows[place] = torch.einsum("n,nd->nd", w, s["X"].double()[token])
        out = {"rows": rows}
    else:
        tokens = torch.zeros(t, d, dtype=torch.float64, device="cuda")
        out = {"tokens": tokens.index_add_(0, token, torch.einsum("n,nd->nd", w, s["Xs"].double()[place]))}
    if c["op"].endswith("backward") and s["weight"] is not None:
        dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        dw[token, choice] = torch.einsum("nd,nd->n", s["X"].double()[token], s["Xs"].double()[place])
        out["dweight"] = dw
    return out


def _exact_sort(c, ids):
    """The same from one unique key for each choice: its expert, then its place in the input."""
    flat = ids.flatten().long()
    n, e = flat.numel(), c["e"]
    slot = torch.arange(n, device="cuda")
    kept = slot[(flat >= 0) & (flat < e)]
    keys = torch.sort(flat[kept] * n + slot[kept])[0]
    order = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    order[: keys.numel()] = (keys % n).int()
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos[keys % n] = torch.arange(keys.numel(), dtype=torch.int32, device="cuda")
    bounds = torch.arange(e + 1, device="cuda") * n
    return {"pos": pos.view(c["t"], c["k"]), "offsets": torch.searchsorted(keys, bounds).int(), "order": order}


def _exact_ortho(c, x):
    a, b, q = COEFFICIENTS
    tall = c["rows"] > c["cols"]
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
    for _ in range(STEPS):
        # the polynomial of the Gram matrix of the shorter side, times x
        g = torch.einsum("bij,bik->bjk", x, x) if tall else torch.einsum("bij,bkj->bik", x, x)
        p = torch.baddbmm(b * g, g, g, alpha=q)
        p.diagonal(dim1=1, dim2=2).add_(a)
        x = torch.bmm(x, p) if tall else torch.bmm(p, x)
    return x
