"""The dense and the per-expert matrix products around the routed-expert layer,
as cases to be measured: what is called, on which inputs, and in plain form.

Four operators, all over 16-bit activations x and row-major weights w [N, K]:

  linear                   y = act(x w^T + b) + r       router logits, shared expert
  linear_backward          dz = dy act'(z); dx = dz w; dw = dz^T x; db = sum of dz
  grouped_linear           the same per expert over rows grouped by expert
                           (offsets [E+1]), rows gathered from the tokens and
                           results scattered back on the way
  grouped_linear_backward  its gradients; dw and db per expert

SwiGLU has two weights, w (gate) and w_up: silu(x w^T + b) * (x w_up^T + b_up).
A case is a dict of plain values; ``run`` computes one pass in plain torch
operations in fp32 or, when ``own`` is set, by the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(name, op, rows, k, n, act="none", dtype="bf16", out="", bias="", residual="", save=False, experts=0,
          topk=0, dw=""):
    """rows: tokens; with experts, every token brings topk rows.  out, bias and
    residual: the types of y (of dx in a backward pass), b and r ("" = x's type
    for out, none for the others).  dw: the type of the weights' gradients."""
    c = {"op": op, "rows": rows, "k": k, "n": n, "act": act, "dtype": dtype, "out": out or dtype, "bias": bias,
         "residual": residual, "save": save, "experts": experts, "topk": topk, "dw": dw or dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the router's product for one decoded token: the smallest call, latency alone counts
        _case("router logits, 1 token", "linear", 1, 5120, 384, out="f32", bias="f32"),
        # gate and up product of a shared expert for a decode batch: bound by reading the weights
        _case("shared up, 64 tokens", "linear", 64, 5120, 2304, act="swiglu"),
        # an adapter of odd sizes: rows of 1001 values are not 16-byte aligned; keeps z for training
        _case("odd sizes, gelu", "linear", 333, 1001, 517, act="gelu", dtype="f16", bias="f16", residual="f16",
              save=True),
        # down product of a shared expert on a long chunk, added to the routed experts' fp32 output
        _case("shared down, 8192 tokens", "linear", 8192, 2304, 5120, residual="f32"),
        # gradients of a small layer of odd sizes
        _case("small gradients", "linear_backward", 129, 256, 131, act="silu", dtype="f16", bias="f16"),
        # gradients of the router's product on one prefill chunk
        _case("router gradients", "linear_backward", 2048, 5120, 384, bias="f32"),
        # gradients of the shared expert's gate and up products on a long chunk
        _case("shared up gradients", "linear_backward", 8192, 5120, 2304, act="swiglu"),
        # routed gate and up products of a decode batch: a row or two for each expert
        _case("expert up, 8 tokens", "grouped_linear", 8, 5120, 2304, act="swiglu", experts=64, topk=6),
        # the same for a prefill chunk
        _case("expert up, 2048 tokens", "grouped_linear", 2048, 5120, 2304, act="swiglu", experts=64, topk=6),
        # routed down product of that chunk into fp32 rows in entry order, as the combine takes them
        _case("expert down, 2048 tokens", "grouped_linear", 2048, 2304, 5120, out="f32", experts=64, topk=6),
        # gradients of a small layer: 16 experts, some without a row, with biases
        _case("small expert gradients", "grouped_linear_backward", 37, 256, 128, act="silu", bias="f32", experts=16,
              topk=2),
        # gradients of the routed gate and up products of a chunk: the largest call
        _case("expert up gradients", "grouped_linear_backward", 2048, 5120, 2304, act="swiglu", experts=64, topk=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "grouped_linear", "grouped_linear_backward"])
    back = op.endswith("backward")
    grouped = op.startswith("grouped")
    act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    k, n = _log(rng, 40, 5120), _log(rng, 24, 5120)
    if rng.random() < 0.7:      # most models' sizes are multiples of 8; the others come odd
        k, n = max(8, k // 8 * 8), max(8, n // 8 * 8)
    if n * k > 5120 * 2304:
        n = max(8, 5120 * 2304 // k // 8 * 8)
    experts = rng.randint(2, 64) if grouped else 0
    topk = rng.randint(1, min(6, experts)) if grouped else 0
    rows = _log(rng, 1, 2048 if grouped else 8192)
    bias = rng.choice(["", "f32", dtype])
    residual = "" if back or grouped else rng.choice(["", "f32", dtype])
    out = dtype if back else rng.choice([dtype, dtype, "f32"])
    save = not back and rng.random() < 0.3
    return _case("", op, rows, k, n, act, dtype, out, bias, residual, save, experts, topk)


_CTX = {}


def _context():
    """A context of the library on the current device; these calls use none of its arena."""
    from fp4_routed_expert_router_b200 import moe
    dev = torch.cuda.current_device()
    if dev not in _CTX:
        _CTX[dev] = moe.Context(hidden=128, inter=128, n_experts=1, top_k=1, n_layers=1, n_slots=1, max_tokens=1,
                                device=dev)
    return _CTX[dev]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    T, K, N, E = case["rows"], case["k"], case["n"], case["experts"]
    two = case["act"] == "swiglu"
    back = case["op"].endswith("backward")

    def normal(*shape, dtype=dt, scale=1.0):
        if len(shape) < 3:
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = {"case": case, "x": normal(T, K)}
    rows = T
    if E:
        # each token's experts by a router with uneven popularity, entries grouped by expert
        kk = case["topk"]
        popular = torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32)) * -0.5
        popular = popular[torch.randperm(E, generator=g, device="cuda")]
        logits = torch.randn(T, E, generator=g, device="cuda") + popular
        ids = torch.topk(logits, kk, dim=1).indices.reshape(-1)
        order = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)
        rows = T * kk
        s["offsets"], s["bounds"] = offsets, offsets.tolist()
        s["entry"] = order.to(torch.int32)             # grouped row -> entry t*k+j
        s["token"] = (order // kk).to(torch.int32)      # grouped row -> token
    lead = (E,) if E else ()
    s["w"] = normal(*lead, N, K, scale=K ** -0.5)
    s["w_up"] = normal(*lead, N, K, scale=K ** -0.5) if two else None
    b = _DT[case["bias"]] if case["bias"] else None
    s["b"] = normal(*lead, N, dtype=b, scale=0.1) if b and not back else None
    s["b_up"] = normal(*lead, N, dtype=b, scale=0.1) if b and two and not back else None
    s["r"] = normal(rows, N, dtype=_DT[case["residual"]]) if case["residual"] else None
    if back:
        s["dy"] = normal(rows, N, scale=0.1)
        s["z"] = normal(rows, N) if case["act"] != "none" else None      # kept by the forward pass, grouped order
        s["z_up"] = normal(rows, N) if two else None
    return s


# ------------------------------------------------------------------ plain form (fp32)
def _act(name, z, z_up):
    if name == "relu":
        return z * (z > 0)
    if name in ("silu", "swiglu"):
        v = z / (1 + torch.exp(-z))
        return v * z_up if name == "swiglu" else v
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _slope(name, z):
    """The derivative of the activation (of the gate's, for swiglu)."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name in ("silu", "swiglu"):
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _spans(s, total):
    """(weight index, first row, last row) of each product: one, or one per expert that has rows."""
    if "bounds" not in s:
        return [((), 0, total)]
    b = s["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _plain_forward(s):
    c, f = s["case"], torch.float32
    x = s["x"] if "token" not in s else s["x"][s["token"].long()]
    rows, two = x.shape[0], s["w_up"] is not None
    z = torch.empty(rows, c["n"], device=x.device)
    z_up = torch.empty_like(z) if two else None
    # a product per expert with rows, as torch has no ragged product among its elementary operations
    for e, lo, hi in _spans(s, rows):
        xe = x[lo:hi].to(f)
        z[lo:hi] = xe @ s["w"][e].to(f).mT
        if two:
            z_up[lo:hi] = xe @ s["w_up"][e].to(f).mT
        if s["b"] is not None:
            z[lo:hi] += s["b"][e].to(f)
            if two:
                z_up[lo:hi] += s["b_up"][e].to(f)
    y = _act(c["act"], z, z_up)
    if s["r"] is not None:
        y = y + s["r"].to(f)
    y = y.to(_DT[c["out"]])
    if "entry" in s:
        y = torch.empty_like(y).index_copy_(0, s["entry"].long(), y)
    dt = _DT[c["dtype"]]
    return (y, z.to(dt), z_up.to(dt) if two else None) if c["save"] else y


def _plain_backward(s):
    c, f = s["case"], torch.float32
    x = s["x"] if "token" not in s else s["x"][s["token"].long()]
    dy = (s["dy"] if "entry" not in s else s["dy"][s["entry"].long()]).to(f)
    two = s["w_up"] is not None
    dz_up = None
    if c["act"] == "none":
        dz = dy
    elif two:
        z = s["z"].to(f)
        dz, dz_up = dy * s["z_up"].to(f) * _slope("swiglu", z), dy * (z / (1 + torch.exp(-z)))
    else:
        dz = dy * _slope(c["act"], s["z"].to(f))
    E = c["experts"]
    lead = (E,) if E else ()
    dt, wt = _DT[c["dtype"]], _DT[c["dw"]]
    dx = torch.empty(x.shape[0], c["k"], dtype=dt, device=x.device)
    dw = torch.zeros(*lead, c["n"], c["k"], dtype=wt, device=x.device)
    dw_up = torch.zeros_like(dw) if two else None
    db = torch.zeros(*lead, c["n"], device=x.device) if c["bias"] else None
    db_up = torch.zeros_like(db) if two and db is not None else None
    for e, lo, hi in _spans(s, x.shape[0]):
        xe, de = x[lo:hi].to(f), dz[lo:hi]
        d = de @ s["w"][e].to(f)
        dw[e] = (de.mT @ xe).to(wt)
        if db is not None:
            db[e] = de.sum(0)
        if two:
            ue = dz_up[lo:hi]
            d += ue @ s["w_up"][e].to(f)
            dw_up[e] = (ue.mT @ xe).to(wt)
            if db is not None:
                db_up[e] = ue.sum(0)
        dx[lo:hi] = d.to(dt)
    if "entry" in s:
        dx = torch.empty_like(dx).index_copy_(0, s["entry"].long(), dx)
    return dx, dw, dw_up, db, db_up


# ------------------------------------------------------------------ the library's calls
def _own(s):
    c = s["case"]
    ctx = _context()
    out = _DT[c["out"]]
    if c["op"] == "linear":
        return ctx.linear(s["x"], s["w"], w_up=s["w_up"], bias=s["b"], bias_up=s["b_up"], act=c["act"],
                          residual=s["r"], out_dtype=out, save=c["save"])
    if c["op"] == "grouped_linear":
        return ctx.grouped_linear(s["x"], s["w"], s["offsets"], w_up=s["w_up"], bias=s["b"], bias_up=s["b_up"],
                                  act=c["act"], x_rows=s["token"], y_rows=s["entry"], out_dtype=out, save=c["save"])
    kw = {"w_up": s["w_up"], "z": s["z"], "z_up": s["z_up"], "act": c["act"], "need_db": bool(c["bias"]),
          "dw_dtype": _DT[c["dw"]]}
    if c["op"] == "linear_backward":
        r = ctx.linear_backward(s["dy"], s["x"], s["w"], **kw)
    else:
        r = ctx.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], x_rows=s["token"],
                                        y_rows=s["entry"], dx_rows=s["entry"], **kw)
    return r.dx, r.dw, r.dw_up, r.db, r.db_up


def run(state):
    if own:
        return _own(state)
    return _plain_backward(state) if state["case"]["op"].endswith("backward") else _plain_forward(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, K, N, E = case["rows"], case["k"], case["n"], case["experts"]
    size = {"bf16": 2, "f16": 2, "f32": 4, "": 0}
    pair = 2 if case["act"] == "swiglu" else 1
    rows, weights, index = T, 1, 0
    if E:
        rows = T * case["topk"]
        weights = min(E, max(1, round(E * (1 - (1 - case["topk"] / E) ** T))))   # experts that get a row
        index = 8 * rows + 4 * (E + 1)
    x, w, e = 2 * T * K, 2 * pair * weights * N * K, rows * N
    product = 2 * rows * N * K * pair
    if case["op"].endswith("backward"):
        zs = 0 if case["act"] == "none" else 2 * pair * e
        grads = pair * (E or 1) * N * (K * size[case["dw"]] + (4 if case["bias"] else 0))
        return {"bytes": x + w + 2 * e + zs + 2 * rows * K + grads + index, "flops": 2 * product}
    kept = 2 * pair * e if case["save"] else 0
    biases = pair * weights * N * size[case["bias"]]
    return {"bytes": x + w + e * size[case["out"]] + e * size[case["residual"]] + biases + kept + index,
            "flops": product}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    E, two, back = case["experts"], case["act"] == "swiglu", case["op"].endswith("backward")
    x = s["x"].to(d)
    if E:
        x = x.index_select(0, s["token"].long())
    n_rows = x.shape[0]

    def sigmoid(v):
        return torch.reciprocal(1 + torch.exp(-v))

    def phi(v):   # the normal distribution function
        return 0.5 * torch.erfc(-v / math.sqrt(2))

    def weight(t, e):
        return (t if e is None else t[e]).to(d)

    groups = [(None, torch.arange(n_rows, device=x.device))]
    if E:
        owner = torch.repeat_interleave(torch.arange(E, device=x.device), torch.diff(s["offsets"].long()))
        groups = [(e, torch.nonzero(owner == e).flatten()) for e in range(E)]

    if not back:
        pre = []
        for t, b in ((s["w"], s["b"]), (s["w_up"], s["b_up"])):
            if t is None:
                pre.append(None)
                continue
            v = torch.zeros(n_rows, case["n"], dtype=d, device=x.device)
            for e, at in groups:
                if at.numel():
                    p = torch.einsum("rk,nk->rn", x[at], weight(t, e))
                    v[at] = p if b is None else p + weight(b, e)
            pre.append(v)
        z, u = pre
        y = {"none": lambda: z, "relu": lambda: torch.clamp(z, min=0), "silu": lambda: z * sigmoid(z),
             "gelu": lambda: z * phi(z), "swiglu": lambda: z * sigmoid(z) * u}[case["act"]]()
        if s["r"] is not None:
            y = y + s["r"].to(d)
        if E:
            placed = torch.empty_like(y)
            placed[s["entry"].long()] = y
            y = placed
        return (y, z, u) if case["save"] else y

    dy = s["dy"].to(d)
    if E:
        dy = dy.index_select(0, s["entry"].long())
    if case["act"] == "none":
        grads = [(dy, s["w"])]
    else:
        z = s["z"].to(d)
        if case["act"] == "relu":
            grads = [(torch.where(z > 0, dy, torch.zeros_like(dy)), s["w"])]
        elif case["act"] == "gelu":
            grads = [(dy * (phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)), s["w"])]
        else:
            slope = sigmoid(z) + z * sigmoid(z) * sigmoid(-z)
            if two:
                grads = [(dy * s["z_up"].to(d) * slope, s["w"]), (dy * z * sigmoid(z), s["w_up"])]
            else:
                grads = [(dy * slope, s["w"])]
    dx = torch.zeros(n_rows, case["k"], dtype=d, device=x.device)
    dws, dbs = [], []
    for dz, t in grads:
        dw = torch.zeros(t.shape, dtype=d, device=x.device)
        db = torch.zeros(t.shape[:-1], dtype=d, device=x.device)
        for e, at in groups:
            if at.numel():
                dx[at] += torch.einsum("rn,nk->rk", dz[at], weight(t, e))
                into = slice(None) if e is None else e
                dw[into] = torch.einsum("rn,rk->nk", dz[at], x[at])
                db[into] = torch.einsum("rn->n", dz[at])
        dws.append(dw)
        dbs.append(db if case["bias"] else None)
    if E:
        placed = torch.empty_like(dx)
        placed[s["entry"].long()] = dx
        dx = placed
    return dx, dws[0], dws[1] if two else None, dbs[0], dbs[1] if two else None
