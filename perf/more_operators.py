"""What the layer norm and the low-rank adapters are measured on.

Four kinds of case, each a call that a user of the package makes:

  norm               h = bf16(x + r) where there is a residual r, else x;
                     mu and v the mean and the mean square deviation of a row of h,
                     y = (h - mu) / sqrt(v + eps) * w + b, with mu and 1 / sqrt(v + eps) kept
  norm backward      xhat = (h - mu) rstd, g = dy w,
                     dx = rstd (g - mean(g) - xhat mean(g xhat)) + dr,
                     dw = sum over the rows of dy xhat, db = sum over the rows of dy
  adapters           y = base + s_a B_a (A_a x) for each row, a the row's adapter: base is
                     what a shared projection of x gave; a = -1: the row keeps base
  adapters backward  with h = A_a x kept from the forward and dh = s_a B_a^T dy:
                     dx = base + A_a^T dh (base: the shared projection's gradient),
                     dA_a = sum over a's rows of dh x^T, dB_a = sum over them of s_a dy h^T

x, y, dy, dx, the adapters and their gradients are bf16, statistics and h fp32; a norm's weight,
bias and their gradients are bf16 or fp32.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # One decoding batch's hidden states after a 4096-wide Linear, added to the residual: latency.
        {"name": "norm 16x4096 residual", "op": "norm", "rows": 16, "cols": 4096, "param": "bf16", "residual": True},
        # The norm before a GPT-1.5B block's Linear, 12 x 1024 tokens.
        {"name": "norm 12288x1600", "op": "norm", "rows": 12288, "cols": 1600, "param": "f32", "residual": False},
        # 65536 tokens of a 4096-wide model, the block's output added to the residual.
        {"name": "norm 65536x4096 residual", "op": "norm", "rows": 65536, "cols": 4096, "param": "bf16", "residual": True},
        # A short training step: few rows for each column's sum.
        {"name": "norm backward 256x4096", "op": "norm_backward", "rows": 256, "cols": 4096, "param": "f32", "residual": False},
        # Rows of odd length.
        {"name": "norm backward 1009x1531", "op": "norm_backward", "rows": 1009, "cols": 1531, "param": "bf16", "residual": True},
        # 65536 tokens, with the gradient that passes the block by.
        {"name": "norm backward 65536x4096 residual", "op": "norm_backward", "rows": 65536, "cols": 4096, "param": "f32",
         "residual": True},
        # A decoding batch of 32 requests, each with an adapter of its own choice, beside the FFN's up projection.
        {"name": "adapters 32x4096x14336 r16", "op": "adapters", "rows": 32, "k": 4096, "n": 14336, "rank": 16, "count": 32,
         "runs": False},
        # A ragged prompt batch into an odd-sized head, rank 8.
        {"name": "adapters 777x1600x4801 r8", "op": "adapters", "rows": 777, "k": 1600, "n": 4801, "rank": 8, "count": 5,
         "runs": True},
        # Prompts of several requests, 8192 tokens in all, rank 64.
        {"name": "adapters 8192x4096x4096 r64", "op": "adapters", "rows": 8192, "k": 4096, "n": 4096, "rank": 64, "count": 8,
         "runs": True},
        # A short training step of one adapter beside a 4096 x 4096 Linear.
        {"name": "adapters backward 256x4096x4096 r16", "op": "adapters_backward", "rows": 256, "k": 4096, "n": 4096, "rank": 16,
         "count": 1, "runs": True},
        # Odd sizes, sequences of four adapters in one batch.
        {"name": "adapters backward 1267x1600x2501 r12", "op": "adapters_backward", "rows": 1267, "k": 1600, "n": 2501, "rank": 12,
         "count": 4, "runs": True},
        # A long training step beside the FFN's up projection.
        {"name": "adapters backward 16384x4096x14336 r16", "op": "adapters_backward", "rows": 16384, "k": 4096, "n": 14336,
         "rank": 16, "count": 4, "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "adapters", "adapters_backward"])
    if op.startswith("norm"):
        return {"op": op, "rows": _log(rng, 1, 32768), "cols": _log(rng, 64, 8192), "param": rng.choice(["bf16", "f32"]),
                "residual": rng.random() < 0.5}
    runs = op == "adapters_backward" or rng.random() < 0.6
    rank = rng.choice([4, 8, 12, 16, 24, 32, 64])
    rows = _log(rng, 64, 8192 if rank < 64 else 4096) if runs else _log(rng, 1, 256)
    return {"op": op, "rows": rows, "k": _log(rng, 64, 8192), "n": _log(rng, 64, 8192), "rank": rank,
            "count": _log(rng, 1, 8 if runs else 64), "runs": runs}


# ---------------------------------------------------------------- inputs


def _values(shape, gen, std, rare=1.0):
    """Normal values of which one in a thousand is ``rare`` times as large, as activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda").mul_(std)
    if rare != 1.0:
        big = torch.rand(shape, generator=gen, device="cuda") < 1e-3
        x = torch.where(big, x * rare, x)
    return x.to(torch.bfloat16)


def _index(case, gen):
    """Each row's adapter: by requests of many rows each, or row by row; one in ten has none, if there are several."""
    rows, count = case["rows"], case["count"]
    if case["runs"]:
        requests = min(rows, 2 * count) if count > 1 else 1
        cuts = torch.rand(rows, generator=gen, device="cuda").argsort()[:requests - 1]
        starts = torch.zeros(rows, dtype=torch.int64, device="cuda")
        starts[cuts] = 1
        request = starts.cumsum(0) - starts[0]
    else:
        requests, request = rows, torch.arange(rows, device="cuda")
    adapter = torch.randint(0, count, (requests + 1,), generator=gen, device="cuda")
    if count > 1:
        none = torch.rand(requests + 1, generator=gen, device="cuda") < 0.1
        adapter = torch.where(none, -1, adapter)
    return adapter[request].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        dtype = torch.bfloat16 if case["param"] == "bf16" else torch.float32
        state["x"] = _values((rows, cols), gen, 1.0, 30.0)
        state["w"] = (torch.randn(cols, generator=gen, device="cuda") * 0.1 + 1.0).to(dtype)
        if op == "norm":
            state["b"] = (torch.randn(cols, generator=gen, device="cuda") * 0.1).to(dtype)
            if case["residual"]:
                state["residual"] = _values((rows, cols), gen, 1.0, 30.0)
            return state
        state["dy"] = _values((rows, cols), gen, 1e-3, 10.0)
        if case["residual"]:
            state["dres"] = _values((rows, cols), gen, 1e-3, 10.0)
        x = state["x"].float()  # the statistics that the forward kept
        mean = x.mean(1)
        state["stats"] = torch.stack([mean, ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()])
        return state
    rows, k, n, r, count = (case[c] for c in ("rows", "k", "n", "rank", "count"))
    state["index"] = _index(case, gen)
    state["x"] = _values((rows, k), gen, 1.0, 30.0)
    state["a"] = _values((count, r, k), gen, k ** -0.5)
    state["b"] = _values((count, n, r), gen, 0.02)
    state["scale"] = 0.5 + torch.rand(count, generator=gen, device="cuda") * 1.5
    if op == "adapters":
        state["base"] = _values((rows, n), gen, 1.0)
        return state
    state["dy"] = _values((rows, n), gen, 1e-3, 10.0)
    state["base"] = _values((rows, k), gen, 1e-3)
    state["h"] = _low(state["x"].float(), state["a"].float(), _chosen(state)).sum(1)  # kept by the forward
    return state


# ---------------------------------------------------------------- the plain form


def _plain_norm(state):
    x = state["x"]
    out = {}
    if "residual" in state:
        x = out["h"] = (x.float() + state["residual"].float()).to(torch.bfloat16)
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / (d.square().mean(1, keepdim=True) + EPS).sqrt()
    out["y"] = (d * rstd * state["w"].float() + state["b"].float()).to(torch.bfloat16)
    out["stats"] = torch.cat([mean, rstd], 1).t().contiguous()
    return out


def _plain_norm_backward(state):
    mean, rstd = state["stats"][0][:, None], state["stats"][1][:, None]
    dy, w = state["dy"].float(), state["w"]
    xhat = (state["x"].float() - mean) * rstd
    g = dy * w.float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    if "dres" in state:
        dx = dx + state["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0).to(w.dtype), "db": dy.sum(0).to(w.dtype)}


def _chosen(state):
    """[rows, count]: 1 where a row has that adapter."""
    adapters = torch.arange(state["case"]["count"], device="cuda", dtype=torch.int32)
    return (state["index"][:, None] == adapters).float()


def _low(x, a, chosen):
    """[rows, count, rank]: x times each adapter's A, 0 where the row has another."""
    count, r, k = a.shape
    return (x @ a.reshape(count * r, k).t()).reshape(-1, count, r) * chosen[:, :, None]


def _plain_adapters(state):
    chosen = _chosen(state)
    a, b = state["a"].float(), state["b"].float()
    low = _low(state["x"].float(), a, chosen) * state["scale"][None, :, None]
    y = state["base"].float() + low.flatten(1) @ b.transpose(1, 2).flatten(0, 1)
    return {"y": y.to(torch.bfloat16)}


def _plain_adapters_backward(state):
    chosen, scale = _chosen(state), state["scale"]
    a, b = state["a"].float(), state["b"].float()
    dy, x = state["dy"].float(), state["x"].float()
    dh = _low(dy, b.transpose(1, 2), chosen) * scale[None, :, None]
    h = state["h"][:, None, :] * chosen[:, :, None] * scale[None, :, None]
    dx = state["base"].float() + dh.flatten(1) @ a.flatten(0, 1)
    da = (dh.flatten(1).t() @ x).reshape(a.shape)
    db = (dy.t() @ h.flatten(1)).reshape(dy.shape[1], *h.shape[1:]).transpose(0, 1).contiguous()
    return {"dx": dx.to(torch.bfloat16), "da": da.to(torch.bfloat16), "db": db.to(torch.bfloat16)}


# ---------------------------------------------------------------- the package's operators


def _kept(state):
    """What a program makes once for these sizes and keeps: outputs, the adapters' handle, the workspace."""
    import quantised_gemm_gb300 as q
    case = state["case"]
    op, like = case["op"], torch.empty_like
    kept = {"ws": q.Workspace()}
    if op == "norm":
        kept["y"] = like(state["x"])
        kept["stats"] = torch.empty((2, case["rows"]), device="cuda")
        kept["h"] = like(state["x"]) if case["residual"] else None
    elif op == "norm_backward":
        kept.update(dx=like(state["x"]), dw=like(state["w"]), db=like(state["w"]))
    else:
        kept["bank"] = q.Adapters(state["a"], state["b"], state["scale"])
        kept["low"] = torch.empty((case["rows"], case["rank"]), device="cuda")
        kept["out"] = like(state["base"])
        if op == "adapters_backward":
            kept.update(da=like(state["a"]), db=like(state["b"]))
    return kept


def _own(state):
    import quantised_gemm_gb300 as q
    if "kept" not in state:
        state["kept"] = _kept(state)
    op, k = state["case"]["op"], state["kept"]
    if op == "norm":
        q.layer_norm(state["x"], state["w"], state["b"], k["y"], k["stats"], eps=EPS, residual=state.get("residual"), h=k["h"])
        out = {"y": k["y"], "stats": k["stats"]}
        if k["h"] is not None:
            out["h"] = k["h"]
        return out
    if op == "norm_backward":
        q.layer_norm_backward(state["dy"], state["x"], state["w"], state["stats"], k["dx"], k["dw"], k["db"], k["ws"],
                              dres=state.get("dres"))
        return {"dx": k["dx"], "dw": k["dw"], "db": k["db"]}
    if op == "adapters":
        q.adapter_linear(state["x"], state["index"], k["bank"], k["out"], k["low"], k["ws"], base=state["base"])
        return {"y": k["out"]}
    q.adapter_backward(state["dy"], state["x"], state["h"], state["index"], k["bank"], k["low"], k["out"], k["da"], k["db"], k["ws"],
                       base=state["base"])
    return {"dx": k["out"], "da": k["da"], "db": k["db"]}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "adapters": _plain_adapters,
          "adapters_backward": _plain_adapters_backward}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the floor


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        m, k = case["rows"], case["cols"]
        size = 2 if case["param"] == "bf16" else 4
        if op == "norm":
            return {"bytes": (8 if case["residual"] else 4) * m * k + 8 * m + 2 * k * size, "flops": 8 * m * k}
        return {"bytes": (8 if case["residual"] else 6) * m * k + 8 * m + 3 * k * size, "flops": 14 * m * k}
    m, k, n, r = (case[c] for c in ("rows", "k", "n", "rank"))
    used = min(case["count"], m)
    weights = 2 * used * r * (k + n)
    if op == "adapters":
        return {"bytes": 2 * m * (k + 2 * n) + weights + 4 * m, "flops": 2 * m * r * (k + n)}
    return {"bytes": 2 * m * (n + 3 * k) + 4 * m * r + weights + 2 * case["count"] * r * (k + n) + 4 * m,
            "flops": 4 * m * r * (k + n)}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_norm(state):
    out = {}
    x = state["x"].double()
    if "residual" in state:
        out["h"] = x + state["residual"].double()
        x = out["h"].to(torch.bfloat16).double()  # what is normalised is the stored sum
    k = x.shape[1]
    mean = x.sum(1) / k
    x -= mean[:, None]
    rstd = 1.0 / torch.sqrt((x * x).sum(1) / k + EPS)
    out["stats"] = torch.stack([mean, rstd])
    out["y"] = torch.addcmul(state["b"].double(), x * rstd[:, None], state["w"].double())
    return out


def _exact_norm_backward(state):
    mean, rstd = state["stats"].double()
    dy, k = state["dy"].double(), state["x"].shape[1]
    xhat = (state["x"].double() - mean[:, None]) * rstd[:, None]
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    dy *= state["w"].double()
    own_part = (dy * xhat).sum(1, keepdim=True) / k
    dx = rstd[:, None] * (dy - dy.sum(1, keepdim=True) / k - xhat * own_part)
    if "dres" in state:
        dx += state["dres"]
    return {"dx": dx, "dw": dw, "db": db}


def _exact_adapters(state, backward):
    index, scale = state["index"].long(), state["scale"].double()
    out = state["base"].double()
    grads = {"da": torch.zeros(state["a"].shape, dtype=torch.float64, device="cuda"),
             "db": torch.zeros(state["b"].shape, dtype=torch.float64, device="cuda")}
    for i in range(state["case"]["count"]):
        rows = (index == i).nonzero()[:, 0]
        a, b, x = state["a"][i].double(), state["b"][i].double(), state["x"][rows].double()
        if not backward:
            out[rows] += torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", x, a) * scale[i], b)
            continue
        dy = state["dy"][rows].double() * scale[i]
        dh = torch.einsum("mn,nr->mr", dy, b)
        out[rows] += torch.einsum("mr,rk->mk", dh, a)
        grads["da"][i] = torch.einsum("mr,mk->rk", dh, x)
        grads["db"][i] = torch.einsum("mn,mr->nr", dy, state["h"][rows].double())
    return {"dx": out, **grads} if backward else {"y": out}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(state)
    if case["op"] == "norm_backward":
        return _exact_norm_backward(state)
    return _exact_adapters(state, case["op"] == "adapters_backward")
