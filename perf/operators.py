"""What the 4-bit operators and the gradient clipping are measured on.

Four kinds of case, each a call that a user of the package makes:

  quantise   bf16 [rows, cols] -> 4-bit codes and block scales (with ``both`` the
             transposed copy too), read back as bf16 values
  product    y = x W^T with x bf16 quantised in the call and W kept in 4 bits
  step       forward and backward of a Linear whose three products run in 4 bits
  clip       the global 2-norm of a list of gradients and the clipped gradients

Formats: "nv" has blocks of 16 values with an e4m3 scale and one fp32 scale a
tensor, "mx" blocks of 32 with a power of two.  In both a value is an e2m1
number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times its scales:

  nv   a = max |x|, S = fl32(448 / max(a, 1e-12)), inv = fl32(1 / S)
       c = e4m3(fl32(b S)), b the block's max |x|;  r = fl32(fl32(6 S) / c), 0 if c is 0
       q = e2m1(fl32(x r)), stands for q c fl32(inv / 6)
  mx   E = max(e - 2, 0), e the exponent field of the block's max |x|
       q = e2m1(x 2^(127 - E)), stands for q 2^(E - 127)

Codes lie two a byte, the even column in the low half, in rows of
ceil(cols / 32) * 16 bytes.  Scales lie in tiles of 512 bytes, one for 128 rows
x 4 blocks: row r, block k of a tile at (r % 32) * 16 + (r // 32) * 4 + k, the
tiles of 128 rows one after another along the row.  Padding is zero.
"""
import math

import torch

own = False

EPS = 1e-12
BLOCK = {"nv": 16, "mx": 32}


def listed():
    return [
        # The activations of one decoding batch, before a 4096-wide Linear: latency.
        {"name": "quantise nv 16x4096", "op": "quantise", "fmt": "nv", "rows": 16, "cols": 4096, "both": False},
        # A GPT-1.5B block's input at batch 12 x 1024 tokens, both copies for training.
        {"name": "quantise nv both 12288x1600", "op": "quantise", "fmt": "nv", "rows": 12288, "cols": 1600, "both": True},
        # The gate weight of a Llama-3-8B FFN, both copies.
        {"name": "quantise mx both 14336x4096", "op": "quantise", "fmt": "mx", "rows": 14336, "cols": 4096, "both": True},
        # Sizes that end inside blocks, vectors and tiles.
        {"name": "quantise nv both 1009x1531", "op": "quantise", "fmt": "nv", "rows": 1009, "cols": 1531, "both": True},
        # One token through the FFN's up projection: the weight is read once.
        {"name": "product nv 1x4096x14336", "op": "product", "fmt": "nv", "m": 1, "k": 4096, "n": 14336},
        # A decoding batch through the down projection.
        {"name": "product mx 32x14336x4096", "op": "product", "fmt": "mx", "m": 32, "k": 14336, "n": 4096},
        # A ragged prompt batch into an odd-sized head.
        {"name": "product nv 777x1600x4801", "op": "product", "fmt": "nv", "m": 777, "k": 1600, "n": 4801},
        # A long prompt through the up projection: the tensor cores.
        {"name": "product nv 8192x4096x14336", "op": "product", "fmt": "nv", "m": 8192, "k": 4096, "n": 14336},
        # A short training step on a 4096 x 4096 Linear: launches and the weight's quantisation.
        {"name": "step nv 256x4096x4096", "op": "step", "fmt": "nv", "m": 256, "k": 4096, "n": 4096},
        # The same Linear with many tokens.
        {"name": "step mx 16384x4096x4096", "op": "step", "fmt": "mx", "m": 16384, "k": 4096, "n": 4096},
        # One GPT-1.5B block's gradients in bf16 (weights, biases and norms), into fp32 for the optimizer.
        {"name": "clip bf16 block", "op": "clip", "dtype": "bf16", "to": "f32", "width": 1600, "ffn": 6400, "layers": 1},
        # Four layers of fp32 gradients of a 4096-wide model: beyond the L2 cache.
        {"name": "clip f32 4 layers", "op": "clip", "dtype": "f32", "to": "f32", "width": 4096, "ffn": 14336, "layers": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "step", "clip"])
    fmt = rng.choice(["nv", "mx"])
    if op == "quantise":
        return {"op": op, "fmt": fmt, "rows": _log(rng, 1, 14336), "cols": _log(rng, 64, 4096), "both": rng.random() < 0.6}
    if op == "clip":
        dtype = rng.choice(["bf16", "f32"])
        width = _log(rng, 61, 2048)
        return {"op": op, "dtype": dtype, "to": rng.choice([dtype, "f32"]), "width": width,
                "ffn": width * rng.choice([3, 4]) + rng.randrange(8), "layers": rng.randint(1, 4)}
    n = _log(rng, 64, 8192)
    k = _log(rng, 64, 8192)
    if op == "product":
        return {"op": op, "fmt": fmt, "m": _log(rng, 1, 8192), "k": k, "n": n}
    return {"op": op, "fmt": fmt, "m": _log(rng, 16, 8192), "k": min(k, 4096), "n": min(n, 4096)}


# ---------------------------------------------------------------- inputs


def _values(shape, gen, std, rare):
    """Normal values of which one in a thousand is ``rare`` times as large, as activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda") * std
    big = torch.rand(shape, generator=gen, device="cuda") < 1e-3
    return torch.where(big, x * rare, x).to(torch.bfloat16)


def _shapes(case):
    w, f = case["width"], case["ffn"]
    block = [(w,), (3 * w, w), (3 * w,), (w, w), (w,), (w,), (f, w), (f,), (w, f), (w,)]
    return block * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "quantise":
        state["x"] = _values((case["rows"], case["cols"]), gen, 1.0, 30.0)
    elif op == "product":
        state["x"] = _values((case["m"], case["k"]), gen, 1.0, 30.0)
        w = _values((case["n"], case["k"]), gen, 0.02, 4.0)
        q, c, inv = _quantise(w.float(), case["fmt"], _amax(w))
        state["codes"] = _pack(q)
        state["scales"] = _tile(_scale_bytes(c, case["fmt"]))
        state["inv"] = inv
    elif op == "step":
        state["x"] = _values((case["m"], case["k"]), gen, 1.0, 30.0)
        state["w"] = _values((case["n"], case["k"]), gen, 0.02, 4.0)
        state["dy"] = _values((case["m"], case["n"]), gen, 1e-3, 10.0)
    else:
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        state["grads"] = [(torch.randn(s, generator=gen, device="cuda") * 10.0 ** (-3 - i % 3)).to(dtype)
                          for i, s in enumerate(_shapes(case))]
        state["max_norm"] = 1e-2
    return state


# ---------------------------------------------------------------- the plain form


def _amax(x):
    return x.abs().amax().float().reshape(1)


def _power(e):
    """2^e in fp32, exactly, for whole e of -149 to 127."""
    return torch.where(e >= -126, (e + 127) << 23, 1 << (e + 149).clamp(0, 30)).to(torch.int32).view(torch.float32)


def _over(number, v):
    """number / v with one rounding: a plain number over a tensor would round twice."""
    return torch.full_like(v, number) / v


def _to_e4m3(v):
    """The nearest e4m3 number (ties to even, at most 448) of v >= 0."""
    step = _power((torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _to_e2m1(v):
    """The nearest e2m1 number (ties to even, at most 6 in magnitude)."""
    y = v.abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return torch.copysign((torch.round(y / step) * step).clamp(max=6.0), v)


def _quantise(x, fmt, amax):
    """e2m1 numbers [rows, blocks, block], block scales [rows, blocks] and the tensor's inverse scale of x (fp32)."""
    block = BLOCK[fmt]
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % block)).reshape(rows, -1, block)
    b = x.abs().amax(dim=2)
    if fmt == "mx":
        e = (torch.frexp(b).exponent - 3).clamp(min=-127)
        e = torch.where(b > 0, e, -127)
        return _to_e2m1(x * _power(-e).unsqueeze(2)), _power(e), None
    s = _over(448.0, amax.clamp(min=EPS))
    c = _to_e4m3(b * s)
    r = torch.where(c > 0, (6.0 * s) / c, torch.zeros_like(c))
    return _to_e2m1(x * r.unsqueeze(2)), c, _over(1.0, s)


def _dequantise(q, c, inv, cols):
    v = (q * c.unsqueeze(2)).reshape(q.shape[0], -1)[:, :cols]
    return v if inv is None else v * (inv / torch.full_like(inv, 6.0))


def _rounded(x, fmt, amax):
    """The fp32 values that the 4-bit form of x stands for, and the tensor's inverse scale."""
    q, c, inv = _quantise(x, fmt, amax)
    return _dequantise(q, c, inv, x.shape[1]), inv


def _pack(q):
    """e2m1 numbers [rows, blocks, block] -> codes, two a byte."""
    rows = q.shape[0]
    q = q.reshape(rows, -1)
    y = q.abs()
    code = torch.where(y < 2, y * 2, torch.where(y < 4, y + 2, y / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    code = torch.nn.functional.pad(code, (0, -code.shape[1] % 32))
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _scale_bytes(c, fmt):
    f, e = torch.frexp(c)
    if fmt == "mx":
        return (e - 1 + 127).to(torch.uint8)
    normal = c >= 2.0 ** -6
    return torch.where(normal, (e - 1 + 7) * 8 + (f * 16 - 8).int(), (c * 512).int()).to(torch.uint8)


def _tile(s):
    rows, blocks = s.shape
    s = torch.nn.functional.pad(s, (0, -blocks % 4, 0, -rows % 128))
    s = s.reshape(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4)
    return s.permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _unpacked(state):
    """The fp32 values of the weight that a product case keeps in 4 bits."""
    case = state["case"]
    rows, cols, block = case["n"], case["k"], BLOCK[case["fmt"]]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    table = torch.cat([table, -table])
    codes = state["codes"]
    q = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=2).reshape(rows, -1)
    s = state["scales"].reshape(-(-rows // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = s.reshape(-(-rows // 128) * 128, -1)[:rows, :-(-cols // block)].int()
    if case["fmt"] == "mx":
        c = _power(s - 127)
    else:
        e, m = s >> 3, (s & 7).float()
        c = torch.where(e > 0, (1 + m / 8) * _power(e - 7), m / 512)
    q = q[:, :c.shape[1] * block].reshape(rows, -1, block)
    return _dequantise(q, c, state["inv"], cols)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "clip":
        norm = torch.stack([g.float().square().sum() for g in state["grads"]]).sum().sqrt().reshape(1)
        coef = _over(state["max_norm"], norm + 1e-6).clamp(max=1.0)
        to = torch.bfloat16 if case["to"] == "bf16" else torch.float32
        return {"norm": norm, "grads": [(g.float() * coef).to(to) for g in state["grads"]]}
    fmt, x = case["fmt"], state["x"]
    amax = _amax(x) if fmt == "nv" else None
    x = x.float()
    v, inv = _rounded(x, fmt, amax)
    if op == "quantise":
        out = {"values": v.to(torch.bfloat16)}
        if case["both"]:
            out["values_t"] = _rounded(x.t(), fmt, amax)[0].to(torch.bfloat16)
        if inv is not None:
            out["inv_scale"] = inv
        return out
    if op == "product":
        return {"y": (v @ _unpacked(state).t()).to(torch.bfloat16)}
    amax_w, amax_dy = (_amax(state[n]) if fmt == "nv" else None for n in ("w", "dy"))
    w, dy = state["w"].float(), state["dy"].float()
    y = v @ _rounded(w, fmt, amax_w)[0].t()
    dx = _rounded(dy, fmt, amax_dy)[0] @ _rounded(w.t(), fmt, amax_w)[0].t()
    dw = _rounded(dy.t(), fmt, amax_dy)[0] @ _rounded(x.t(), fmt, amax)[0].t()
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ---------------------------------------------------------------- the package's operators


def _kept(state):
    """What a program makes once for these sizes and keeps: 4-bit tensors, outputs, workspace."""
    import quantised_gemm_gb300 as q
    case = state["case"]
    op = case["op"]
    if op == "clip":
        to = torch.bfloat16 if case["to"] == "bf16" else torch.float32
        return {"outs": [torch.empty(g.shape, dtype=to, device=g.device) for g in state["grads"]],
                "norm": torch.empty(1, device="cuda"), "ws": q.Workspace()}
    fmt = q.NVFP4 if case["fmt"] == "nv" else q.MXFP4
    if op == "step":
        return {"lin": q.Fp4Linear(case["m"], case["k"], case["n"], fmt=fmt)}
    rows, cols = state["x"].shape
    kept = {"x4": q.Fp4Tensor(rows, cols, fmt), "ws": q.Workspace()}
    if op == "product":
        kept["w4"] = q.Fp4Tensor(case["n"], case["k"], fmt, codes=state["codes"], scales=state["scales"],
                                 inv_scale=state["inv"])
        kept["y"] = torch.empty((rows, case["n"]), dtype=torch.bfloat16, device="cuda")
        return kept
    kept["values"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    kept["x4t"] = None
    if case["both"]:
        kept["x4t"] = q.Fp4Tensor(cols, rows, fmt, state=kept["x4"].state)
        kept["values_t"] = torch.empty((cols, rows), dtype=torch.bfloat16, device="cuda")
    return kept


def _own(state):
    import quantised_gemm_gb300 as q
    if "kept" not in state:
        state["kept"] = _kept(state)
    op, k = state["case"]["op"], state["kept"]
    if op == "clip":
        q.clip_grad_norm(state["grads"], state["max_norm"], k["norm"], k["ws"], outs=k["outs"])
        return {"norm": k["norm"], "grads": k["outs"]}
    if op == "step":
        y = k["lin"].forward(state["x"], state["w"])
        dx, dw = k["lin"].backward(state["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    if op == "product":
        return {"y": q.fp4_linear(state["x"], k["x4"], k["w4"], k["y"], k["ws"])}
    q.fp4_quantise(state["x"], k["x4"], k["x4t"], k["ws"])
    out = {"values": q.fp4_dequantise(k["x4"], k["values"])}
    if k["x4t"] is not None:
        out["values_t"] = q.fp4_dequantise(k["x4t"], k["values_t"])
    if k["x4"].state is not None:
        out["inv_scale"] = k["x4"].state.inv_scale
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the floor


def _held(rows, cols, fmt):
    """Bytes of a [rows, cols] tensor in 4 bits, scales included."""
    return rows * cols / 2 + rows * -(-cols // BLOCK[fmt])


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        size = {"bf16": 2, "f32": 4}
        return {"bytes": n * (size[case["dtype"]] + size[case["to"]]), "flops": 3 * n}
    fmt = case["fmt"]
    if op == "quantise":
        r, c = case["rows"], case["cols"]
        total = 2 * r * c + _held(r, c, fmt) + 2 * r * c
        if case["both"]:
            total += _held(c, r, fmt) + 2 * r * c
        return {"bytes": total, "flops": 4 * r * c}
    m, k, n = case["m"], case["k"], case["n"]
    if op == "product":
        return {"bytes": 2 * m * k + _held(n, k, fmt) + 2 * m * n, "flops": 2 * m * k * n}
    return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * k * n}


# ---------------------------------------------------------------- the definition in 64 bits


def _nearest(v, grid):
    """The nearest of the non-negative numbers ``grid`` (ascending, every other one even) of |v|, with v's sign."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    y = v.abs().contiguous()
    lo, hi = torch.searchsorted(mid, y), torch.searchsorted(mid, y, right=True)
    return torch.copysign(grid[torch.where(lo % 2 == 0, lo, hi)], v)


def _fl(v):
    """Where the definition rounds to fp32."""
    return v.float().double()


def _exact_values(x, fmt, amax):
    rows, cols = x.shape
    block = BLOCK[fmt]
    full = torch.zeros((rows, -(-cols // block) * block), dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    full = full.reshape(rows, -1, block)
    top = full.abs().amax(dim=2, keepdim=True)
    e2m1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    if fmt == "mx":
        powers = torch.tensor([2.0 ** e for e in range(-125, 128)], dtype=torch.float64, device=x.device)
        size = torch.cat([powers[:1], powers])[torch.searchsorted(powers, top, right=True)] / 4
        return (_nearest(full / size, e2m1) * size).reshape(rows, -1)[:, :cols], None
    s = _fl(torch.full_like(amax, 448.0) / amax.clamp(min=float(torch.tensor(EPS))))
    inv = _fl(torch.ones_like(s) / s)
    e4m3 = [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
    c = _nearest(_fl(top * s), e4m3)
    r = torch.where(c > 0, _fl(_fl(6.0 * s) / c), 0.0)
    return (_nearest(_fl(full * r), e2m1) * c * _fl(inv / torch.full_like(inv, 6.0))).reshape(rows, -1)[:, :cols], inv


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        grads = [g.double() for g in state["grads"]]
        norm = torch.stack([g.square().sum() for g in grads]).sum().sqrt()
        coef = min(1.0, state["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm.reshape(1), "grads": [g * coef for g in grads]}
    fmt = case["fmt"]
    both = {n: state[n].double() for n in ("x", "w", "dy") if n in state}
    top = {n: t.abs().max() for n, t in both.items()}
    x, inv = _exact_values(both["x"], fmt, top["x"])
    if op == "quantise":
        out = {"values": x}
        if case["both"]:
            out["values_t"] = _exact_values(both["x"].t(), fmt, top["x"])[0]
        if inv is not None:
            out["inv_scale"] = inv.reshape(1)
        return out
    if op == "product":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        _values((case["m"], case["k"]), gen, 1.0, 30.0)
        w = _values((case["n"], case["k"]), gen, 0.02, 4.0).double()
        return {"y": x @ _exact_values(w, fmt, w.abs().max())[0].t()}
    pick = lambda n, t: _exact_values(both[n].t() if t else both[n], fmt, top[n])[0]  # noqa: E731
    return {"y": x @ pick("w", False).t(), "dx": pick("dy", False) @ pick("w", True).t(),
            "dw": pick("dy", True) @ pick("x", True).t()}
