"""Cases for the block operators: Newton-Schulz orthogonalisation of stacks of small blocks
(attention heads, low-rank factors, narrow experts), its gradient, and the Muon step on such
stacks.

A case describes the matrices of `layers` layers.  Each layer has `rows_mats` matrices whose
`heads` blocks are consecutive rows (a query, key or value projection: heads*dim x width, block
dim x width) and `cols_mats` matrices whose blocks are consecutive columns (an output
projection: width x heads*dim, block width x dim).  Every matrix is one stack of `heads` blocks
in the call; all stacks of a case go through one call.  `pad` widens every row by that many
elements that belong to no block.

Per block, with X oriented so that rows <= columns:
  ns    X = x / (|x| + 1e-7); `steps` times: A = X X^T, X = a X + (b A + c A A) X; output X
  vjp   the gradient with respect to x of <ns(x), y> for a given y
  step  m = beta m + g; u = g + beta m (Nesterov); w = w - lr * ns(u)
"""
import math

import torch

own = False

MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
COEFFS = {"muon": MUON, "cubic": CUBIC}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LR, BETA, EPS = 0.02, 0.95, 1e-7


def _case(name, op, layers, heads, dim, width, dtype="bf16", out="bf16", rows_mats=1, cols_mats=0, steps=5,
          coeffs="muon", pad=0, values="noise"):
    return {"name": name, "op": op, "layers": layers, "heads": heads, "dim": dim, "width": width, "dtype": dtype,
            "out": out, "rows_mats": rows_mats, "cols_mats": cols_mats, "steps": steps, "coeffs": coeffs,
            "pad": pad, "values": values}


def listed():
    return [
        # one GPT-2-small-sized query projection: 12 heads of 64; latency
        _case("ns_gpt2s_layer", "ns", 1, 12, 64, 768),
        # query and key projections of all 24 d24 layers, 12 heads of 128
        _case("ns_d24_qk", "ns", 24, 12, 128, 1536, rows_mats=2, values="spiked"),
        # binary32 weights, 12 layers of GPT-2-small size, heads in rows and in columns
        _case("ns_gpt2s_f32", "ns", 12, 12, 64, 768, dtype="f32", out="f32", rows_mats=3, cols_mats=1),
        # odd sizes, strided rows, tall blocks, cubic iteration
        _case("ns_ragged", "ns", 5, 7, 1001, 51, rows_mats=1, cols_mats=1, steps=4, coeffs="cubic", pad=3),
        # rank-16 factors of one layer's four projections; latency
        _case("vjp_lowrank_layer", "vjp", 1, 1, 16, 1536, rows_mats=4, cols_mats=4, dtype="f32", out="f32"),
        # heads of 12 d24 layers
        _case("vjp_d24_qk", "vjp", 12, 12, 128, 1536, rows_mats=2, values="spiked"),
        # binary32 gradients, GPT-2-small heads
        _case("vjp_gpt2s_f32", "vjp", 6, 12, 64, 768, dtype="f32", out="f32", rows_mats=2, cols_mats=1),
        # odd sizes, strided rows
        _case("vjp_ragged", "vjp", 3, 5, 77, 333, rows_mats=2, cols_mats=1, pad=1),
        # the step of one d24 layer's attention, as submitted behind backward
        _case("step_d24_layer", "step", 1, 12, 128, 1536, rows_mats=3, cols_mats=1, values="spiked"),
        # every attention projection of d24 in one call
        _case("step_d24_heads", "step", 24, 12, 128, 1536, rows_mats=3, cols_mats=1, values="spiked"),
        # binary32 weights and gradients, GPT-2-small
        _case("step_gpt2s_f32", "step", 12, 12, 64, 768, dtype="f32", out="f32", rows_mats=3, cols_mats=1),
        # odd sizes, strided rows
        _case("step_ragged", "step", 9, 11, 90, 1111, rows_mats=1, cols_mats=2, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ns", "vjp", "step"))
    small, large = _log(rng, 1, 128), _log(rng, 64, 4096)
    dim, width = (small, large) if rng.random() < 0.75 else (large, small)
    rows_mats = rng.randint(0, 3)
    cols_mats = rng.randint(0 if rows_mats else 1, 2)
    dtype = rng.choice(("bf16", "f32"))
    out = dtype if op == "step" or rng.random() < 0.7 else rng.choice(("bf16", "f32"))
    most = 100_000_000 // (dim * width * (rows_mats + cols_mats))  # blocks of each kind
    heads = _log(rng, 1, min(40, most))
    layers = _log(rng, 1, max(1, min(24, most // heads)))
    return {"op": op, "layers": layers, "heads": heads, "dim": dim, "width": width, "dtype": dtype, "out": out,
            "rows_mats": rows_mats, "cols_mats": cols_mats, "steps": rng.choice((3, 4, 5, 5, 5, 6)),
            "coeffs": rng.choice(("muon", "muon", "cubic")), "pad": rng.choice((0, 0, 0, 1, 8)),
            "values": rng.choice(("noise", "spiked"))}


# ------------------------------------------------------------------ inputs

def _shapes(case):
    """(matrices, rows, columns) of the two kinds, blocks in rows and blocks in columns."""
    inner = case["heads"] * case["dim"]
    return ((case["layers"] * case["rows_mats"], inner, case["width"]),
            (case["layers"] * case["cols_mats"], case["width"], inner))


def _blocks(t, case, kind):
    """The blocks of a kind's matrices: one strided view (matrices, heads, rows, columns)."""
    n, rows, cols = t.shape
    if kind == 0:
        return t.unflatten(1, (case["heads"], case["dim"]))
    return t.unflatten(2, (case["heads"], case["dim"])).permute(0, 2, 1, 3)


def _empty(shape, pad, dtype):
    n, rows, cols = shape
    return torch.zeros(n, rows, cols + pad, dtype=dtype, device="cuda")[:, :, :cols]


def _fill(shape, pad, dtype, gen, scale, values):
    """N(0, scale^2) noise; "spiked" adds a rank-16 part whose top singular value is about 100
    times the edge of the noise, as gradients early in training have."""
    n, rows, cols = shape
    x = torch.randn(n, rows, cols, generator=gen, device="cuda")
    if values == "spiked":
        a = torch.randn(n, rows, 16, generator=gen, device="cuda")
        b = torch.randn(n, 16, cols, generator=gen, device="cuda")
        x.baddbmm_(a, b, alpha=100.0 * (math.sqrt(rows) + math.sqrt(cols)) / math.sqrt(rows * cols))
    t = _empty(shape, pad, dtype)
    t.copy_(x.mul_(scale))
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, out, pad, op = DTYPES[case["dtype"]], DTYPES[case["out"]], case["pad"], case["op"]
    state = {"case": case, "kinds": []}
    for kind, shape in enumerate(_shapes(case)):
        if shape[0] == 0:
            continue
        k = {"kind": kind, "x": _fill(shape, pad, dt, gen, 1e-3, case["values"])}
        if op == "vjp":
            k["y"] = _fill(shape, pad, dt, gen, 1.0, "noise")
        if op == "step":
            k["m"] = _fill(shape, pad, torch.float32, gen, 1e-2, case["values"])
            k["w"] = _fill(shape, pad, out, gen, 0.02, "noise")
        else:
            k["out"] = _empty(shape, pad, out)
        state["kinds"].append(k)
    if own:
        state["call"] = _arguments(state)
    return state


# ------------------------------------------------- the framework's operators

def _stacks(state, key):
    """One (heads, rows, columns) view for each matrix of the case."""
    case = state["case"]
    return [s for k in state["kinds"] for s in _blocks(k[key], case, k["kind"]).unbind(0)]


def _arguments(state):
    """The pointer and descriptor arrays that a program builds once for its tensors."""
    from muon_newton_schulz_02_amd import binding as mb
    op = state["case"]["op"]
    if op == "step":
        return mb.StepBlocksArgs(_stacks(state, "w"), _stacks(state, "x"), _stacks(state, "m"))
    if op == "vjp":
        return mb.VjpBlocksArgs(_stacks(state, "x"), _stacks(state, "y"), _stacks(state, "out"))
    return mb.NsBlocksArgs(_stacks(state, "x"), _stacks(state, "out"))


def _run_own(state):
    from muon_newton_schulz_02_amd import binding as mb
    case = state["case"]
    ns = {"ns_coeffs": COEFFS[case["coeffs"]], "ns_steps": case["steps"]}
    if case["op"] == "step":
        mb.muon_step_blocks(state["call"], lr=LR, beta=BETA, nesterov=True, **ns)
    elif case["op"] == "vjp":
        mb.muon_ns_blocks_vjp(state["call"], **ns)
    else:
        mb.muon_ns_blocks(state["call"], **ns)


# ------------------------------------------------------------ the plain form

def _wide(x):
    """Blocks in 32 bits, oriented so that rows <= columns."""
    x = x.float()
    return x if x.shape[-2] <= x.shape[-1] else x.transpose(-1, -2)


def _plain_ns(x, steps, coeffs):
    """All iterates of the orthogonalisation, the last one being its result."""
    a, b, c = coeffs
    norm = x.square().sum((-2, -1), keepdim=True).sqrt()
    xs = [x / (norm + EPS)]
    for _ in range(steps):
        x = xs[-1]
        g = x @ x.transpose(-1, -2)
        xs.append(a * x + (b * g + c * (g @ g)) @ x)
    return xs, norm


def _plain_vjp(x, y, steps, coeffs):
    a, b, c = coeffs
    xs, norm = _plain_ns(x, steps, coeffs)
    for z in reversed(xs[:-1]):
        g = z @ z.transpose(-1, -2)
        s = y @ z.transpose(-1, -2)
        s = s + s.transpose(-1, -2)
        t = b * s + c * (s @ g + g @ s)
        y = a * y + (b * g + c * (g @ g)) @ y + t @ z
    inv = 1 / (norm + EPS)
    return inv * (y - xs[0] * (y * x).sum((-2, -1), keepdim=True) / norm)


def _plain(state, k):
    case = state["case"]
    steps, coeffs, kind = case["steps"], COEFFS[case["coeffs"]], k["kind"]
    x = _blocks(k["x"], case, kind)
    tall = x.shape[-2] > x.shape[-1]
    if case["op"] == "step":
        k["m"].mul_(BETA).add_(k["x"].float())
        x = _blocks(k["x"].float() + BETA * k["m"], case, kind)
        o = _plain_ns(_wide(x), steps, coeffs)[0][-1]
    elif case["op"] == "vjp":
        o = _plain_vjp(_wide(x), _wide(_blocks(k["y"], case, kind)), steps, coeffs)
    else:
        o = _plain_ns(_wide(x), steps, coeffs)[0][-1]
    o = o.transpose(-1, -2) if tall else o
    if case["op"] == "step":
        w = _blocks(k["w"], case, kind)
        w.copy_(w.float() - LR * o)
    else:
        _blocks(k["out"], case, kind).copy_(o)


def run(state):
    if own:
        _run_own(state)
    else:
        [_plain(state, k) for k in state["kinds"]]
    if state["case"]["op"] == "step":
        return {"w": [k["w"] for k in state["kinds"]], "m": [k["m"] for k in state["kinds"]]}
    return [k["out"] for k in state["kinds"]]


# ---------------------------------------------------------------- accounting

def work(case):
    m, n = sorted((case["dim"], case["width"]))
    blocks = case["layers"] * case["heads"] * (case["rows_mats"] + case["cols_mats"])
    size, osize = (2 if d == "bf16" else 4 for d in (case["dtype"], case["out"]))
    five = case["coeffs"] == "muon"
    # X enters through its m x m Gram matrix alone, and the result is a matrix function of that
    # matrix times X: one symmetric product over n, (3 or 2) symmetric m x m products a step
    # beside the accumulation of the function, and one product over n
    gram, apply = m * m * n, 2 * m * m * n
    square = case["steps"] * (4 if five else 3) * m ** 3
    if case["op"] == "ns":
        per = size + osize
        flops = gram + apply + square
    elif case["op"] == "vjp":
        per = 2 * size + osize
        flops = gram + 2 * m * m * n + 2 * apply + 3 * square
    else:
        per = size + 8 + 2 * osize
        flops = gram + apply + square
    return {"bytes": float(blocks * m * n * per), "flops": float(blocks * flops)}


# ------------------------------------------------- the definition in 64 bits

def _exact_ns(x, case):
    """ns(x) as z <- (a I + g (b I + c g)) z with g = z z^T, or from the right for tall blocks."""
    a, b, c = (float(torch.tensor(v)) for v in COEFFS[case["coeffs"]])
    z = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + EPS)
    tall = z.shape[-2] > z.shape[-1]
    eye = torch.eye(min(z.shape[-2:]), dtype=z.dtype, device=z.device)
    for _ in range(case["steps"]):
        g = z.mT @ z if tall else z @ z.mT
        q = a * eye + g @ (b * eye + c * g)
        z = z @ q if tall else q @ z
    return z


def exact(case, seed):
    state = prepare(case, seed)
    res, mom = [], []
    for k in state["kinds"]:
        x = _blocks(k["x"], case, k["kind"]).double()
        if case["op"] == "ns":
            res.append(_back(_exact_ns(x, case), case, k["kind"]))
        elif case["op"] == "vjp":
            y = _blocks(k["y"], case, k["kind"]).double()
            x.requires_grad_(True)
            (_exact_ns(x, case) * y).sum().backward()
            res.append(_back(x.grad, case, k["kind"]))
        else:
            beta = float(torch.tensor(BETA))
            m = beta * k["m"].double() + k["x"].double()
            u = _blocks(k["x"].double() + beta * m, case, k["kind"])
            res.append(k["w"].double() - float(torch.tensor(LR)) * _back(_exact_ns(u, case), case, k["kind"]))
            mom.append(m)
    return {"w": res, "m": mom} if case["op"] == "step" else res


def _back(blocks, case, kind):
    """The matrices that the blocks (matrices, heads, rows, columns) are parts of."""
    return blocks.flatten(1, 2) if kind == 0 else blocks.permute(0, 2, 1, 3).flatten(2, 3)
