"""Cases for the operators that make the gradients the optimizer reads: products grouped by expert
over packed rows of ragged counts, with their gradients, and the softmax cross entropy of an
output head over a large vocabulary, with its gradient.

Experts: rows of x (tokens x inner, sorted by expert) meet the weight of their expert,
  fwd   y[r] = W_e x[r]                      for offsets[e] <= r < offsets[e + 1]
  dx    grad_x[r] = W_e^T grad_y[r]
  dw    grad_W_e = sum over its rows of grad_y[r] x[r]^T
Rows behind the last offset belong to no expert: their outputs stay as they were.

Head: logits l = x W^T over `vocab` rows of W, z = cap tanh(l / cap) with a soft cap, else l,
  loss  lse[r] = log sum_j exp z_rj, loss[r] = lse[r] - z_r,target; both 0 for ignored rows
  grad  the same, and from grad_loss the gradients with respect to x and W
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100


def _experts(name, op, tokens, experts, inner, outer, dtype="bf16", out="bf16", skew=1.0, spare=0, pad=0):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "inner": inner, "outer": outer,
            "dtype": dtype, "out": out, "skew": skew, "spare": spare, "pad": pad}


def _head(name, op, tokens, inner, vocab, dtype="bf16", cap=0.0, ignored=0.0, pad=0):
    return {"name": name, "op": op, "tokens": tokens, "inner": inner, "vocab": vocab, "dtype": dtype, "cap": cap,
            "ignored": ignored, "pad": pad}


def listed():
    return [
        # one token through two of eight experts of a d24-wide layer: latency, two weights read
        _experts("fwd_token", "fwd", 2, 8, 1536, 6144, skew=0.0),
        # a short batch, down projection: every expert's weight read for a few rows
        _experts("fwd_few", "fwd", 96, 32, 6144, 1536, spare=7),
        # a training batch of the d24 width, up projection, each direction
        _experts("fwd_up", "fwd", 16384, 8, 1536, 6144),
        _experts("dx_up", "dx", 16384, 8, 1536, 6144),
        _experts("dw_up", "dw", 16384, 8, 1536, 6144),
        # many narrow experts, binary32 gradients for the block step, some experts without rows
        _experts("dw_narrow", "dw", 8192, 64, 1536, 128, out="f32", skew=2.0, spare=100),
        # odd sizes, binary32, strided rows
        _experts("dx_ragged_f32", "dx", 3001, 5, 777, 1003, dtype="f32", out="f32", pad=3),
        # one token's loss over the vocabulary of the d24 head: the weight read once
        _head("loss_token", "loss", 1, 1536, 32768, cap=15.0),
        # the loss of a batch, as an evaluation has it
        _head("loss_d24", "loss", 8192, 1536, 32768, cap=15.0),
        # the head's part of a training step
        _head("grad_d24", "grad", 8192, 1536, 32768, cap=15.0, ignored=0.05),
        # a small model in binary32, odd vocabulary
        _head("grad_small_f32", "grad", 1024, 768, 10007, dtype="f32", ignored=0.3),
        # odd sizes, strided rows, most rows ignored
        _head("grad_ragged", "grad", 1337, 333, 20011, ignored=0.6, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    # binary32 products cost several times as much: their cases are smaller
    most = 300e9 if dtype == "bf16" else 60e9
    pad = rng.choice((0, 0, 0, 1, 8))
    if rng.random() < 0.6:
        op = rng.choice(("fwd", "dx", "dw"))
        inner, outer = _log(rng, 24, 6144), _log(rng, 24, 6144)
        experts = _log(rng, 1, min(64, max(1, 150_000_000 // (inner * outer))))
        tokens = _log(rng, 1, max(1, min(16384, int(most / (2 * inner * outer)))))
        out = dtype if op != "dw" or rng.random() < 0.5 else "f32"
        return {"op": op, "tokens": tokens, "experts": experts, "inner": inner, "outer": outer, "dtype": dtype,
                "out": out, "skew": rng.choice((0.0, 1.0, 2.0)), "spare": rng.choice((0, 0, 1, 77)), "pad": pad}
    op = rng.choice(("loss", "grad", "grad"))
    inner, vocab = _log(rng, 24, 2048), _log(rng, 500, 50000)
    tokens = _log(rng, 1, max(1, min(8192, int(2 * most / (2 * inner * vocab)))))
    return {"op": op, "tokens": tokens, "inner": inner, "vocab": vocab, "dtype": dtype,
            "cap": rng.choice((0.0, 15.0, 30.0)), "ignored": rng.choice((0.0, 0.1, 0.7)), "pad": pad}


# ------------------------------------------------------------------ inputs

def _is_head(case):
    return case["op"] in ("loss", "grad")


def _rows(n, cols, pad, dtype, device="cuda"):
    """n zeroed rows of `cols` elements, `pad` more between one row and the next."""
    return torch.zeros(n, cols + pad, dtype=dtype, device=device)[:, :cols]


def _put(values, pad, dtype):
    t = _rows(values.shape[0], values.shape[1], pad, dtype)
    t.copy_(values)
    return t


def _normed(x):
    """Rows of unit root mean square, as a model's norms leave them, a few channels larger than the rest."""
    x[:, ::97] *= 6.0
    return x / x.square().mean(1, keepdim=True).sqrt()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, t, pad = DTYPES[case["dtype"]], case["tokens"], case["pad"]
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if _is_head(case):
        inner, vocab = case["inner"], case["vocab"]
        w = normal(vocab, inner) * inner ** -0.5
        targets = torch.randint(vocab, (t,), generator=gen, device="cuda")
        # some tokens are foreseen well, some badly: the share of the target's direction in x differs by row
        share = 6.0 * torch.rand(t, 1, generator=gen, device="cuda")
        x = _normed(1.5 * normal(t, inner)) + share * w[targets]
        ignored = torch.rand(t, generator=gen, device="cuda") < case["ignored"]
        state["targets"] = torch.where(ignored, IGNORE, targets)
        state["x"], state["w"] = _put(x, pad, dt), _put(w, pad, dt)
        state["loss"], state["lse"] = (torch.zeros(t, device="cuda") for _ in range(2))
        if case["op"] == "grad":
            state["grad_loss"] = torch.full((t,), 1.0 / t, device="cuda")
            state["grad_x"], state["grad_w"] = _rows(t, inner, pad, dt), _rows(vocab, inner, pad, dt)
    else:
        inner, outer, experts, all_rows = case["inner"], case["outer"], case["experts"], t + case["spare"]
        # a router's choice: how well liked an expert is differs by exp(skew N(0, 1))
        liked = torch.exp(case["skew"] * normal(experts))
        chosen = torch.multinomial(liked, t, replacement=True, generator=gen)
        counts = torch.bincount(chosen, minlength=experts)
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        if case["op"] != "dw":
            w = torch.empty(experts, outer, inner + pad, dtype=dt, device="cuda")
            for e in range(experts):
                w[e] = normal(outer, inner + pad) * inner ** -0.5
            state["w"] = w[:, :, :inner]
        if case["op"] != "dx":
            state["x"] = _put(_normed(normal(all_rows, inner)), pad, dt)
        if case["op"] != "fwd":
            state["grad_y"] = _put(1e-3 * normal(all_rows, outer), pad, dt)
        if case["op"] == "dw":
            state["out"] = torch.zeros(experts, outer, inner, dtype=DTYPES[case["out"]], device="cuda")
        else:
            state["out"] = _rows(all_rows, outer if case["op"] == "fwd" else inner, pad, dt)
    if own:
        state["call"] = _arguments(state)
    return state


# ------------------------------------------------- the framework's operators

def _arguments(state):
    """The arguments that a program builds once for its tensors."""
    from muon_newton_schulz_02_amd import binding as mb
    op = state["case"]["op"]
    if op == "fwd":
        return mb.ExpertsArgs(state["x"], state["w"], state["offsets"], state["out"])
    if op == "dx":
        return mb.ExpertsVjpArgs(None, state["w"], state["offsets"], state["grad_y"], grad_x=state["out"])
    if op == "dw":
        return mb.ExpertsVjpArgs(state["x"], None, state["offsets"], state["grad_y"], grad_w=state["out"])
    args = [mb.HeadLossArgs(state["x"], state["w"], state["targets"], state["loss"], state["lse"])]
    if op == "grad":
        args.append(mb.HeadLossVjpArgs(state["x"], state["w"], state["targets"], state["lse"], state["grad_loss"],
                                       grad_x=state["grad_x"], grad_w=state["grad_w"]))
    return args


def _run_own(state):
    from muon_newton_schulz_02_amd import binding as mb
    case = state["case"]
    if case["op"] == "fwd":
        mb.muon_experts_product(state["call"])
    elif case["op"] in ("dx", "dw"):
        mb.muon_experts_product_vjp(state["call"])
    else:
        mb.muon_head_loss(state["call"][0], softcap=case["cap"], ignore_index=IGNORE)
        if case["op"] == "grad":
            mb.muon_head_loss_vjp(state["call"][1], softcap=case["cap"], ignore_index=IGNORE)


# ------------------------------------------------------------ the plain form

def _plain_experts(state):
    op, at = state["case"]["op"], state["offsets"].tolist()
    for e in range(state["case"]["experts"]):
        r = slice(at[e], at[e + 1])
        if op == "fwd":
            state["out"][r] = (state["x"][r].float() @ state["w"][e].float().t()).to(state["out"].dtype)
        elif op == "dx":
            state["out"][r] = (state["grad_y"][r].float() @ state["w"][e].float()).to(state["out"].dtype)
        else:
            state["out"][e] = (state["grad_y"][r].float().t() @ state["x"][r].float()).to(state["out"].dtype)


def _plain_head(state):
    case = state["case"]
    x, w, targets = state["x"].float(), state["w"].float(), state["targets"]
    seen = targets != IGNORE
    at = targets.clamp(min=0)[:, None]
    z = x @ w.t()
    if case["cap"]:
        z = case["cap"] * torch.tanh(z / case["cap"])
    most = z.amax(1, keepdim=True)
    lse = most + (z - most).exp().sum(1, keepdim=True).log()
    state["lse"].copy_(torch.where(seen, lse[:, 0], 0.0))
    state["loss"].copy_(torch.where(seen, (lse - z.gather(1, at))[:, 0], 0.0))
    if case["op"] == "loss":
        return
    g = torch.where(seen, state["grad_loss"], 0.0)[:, None]
    slope = 1 - (z / case["cap"]).square() if case["cap"] else None
    d = z.sub_(lse).exp_().mul_(g)
    d.scatter_add_(1, at, -g)
    if case["cap"]:
        d *= slope
    state["grad_x"].copy_(d @ w)
    state["grad_w"].copy_(d.t() @ x)


def run(state):
    case = state["case"]
    if own:
        _run_own(state)
    elif _is_head(case):
        _plain_head(state)
    else:
        _plain_experts(state)
    if case["op"] == "grad":
        return {k: state[k] for k in ("loss", "lse", "grad_x", "grad_w")}
    if case["op"] == "loss":
        return {k: state[k] for k in ("loss", "lse")}
    return state["out"]


# ---------------------------------------------------------------- accounting

def _used(case):
    """Experts that have rows, on average over the router's choices (exact where all are liked alike)."""
    return case["experts"] * (1 - (1 - 1 / case["experts"]) ** case["tokens"])


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    t, inner = case["tokens"], case["inner"]
    if _is_head(case):
        v = case["vocab"]
        flops, read, rows = 2 * t * v * inner, size * inner * (t + v), 16 * t
        if case["op"] == "loss":
            return {"bytes": float(read + rows), "flops": float(flops)}
        return {"bytes": float(2 * read + rows + 4 * t), "flops": float(3 * flops)}
    outer = case["outer"]
    if case["op"] == "dw":
        w = (2 if case["out"] == "bf16" else 4) * inner * outer * case["experts"]
    else:
        w = size * inner * outer * _used(case)
    return {"bytes": float(w + size * t * (inner + outer)), "flops": float(2 * t * inner * outer)}


# ------------------------------------------------- the definition in 64 bits

def _exact_experts(state):
    case, ends = state["case"], state["offsets"][1:].long()
    out = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    # the expert of every row that has one
    owner = torch.bucketize(torch.arange(case["tokens"], device="cuda"), ends, right=True)
    for e in range(case["experts"]):
        rows = (owner == e).nonzero()[:, 0]
        if case["op"] == "dw":
            out[e] = torch.mm(state["x"][rows].double().t(), state["grad_y"][rows].double()).t()
        elif case["op"] == "fwd":
            out[rows] = torch.mm(state["w"][e].double(), state["x"][rows].double().t()).t()
        else:
            out[rows] = torch.mm(state["w"][e].double().t(), state["grad_y"][rows].double().t()).t()
    return out


def _exact_head(state):
    """Row by row blocks, the gradient through autograd."""
    case, cap = state["case"], state["case"]["cap"]
    grads = case["op"] == "grad"
    w = state["w"].double().requires_grad_(grads)
    loss, lse, grad_x = [], [], []
    step = max(1, 100_000_000 // case["vocab"])
    for r in range(0, case["tokens"], step):
        x = state["x"][r:r + step].double().requires_grad_(grads)
        target = state["targets"][r:r + step]
        with torch.set_grad_enabled(grads):
            z = torch.mm(x, w.t())
            if cap:
                z = torch.tanh(z / cap) * cap
            n = torch.logsumexp(z, 1)
            picked = z[torch.arange(len(target), device="cuda"), target.clamp(min=0)]
            value = (n - picked) * (target != IGNORE)
        loss.append(value.detach())
        lse.append(n.detach() * (target != IGNORE))
        if grads:
            (value * state["grad_loss"][r:r + step].double()).sum().backward()
            grad_x.append(x.grad)
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if grads:
        out.update(grad_x=torch.cat(grad_x), grad_w=w.grad)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_head(state) if _is_head(case) else _exact_experts(state)
