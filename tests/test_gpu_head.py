"""The head's loss and its gradient on the GPU, against float64, with the bounds
that oracle/training_oracle.py derives; and one training step of experts and head
through to the optimizer's calls."""
import numpy as np
import pytest
import torch

import oracle as orc
from muon_newton_schulz_02_amd import binding as mb
from training_cases import HEAD_LARGE, HEAD_LONG, HEAD_TILES, HEAD_TILES_CAPS

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, dtype, gen, pad=0, scale=1.0, lead=0):
    """rows x cols in a wider buffer whose padding holds NaN, `lead` elements after its start."""
    buf = torch.full((lead + rows * (cols + pad),), float("nan"), dtype=dtype)
    t = buf[lead:].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=gen) * scale)
    return buf.cuda()[lead:].view(rows, cols + pad)[:, :cols]


def check(got, want, tol, dtype, what):
    step = torch.finfo(dtype).eps / 2
    tol = tol + step * (np.abs(want) + tol) + 1e-45
    g = np64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN in other places"
    with np.errstate(invalid="ignore"):
        worst = np.nanmax(np.abs(g - want) / tol) if g.size else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} times the tolerance"


def case(rows, dim, vocab, dtype, *, cap=0.0, ignored=0.0, pad=0, lead=0, scale=1.0, seed=0, lse_too=True, stray=False):
    dt = DTYPES[dtype]
    gen = torch.Generator().manual_seed(seed)
    x, w = matrix(rows, dim, dt, gen, pad, scale, lead), matrix(vocab, dim, dt, gen, pad, dim ** -0.5 * 2, lead)
    t = torch.randint(vocab, (rows,), generator=gen)
    t[torch.rand(rows, generator=gen) < ignored] = -100
    if stray and rows > 2:
        t[0], t[rows // 2] = vocab, -5
    off = (t < 0) | (t >= vocab)
    x[off.cuda()] = float("nan")                   # what ignored rows hold does not matter
    g, h = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
    g[off] = float("nan")
    h[off] = float("inf")
    t, g, h = t.cuda(), g.cuda(), (h.cuda() if lse_too else None)
    loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    gx, gw = matrix(rows, dim, dt, gen, pad, lead=lead), matrix(vocab, dim, dt, gen, pad, lead=lead)
    mb.muon_head_loss(x, w, t, loss, lse, softcap=cap)
    mb.muon_head_loss_vjp(x, w, t, lse, g, gx, gw, grad_lse=h, softcap=cap)
    torch.cuda.synchronize()
    want = orc.training.head(np.nan_to_num(np64(x)), np64(w), t.cpu().numpy(), cap, -100, np.nan_to_num(np64(g)),
                             None if h is None else np.nan_to_num(np64(h), posinf=0.0),
                             half_step=torch.finfo(dt).eps / 2)
    for name, got, odt in (("loss", loss, torch.float32), ("lse", lse, torch.float32), ("grad_x", gx, dt), ("grad_w", gw, dt)):
        check(got, want[name], want["tol_" + name], odt, name)
    return x, w, t, lse, g, h, gx, gw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("rows,dim,vocab", [
    (1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (5, 40, 257), (64, 64, 256), (65, 129, 1023), (300, 96, 2500),
    (257, 200, 4097),
])
def test_sizes(rows, dim, vocab, cap, dtype):
    case(rows, dim, vocab, dtype, cap=cap)


@pytest.mark.parametrize("rows,dim,vocab", HEAD_TILES)
@pytest.mark.parametrize("dtype,cap", [(d, c) for d, caps in HEAD_TILES_CAPS.items() for c in caps])
def test_tiles_of_each_size(rows, dim, vocab, dtype, cap):
    x, w, t, *_ = case(rows, dim, vocab, dtype, cap=cap, ignored=0.2, pad=1 if dim % 8 else 0, stray=True, seed=rows)
    assert ((t >= vocab - 131) & (t < vocab)).any()         # targets in the last tile


@pytest.mark.parametrize("rows,dim,vocab", HEAD_LARGE)
@pytest.mark.parametrize("dtype,cap", [("bf16", 15.0), ("bf16", 0.0), ("f32", 15.0)])
def test_gradients_on_the_largest_tiles(rows, dim, vocab, dtype, cap):
    """Against float64 on the GPU; the bounds of oracle/training_oracle.py, element by element."""
    dt, u = DTYPES[dtype], 2.0 ** -24
    gen = torch.Generator().manual_seed(77)
    x, w = matrix(rows, dim, dt, gen), matrix(vocab, dim, dt, gen, scale=dim ** -0.5 * 2)
    t = torch.randint(vocab, (rows,), generator=gen)
    t[torch.rand(rows, generator=gen) < 0.1] = -100
    t, g = t.cuda(), torch.randn(rows, generator=gen).cuda()
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gx, gw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    mb.muon_head_loss(x, w, t, loss, lse, softcap=cap)
    mb.muon_head_loss_vjp(x, w, t, lse, g, gx, gw, softcap=cap)
    seen = t >= 0
    assert (gx[~seen] == 0).all() and (loss[~seen] == 0).all()
    xd, wd, at, gd = x.double()[seen], w.double(), t[seen], g.double()[seen, None]
    row = torch.arange(len(at), device="cuda")
    z = xd @ wd.t()
    tol_z = (dim + 4) * u * (xd.abs() @ wd.abs().t())
    if cap:
        z = cap * torch.tanh(z / cap)
        tol_z += 6 * u * cap
    want = torch.logsumexp(z, 1, keepdim=True)
    d = torch.exp(z - want)
    tol_lse = (d * (tol_z + ((z - z.amax(1, keepdim=True)).abs() + 4) * u)).sum(1, keepdim=True) + 320 * u + 2 * u * want.abs()
    assert ((lse[seen].double() - want[:, 0]).abs() <= 1.01 * tol_lse[:, 0]).all()
    picked = z[row, at]
    assert ((loss[seen].double() - (want[:, 0] - picked)).abs() <= 1.01 * (tol_lse[:, 0] + tol_z[row, at] + 2 * u * picked.abs())
            + u * want[:, 0].abs()).all()
    d *= gd
    tol = d.abs() * (tol_z + tol_lse + ((z - want).abs() + 10) * u)
    d[row, at] -= gd[:, 0]
    tol[row, at] += 2 * u * gd[:, 0].abs()
    if cap:
        slope = 1 - (z / cap) ** 2
        tol = tol * slope + d.abs() * (2 * z.abs() / cap ** 2 * tol_z + 6 * u)
        d *= slope
    step = torch.finfo(dt).eps / 2
    tol += step * (d.abs() + tol) + 2.0 ** -126 * (gd.abs() + 2)
    for got, ref, off in ((gx[seen], d @ wd, tol @ wd.abs() + (vocab + 68) * u * (d.abs() @ wd.abs())),
                          (gw, d.t() @ xd, tol.t() @ xd.abs() + (len(at) + 4) * u * (d.abs().t() @ xd.abs()))):
        off = off + step * (ref.abs() + off) + 1e-30
        assert ((got.double() - ref).abs() <= off).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,lead", [(1, 0), (8, 0), (3, 1), (0, 1)])
def test_strides_and_alignment(pad, lead, dtype):
    case(70, 72, 600, dtype, cap=15.0, ignored=0.2, pad=pad, lead=lead)
    case(33, 77, 515, dtype, ignored=0.2, pad=pad, lead=lead)


@pytest.mark.parametrize("ignored", [0.1, 0.9, 1.1])
@pytest.mark.parametrize("rows", [7, 700])
def test_ignored_rows(rows, ignored):
    case(rows, 48, 900, "bf16", ignored=ignored, stray=True)
    case(rows, 48, 900, "f32", ignored=ignored, stray=True, lse_too=False)


@pytest.mark.parametrize("dtype,rows,vocab", [("f32", 600, 450_001), ("bf16", 1210, 230_000)])
def test_a_vocabulary_in_pieces(dtype, rows, vocab):
    """More columns than one piece of the gradient holds (512 MiB); against float64 on the GPU, elements' bounds as in
    oracle/training_oracle.py: 2^-8 (binary32 (16 + 60) 2^-24) of sum |dl| |w| for what is rounded, and the result's own
    half step."""
    dt = DTYPES[dtype]
    gen = torch.Generator().manual_seed(5)
    x, w = matrix(rows, 16, dt, gen, pad=8), matrix(vocab, 16, dt, gen)
    t = torch.randint(vocab, (rows,), generator=gen).cuda()
    t[::9] = -100
    g = torch.randn(rows, generator=gen).cuda()
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gx, gw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    mb.muon_head_loss(x, w, t, loss, lse)
    args = mb.HeadLossVjpArgs(x, w, t, lse, g, gx, gw)
    assert args.workspace_bytes() < rows * vocab * x.element_size()
    mb.muon_head_loss_vjp(args)
    seen = t >= 0
    xd, wd, at = x.double()[seen], w.double(), t[seen]
    d = xd @ wd.t()
    want = torch.logsumexp(d, 1)
    # the logits' 20 u sum |x| |w| (130 at most), the exponentials' 100 u, the sums' 320 u
    assert (lse[seen].double() - want).abs().max() < (20 * 130 + 420 + 40) * 2.0 ** -24
    d = torch.exp(d - want[:, None]) * g.double()[seen, None]
    d[torch.arange(len(at)), at] -= g.double()[seen]
    part = 2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else (20 * 130 + 900) * 2.0 ** -24
    step = torch.finfo(dt).eps / 2
    for got, ref, reach in ((gx[seen], d @ wd, d.abs() @ wd.abs()), (gw, d.t() @ xd, d.abs().t() @ xd.abs())):
        tol = part * reach + step * (ref.abs() + part * reach) + 1e-30
        assert ((got.double() - ref).abs() <= tol).all()
    assert (gx[~seen] == 0).all()


def test_a_long_vocabulary():
    case(3, 16, 300_001, "bf16", cap=30.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [33.0, 1e3, 1e6, 1e8, 1e20, 3.3e38])
@pytest.mark.parametrize("rows,dim,vocab", [(3, 5, 40), (40, 64, 300), (300, 72, 1030), (1900, 200, 4099)])
def test_large_soft_caps(rows, dim, vocab, cap, dtype):
    """A cap far above the logits leaves them as they are: what its evaluation may be off by goes with the logit, not
    with the cap (oracle/training_oracle.py)."""
    case(rows, dim, vocab, dtype, cap=cap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 64), (300, 64), (600, 2050)])
@pytest.mark.parametrize("far", [2.0, -2.0, 4.0, -4.0, 6.0, -6.0, 8.0, -8.0])
def test_slope_of_the_soft_cap_far_out(far, rows, vocab, dtype):
    """The target's logit at `far` caps, all others 0: its gradient is (p - 1) times a slope of 4 e^(-2 |far|) or so.  The
    slope's relative error is that of e^(2 |l| / cap), four roundings of the exponent and eight more of 2^-24; p's is some
    20 of them; bfloat16: two roundings of half a step.  The gradients of `rows` equal rows are added: as many 2^-24."""
    dt = DTYPES[dtype]
    cap = 2.0
    x, w = torch.ones(rows, 16, dtype=dt, device="cuda"), torch.zeros(vocab, 16, dtype=dt, device="cuda")
    w[33, 5] = far * cap
    t = torch.full((rows,), 33, device="cuda")
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gw = torch.zeros_like(w)
    mb.muon_head_loss(x, w, t, loss, lse, softcap=cap)
    mb.muon_head_loss_vjp(x, w, t, lse, torch.ones(rows, device="cuda"), None, gw, softcap=cap)
    z = cap * np.tanh(far)
    p = np.exp(z) / (vocab - 1 + np.exp(z))
    want = rows * (p - 1) / np.cosh(far) ** 2
    tol = (8 * abs(far) + 28 + rows) * 2.0 ** -24 + (2 * torch.finfo(dt).eps / 2 * 1.01 if dtype == "bf16" else 0.0)
    assert np.abs(np64(gw)[33] / want - 1).max() <= tol


def test_large_logits_and_sure_rows():
    """Logits up to some hundreds: no overflow, p of 1 and 0."""
    case(64, 64, 700, "f32", scale=60.0)
    case(64, 64, 700, "bf16", scale=60.0, cap=15.0)


def test_non_finite_logits():
    gen = torch.Generator().manual_seed(3)
    x, w = matrix(6, 32, torch.float32, gen), matrix(90, 32, torch.float32, gen)
    x[1, 3] = float("nan")
    x[2, 0] = float("inf")
    t = torch.zeros(6, dtype=torch.int64, device="cuda")
    loss, lse = torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda")
    mb.muon_head_loss(x, w, t, loss, lse)
    assert torch.isfinite(loss[[0, 3, 4, 5]]).all() and torch.isnan(loss[1]) and not torch.isfinite(loss[2])
    gx = torch.zeros_like(x)
    mb.muon_head_loss_vjp(x, w, t, lse, torch.ones(6, device="cuda"), gx)
    assert torch.isfinite(gx[[0, 3, 4, 5]]).all() and torch.isnan(gx[1]).all() and torch.isnan(gx[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 15.0, 50.0])
@pytest.mark.parametrize("rows,dim,vocab", [(6, 32, 90), (6, 6, 90), (300, 72, 3000), (900, 200, 4227), (1030, 200, 7299)])
def test_nan_and_infinity_stay_in_their_rows(rows, dim, vocab, cap, dtype):
    """A row with a NaN is NaN.  One with an infinity has infinite logits: without a soft cap its results are not finite;
    with one, for bfloat16, the logits are the cap or minus it, and their slope is 0.  Other rows keep their bits."""
    dt = DTYPES[dtype]
    gen = torch.Generator().manual_seed(51)
    x, w = matrix(rows, dim, dt, gen), matrix(vocab, dim, dt, gen)
    w[w == 0] = 1.0
    t = torch.randint(vocab, (rows,), generator=gen).cuda()
    ones = torch.ones(rows, device="cuda")

    def run(x):
        loss, lse, gx = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(rows, dim, dtype=dt, device="cuda")
        mb.muon_head_loss(x, w, t, loss, lse, softcap=cap)
        mb.muon_head_loss_vjp(x, w, t, lse, ones, gx, softcap=cap)
        return loss, lse, gx

    clean = run(x)
    bad = x.clone()
    a, b, c = 1, rows // 2, rows - 1
    bad[a, dim - 1], bad[b, 0], bad[c, 3] = float("nan"), float("inf"), float("-inf")
    got = run(bad)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[a, b, c]] = False
    for u, v in zip(clean, got):
        assert torch.equal(u[keep], v[keep]) and torch.isfinite(u).all()
    assert torch.isnan(got[0][a]) and torch.isnan(got[1][a]) and torch.isnan(got[2][a]).all()
    for r, column, sign in ((b, 0, 1.0), (c, 3, -1.0)):
        if cap and dtype == "bf16":
            z = cap * np.sign(sign * np64(w)[:, column])
            lse = z.max() + np.log(np.exp(z - z.max()).sum())
            # the cap to 6 u, the exponentials and their sum to 400
            tol = 6 * cap * 2.0 ** -24 + 400 * 2.0 ** -24 + 4 * 2.0 ** -24 * abs(lse)
            assert abs(got[1][r].item() - lse) <= tol and abs(got[0][r].item() - (lse - z[t[r].item()])) <= 2 * tol
            assert (got[2][r] == 0).all()
        elif not cap:
            assert not torch.isfinite(got[1][r]) and not torch.isfinite(got[0][r]) and torch.isnan(got[2][r]).all()


def test_gradient_against_differences():
    """binary32, a step of 2^-6 along a direction: the central difference is off by its third derivative, h^2 / 6 times
    some units, 4e-5 times 10, and the rounding of the loss over the step, 40 rows of 2^-23 * 8 / 2^-6 = 2.4e-3."""
    gen = torch.Generator().manual_seed(8)
    x, w = matrix(40, 24, torch.float32, gen), matrix(300, 24, torch.float32, gen, scale=0.3)
    t = torch.randint(300, (40,), generator=gen).cuda()
    g = torch.rand(40, generator=gen).cuda()

    def value(x, w):
        loss, lse = torch.zeros(40, device="cuda"), torch.zeros(40, device="cuda")
        mb.muon_head_loss(x, w, t, loss, lse, softcap=4.0)
        return (loss.double() * g.double()).sum().item(), lse

    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    mb.muon_head_loss_vjp(x, w, t, value(x, w)[1], g, gx, gw, softcap=4.0)
    h = 2.0 ** -6
    for a, grad in ((0, gx), (1, gw)):
        d = torch.randn(*grad.shape, generator=gen).cuda()
        d /= d.norm()
        up, down = ((x + s * h * d, w) if a == 0 else (x, w + s * h * d) for s in (1, -1))
        assert abs((value(*up)[0] - value(*down)[0]) / (2 * h) - (grad.double() * d.double()).sum().item()) < 3e-3


@pytest.mark.parametrize("g", [1.0 + 2.0 ** -8 + 2.0 ** -12, -(1.0 + 2.0 ** -8 + 2.0 ** -12) / 4096, 1.0 / 1859, 2.0 ** -120 * 1.99, 0.0])
@pytest.mark.parametrize("first", [0, 3])
def test_one_gradient_of_the_loss_for_all_rows_is_not_rounded(g, first):
    """bfloat16.  With small logits p is below 2^-11 and the target's element is -g (1 - p).  Rounded as it is, it
    could be 2^-8 off for all rows alike (the first g here: 2^-8 - 2^-12); in units of g's significand it is -1 or
    next below, off by p or less.  The scale of the result, <got, want> / <want, want>, then is off by 2^-11, and by
    the roundings of 300 x 64 results (and 64 x as many of grad_w's): 2^-8 each at most, independent, 2^-8 / sqrt(19200)
    = 3e-5 together, of which ten times are allowed."""
    gen = torch.Generator().manual_seed(21)
    rows, dim, vocab = 300, 64, 5000
    x, w = matrix(rows, dim, torch.bfloat16, gen, scale=0.05), matrix(vocab, dim, torch.bfloat16, gen, scale=dim ** -0.5)
    t = torch.randint(vocab, (rows,), generator=gen).cuda()
    t[:first] = -100                       # the first rows take no part
    grad = torch.full((rows,), g, device="cuda")
    grad[:first] = float("nan")
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    mb.muon_head_loss(x, w, t, loss, lse)
    mb.muon_head_loss_vjp(x, w, t, lse, grad, gx, gw)
    seen = (t >= 0).cpu().numpy()
    at = t.cpu().numpy()[seen]
    xd, wd = np64(x)[seen], np64(w)
    d = np.exp(xd @ wd.T - np64(lse)[seen, None])
    assert d.max() < 2.0 ** -11
    d[np.arange(len(at)), at] -= 1
    unit = np.float64(np.float32(g))
    for got, want in ((np64(gx)[seen], unit * (d @ wd)), (np64(gw), unit * (d.T @ xd))):
        if g == 0.0:
            assert (got == 0).all()
        else:
            scale = (got / unit * (want / unit)).sum() / np.square(want / unit).sum()
            assert abs(scale - 1) < 2.0 ** -11 + 3e-4


# rows, dim, vocabulary; the products' shapes as in tests/training_cases.py
ROUNDED_ONCE = [(50, 24, 300), (700, 200, 3000), (1030, 333, 7299), (1300, 45, 230_000), *HEAD_LARGE, *HEAD_LONG]


@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("targets", ["any", "few", "one"])
@pytest.mark.parametrize("rows,dim,vocab", ROUNDED_ONCE)
def test_bfloat16_gradients_are_off_by_their_own_rounding_alone(rows, dim, vocab, targets, cap):
    """The gradient with respect to a logit is bfloat16 between the products, but the target's, by far the largest, is
    kept in two parts.  With p of the others at most 0.1 and a sum of their squares of some hundredths, what their rounding
    adds to the gradients is below 2^-8 / sqrt(3) 0.2 of them, against 2^-9.2 for the results' own rounding: 1.03 times
    their error at most, in the mean square.  One target for all rows: the sum of all rows' rests in one row of grad_w."""
    gen = torch.Generator().manual_seed(rows)
    x = matrix(rows, dim, torch.bfloat16, gen, pad=dim % 2)
    w = matrix(vocab, dim, torch.bfloat16, gen, scale=dim ** -0.5)
    t = torch.randint(vocab, (rows,), generator=gen)
    if targets != "any":
        t = torch.tensor([vocab - 2, vocab // 3, 0])[t % 3] if targets == "few" else torch.full_like(t, vocab - 1)
    t[3::10] = -100
    t, g = t.cuda(), (torch.rand(rows, generator=gen) + 0.5).cuda() / rows
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    mb.muon_head_loss(x, w, t, loss, lse, softcap=cap)
    mb.muon_head_loss_vjp(x, w, t, lse, g, gx, gw, softcap=cap)
    seen = t >= 0
    xd, wd, at = x.double()[seen], w.double(), t[seen]
    z = xd @ wd.t()
    if cap:
        z = cap * torch.tanh(z / cap)
    d = torch.softmax(z, 1)
    assert d.amax() < 0.2 and d.square().sum(1).mean() < 0.04
    d[torch.arange(len(at), device="cuda"), at] -= 1
    d *= g.double()[seen, None]
    if cap:
        d *= 1 - (z / cap) ** 2
    for got, want in ((gx[seen], d @ wd), (gw, d.t() @ xd)):
        off, own = (got.double() - want).norm(), (want.bfloat16().double() - want).norm()
        assert off <= 1.03 * own, (off / own).item()


def test_one_gradient_at_a_time_is_the_same():
    x, w, t, lse, g, h, gx, gw = case(130, 96, 1500, "bf16", ignored=0.2)
    a, b = torch.zeros_like(gx), torch.zeros_like(gw)
    mb.muon_head_loss_vjp(x, w, t, lse, g, a, None, grad_lse=h)
    mb.muon_head_loss_vjp(x, w, t, lse, g, None, b, grad_lse=h)
    assert torch.equal(a, gx) and torch.equal(b, gw)


def test_no_rows():
    w, gw = torch.ones(30, 16, device="cuda"), torch.full((30, 16), 3.0, device="cuda")
    x, t, f = torch.zeros(0, 16, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, device="cuda")
    mb.muon_head_loss(x, w, t, f, f.clone())
    mb.muon_head_loss_vjp(x, w, t, f, f, None, gw)
    assert (gw == 0).all()


def test_captured_with_workspaces_and_streams():
    gen = torch.Generator().manual_seed(6)
    rows, dim, vocab = 150, 72, 1300
    x, w = matrix(rows, dim, torch.bfloat16, gen), matrix(vocab, dim, torch.bfloat16, gen)
    t = torch.randint(vocab, (rows,), generator=gen).cuda()
    t[::7] = -100
    g = torch.full((rows,), 1 / rows, device="cuda")
    sets = []
    for _ in range(3):
        loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        gx, gw = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda"), torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
        sets.append((mb.HeadLossArgs(x, w, t, loss, lse), mb.HeadLossVjpArgs(x, w, t, lse, g, gx, gw), (loss, lse, gx, gw)))
    need = max(sets[0][0].workspace_bytes(), sets[0][1].workspace_bytes())
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def both(i, ws=None, stream=None):
        mb.muon_head_loss(sets[i][0], softcap=15.0, workspace=ws, stream=stream)
        mb.muon_head_loss_vjp(sets[i][1], softcap=15.0, workspace=ws, stream=stream)

    both(0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(2, ws[1])
    for _ in range(3):
        for o in sets[2][2]:
            o.fill_(9.0)
        graph.replay()
        both(1, ws[0], side)
        both(0)
        torch.cuda.synchronize()
        for i in (1, 2):
            assert all(torch.equal(a, b) for a, b in zip(sets[0][2], sets[i][2]))
    with pytest.raises(mb.MuonError, match="holds"):
        mb.muon_head_loss(sets[0][0], workspace=ws[0][:256])
    with pytest.raises(mb.MuonError, match="captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            mb.muon_head_loss(sets[0][0])
    torch.cuda.synchronize()


def test_library_workspace_orders_streams_and_is_released():
    gen = torch.Generator().manual_seed(7)
    x, w = matrix(200, 64, torch.float32, gen), matrix(900, 64, torch.float32, gen)
    t = torch.randint(900, (200,), generator=gen).cuda()
    outs = [(torch.zeros(200, device="cuda"), torch.zeros(200, device="cuda")) for _ in range(6)]
    torch.cuda.synchronize()
    for i, (loss, lse) in enumerate(outs):
        if i == 3:
            torch.cuda.synchronize()
            mb.muon_release_workspace()
        mb.muon_head_loss(x, w, t, loss, lse, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0][k], o[k]) for o in outs for k in (0, 1))


def test_allocation_failure_changes_nothing(monkeypatch):
    gen = torch.Generator().manual_seed(9)
    x, w = matrix(20, 16, torch.float32, gen), matrix(50, 16, torch.float32, gen)
    t = torch.randint(50, (20,), generator=gen).cuda()
    loss, lse = torch.full((20,), 4.0, device="cuda"), torch.full((20,), 4.0, device="cuda")
    mb.muon_release_workspace()
    monkeypatch.setenv("MUON_FAULT_ALLOC", "1")
    with pytest.raises(mb.MuonError) as e:
        mb.muon_head_loss(x, w, t, loss, lse)
    assert e.value.status == mb.MUON_ERR_OUT_OF_MEMORY and (loss == 4.0).all()
    monkeypatch.delenv("MUON_FAULT_ALLOC")
    mb.muon_head_loss(x, w, t, loss, lse)
    assert (loss != 4.0).all()


def test_binding_refusals():
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(9, 8, device="cuda")
    t, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    for bad in [dict(t=t.int()), dict(t=t[:3]), dict(w=w.bfloat16()), dict(loss=f.double()), dict(lse=f[:2]), dict(x=x.t()),
                dict(w=w.cpu()), dict(loss=torch.zeros(8, device="cuda")[::2])]:
        a = dict(dict(x=x, w=w, t=t, loss=f, lse=f.clone()), **bad)
        with pytest.raises((ValueError, TypeError)):
            mb.muon_head_loss(a["x"], a["w"], a["t"], a["loss"], a["lse"])
    with pytest.raises(ValueError, match="both None"):
        mb.muon_head_loss_vjp(x, w, t, f, f)
    with pytest.raises(mb.MuonError, match="softcap"):
        mb.muon_head_loss(x, w, t, f, f.clone(), softcap=-1.0)


def test_prebuilt_arguments_hold_the_soft_cap():
    """As a program uses them: softcap and ignore_index given once, with the tensors; gradients of that loss."""
    gen = torch.Generator().manual_seed(41)
    h, head = matrix(60, 48, torch.float32, gen, scale=4.0), matrix(500, 48, torch.float32, gen)
    targets = torch.randint(500, (60,), generator=gen).cuda()
    targets[::6] = 7
    loss, lse, grad_loss = torch.zeros(60, device="cuda"), torch.zeros(60, device="cuda"), torch.ones(60, device="cuda")
    grad_h, grad_head = torch.zeros(60, 48, device="cuda"), torch.zeros(500, 48, device="cuda")
    mb.muon_head_loss(mb.HeadLossArgs(h, head, targets, loss, lse, softcap=5.0, ignore_index=7))
    args = mb.HeadLossVjpArgs(h, head, targets, lse, grad_loss, grad_h, grad_head, softcap=5.0, ignore_index=7)
    ws = torch.empty(args.workspace_bytes(), dtype=torch.uint8, device="cuda")
    mb.muon_head_loss_vjp(args, workspace=ws)
    want = orc.training.head(np64(h), np64(head), targets.cpu().numpy(), 5.0, 7, np64(grad_loss))
    for name, got in (("loss", loss), ("lse", lse), ("grad_x", grad_h), ("grad_w", grad_head)):
        check(got, want[name], want["tol_" + name], torch.float32, name)
    # the same with the call's, and refused where the two differ
    again = [torch.zeros_like(grad_h), torch.zeros_like(grad_head)]
    mb.muon_head_loss_vjp(h, head, targets, lse, grad_loss, *again, softcap=5.0, ignore_index=7)
    mb.muon_head_loss_vjp(args, softcap=5.0, ignore_index=7)
    assert torch.equal(again[0], grad_h) and torch.equal(again[1], grad_head)
    with pytest.raises(ValueError, match="softcap is 4.0 in the call and 5.0"):
        mb.muon_head_loss_vjp(args, softcap=4.0)
    with pytest.raises(ValueError, match="ignore_index"):
        mb.muon_head_loss_vjp(args, ignore_index=-100)
    # built without: the call's, or its defaults
    bare = mb.HeadLossVjpArgs(h, head, targets, lse, grad_loss, *again)
    mb.muon_head_loss_vjp(bare, softcap=5.0, ignore_index=7)
    assert torch.equal(again[0], grad_h) and torch.equal(again[1], grad_head)


def test_a_training_step_from_experts_to_the_optimizer():
    """Experts, the head's loss, their gradients, then the Muon step on the experts and AdamW on the head, as a program
    has them; the gradients against float64 through the whole chain."""
    gen = torch.Generator().manual_seed(11)
    experts, inner, outer, vocab, rows = 4, 96, 64, 700, 240
    counts = [100, 0, 90, 50]
    off = torch.tensor(np.cumsum([0] + counts).astype(np.int32), device="cuda")
    w = matrix(experts * outer, inner, torch.float32, gen, scale=inner ** -0.5).view(experts, outer, inner)
    head = matrix(vocab, outer, torch.float32, gen, scale=outer ** -0.5)
    x = matrix(rows, inner, torch.float32, gen)
    t = torch.randint(vocab, (rows,), generator=gen).cuda()
    t[::5] = -100
    g = torch.full((rows,), 1.0 / int((t >= 0).sum()), device="cuda")
    y, gy = torch.zeros(rows, outer, device="cuda"), torch.zeros(rows, outer, device="cuda")
    loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    gw, gh, gx = torch.zeros_like(w), torch.zeros_like(head), torch.zeros_like(x)
    mb.muon_experts_product(x, w, off, y)
    mb.muon_head_loss(y, head, t, loss, lse, softcap=15.0)
    mb.muon_head_loss_vjp(y, head, t, lse, g, gy, gh, softcap=15.0)
    mb.muon_experts_product_vjp(x, w, off, gy, gx, gw)
    xd, wd, hd = (v.detach().double().cpu().requires_grad_(True) for v in (x, w, head))
    yd = torch.cat([xd[a:b] @ wd[e].t() for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist()))])
    z = 15.0 * torch.tanh(yd @ hd.t() / 15.0)
    ref = torch.nn.functional.cross_entropy(z, t.cpu(), ignore_index=-100)
    ref.backward()
    assert abs((loss.double() * g.double()).sum().item() - ref.item()) < 1e-5     # 192 losses of 7, 2^-22 relative each
    for name, got, want in (("head", gh, hd.grad), ("experts", gw, wd.grad), ("x", gx, xd.grad)):
        # binary32 through three products of 64 to 700 terms: (64 + 700 + 96) 2^-24 = 5e-5 at the very most
        err = (got.double().cpu() - want).norm() / want.norm()
        assert err < 5e-5, (name, err)
    w0, h0 = w.clone(), head.clone()
    mom, m1, m2 = torch.zeros_like(w), torch.zeros_like(head), torch.zeros_like(head)
    mb.muon_step_blocks([w], [gw], [mom], lr=0.02, beta=0.95, nesterov=True, ns_coeffs=(3.4445, -4.7750, 2.0315), ns_steps=5)
    mb.muon_adamw_batched([head.view(-1)], [gh.view(-1)], [m1.view(-1)], [m2.view(-1)], lr=1e-3, beta1=0.9, beta2=0.95,
                          eps=1e-8, weight_decay=0.0, step=1)
    torch.cuda.synchronize()
    assert torch.equal(mom, gw) and not torch.equal(w[0], w0[0]) and torch.equal(w[1], w0[1])   # expert 1 had no rows
    assert not torch.equal(head, h0) and torch.isfinite(w).all() and torch.isfinite(head).all()
