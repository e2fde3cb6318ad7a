"""The block operators on the GPU against the float64 oracle: orthogonalisation
of stacks of small blocks, its gradient, and the Muon step on stacks.

Tolerances (relative Frobenius error of one block).  With G the product over
the steps of max(1, |a|, ...), the growth of a small singular value:

* binary32 results: the values a step stores carry 2^-24 of the iterate's
  norm, which the later steps multiply by at most G; a result of m rows has
  norm about sqrt(m).  Some tens of such roundings (Gram sums, P, the apply
  product) give T32 = 2^-24 (64 + 16 G / sqrt(m)).  A gradient passes the
  same steps twice, and its Gram product with the cotangent: 4 T32.
* bfloat16 results: half a step, 2^-8 of the value, plus what one stage of
  growth up to 512 leaves of the Gram matrix's 2^-24: the Gram error is
  carried on with the square of the growth at the singular values 1/512 and
  less, 512^2 2^-24 = 2^-6 in the worst direction, and on a spectrum without
  a preferred direction 1/sqrt(m) of that in norm, at most 2^-6 / sqrt(m);
  blocks of a few rows, where one direction counts, start again after a growth
  of 48.  TB = 2^-8 + 2^-9.
"""
import ctypes
import sys

import numpy as np
import pytest
import torch

import oracle as orc
from muon_newton_schulz_02_amd import binding as mb

from gpu_helpers import CUBIC, MUON, bits, f32, to_np

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
TB = 2.0 ** -8 + 2.0 ** -9


def _announce(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def _co(coeffs):
    return np.float32(np.asarray(coeffs, dtype=np.float64)).astype(np.float64)


def _gain(coeffs, steps):
    g = 1.0
    for a, b, c in orc.schedule(_co(coeffs), steps):
        g *= max(1.0, max(abs(a + b * x + c * x * x) for x in np.linspace(0, 1.5, 31)))
    return g


def _tol(dtype, m, coeffs, steps, grad=False):
    if dtype == BF:
        return TB
    return 2.0 ** -24 * (64 + 16 * _gain(coeffs, steps) / np.sqrt(m)) * (4 if grad else 1)


def _make(blocks, rows, cols, dtype, gen, kind="dense", pad=0, scale=1.0):
    """A stack view and the tensor it lies in: "dense" blocks in rows, "cols"
    blocks side by side in the columns, "odd" with an odd element offset."""
    val = torch.randn(blocks, rows, cols, generator=gen) * scale
    if kind == "cols":
        base = torch.full((rows, blocks * cols + pad), 7.0).to(dtype).cuda()
        view = base[:, :blocks * cols].unflatten(1, (blocks, cols)).transpose(0, 1)
    elif kind == "odd":
        flat = torch.full((1 + blocks * rows * (cols + pad) + 5,), 7.0).to(dtype).cuda()
        base = flat
        view = flat[1:1 + blocks * rows * (cols + pad)].view(blocks, rows, cols + pad)[:, :, :cols]
    else:
        base = torch.full((blocks, rows, cols + pad), 7.0).to(dtype).cuda()
        view = base[:, :, :cols]
    view.copy_(val.to(dtype))
    return view, base


def _untouched(view, base):
    """Every element of `base` outside `view` still holds 7."""
    rest = base.clone()
    rest.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(7.0)
    assert bool((rest == 7.0).all()), "elements outside the blocks were written"


def _check_blocks(got, ref, tol, what):
    got = to_np(got)
    for b in range(len(ref)):
        e, n = np.linalg.norm(got[b] - ref[b]), np.linalg.norm(ref[b])
        assert np.isfinite(got[b]).all() and e <= tol * n, f"{what} block {b}: {e / max(n, 1e-300):.3e} > {tol:.3e}"


SHAPES = [
    # blocks, rows, cols, kind, pad
    (1, 1, 1, "dense", 0),
    (3, 1, 64, "dense", 0),
    (3, 64, 1, "dense", 0),
    (5, 2, 7, "odd", 1),
    (2, 15, 300, "dense", 0),
    (2, 16, 257, "odd", 0),
    (2, 300, 17, "dense", 3),
    (3, 31, 129, "cols", 0),
    (3, 129, 32, "cols", 0),
    (3, 200, 33, "cols", 5),
    (2, 33, 40, "dense", 0),
    (2, 48, 48, "odd", 3),
    (2, 63, 1000, "dense", 8),
    (2, 64, 64, "dense", 0),
    (12, 64, 768, "dense", 0),
    (2, 65, 96, "dense", 0),
    (2, 90, 1111, "dense", 5),
    (2, 1111, 90, "cols", 2),
    (3, 127, 255, "odd", 0),
    (2, 128, 1536, "dense", 0),
    (2, 1536, 128, "cols", 0),
    (1, 128, 128, "dense", 0),
    (2, 4097, 5, "dense", 0),
]


def _run_ns(x, out, coeffs, steps, **kw):
    mb.muon_ns_blocks([x], [out], ns_coeffs=coeffs if np.ndim(coeffs) == 1 else coeffs[0], ns_steps=steps,
                      ns_schedule=None if np.ndim(coeffs) == 1 else coeffs, **kw)


def _run_vjp(x, y, dx, coeffs, steps, **kw):
    mb.muon_ns_blocks_vjp([x], [y], [dx], ns_coeffs=coeffs if np.ndim(coeffs) == 1 else coeffs[0], ns_steps=steps,
                          ns_schedule=None if np.ndim(coeffs) == 1 else coeffs, **kw)


@pytest.mark.parametrize("xdt,odt", [(BF, BF), (F, F), (F, BF), (BF, F)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}-{s[3]}{s[4]}")
def test_ns_shapes(shape, xdt, odt):
    blocks, rows, cols, kind, pad = shape
    _announce(f"ns {shape} {xdt} {odt}")
    gen = torch.Generator().manual_seed(rows * 7 + cols)
    x, _ = _make(blocks, rows, cols, xdt, gen, kind, pad)
    out, base = _make(blocks, rows, cols, odt, gen, kind, pad)
    _run_ns(x, out, MUON, 5)
    torch.cuda.synchronize()
    ref = [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)]
    _check_blocks(out, ref, _tol(odt, min(rows, cols), MUON, 5), "NS")
    _untouched(out, base)


@pytest.mark.parametrize("xdt,odt", [(BF, BF), (F, F), (F, BF), (BF, F)])
@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}-{s[3]}{s[4]}")
def test_vjp_shapes(shape, xdt, odt):
    blocks, rows, cols, kind, pad = shape
    _announce(f"vjp {shape} {xdt} {odt}")
    gen = torch.Generator().manual_seed(rows * 7 + cols + 1)
    x, _ = _make(blocks, rows, cols, xdt, gen, kind, pad)
    y, _ = _make(blocks, rows, cols, xdt, gen, kind, pad)
    dx, base = _make(blocks, rows, cols, odt, gen, kind, pad)
    _run_vjp(x, y, dx, MUON, 5)
    torch.cuda.synchronize()
    ref = [orc.orthogonalise_vjp(v, w, _co(MUON), 5) for v, w in zip(to_np(x), to_np(y))]
    _check_blocks(dx, ref, _tol(odt, min(rows, cols), MUON, 5, grad=True), "gradient")
    _untouched(dx, base)


SCHEDULE = [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), MUON, (15 / 8, -5 / 4, 3 / 8)]


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("coeffs,steps", [(MUON, 0), (MUON, 1), (MUON, 2), (MUON, 10), (CUBIC, 1), (CUBIC, 12),
                                          (SCHEDULE, 4), ([CUBIC] * 40, 40)],
                         ids=lambda v: str(v) if isinstance(v, int) else "s" if np.ndim(v) > 1 else f"{v[0]}")
def test_steps_and_schedules(coeffs, steps, dt):
    _announce(f"steps {steps} {coeffs[:1]} {dt}")
    gen = torch.Generator().manual_seed(steps)
    for rows, cols in ((20, 100), (100, 700), (300, 50)):
        x, _ = _make(3, rows, cols, dt, gen, scale=1e-3)
        y, _ = _make(3, rows, cols, dt, gen)
        out, dx = torch.empty_like(x), torch.empty_like(x)
        _run_ns(x, out, coeffs, steps)
        _run_vjp(x, y, dx, coeffs, steps)
        torch.cuda.synchronize()
        xs, ys = to_np(x), to_np(y)
        m = min(rows, cols)
        _check_blocks(out, [orc.orthogonalise(v, _co(coeffs), steps) for v in xs], _tol(dt, m, coeffs, steps), "NS")
        _check_blocks(dx, [orc.orthogonalise_vjp(v, w, _co(coeffs), steps) for v, w in zip(xs, ys)],
                      _tol(dt, m, coeffs, steps, grad=True), "gradient")


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("power", [1.0, 2.0])
def test_decaying_spectra(dt, power):
    """Singular values i^-power: the smallest grow by the whole gain."""
    _announce(f"spectra {power} {dt}")
    gen = torch.Generator().manual_seed(5)
    m, n = 96, 400
    u = torch.linalg.qr(torch.randn(2, m, m, generator=gen, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(2, n, m, generator=gen, dtype=torch.float64))[0]
    s = torch.arange(1, m + 1, dtype=torch.float64) ** -power
    x = ((u * s) @ v.transpose(1, 2)).to(dt).cuda()
    y = torch.randn(2, m, n, generator=gen).to(dt).cuda()
    out, dx = torch.empty_like(x), torch.empty_like(x)
    _run_ns(x, out, MUON, 5)
    _run_vjp(x, y, dx, MUON, 5)
    torch.cuda.synchronize()
    _check_blocks(out, [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)], _tol(dt, m, MUON, 5), "NS")
    _check_blocks(dx, [orc.orthogonalise_vjp(v, w, _co(MUON), 5) for v, w in zip(to_np(x), to_np(y))],
                  _tol(dt, m, MUON, 5, grad=True), "gradient")


@pytest.mark.parametrize("xdt,odt", [(BF, BF), (F, BF), (F, F)])
@pytest.mark.parametrize("m,n", [(4, 64), (16, 1024), (64, 768), (128, 300)])
@pytest.mark.parametrize("ratio", [50, 200, 1000])
def test_one_large_singular_value(m, n, ratio, xdt, odt):
    """One singular value and m - 1 at 1/ratio of it: the Gram matrix holds the others' squares least exactly.

    With O = p(A_0) X_0, an error E of A_0 gives p'(l) s E in the m - 1 small directions (s the small singular value
    of X_0, l = s^2).  E is a few roundings of the trace, 1: four of 2^-24 a direction.  O has norm f(s) sqrt(m - 1)
    at least.  Binary32 results start again before the growth passes 48, where E counts (48 / G)^2 as much."""
    _announce(f"one large {m} {n} {ratio} {xdt} {odt}")
    gen = torch.Generator().manual_seed(m + ratio)
    u = torch.linalg.qr(torch.randn(8, m, m, generator=gen, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(8, n, m, generator=gen, dtype=torch.float64))[0]
    sv = torch.full((m,), 1.0 / ratio, dtype=torch.float64)
    sv[0] = 1
    x = ((u * sv) @ v.transpose(1, 2)).to(xdt).cuda()
    out = torch.empty_like(x, dtype=odt)
    _run_ns(x, out, MUON, 5)
    torch.cuda.synchronize()

    def f(s):
        for a, b, c in orc.schedule(_co(MUON), 5):
            s = s * (a + b * s * s + c * s ** 4)
        return s

    s = 1 / ratio / np.sqrt(1 + (m - 1) / ratio ** 2)
    # p(l) = f(s) / s; p'(l) = (f'(s) - f(s) / s) / (2 l), over the values that rounding x spreads s to
    worst = 0.0
    for t in np.linspace(0.8, 1.25, 91) * s:
        h = t * 1e-6
        worst = max(worst, abs((f(t + h) - f(t - h)) / (2 * h) - f(t) / t) / (2 * t) / abs(f(t)))
    e = 4 * 2.0 ** -24 * worst
    tol = TB + e if odt == BF else _tol(F, m, MUON, 5) + e * (48 / 485) ** 2
    _check_blocks(out, [orc.orthogonalise(w, _co(MUON), 5) for w in to_np(x)], tol, "NS")


def test_gradient_against_differences():
    """<dx, d> against central differences of the library's own forward pass (binary32)."""
    _announce("differences")
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(2, 24, 200, generator=gen).cuda()
    y = torch.randn(2, 24, 200, generator=gen).cuda()
    dx, o1, o2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    _run_vjp(x, y, dx, MUON, 5)
    for k in range(4):
        d = torch.randn(2, 24, 200, generator=gen).cuda()
        h = 2.0 ** -7
        _run_ns(x + h * d, o1, MUON, 5)
        _run_ns(x - h * d, o2, MUON, 5)
        torch.cuda.synchronize()
        fd = ((o1 - o2).double() * y.double()).sum((1, 2)) / (2 * h)
        an = (dx.double() * d.double()).sum((1, 2))
        # the outputs are off by T32 of their norm sqrt(24), against y of norm
        # sqrt(24 * 200) in a random direction: about T32 sqrt(24); truncation
        # h^2 times the third derivative along d (relative size 1/14 of x)
        lim = _tol(F, 24, MUON, 5) * 24 ** 0.5 * 4 / h + h * h * dx.double().norm().item() * d.double().norm().item()
        assert (fd - an).abs().max().item() <= lim


def test_zero_nan_and_infinite_blocks_stay_apart():
    _announce("non-finite blocks")
    gen = torch.Generator().manual_seed(2)
    for dt in (BF, F):
        for rows, cols in ((64, 200), (200, 20)):
            x, _ = _make(5, rows, cols, dt, gen)
            y, _ = _make(5, rows, cols, dt, gen)
            x[1] = 0
            x[2, 3, 4] = float("nan")
            x[3, rows - 1, cols - 1] = float("inf")
            out, dx = torch.empty_like(x), torch.empty_like(x)
            _run_ns(x, out, MUON, 5)
            _run_vjp(x, y, dx, MUON, 5)
            torch.cuda.synchronize()
            xs, ys, m = to_np(x), to_np(y), min(rows, cols)
            for b in (0, 4):
                _check_blocks(out[b:b + 1], [orc.orthogonalise(xs[b], _co(MUON), 5)], _tol(dt, m, MUON, 5), "NS")
                _check_blocks(dx[b:b + 1], [orc.orthogonalise_vjp(xs[b], ys[b], _co(MUON), 5)],
                              _tol(dt, m, MUON, 5, grad=True), "gradient")
            assert bool((out[1] == 0).all())
            _check_blocks(dx[1:2], [orc.orthogonalise_vjp(xs[1], ys[1], _co(MUON), 5)], _tol(dt, m, MUON, 5, True), "0")
            for b in (2, 3):
                assert bool(out[b].isnan().all()) and bool(dx[b].isnan().all())


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows,cols", [(40, 90), (64, 768), (128, 200), (300, 100)])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -60, 2.0 ** -110])
def test_rows_of_zeros_and_tiny_rows(rows, cols, dt, small):
    """Whole groups of rows of x (of columns where rows > cols) that are zero, or 2^-60 and 2^-110 of the others: y is
    not, and the gradient there is P y."""
    _announce(f"zero rows {rows} {cols} {dt} {small}")
    gen = torch.Generator().manual_seed(rows)
    x, _ = _make(3, rows, cols, dt, gen)
    y, _ = _make(3, rows, cols, dt, gen)
    part = x if rows <= cols else x.transpose(1, 2)
    part[0, 16:32] *= small
    part[1, :32] *= small
    part[2, 5:6] *= small
    part[2, 20:] *= small
    out, dx = torch.empty_like(x), torch.empty_like(x)
    _run_ns(x, out, MUON, 5)
    _run_vjp(x, y, dx, MUON, 5)
    torch.cuda.synchronize()
    xs, ys, m = to_np(x), to_np(y), min(rows, cols)
    _check_blocks(out, [orc.orthogonalise(v, _co(MUON), 5) for v in xs], _tol(dt, m, MUON, 5), "NS")
    _check_blocks(dx, [orc.orthogonalise_vjp(v, w, _co(MUON), 5) for v, w in zip(xs, ys)],
                  _tol(dt, m, MUON, 5, grad=True), "gradient")


@pytest.mark.parametrize("e", [-100, -60, 60])
@pytest.mark.parametrize("m,n", [(20, 100), (64, 768), (100, 130)])
def test_scale_of_the_cotangent(m, n, e):
    """The gradient is linear in y: 2^e y gives 2^e times it.  The parts of 2^-100 y that leave the range of bfloat16
    are 2^-18 of it at most."""
    _announce(f"cotangent 2^{e} {m} {n}")
    gen = torch.Generator().manual_seed(m)
    x, y = (torch.randn(3, m, n, generator=gen).cuda() for _ in range(2))
    d0, d1 = torch.empty_like(x), torch.empty_like(x)
    _run_vjp(x, y, d0, MUON, 5)
    _run_vjp(x, y * 2.0 ** e, d1, MUON, 5)
    torch.cuda.synchronize()
    _check_blocks(d1, [to_np(d) * 2.0 ** e for d in d0], 2.0 ** -16, "gradient")


def test_tiny_and_large_scales():
    """NS(s x) for s from 2^-40 to 2^40: eps matters below, nothing above."""
    _announce("scales")
    gen = torch.Generator().manual_seed(3)
    x0 = torch.randn(2, 40, 90, generator=gen)
    for e in (-40, -20, 20, 40):
        for dt in (BF, F):
            x = (x0 * 2.0 ** e).to(dt).cuda()
            out = torch.empty(2, 40, 90, dtype=F, device="cuda")
            _run_ns(x, out, MUON, 5)
            torch.cuda.synchronize()
            _check_blocks(out, [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)], _tol(F, 40, MUON, 5), "NS")


def _many(seed, dt, count=37):
    gen = torch.Generator().manual_seed(seed)
    xs, ys = [], []
    for i in range(count):
        blocks, rows, cols = 1 + i % 4, (8, 40, 128, 300)[i % 4], (100, 40, 200, 64)[(i // 2) % 4]
        if min(rows, cols) > 128:
            cols = 100
        xs.append(torch.randn(blocks, rows, cols, generator=gen).to(dt).cuda())
        ys.append(torch.randn(blocks, rows, cols, generator=gen).to(dt).cuda())
    return xs, ys


@pytest.mark.parametrize("dt", [BF, F])
def test_many_stacks_of_mixed_sizes(dt):
    """More stacks than a launch carries in its arguments, in several groups; an empty stack among them."""
    _announce(f"many stacks {dt}")
    xs, ys = _many(4, dt)
    xs.insert(5, torch.empty(0, 8, 100, dtype=dt, device="cuda"))
    ys.insert(5, torch.empty(0, 8, 100, dtype=dt, device="cuda"))
    outs, dxs = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
    mb.muon_ns_blocks(xs, outs, ns_coeffs=MUON, ns_steps=5)
    mb.muon_ns_blocks_vjp(xs, ys, dxs, ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    for x, y, o, d in zip(xs, ys, outs, dxs):
        m = min(x.shape[1:])
        _check_blocks(o, [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)], _tol(dt, m, MUON, 5), "NS")
        _check_blocks(d, [orc.orthogonalise_vjp(v, w, _co(MUON), 5) for v, w in zip(to_np(x), to_np(y))],
                      _tol(dt, m, MUON, 5, grad=True), "gradient")


def test_shared_and_broadcast_inputs():
    """One block read by every block of a stack (stride 0), one cotangent for all."""
    _announce("broadcast")
    gen = torch.Generator().manual_seed(6)
    x1, y1 = torch.randn(1, 30, 70, generator=gen).cuda(), torch.randn(1, 30, 70, generator=gen).cuda()
    x, y = x1.expand(4, 30, 70), y1.expand(4, 30, 70)
    out, dx = torch.empty(4, 30, 70, device="cuda"), torch.empty(4, 30, 70, device="cuda")
    _run_ns(x, out, MUON, 5)
    _run_vjp(x, y, dx, MUON, 5)
    torch.cuda.synchronize()
    _check_blocks(out, [orc.orthogonalise(to_np(x1)[0], _co(MUON), 5)] * 4, _tol(F, 30, MUON, 5), "NS")
    _check_blocks(dx, [orc.orthogonalise_vjp(to_np(x1)[0], to_np(y1)[0], _co(MUON), 5)] * 4,
                  _tol(F, 30, MUON, 5, grad=True), "gradient")


# ------------------------------------------------------------------ the step

def _step_case(shape, wdt, gdt, seed, count=1):
    blocks, rows, cols, kind, pad = shape
    gen = torch.Generator().manual_seed(seed)
    st = []
    for _ in range(count):
        w, wb = _make(blocks, rows, cols, wdt, gen, kind, pad, 0.02)
        g, _ = _make(blocks, rows, cols, gdt, gen, kind, pad)
        m, mbase = _make(blocks, rows, cols, F, gen, kind, pad)
        st.append((w, g, m, wb, mbase))
    return st


def _check_step_stack(w0, g0, m0, w, m, o, *, lr, beta, nesterov, coeffs, steps, scale, wd, kind, wdt):
    for b in range(w0.shape[0]):
        m_ref, u = orc.momentum(m0[b], g0[b], beta, bool(nesterov), kind)
        assert np.array_equal(bits(m[b]), bits(m_ref)), "momentum not bit-exact"
        ref = orc.orthogonalise(u, _co(coeffs), steps)
        tol = TB if wdt == BF else _tol(F, min(ref.shape), coeffs, steps)
        e = orc.rel_frobenius(o[b], ref)
        assert e <= tol, f"update of block {b}: {e:.3e} > {tol:.3e}"
        w_ref = orc.write_back(w0[b], o[b], lr, scale, wdt == BF, wd)
        assert np.array_equal(bits(w[b]), bits(w_ref)), "write-back not bit-exact given O"


@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F, F), (BF, F), (F, BF)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}-{s[3]}{s[4]}")
def test_step_shapes(shape, wdt, gdt):
    _announce(f"step {shape} {wdt} {gdt}")
    lr = f32(0.02)
    (w, g, m, wb, mbase), = _step_case(shape, wdt, gdt, shape[1] * 3 + shape[2])
    w0, g0, m0 = to_np(w), to_np(g), to_np(m)
    o = torch.full(tuple(w.shape), float("nan"), device="cuda")
    mb.muon_step_blocks([w], [g], [m], lr=lr, beta=0.95, nesterov=True, ns_coeffs=MUON, ns_steps=5, updates_out=[o])
    torch.cuda.synchronize()
    _check_step_stack(w0, g0, m0, to_np(w), to_np(m), to_np(o), lr=lr, beta=f32(0.95), nesterov=1, coeffs=MUON,
                      steps=5, scale=1.0, wd=0.0, kind=0, wdt=wdt)
    _untouched(w, wb)
    _untouched(m, mbase)


@pytest.mark.parametrize("wdt", [BF, F])
@pytest.mark.parametrize("nesterov", [0, 1])
@pytest.mark.parametrize("kind", [0, 1])
def test_step_variants(wdt, nesterov, kind):
    """EMA, plain momentum, weight decay, scale rules, per-stack rates and scales, schedules, no steps."""
    _announce(f"step variants {wdt} {nesterov} {kind}")
    cases = [
        dict(scale_rule=mb.SCALE_RMS_MATCH, weight_decay=f32(0.1)),
        dict(scale_rule=mb.SCALE_SQRT_ASPECT, lr_per_stack=[f32(0.01), f32(0.03)]),
        dict(scale_per_stack=[f32(0.5), f32(2.0)], weight_decay=f32(0.01), ns_schedule=SCHEDULE),
        dict(steps=0),
        dict(steps=10),
    ]
    for i, kw in enumerate(cases):
        st = _step_case((3, 200, 48, "cols", 0), wdt, BF, 50 + i) + _step_case((2, 60, 129, "dense", 3), wdt, BF, 60 + i)
        before = [tuple(to_np(t) for t in s[:3]) for s in st]
        outs = [torch.full(tuple(s[0].shape), float("nan"), device="cuda") for s in st]
        kw = dict(kw)
        steps = kw.pop("steps", len(kw["ns_schedule"]) if "ns_schedule" in kw else 5)
        mb.muon_step_blocks([s[0] for s in st], [s[1] for s in st], [s[2] for s in st], lr=f32(0.02), beta=f32(0.9),
                            nesterov=nesterov, ns_coeffs=MUON, ns_steps=steps, momentum_kind=kind,
                            updates_out=outs, **kw)
        torch.cuda.synchronize()
        for k, (s, (w0, g0, m0)) in enumerate(zip(st, before)):
            lr = kw["lr_per_stack"][k] if "lr_per_stack" in kw else f32(0.02)
            sc = kw["scale_per_stack"][k] if "scale_per_stack" in kw else \
                orc.scale_factor(kw.get("scale_rule", 0), *w0.shape[1:])
            _check_step_stack(w0, g0, m0, to_np(s[0]), to_np(s[2]), to_np(outs[k]), lr=lr, beta=f32(0.9),
                              nesterov=nesterov, coeffs=kw.get("ns_schedule", MUON), steps=steps, scale=sc,
                              wd=kw.get("weight_decay", 0.0), kind=kind, wdt=wdt)


def test_step_is_ns_of_the_momentum():
    """The step's exported update equals muon_ns_blocks of U with binary32 results, and
    muon_step_batched on the same blocks gives the same momentum and nearly the same weights."""
    _announce("step against ns and against the whole-matrix step")
    lr = f32(0.02)
    (w, g, m, _, _), = _step_case((4, 128, 512, "dense", 0), F, F, 77)
    w2, m2 = w.clone(), m.clone()
    o = torch.empty(4, 128, 512, device="cuda")
    mb.muon_step_blocks([w], [g], [m], lr=lr, beta=0.95, nesterov=False, ns_coeffs=MUON, ns_steps=5, updates_out=[o])
    ns = torch.empty_like(o)
    _run_ns(m, ns, MUON, 5)  # without Nesterov U is the updated momentum
    mb.muon_step_batched(list(w2), list(g), list(m2), lr=lr, beta=0.95, nesterov=False, ns_coeffs=MUON, ns_steps=5,
                         precision=mb.NS_F32)
    torch.cuda.synchronize()
    assert torch.equal(o, ns)
    assert torch.equal(m, m2)
    t = _tol(F, 128, MUON, 5)
    assert ((w - w2).norm() / (lr * o.norm())).item() <= t + 1e-4  # muon_step_batched's own binary32 gate


# ------------------------------------------- streams, graphs and workspaces

def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32).cpu().numpy()


def test_same_call_same_bits():
    _announce("determinism")
    xs, ys = _many(8, BF, 20)
    outs = []
    for _ in range(3):
        o, d = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
        mb.muon_ns_blocks(xs, o, ns_coeffs=MUON, ns_steps=5)
        mb.muon_ns_blocks_vjp(xs, ys, d, ns_coeffs=MUON, ns_steps=5)
        torch.cuda.synchronize()
        outs.append([_bits(t) for t in o + d])
    for other in outs[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(outs[0], other))


def test_calls_on_two_streams_run_in_call_order():
    """The library's workspace is one per device: calls on two streams follow each other."""
    _announce("two streams")
    xs, ys = _many(11, BF, 24)
    ref = [torch.empty_like(x) for x in xs]
    refd = [torch.empty_like(x) for x in xs]
    mb.muon_ns_blocks(xs, ref, ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    mb.muon_ns_blocks_vjp(xs, ys, refd, ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    sink = torch.zeros(1, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    out, dx = [torch.zeros_like(x) for x in xs], [torch.zeros_like(x) for x in xs]
    torch.cuda.synchronize()
    mb.muon_mfma_probe(200_000, sink, stream=s1)
    mb.muon_ns_blocks(xs, out, ns_coeffs=MUON, ns_steps=5, stream=s1)
    mb.muon_ns_blocks_vjp(xs, ys, dx, ns_coeffs=MUON, ns_steps=5, stream=s2)
    torch.cuda.synchronize()
    assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(out + dx, ref + refd))


def _workspace(args, steps=5, extra=0, **kw):
    return torch.empty(args.workspace_bytes(ns_coeffs=MUON, ns_steps=steps, **kw) + extra, dtype=torch.uint8,
                       device="cuda")


def test_own_workspace_and_its_size():
    _announce("own workspace")
    xs, ys = _many(12, F, 20)
    ref, out = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
    mb.muon_ns_blocks_vjp(xs, ys, ref, ns_coeffs=MUON, ns_steps=5)
    args = mb.VjpBlocksArgs(xs, ys, out)
    ws = _workspace(args, extra=4096)
    n = ws.numel() - 4096
    ws.fill_(0xA5)
    mb.muon_ns_blocks_vjp(args, ns_coeffs=MUON, ns_steps=5, workspace=ws[:n])
    torch.cuda.synchronize()
    assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(out, ref))
    assert bool((ws[n:] == 0xA5).all()), "written past the workspace"
    with pytest.raises(mb.MuonError, match="INVALID_ARGUMENT"):
        mb.muon_ns_blocks_vjp(args, ns_coeffs=MUON, ns_steps=5, workspace=ws[:n - 256])
    with pytest.raises(mb.MuonError, match="UNSUPPORTED"):
        mb.muon_ns_blocks_vjp(args, ns_coeffs=MUON, ns_steps=5, workspace=ws[64:])


def test_captured_calls():
    """Two graphs with workspaces of their own, replayed several times between eager calls."""
    _announce("graphs")
    xs, ys = _many(13, BF, 20)
    outs = [torch.empty_like(x) for x in xs]
    dxs = [torch.empty_like(x) for x in xs]
    st = _step_case((12, 64, 768, "dense", 0), BF, BF, 14, count=3)
    w, g, m = ([s[k] for s in st] for k in range(3))
    hp = dict(lr=f32(0.02), beta=0.95, nesterov=True, ns_coeffs=MUON, ns_steps=5)
    a1, a2, a3 = mb.NsBlocksArgs(xs, outs), mb.VjpBlocksArgs(xs, ys, dxs), mb.StepBlocksArgs(w, g, m)
    ws1, ws2 = _workspace(a1), torch.empty(max(_workspace(a).numel() for a in (a2, a3)), dtype=torch.uint8,
                                           device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with pytest.raises(mb.MuonError, match="UNSUPPORTED"):
        bad = torch.cuda.CUDAGraph()
        with torch.cuda.graph(bad, stream=s):
            mb.muon_ns_blocks(a1, ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s):
        mb.muon_ns_blocks(a1, ns_coeffs=MUON, ns_steps=5, workspace=ws1)
    with torch.cuda.graph(g2, stream=s):
        mb.muon_ns_blocks_vjp(a2, ns_coeffs=MUON, ns_steps=5, workspace=ws2)
        mb.muon_step_blocks(a3, workspace=ws2, **hp)
    # the same calls eagerly on copies, with the library's workspace
    we, me = [t.clone() for t in w], [t.clone() for t in m]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(4):
        for x in xs + ys:
            x.mul_(1.25 if k % 2 else -0.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(side[0]):
            g1.replay()
        with torch.cuda.stream(side[1]):
            g2.replay()
        ref, refd = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
        mb.muon_ns_blocks(xs, ref, ns_coeffs=MUON, ns_steps=5)
        mb.muon_ns_blocks_vjp(xs, ys, refd, ns_coeffs=MUON, ns_steps=5)
        mb.muon_step_blocks(we, g, me, **hp)
        torch.cuda.synchronize()
        for a, b in zip(outs + dxs + w + m, ref + refd + we + me):
            assert np.array_equal(_bits(a), _bits(b)), f"replay {k}"


# Groups of stacks about as large as those that the library runs in two or three
# parts, all but the first on streams of their own: op, result type, stacks
# (blocks, rows, cols).  The parts meet inside a stack, or between two of a
# table in device memory.
PARTED = [
    ("ns", F, [(77, 40, 64), (61, 64, 40)]),
    ("ns", F, [(9, 20, 100)] * 20),
    ("ns", BF, [(530, 70, 80)]),
    ("vjp", F, [(150, 16, 20)]),
    ("vjp", F, [(67, 100, 20), (68, 18, 70)]),
    ("vjp", BF, [(201, 66, 90)]),
    ("step", F, [(131, 33, 70)]),
    ("step", F, [(140, 128, 64)]),
    ("step", BF, [(17, 130, 65)] * 32),
    ("ns", F, [(9, 70, 150)] * 30),
    ("ns", F, [(1030, 12, 30)]),
    ("vjp", F, [(197, 16, 20)]),
    ("vjp", BF, [(129, 66, 90), (130, 100, 70)]),
    ("step", F, [(260, 128, 64)]),
]


def _parted(op, dt, stacks, seed):
    """Arguments, the call and its written tensors."""
    gen = torch.Generator().manual_seed(seed)
    xs = [torch.randn(s, generator=gen).to(dt).cuda() for s in stacks]
    if op == "step":
        ws = [(torch.randn(s, generator=gen) * 0.02).to(dt).cuda() for s in stacks]
        ms = [torch.randn(s, generator=gen).cuda() for s in stacks]
        args = mb.StepBlocksArgs(ws, xs, ms)
        return args, lambda **k: mb.muon_step_blocks(args, lr=f32(0.02), beta=0.95, nesterov=True, ns_coeffs=MUON,
                                                     ns_steps=5, **k), ws + ms, xs
    outs = [torch.empty_like(x) for x in xs]
    if op == "ns":
        args = mb.NsBlocksArgs(xs, outs)
        return args, lambda **k: mb.muon_ns_blocks(args, ns_coeffs=MUON, ns_steps=5, **k), outs, xs
    ys = [torch.randn(s, generator=gen).to(dt).cuda() for s in stacks]
    args = mb.VjpBlocksArgs(xs, ys, outs)
    return args, lambda **k: mb.muon_ns_blocks_vjp(args, ns_coeffs=MUON, ns_steps=5, **k), outs, (xs, ys)


@pytest.mark.parametrize("op,dt,stacks", PARTED, ids=lambda v: v if isinstance(v, str) else f"{len(v)}-{v[0]}"
                         if isinstance(v, list) else str(v)[6:])
def test_parts_on_two_streams_keep_the_bits(op, dt, stacks):
    """A captured call runs on one stream, an eager one in two parts: the same bits, whatever else runs."""
    _announce(f"parted {op} {dt} {stacks[0]} x {len(stacks)}")
    args, call, written, inputs = _parted(op, dt, stacks, 31)
    start = [t.clone() for t in written]
    ws = _workspace(args)

    def reset():
        for t, t0 in zip(written, start):
            t.copy_(t0)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(workspace=ws)
    reset()
    graph.replay()
    torch.cuda.synchronize()
    ref = [t.clone() for t in written]
    if op != "step":
        for k, i in ((0, 0), (0, stacks[0][0] // 2), (len(stacks) - 1, stacks[-1][0] - 1)):
            tol = _tol(dt, min(stacks[k][1:]), MUON, 5, grad=op == "vjp")
            if op == "ns":
                r = orc.orthogonalise(to_np(inputs[k][i]), _co(MUON), 5)
            else:
                r = orc.orthogonalise_vjp(to_np(inputs[0][k][i]), to_np(inputs[1][k][i]), _co(MUON), 5)
            _check_blocks(ref[k][i:i + 1], [r], tol, op)
    # with the library's workspace, its own, and timed; another call of the same kind beside it
    other, call2, written2, _ = _parted(op, dt, stacks, 31)
    ws2 = _workspace(other)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for kw in (dict(), dict(workspace=ws)):
        reset()
        for t, t0 in zip(written2, start):
            t.copy_(t0)
        torch.cuda.synchronize()
        call(stream=s1, **kw)
        call2(stream=s2, workspace=ws2)
        torch.cuda.synchronize()
        for a, b, r in zip(written, written2, ref):
            assert np.array_equal(_bits(a), _bits(r)) and np.array_equal(_bits(b), _bits(r))
    # the parts are joined: work that follows on the stream finds the whole result
    reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        call(stream=s1)
        after = [t.clone() for t in written]
        for t in written:
            t.zero_()
    torch.cuda.synchronize()
    assert all(np.array_equal(_bits(a), _bits(r)) for a, r in zip(after, ref))
    assert all(bool((t == 0).all()) for t in written)


@pytest.mark.parametrize("blocks,m,n", [(300, 64, 768), (301, 40, 768), (200, 100, 300)])
def test_parts_of_a_gradient_at_different_stages(blocks, m, n):
    """One part of a gradient may be at a backward stage while the other is at a forward one, whose Gram partials are
    shorter: neither touches the other's."""
    _announce(f"stages apart {blocks} {m} {n}")
    args, call, (dx,), _ = _parted("vjp", F, [(blocks, m, n)], 32)
    ws = _workspace(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    ref = _bits(dx)
    for _ in range(8):
        dx.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert np.array_equal(_bits(dx), ref)


def _plain64(x, coeffs, steps):
    """NS of a batch in float64 (wide or tall)."""
    x = x.double()
    if x.shape[1] > x.shape[2]:
        return _plain64(x.transpose(1, 2), coeffs, steps).transpose(1, 2)
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    for a, b, c in orc.schedule(_co(coeffs), steps):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("blocks,rows,cols", [(300_001, 2, 3), (1 << 20, 1, 1), (2, 64, 65536), (1, 65536, 3),
                                              (1, 128, 65536)])
def test_largest_sizes(blocks, rows, cols, dt):
    _announce(f"large {blocks} {rows} {cols} {dt}")
    gen = torch.Generator().manual_seed(15)
    x = torch.randn(blocks, rows, cols, generator=gen).to(dt).cuda()
    out = torch.empty_like(x)
    _run_ns(x, out, MUON, 5)
    ref = _plain64(x, MUON, 5)
    err = (out.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert err.max().item() <= _tol(dt, min(rows, cols), MUON, 5)
    mb.muon_release_workspace()


@pytest.mark.parametrize("dt", [BF, F])
def test_offsets_past_32_bits(dt):
    """Blocks more than 2^32 elements apart, and the longest row stride in both orientations."""
    _announce(f"offsets {dt}")
    gen = torch.Generator().manual_seed(16)
    far = 2 ** 32 + 24
    for rows, cols in ((40, 200), (200, 40)):
        bufs = [torch.empty(far + rows * cols, dtype=dt, device="cuda") for _ in range(2)]
        x, out = (b.as_strided((2, rows, cols), (far, cols, 1)) for b in bufs)
        x.copy_(torch.randn(2, rows, cols, generator=gen).to(dt))
        _run_ns(x, out, MUON, 5)
        torch.cuda.synchronize()
        _check_blocks(out, [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)], _tol(dt, 40, MUON, 5), "far")
        del x, out, bufs
    ld = 2 ** 21
    for rows, cols in ((300, 20), (120, 300)):
        bufs = [torch.empty((rows - 1) * ld + cols, dtype=dt, device="cuda") for _ in range(3)]
        x, y, out = (b.as_strided((1, rows, cols), (0, ld, 1)) for b in bufs)
        x.copy_(torch.randn(1, rows, cols, generator=gen).to(dt))
        y.copy_(torch.randn(1, rows, cols, generator=gen).to(dt))
        _run_vjp(x, y, out, MUON, 5)
        torch.cuda.synchronize()
        ref = [orc.orthogonalise_vjp(to_np(x)[0], to_np(y)[0], _co(MUON), 5)]
        _check_blocks(out, ref, _tol(dt, min(rows, cols), MUON, 5, grad=True), "stride")
        del x, y, out, bufs
    torch.cuda.empty_cache()


@pytest.mark.parametrize("count", [16, 17, 96, 97, 230])
def test_table_launches(count):
    """Up to 16 stacks in a launch's arguments, 96 pointers and four shapes a table launch above."""
    _announce(f"tables {count}")
    gen = torch.Generator().manual_seed(count)
    xs = [torch.randn(1 + i % 2, 9 + i % 7, 17 + i % 5, generator=gen).cuda() for i in range(count)]
    outs = [torch.empty_like(x) for x in xs]
    mb.muon_ns_blocks(xs, outs, ns_coeffs=CUBIC, ns_steps=3)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        _check_blocks(o, [orc.orthogonalise(v, _co(CUBIC), 3) for v in to_np(x)],
                      _tol(F, min(x.shape[1:]), CUBIC, 3), "NS")


def test_thousands_of_stacks():
    _announce("20000 stacks")
    gen = torch.Generator().manual_seed(40)
    base = torch.randn(20000, 1, 6, 9, generator=gen).cuda()
    out = torch.empty_like(base)
    mb.muon_ns_blocks(list(base), list(out), ns_coeffs=MUON, ns_steps=5)
    ref = _plain64(base[:, 0], MUON, 5)
    err = (out[:, 0].double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
    assert err.max().item() <= _tol(F, 6, MUON, 5)


def test_calls_from_two_threads():
    """Calls made at once share the library's workspace one after another."""
    import threading

    _announce("threads")
    cases = [_parted("ns", F, [(77, 40, 64), (61, 64, 40)], 41), _parted("vjp", BF, [(30, 66, 90), (5, 20, 300)], 42)]
    ref = []
    for _, call, written, _ in cases:
        call()
        torch.cuda.synchronize()
        ref.append([_bits(t) for t in written])
        for t in written:
            t.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(k):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for _ in range(20):
                cases[k][1](stream=stream)
            stream.synchronize()
        except Exception as e:  # handed to the test below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, _, written, _), r in zip(cases, ref):
        assert all(np.array_equal(_bits(t), b) for t, b in zip(written, r))


def test_timing_counts_the_passes():
    """With per-kernel timing a call runs on one stream, in the classes of the whole-matrix step, to the same bits."""
    _announce("timing")
    args, call, written, _ = _parted("step", F, [(131, 33, 70)], 43)
    start = [t.clone() for t in written]
    call()
    torch.cuda.synchronize()
    ref = [_bits(t) for t in written]
    for t, t0 in zip(written, start):
        t.copy_(t0)
    mb.muon_timing_enable(True)
    try:
        call()
        torch.cuda.synchronize()
        launches = {k: n for k, (_, n) in mb.muon_timing_read().items()}
    finally:
        mb.muon_timing_enable(False)
    assert all(np.array_equal(_bits(t), r) for t, r in zip(written, ref))
    assert launches["momentum"] == 1 and launches["gram"] == 1  # two stages: the first one's gram pass has the momentum
    assert launches["poly"] == 2 and launches["combine"] == 2


def test_fault_hook_changes_nothing(monkeypatch):
    _announce("allocation failure")
    x = torch.randn(3, 50, 80).cuda()
    out = torch.full((3, 50, 80), 3.0, device="cuda")
    torch.cuda.synchronize()
    mb.muon_release_workspace()
    monkeypatch.setenv("MUON_FAULT_ALLOC", "1")
    with pytest.raises(mb.MuonError, match="OUT_OF_MEMORY"):
        _run_ns(x, out, MUON, 5)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    monkeypatch.delenv("MUON_FAULT_ALLOC")
    _run_ns(x, out, MUON, 5)
    torch.cuda.synchronize()
    _check_blocks(out, [orc.orthogonalise(v, _co(MUON), 5) for v in to_np(x)], _tol(F, 50, MUON, 5), "NS")


def test_training_with_heads_and_the_rest():
    """A run of them together: the attention heads of a layer by muon_step_blocks, its MLP by
    muon_step_batched, the embedding by muon_adamw_batched, three steps; and the gradient of the
    heads' orthogonalisation as a weight parametrisation."""
    _announce("together")
    gen = torch.Generator().manual_seed(21)
    heads, dim, width = 4, 32, 96
    q = (torch.randn(heads * dim, width, generator=gen) * 0.1).cuda()
    o = (torch.randn(width, heads * dim, generator=gen) * 0.1).cuda()
    up = (torch.randn(2 * width, width, generator=gen) * 0.1).cuda()
    emb = (torch.randn(50, width, generator=gen) * 0.1).cuda()
    mom = [torch.zeros_like(t) for t in (q, o, up)]
    av, sq = torch.zeros_like(emb), torch.zeros_like(emb)

    def rows(t):
        return t.view(heads, dim, width)

    def cols(t):
        return t.unflatten(1, (heads, dim)).transpose(0, 1)

    ref = {"q": to_np(q), "o": to_np(o), "mq": to_np(mom[0]), "mo": to_np(mom[1])}
    hp = dict(lr=f32(0.02), beta=f32(0.95), nesterov=True, ns_coeffs=MUON, ns_steps=5)
    for step in range(1, 4):
        gs = [torch.randn(t.shape, generator=gen).cuda() for t in (q, o, up, emb)]
        mb.muon_step_blocks([rows(q), cols(o)], [rows(gs[0]), cols(gs[1])], [rows(mom[0]), cols(mom[1])],
                            weight_decay=f32(0.1), **hp)
        mb.muon_step_batched([up], [gs[2]], [mom[2]], precision=mb.NS_F32, **hp)
        mb.muon_adamw_batched([emb], [gs[3]], [av], [sq], lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=step)
        torch.cuda.synchronize()
        gq, go = to_np(gs[0]), to_np(gs[1])
        for h in range(heads):
            for name, mname, g, sl in (("q", "mq", gq, np.s_[h * dim:(h + 1) * dim, :]),
                                       ("o", "mo", go, np.s_[:, h * dim:(h + 1) * dim])):
                r = orc.muon_step(ref[name][sl], g[sl], ref[mname][sl], lr=hp["lr"], beta=hp["beta"], nesterov=True,
                                  coeffs=_co(MUON), steps=5, weight_decay=f32(0.1), param_bf16=False)
                ref[name][sl], ref[mname][sl] = r.w, r.m
        for name, t in (("q", q), ("o", o)):
            # three updates of norm lr |O|, each off by T32
            lim = 3 * hp["lr"] * _tol(F, dim, MUON, 5) * np.sqrt(heads * dim) * 2 + 1e-6 * np.linalg.norm(ref[name])
            assert np.linalg.norm(to_np(t) - ref[name]) <= lim
    # q as NS(v), loss <NS(v) t, t'>: the gradient with respect to v
    t, t2 = torch.randn(width, 7, generator=gen).cuda(), torch.randn(heads * dim, 7, generator=gen).cuda()
    out, dv = torch.empty_like(q), torch.empty_like(q)
    mb.muon_ns_blocks([rows(q)], [rows(out)], ns_coeffs=MUON, ns_steps=5)
    mb.muon_ns_blocks_vjp([rows(q)], [rows(t2 @ t.T)], [rows(dv)], ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    qn, yn = to_np(q), to_np(t2 @ t.T)
    for h in range(heads):
        sl = np.s_[h * dim:(h + 1) * dim]
        _check_blocks(dv[None, sl], [orc.orthogonalise_vjp(qn[sl], yn[sl], _co(MUON), 5)],
                      _tol(F, dim, MUON, 5, grad=True), "gradient")


# ------------------------------------------------- norms that leave the range

@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows,cols", [(64, 768), (768, 128), (20, 30)])
@pytest.mark.parametrize("coeffs,steps", [(MUON, 5), (MUON, 0), (CUBIC, 1)], ids=lambda v: str(v))
def test_norm_that_overflows_gives_nan(rows, cols, dt, coeffs, steps):
    """A block whose elements, and whose rows' squared norms, are finite while the sum of the squares is not; a block
    with an infinite element.  Both are NaN throughout, after any number of steps; the blocks beside them are not."""
    _announce(f"norm overflow {rows} {cols} {dt} {steps}")
    gen = torch.Generator().manual_seed(rows + steps)
    val = torch.randn(4, rows, cols, generator=gen)
    # a row's (or column's) squared norm stays below 2^127 and that of the whole block is above 2^128
    short, long = min(rows, cols), max(rows, cols)
    e = int(np.floor((127 - np.log2(long)) / 2))
    assert 2 * e + np.log2(long) < 127.5 and 2 * e + np.log2(rows * cols) > 128, "block too small for the case"
    val[1] = torch.sign(val[1]) * 2.0 ** e
    val[2, rows - 1, 0] = float("inf")
    x, y = val.to(dt).cuda(), torch.randn(4, rows, cols, generator=gen).to(dt).cuda()
    assert bool(x[1].isfinite().all())
    out, dx = torch.empty_like(x), torch.empty_like(x)
    _run_ns(x, out, coeffs, steps)
    _run_vjp(x, y, dx, coeffs, steps)
    # the step: U = g where the momentum starts at zero without Nesterov
    w, m, o = torch.zeros_like(x), torch.zeros(4, rows, cols, device="cuda"), torch.zeros(4, rows, cols, device="cuda")
    mb.muon_step_blocks([w], [x], [m], lr=f32(0.5), beta=0.5, nesterov=False, ns_coeffs=coeffs, ns_steps=steps,
                        updates_out=[o])
    torch.cuda.synchronize()
    assert torch.equal(m, x.float())
    for t in (out, dx, w, o):
        assert bool(t[1].isnan().all()) and bool(t[2].isnan().all())
    xs, ys = to_np(x), to_np(y)
    for b in (0, 3):
        ref = [orc.orthogonalise(xs[b], _co(coeffs), steps)]
        _check_blocks(out[b:b + 1], ref, _tol(dt, short, coeffs, steps), "NS")
        _check_blocks(o[b:b + 1], ref, _tol(dt, short, coeffs, steps), "step")
        _check_blocks(dx[b:b + 1], [orc.orthogonalise_vjp(xs[b], ys[b], _co(coeffs), steps)],
                      _tol(dt, short, coeffs, steps, grad=True), "gradient")


def test_more_threads_than_a_launch_takes():
    """2^21 blocks of 1 x 5000 take 2^23 apply workgroups of 512 threads, 2^32 in all: they run in slices.  Block b reads
    elements b .. b + 4999 of one buffer, and a row's result is a multiple of the row."""
    n, blocks = 5000, 1 << 20
    _announce(f"2 x {blocks} blocks of 1 x {n}")
    gen = torch.Generator().manual_seed(61)
    base = torch.randn(2 * blocks + n, generator=gen).to(BF).cuda()
    xs = [base[k * blocks:].as_strided((blocks, 1, n), (1, n, 1)) for k in range(2)]
    outs = [torch.empty(blocks, 1, n, dtype=BF, device="cuda") for _ in range(2)]
    mb.muon_ns_blocks(xs, outs, ns_coeffs=CUBIC, ns_steps=3)
    s = 1.0
    for a, b, c in orc.schedule(_co(CUBIC), 3):
        s = s * (a + b * s * s + c * s ** 4)
    worst, chunk = 0.0, 1 << 14
    for x, out in zip(xs, outs):
        for b in range(0, blocks, chunk):
            u, o = x[b:b + chunk, 0].double(), out[b:b + chunk, 0].double()
            o -= u * (s / u.norm(dim=1, keepdim=True))
            worst = max(worst, (o.norm(dim=1).max() / s).item())
    del outs, out, o, u
    mb.muon_release_workspace()
    torch.cuda.empty_cache()
    assert worst <= TB


@pytest.mark.parametrize("kind", ["rows", "cols"])
@pytest.mark.parametrize("dt", [BF, F])
def test_parts_of_one_weight_kept_per_head(dt, kind):
    """Query, key and value of each head one after another in one weight, as three stacks of a call: the bits of the same
    blocks in tensors of their own."""
    _announce(f"fused weight {kind} {dt}")
    heads, dim, width = 5, 24, 70
    gen = torch.Generator().manual_seed(71)
    shape = (heads, 3, dim, width) if kind == "rows" else (width, heads, 3, dim)

    def parts(t):
        return list(t.unbind(1)) if kind == "rows" else [t[:, :, k].transpose(0, 1) for k in range(3)]

    w, g = (torch.randn(shape, generator=gen).to(dt).cuda() for _ in range(2))
    m = torch.randn(shape, generator=gen).cuda()
    own = [[p.contiguous() for p in parts(t)] for t in (w, g, m)]
    hp = dict(lr=f32(0.02), beta=f32(0.95), nesterov=True, ns_coeffs=MUON, ns_steps=5)
    mb.muon_step_blocks(parts(w), parts(g), parts(m), **hp)
    mb.muon_step_blocks(*own, **hp)
    out, dx = torch.zeros_like(w), torch.zeros_like(w)
    ref, refd = ([torch.zeros_like(p) for p in own[0]] for _ in range(2))
    mb.muon_ns_blocks(parts(g), parts(out), ns_coeffs=MUON, ns_steps=5)
    mb.muon_ns_blocks_vjp(parts(g), parts(w), parts(dx), ns_coeffs=MUON, ns_steps=5)
    mb.muon_ns_blocks(own[1], ref, ns_coeffs=MUON, ns_steps=5)
    mb.muon_ns_blocks_vjp(own[1], own[0], refd, ns_coeffs=MUON, ns_steps=5)
    torch.cuda.synchronize()
    for t, r in ((w, own[0]), (m, own[2]), (out, ref), (dx, refd)):
        assert all(np.array_equal(_bits(a), _bits(b)) for a, b in zip(parts(t), r))


@pytest.mark.parametrize("dt", [BF, F])
def test_single_rows_of_any_row_stride(dt):
    """(blocks, 1, cols) views whose row stride, never used, is 0 or the whole matrix."""
    _announce(f"single rows {dt}")
    gen = torch.Generator().manual_seed(72)
    n, cols = 3000, 750  # 2.25 million elements, past the largest row stride
    x, y, out, dx = (torch.randn(n, cols, generator=gen).to(dt).cuda() for _ in range(4))
    views = [t.view(1, n, cols).transpose(0, 1) for t in (x, y, out, dx)]
    assert views[0].stride(1) > 2 ** 21
    _run_ns(views[0], views[2], CUBIC, 3)
    _run_vjp(views[0], views[1], views[3], CUBIC, 3)
    ref, refd = torch.empty_like(x), torch.empty_like(x)
    _run_ns(x.as_strided((n, 1, cols), (cols, 0, 1)), ref.view(n, 1, cols), CUBIC, 3)
    _run_vjp(x.view(n, 1, cols), y.view(n, 1, cols), refd.as_strided((n, 1, cols), (cols, 1, 1)), CUBIC, 3)
    torch.cuda.synchronize()
    assert np.array_equal(_bits(out), _bits(ref)) and np.array_equal(_bits(dx), _bits(refd))
    _check_blocks(out[:5, None], [orc.orthogonalise(v[None], _co(CUBIC), 3) for v in to_np(x[:5])],
                  _tol(dt, 1, CUBIC, 3), "NS")


def test_a_held_back_call_holds_no_other():
    """A large call on a stream that waits for a long time (one spinning thread), and another on a stream of its own, each
    with a workspace of its own: the second ends before the wait does.  Streams may share a hardware queue, whose order
    they then keep, so one of four other streams has to show it."""
    _announce("held back")
    (a, call_a, _, _), (b, call_b, out_b, _) = (_parted("ns", F, [(600, 128, 256)], seed) for seed in (81, 82))
    ws_a, ws_b = _workspace(a), _workspace(b)
    streams = [torch.cuda.Stream() for _ in range(5)]
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    call_b(workspace=ws_b)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    ref = [_bits(t) for t in out_b]
    ev[0].record()
    torch.cuda._sleep(1_000_000)
    ev[1].record()
    torch.cuda.synchronize()
    cycles = int(1_000_000 * 100 / ev[0].elapsed_time(ev[1]))  # 100 ms
    before = 0
    for s in streams[1:]:
        for t in out_b:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            torch.cuda._sleep(cycles)
        waited, done_b = torch.cuda.Event(), torch.cuda.Event()
        waited.record(streams[0])
        call_a(workspace=ws_a, stream=streams[0])
        call_b(workspace=ws_b, stream=s)
        done_b.record(s)
        done_b.synchronize()
        before += not waited.query()
        torch.cuda.synchronize()
        assert all(np.array_equal(_bits(t), r) for t, r in zip(out_b, ref))
    assert before > 0


def test_an_earlier_error_is_not_this_call_s():
    """HIP keeps a thread's last error until it is asked for: a refused call before (a device that is not there) is not
    taken for a failed launch."""
    _announce("earlier error")
    hip = ctypes.CDLL("libamdhip64.so")
    lr = f32(0.02)
    (w, g, m, _, _), = _step_case((4, 40, 96, "dense", 0), BF, BF, 91)
    w2, m2 = w.clone(), m.clone()
    outs = [torch.full((4, 40, 96), float("nan"), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for t in ((w, m, outs[0]), (w2, m2, outs[1])):
        if t[0] is w:
            assert hip.hipSetDevice(999) != 0
        mb.muon_step_blocks([t[0]], [g], [t[1]], lr=lr, beta=0.95, nesterov=True, ns_coeffs=MUON, ns_steps=5,
                            updates_out=[t[2]])
    torch.cuda.synchronize()
    for a, b in ((w, w2), (m, m2), (outs[0], outs[1])):
        assert np.array_equal(_bits(a), _bits(b))


# -------------------------------------- the stages, against binary32 iterates

def _iterates(x, y, coeffs, steps):
    """NS of a batch and its gradient along y, by the iteration and its reverse, in the batch's type."""
    if x.shape[1] > x.shape[2]:
        return tuple(t.transpose(1, 2) for t in _iterates(x.transpose(1, 2), y.transpose(1, 2), coeffs, steps))
    norm = x.flatten(1).norm(dim=1)[:, None, None]
    xs = [x / (norm + 1e-7)]
    sched = orc.schedule(_co(coeffs), steps)
    for a, b, c in sched:
        z = xs[-1]
        g = z @ z.transpose(1, 2)
        xs.append(a * z + (b * g + c * (g @ g)) @ z)
    for (a, b, c), z in zip(reversed(sched), reversed(xs[:-1])):
        g = z @ z.transpose(1, 2)
        s = y @ z.transpose(1, 2)
        s = s + s.transpose(1, 2)
        y = a * y + (b * g + c * (g @ g)) @ y + (b * s + c * (s @ g + g @ s)) @ z
    inv = 1 / (norm + 1e-7)
    return xs[-1], inv * (y - xs[0] * (y * x).sum((1, 2), keepdim=True) / norm)


def _structured(rows, cols, gen):
    """Blocks with a few large directions: name, batch of four."""
    m, n = sorted((rows, cols))
    r = torch.randn(4, m, n, generator=gen)
    one = torch.randn(4, m, 1, generator=gen) @ torch.randn(4, 1, n, generator=gen)
    many = torch.randn(4, m, 16, generator=gen) @ torch.randn(4, 16, n, generator=gen)
    u = torch.linalg.qr(torch.randn(4, m, m, generator=gen, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(4, n, m, generator=gen, dtype=torch.float64))[0]
    out = {"noise": r, "plus 1": r + 1, "plus 10": r + 10, "plus 100": r + 100, "rank 1 and noise": one + 0.01 * r,
           "rank 16 and noise": r + many * (100 * (m ** 0.5 + n ** 0.5) / (m * n) ** 0.5)}
    for ratio in (20, 200, 1000):
        sv = torch.full((m,), 1.0 / ratio, dtype=torch.float64)
        sv[0] = 1
        out[f"one {ratio} times the rest"] = ((u * sv) @ v.transpose(1, 2)).float()
    return {k: t if rows <= cols else t.transpose(1, 2).contiguous() for k, t in out.items()}


def _worst(got, ref):
    return ((got.double().cpu() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)).max().item()


STAGED = [(CUBIC, 8), (CUBIC, 9), (MUON, 3), (MUON, 6), (MUON, 8), (MUON, 10)]


@pytest.mark.parametrize("coeffs,steps", STAGED, ids=lambda v: str(v) if isinstance(v, int) else f"{v[0]}")
@pytest.mark.parametrize("rows,cols", [(64, 200), (300, 40), (100, 801), (16, 128), (128, 257)])
def test_binary32_results_against_binary32_iterates(rows, cols, coeffs, steps):
    """Both forms round to 2^-24 of an iterate a few times a step, and what follows multiplies these alike.  The staged one
    rounds a Gram matrix, P and P x beside, once a stage; they are carried on with the stage's growth squared, which its
    limit keeps to 3.5 times the growth of all steps, or to 12^2.  Its products are of operands in two parts: 2^-24 for
    each of two operands, for the product of the low parts, which is left out, and for the sum, where the iterates'
    have the sum's alone.  So four times the iterates' error, and 64 roundings; the tangents of the gradient are sums of
    two products each, so twice that for it."""
    _announce(f"binary32 stages {rows} {cols} {coeffs} {steps}")
    gen = torch.Generator().manual_seed(rows + steps)
    for name, x in _structured(rows, cols, gen).items():
        y = torch.randn(x.shape, generator=gen)
        xg, yg = x.cuda(), y.cuda()
        out, dx = torch.empty_like(xg), torch.empty_like(xg)
        _run_ns(xg, out, coeffs, steps)
        _run_vjp(xg, yg, dx, coeffs, steps)
        torch.cuda.synchronize()
        refs = _iterates(x.double(), y.double(), coeffs, steps)
        for what, got, ref, it in zip(("NS", "gradient"), (out, dx), refs, _iterates(x, y, coeffs, steps)):
            e, e32 = _worst(got, ref), _worst(it, ref)
            factor = 4 if what == "NS" else 8
            assert e <= factor * e32 + 64 * 2.0 ** -24, f"{what}, {name}: {e:.2e}, iterates {e32:.2e}"


@pytest.mark.parametrize("coeffs,steps", [(CUBIC, 8), (CUBIC, 9), (MUON, 3), (MUON, 5)],
                         ids=lambda v: str(v) if isinstance(v, int) else f"{v[0]}")
@pytest.mark.parametrize("rows,cols", [(64, 200), (300, 40), (128, 128)])
def test_blocks_of_rank_one(rows, cols, coeffs, steps):
    """All ones, and rank one: beside one direction nothing but the rounding of X_0 and of the sums, which the steps
    multiply by their whole growth, while the result has the norm of that one direction: T32 with |O| for sqrt(m)."""
    _announce(f"rank one {rows} {cols} {coeffs} {steps}")
    gen = torch.Generator().manual_seed(rows)
    one = torch.randn(4, rows, 1, generator=gen) @ torch.randn(4, 1, cols, generator=gen)
    for name, x in (("ones", torch.ones(4, rows, cols)), ("rank one", one)):
        out = torch.empty_like(x.cuda())
        _run_ns(x.cuda(), out, coeffs, steps)
        torch.cuda.synchronize()
        ref = _iterates(x.double(), x.double(), coeffs, steps)[0]
        tol = 2.0 ** -24 * (64 + 16 * _gain(coeffs, steps) / ref.flatten(1).norm(dim=1).min().item())
        e = _worst(out, ref)
        assert e <= tol, f"{name}: {e:.2e} > {tol:.2e}"


@pytest.mark.parametrize("steps", [6, 7, 8, 9, 10])
@pytest.mark.parametrize("m,n", [(16, 64), (16, 1024), (64, 768), (128, 300)])
def test_bfloat16_results_of_many_steps(m, n, steps):
    """More growth than one stage takes: results and gradients of blocks with large directions stay within TB, and with
    what binary32 iterates lose where that counts beside it."""
    _announce(f"bfloat16 stages {m} {n} {steps}")
    gen = torch.Generator().manual_seed(m + steps)
    for name, x in _structured(m, n, gen).items():
        x, y = x.to(BF), torch.randn(x.shape, generator=gen).to(BF)
        xg, yg = x.cuda(), y.cuda()
        out, dx = torch.empty_like(xg), torch.empty_like(xg)
        _run_ns(xg, out, MUON, steps)
        _run_vjp(xg, yg, dx, MUON, steps)
        torch.cuda.synchronize()
        refs = _iterates(x.double(), y.double(), MUON, steps)
        for what, got, ref, it in zip(("NS", "gradient"), (out, dx), refs, _iterates(x.float(), y.float(), MUON, steps)):
            e, e32 = _worst(got, ref), _worst(it, ref)
            assert e <= TB + 4 * e32, f"{what}, {name}: {e:.2e}, iterates {e32:.2e}"


# ------------------------- the binary32 update of a step on bfloat16 weights

def _tol_update(m, coeffs, steps, norm=None):
    """Of an update that is not rounded to bfloat16: U and P are 17 bits each, so off by 2^-18.  The steps multiply an error
    of U, of norm 2^-18 beside X_0's 1, by G at most, and a result has norm sqrt(m) (`norm`, where that is known and
    less).  P, of norm G at most in every direction, is off by 2^-18 of that and acts on singular values of up to 2 /
    sqrt(m) of noise (1 of other blocks).  No more than 2^-9, what one stage leaves of its Gram matrix."""
    size = norm if norm is not None else np.sqrt(m)
    return min(2.0 ** -9, 3 * 2.0 ** -18 * _gain(coeffs, steps) / size)


@pytest.mark.parametrize("gdt", [BF, F])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}-{s[3]}{s[4]}")
def test_update_of_bfloat16_weights(shape, gdt):
    """One bfloat16 part of U would leave 1.6e-3 to 3.6e-3."""
    _announce(f"update {shape} {gdt}")
    (w, g, m, _, _), = _step_case(shape, BF, gdt, shape[1] * 5 + shape[2])
    g0, m0 = to_np(g), to_np(m)
    o = torch.full(tuple(w.shape), float("nan"), device="cuda")
    mb.muon_step_blocks([w], [g], [m], lr=f32(0.02), beta=0.95, nesterov=True, ns_coeffs=MUON, ns_steps=5,
                        updates_out=[o])
    torch.cuda.synchronize()
    got, tol = to_np(o), _tol_update(min(shape[1:3]), MUON, 5)
    for b in range(shape[0]):
        ref = orc.orthogonalise(orc.momentum(m0[b], g0[b], f32(0.95), True, 0)[1], _co(MUON), 5)
        e = orc.rel_frobenius(got[b], ref)
        assert e <= tol, f"block {b}: {e:.2e} > {tol:.2e}"


@pytest.mark.parametrize("wdt", [BF, F])
@pytest.mark.parametrize("rows,cols", [(16, 128), (64, 200), (300, 100), (128, 300)])
def test_step_on_structured_gradients(rows, cols, wdt):
    """The step's own kernels on blocks with a few large directions (U is the gradient): the update of bfloat16 weights
    within the roundings of _tol_update and four of 2^-24 of the Gram matrix, carried on by the stage; that of binary32
    ones the same as muon_ns_blocks."""
    _announce(f"structured step {rows} {cols} {wdt}")
    gen = torch.Generator().manual_seed(rows)
    for name, x in _structured(rows, cols, gen).items():
        g = x.cuda()
        w, m, o = torch.zeros_like(g, dtype=wdt), torch.zeros_like(g), torch.empty_like(g)
        mb.muon_step_blocks([w], [g], [m], lr=f32(0.5), beta=0.0, nesterov=False, ns_coeffs=MUON, ns_steps=5,
                            updates_out=[o])
        torch.cuda.synchronize()
        assert torch.equal(m, g)
        if wdt == F:
            out = torch.empty_like(g)
            _run_ns(g, out, MUON, 5)
            assert np.array_equal(_bits(o), _bits(out)), name
            continue
        ref = _iterates(x.double(), x.double(), MUON, 5)[0]
        for b in range(4):
            # s |p'(s^2)| over the singular values that an iterate may have: what a unit error of A_0 gives
            t = np.logspace(-5, 0, 2001)
            f = [t * (1 + d) for d in (-1e-6, 0.0, 1e-6)]
            for a, bb, c in orc.schedule(_co(MUON), 5):
                f = [v * (a + bb * v * v + c * v ** 4) for v in f]
            dp = np.abs(((f[2] - f[0]) / (2e-6 * t) - f[1] / t) / (2 * t)).max()
            size = ref[b].norm().item()
            tol = 3 * 2.0 ** -18 * _gain(MUON, 5) / size + 4 * 2.0 ** -24 * dp / size
            e = _worst(o[b:b + 1], ref[b:b + 1])
            assert e <= tol, f"{name}, block {b}: {e:.2e} > {tol:.2e}"
