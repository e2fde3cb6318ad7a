"""The block operators without a GPU: exported names, refusals on the host
before any HIP call, the overlap rules for stacks, and the oracle's pins."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from muon_newton_schulz_02_amd import binding as mb
from muon_newton_schulz_02_amd import build as mbuild

HEADER = os.path.join(os.path.dirname(mb.HEADER), "muon_blocks.h")
BASE = 0x7F0000000000
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mb.LIB_PATH):
        mbuild.build(verbose=False)
    return mb.lib()


def test_exports(L):
    names = sorted(set(re.findall(r"^(?:muon_status|uint64_t) (muon_[a-z0-9_]+)\(", open(HEADER).read(), re.M)))
    assert names == ["muon_blocks_workspace_bytes", "muon_ns_blocks", "muon_ns_blocks_vjp", "muon_step_blocks"]
    out = subprocess.run(["nm", "-D", "--defined-only", mb.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(names) <= exported


def _desc(blocks=4, rows=16, cols=96, ld=None, stride=None, pdt=mb.DTYPE_BF16, gdt=mb.DTYPE_BF16, mdt=mb.DTYPE_F32,
          **kw):
    d = mb.BlockDesc()
    d.blocks, d.rows, d.cols = blocks, rows, cols
    d.ld_param = d.ld_grad = d.ld_mom = cols if ld is None else ld
    d.stride_param = d.stride_grad = d.stride_mom = rows * d.ld_param if stride is None else stride
    d.param_dtype, d.grad_dtype, d.mom_dtype = pdt, gdt, mdt
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _three(i=0):
    return tuple(BASE + ((3 * i + k) << 40) for k in range(3))


def _call(L, op, descs, ptrs=None, coeffs=MUON, steps=5, sched=None, ws=None, ws_bytes=0, updates=None, **hp):
    """The C entry point of `op` on made-up addresses (validation never reads them)."""
    n = len(descs)
    D = (mb.BlockDesc * max(n, 1))(*descs)
    ptrs = [_three(i) for i in range(n)] if ptrs is None else ptrs
    p, g, m = (mb._ptr_array([t[k] for t in ptrs]) for k in range(3))
    co = mb.NsCoeffs(*coeffs)
    if op == mb.BLOCKS_NS:
        return L.muon_ns_blocks(g, p, D, n, co, steps, sched, ws, ws_bytes, None)
    if op == mb.BLOCKS_VJP:
        return L.muon_ns_blocks_vjp(g, m, p, D, n, co, steps, sched, ws, ws_bytes, None)
    opt = hp.pop("options", None)
    h = mb.StepHparams(hp.get("lr", 0.02), hp.get("beta", 0.95), hp.get("nesterov", 1), co, steps,
                       hp.get("scale_rule", 0), ctypes.pointer(opt) if opt is not None else None)
    return L.muon_step_blocks(p, g, m, D, n, ctypes.byref(h),
                              None if updates is None else mb._ptr_array(updates), ws, ws_bytes, None)


OPS = (mb.BLOCKS_NS, mb.BLOCKS_VJP, mb.BLOCKS_STEP)
PASSES = (mb.MUON_OK, mb.MUON_ERR_HIP)  # validation passed (no GPU here)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("bad,status", [
    (dict(blocks=-1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(blocks=(1 << 20) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(rows=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(cols=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(rows=65537), mb.MUON_ERR_UNSUPPORTED),
    (dict(rows=129, cols=129), mb.MUON_ERR_UNSUPPORTED),
    (dict(ld_grad=95), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_param=95), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_param=(1 << 21) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(stride_grad=-1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(stride_param=16 * 96 - 1), mb.MUON_ERR_ALIAS),
    (dict(stride_param=0), mb.MUON_ERR_ALIAS),
    (dict(param_dtype=2), mb.MUON_ERR_UNSUPPORTED),
    (dict(grad_dtype=-1), mb.MUON_ERR_UNSUPPORTED),
    (dict(reserved=1), mb.MUON_ERR_INVALID_ARGUMENT),
])
def test_descriptor_refusals(L, op, bad, status):
    assert _call(L, op, [_desc(**{k: v for k, v in bad.items() if k in ("blocks", "rows", "cols")},
                               **{k: v for k, v in bad.items() if k not in ("blocks", "rows", "cols")})]) == status
    assert "stack 0" in mb.muon_last_error()


def test_accepted_descriptors(L):
    for op in OPS:
        assert _call(L, op, []) == mb.MUON_OK
        assert _call(L, op, [_desc(blocks=0)], ptrs=[(0, 0, 0)]) == mb.MUON_OK
    if torch.cuda.is_available():
        pytest.skip("the rest would launch on made-up addresses")
    for op in OPS:
        for d in (_desc(), _desc(blocks=1, stride=0), _desc(rows=65536, cols=128), _desc(rows=1, cols=1),
                  # heads side by side in the columns of a 96-wide matrix
                  _desc(blocks=6, rows=64, cols=16, ld=96, stride=16),
                  # one gradient for every block
                  _desc(stride_grad=0)):
            assert _call(L, op, [d]) == mb.MUON_ERR_HIP, mb.muon_last_error()


@pytest.mark.parametrize("op", OPS)
def test_pointer_refusals(L, op):
    p, g, m = _three()
    assert _call(L, op, [_desc()], ptrs=[(0, g, m)]) == mb.MUON_ERR_INVALID_ARGUMENT
    assert _call(L, op, [_desc()], ptrs=[(p, 0, m)]) == mb.MUON_ERR_INVALID_ARGUMENT
    assert _call(L, op, [_desc()], ptrs=[(p + 1, g, m)]) == mb.MUON_ERR_UNSUPPORTED
    assert _call(L, op, [_desc()], ptrs=[(p, g + 1, m)]) == mb.MUON_ERR_UNSUPPORTED
    if op != mb.BLOCKS_NS:
        assert _call(L, op, [_desc()], ptrs=[(p, g, 0)]) == mb.MUON_ERR_INVALID_ARGUMENT
        assert _call(L, op, [_desc()], ptrs=[(p, g, m + 2)]) == mb.MUON_ERR_UNSUPPORTED
    # output over an input, over another stack's output, over the workspace
    assert _call(L, op, [_desc()], ptrs=[(g + 2 * 96, g, m)]) == mb.MUON_ERR_ALIAS
    size = 4 * 16 * 96 * 2
    two = [_desc(), _desc()]
    p1, g1, m1 = _three(1)
    assert _call(L, op, two, ptrs=[(p, g, m), (p + size - 2, g1, m1)]) == mb.MUON_ERR_ALIAS
    assert _call(L, op, [_desc()], ws=p, ws_bytes=1 << 20) == mb.MUON_ERR_ALIAS
    assert _call(L, op, [_desc()], ws=BASE + (50 << 40) + 128, ws_bytes=1 << 20) == mb.MUON_ERR_UNSUPPORTED
    # two stacks may read one input (the step writes each momentum: not shared)
    if not torch.cuda.is_available():
        assert _call(L, op, two, ptrs=[(p, g, m), (p + size, g, m1)]) == mb.MUON_ERR_HIP
        st = _call(L, op, two, ptrs=[(p, g, m), (p + size, g1, m)])
        assert st == (mb.MUON_ERR_ALIAS if op == mb.BLOCKS_STEP else mb.MUON_ERR_HIP)


def test_stacks_side_by_side(L):
    """Two stacks in the columns of one matrix (row stride 256): columns 0-95 and 96-191 or later."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    d = [_desc(blocks=6, rows=64, cols=16, ld=256, stride=16) for _ in range(2)]
    (p, g, m), (_, g1, m1) = _three(), _three(1)
    for off, status in ((96, mb.MUON_ERR_HIP), (160, mb.MUON_ERR_HIP), (95, mb.MUON_ERR_ALIAS),
                        (161, mb.MUON_ERR_ALIAS), (64 * 256, mb.MUON_ERR_HIP), (63 * 256 + 95, mb.MUON_ERR_ALIAS),
                        (63 * 256 + 96, mb.MUON_ERR_HIP)):
        assert _call(L, mb.BLOCKS_STEP, d, ptrs=[(p, g, m), (p + 2 * off, g1, m1)]) == status, off
    # another row stride: the intervals decide
    d[1] = _desc(blocks=6, rows=64, cols=16, ld=128, stride=16)
    assert _call(L, mb.BLOCKS_STEP, d, ptrs=[(p, g, m), (p + 2 * 96, g1, m1)]) == mb.MUON_ERR_ALIAS


@pytest.mark.parametrize("op", OPS)
def test_coefficient_refusals(L, op):
    nan, inf = float("nan"), float("inf")
    for co in ((nan, 0, 0), (1, inf, 0), (1, 0, -inf)):
        assert _call(L, op, [_desc()], coeffs=co) == mb.MUON_ERR_INVALID_ARGUMENT
    for steps in (-1, 1001):
        assert _call(L, op, [_desc()], steps=steps) == mb.MUON_ERR_INVALID_ARGUMENT
    if op != mb.BLOCKS_STEP:
        sched, keep = mb._schedule([MUON, (nan, 0, 0)], 2)
        assert _call(L, op, [_desc()], steps=2, sched=sched) == mb.MUON_ERR_INVALID_ARGUMENT
        assert "ns_schedule[1]" in mb.muon_last_error()
        del keep


def test_hparam_refusals(L):
    def st(**kw):
        return _call(L, mb.BLOCKS_STEP, [_desc()], **kw)

    bad = mb.MUON_ERR_INVALID_ARGUMENT
    assert st(lr=float("nan")) == bad and st(beta=1.0) == bad and st(beta=-0.1) == bad
    assert st(nesterov=2) == bad and st(scale_rule=3) == bad
    for field, value, status in (("weight_decay", -1.0, bad), ("weight_decay", float("inf"), bad),
                                 ("momentum_kind", 2, bad), ("launch_mode", 3, bad), ("tile_mode", -1, bad),
                                 ("launch_mode", mb.LAUNCH_CHAIN, mb.MUON_ERR_UNSUPPORTED),
                                 ("tile_mode", mb.TILES_SMALL, mb.MUON_ERR_UNSUPPORTED)):
        o = mb.StepOptions()
        setattr(o, field, value)
        assert st(options=o) == status, field
    arr = (ctypes.c_float * 1)(float("nan"))
    for field in ("lr_per_matrix", "scale_per_matrix"):
        o = mb.StepOptions()
        setattr(o, field, ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)))
        assert st(options=o) == bad
    # momentum is binary32; the exported update may not overlap a weight
    assert _call(L, mb.BLOCKS_STEP, [_desc(mdt=mb.DTYPE_BF16)]) == mb.MUON_ERR_UNSUPPORTED
    p, _, _ = _three()
    assert st(updates=[p + 64]) == mb.MUON_ERR_ALIAS
    D = (mb.BlockDesc * 1)(_desc())
    arr = mb._ptr_array([BASE])
    assert L.muon_step_blocks(arr, arr, arr, D, 1, None, None, None, 0, None) == bad
    assert L.muon_ns_blocks(None, arr, D, 1, mb.NsCoeffs(*MUON), 5, None, None, 0, None) == bad
    assert L.muon_ns_blocks(arr, arr, None, 1, mb.NsCoeffs(*MUON), 5, None, None, 0, None) == bad
    assert L.muon_ns_blocks(arr, arr, D, -1, mb.NsCoeffs(*MUON), 5, None, None, 0, None) == bad


def test_workspace_query_refusals(L):
    D = (mb.BlockDesc * 1)(_desc(rows=200, cols=200))
    assert L.muon_blocks_workspace_bytes(mb.BLOCKS_NS, D, 1, mb.NsCoeffs(*MUON), 5, None) == 0
    assert "128" in mb.muon_last_error()
    assert L.muon_blocks_workspace_bytes(3, D, 1, mb.NsCoeffs(*MUON), 5, None) == 0
    assert L.muon_blocks_workspace_bytes(mb.BLOCKS_NS, None, 1, mb.NsCoeffs(*MUON), 5, None) == 0


def test_binding_refusals():
    x = torch.zeros(4, 16, 96)
    with pytest.raises(ValueError, match="not on a GPU"):
        mb.muon_ns_blocks([x], [x.clone()], ns_coeffs=MUON, ns_steps=5)
    with pytest.raises(ValueError, match="3-D"):
        mb.NsBlocksArgs([x[0]], [x[0]])
    with pytest.raises(ValueError, match="unit column stride"):
        mb.NsBlocksArgs([x.transpose(1, 2)], [x.transpose(1, 2)])
    with pytest.raises(ValueError, match="stacks where"):
        mb.NsBlocksArgs([x], [])
    with pytest.raises(TypeError):
        mb.NsBlocksArgs([x.half()], [x])
    mb.muon_ns_blocks([], [], ns_coeffs=MUON, ns_steps=5)
    with pytest.raises(ValueError, match="StepBlocksArgs holds every tensor"):
        mb.muon_step_blocks(mb.StepBlocksArgs([], [], []), updates_out=[], lr=0.02, beta=0.95, nesterov=True,
                            ns_coeffs=MUON, ns_steps=5)


def _touched(d, base, esz):
    """Bytes that the blocks of a written tensor cover."""
    return {base + esz * (b * d.stride_param + r * d.ld_param + c) + k
            for b in range(d.blocks) for r in range(d.rows) for c in range(d.cols) for k in range(esz)}


def _two_written(L, d0, d1, off, esz=2):
    """Status of an NS call whose two stacks' outputs start `off` elements apart."""
    g0, g1 = BASE + (8 << 40), BASE + (9 << 40)
    return _call(L, mb.BLOCKS_NS, [d0, d1], ptrs=[(BASE, g0, 0), (BASE + esz * off, g1, 0)])


def test_interleaved_stacks(L):
    """Stacks whose blocks lie between each other's: parts of one weight kept per head, (heads, 3, dim, width) or
    (width, heads, 3, dim), and the even and odd heads of one."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    heads, dim, width = 12, 64, 768
    cases = [
        # blocks of rows: q, k and v of each head, one after another
        (_desc(heads, dim, width, ld=width, stride=3 * dim * width), dim * width, 2 * dim * width),
        # blocks of columns, (width, heads, 3, dim)
        (_desc(heads, width, dim, ld=3 * heads * dim, stride=3 * dim), dim, 2 * dim),
        # even and odd heads
        (_desc(heads // 2, dim, width, ld=width, stride=2 * dim * width), dim * width, dim * width),
        (_desc(heads // 2, width, dim, ld=heads * dim, stride=2 * dim), dim, dim),
        # padded rows, of which one head's are between another's: columns 0-99 and 100-199 of 256
        (_desc(heads, dim, 100, ld=256, stride=2 * dim * 256), 100, dim * 256),
    ]
    for d, lo, hi in cases:
        for off in (lo, hi):
            for first, second in ((0, off), (off, 0)):
                assert _two_written(L, d, d, second - first) == mb.MUON_ERR_HIP, mb.muon_last_error()
        # an element before the first place that is free, and one behind the last
        assert _two_written(L, d, d, lo - 1) == mb.MUON_ERR_ALIAS
        assert _two_written(L, d, d, 1 - lo) == mb.MUON_ERR_ALIAS
        assert _two_written(L, d, d, 0) == mb.MUON_ERR_ALIAS
    d, lo, hi = cases[0]
    assert _two_written(L, d, d, hi + 1) == mb.MUON_ERR_ALIAS
    # three parts in one call of every operator
    st = [_desc(heads, dim, width, ld=width, stride=3 * dim * width) for _ in range(3)]
    ptrs = [tuple(BASE + (k << 40) + e * i * dim * width for k, e in ((0, 2), (1, 2), (2, 4))) for i in range(3)]
    for op in OPS:
        assert _call(L, op, st, ptrs=ptrs) == mb.MUON_ERR_HIP, mb.muon_last_error()


def test_overlap_rule_against_sets_of_bytes(L):
    """Random pairs of small written stacks: a pair that shares a byte is refused, whatever its strides; one with equal
    strides is refused for that alone."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    import random
    rng = random.Random(5)
    seen = {(beside, overlap): 0 for beside in (True, False) for overlap in (True, False)}
    for _ in range(4000):
        descs = []
        rows, cols, ld = rng.randint(1, 4), rng.randint(1, 4), rng.randint(4, 16)
        beside = rng.random() < 0.5
        blocks = rng.randint(1, max(1, ld // cols)) if beside else rng.randint(1, 4)
        stride = rng.randint(cols, max(cols, (ld - cols) // max(blocks - 1, 1))) if beside else \
            rng.randint((rows - 1) * ld + cols, 3 * rows * ld)
        for k in range(2):
            # the second stack differs in its extents alone, or (every fourth) in its strides too
            r, c, b = (rows, cols, blocks) if k == 0 else (rng.randint(1, rows), rng.randint(1, cols), rng.randint(1, blocks))
            same = k == 0 or rng.random() < 0.75
            descs.append(_desc(b, r, c, ld=ld if same else ld + 4, stride=stride if same else stride + 5 * (ld + 4),
                               pdt=mb.DTYPE_F32, gdt=mb.DTYPE_F32))
        if any(d.blocks > 1 and not (d.stride_param >= (d.rows - 1) * d.ld_param + d.cols or
                                     (d.stride_param >= d.cols and (d.blocks - 1) * d.stride_param + d.cols <= d.ld_param))
               for d in descs):
            continue  # a stack that overlaps itself
        off = rng.randint(-3 * ld, 3 * ld)
        for d in descs:
            d.stride_grad, d.ld_grad = 0, d.cols
        overlap = bool(_touched(descs[0], 0, 4) & _touched(descs[1], 4 * off, 4))
        got = _two_written(L, *descs, off, esz=4)
        assert got in (mb.MUON_ERR_ALIAS, mb.MUON_ERR_HIP)
        if overlap:
            assert got == mb.MUON_ERR_ALIAS, ([(d.blocks, d.rows, d.cols, d.ld_param, d.stride_param) for d in descs], off)
        a, b = descs
        if (a.ld_param, a.stride_param) == (b.ld_param, b.stride_param):
            seen[beside, overlap] += 1
            assert got == (mb.MUON_ERR_ALIAS if overlap else mb.MUON_ERR_HIP), off
    assert min(seen.values()) >= 100


@pytest.mark.parametrize("op", OPS)
def test_row_stride_of_single_rows(L, op):
    """Blocks of one row have no next row: their row stride is not looked at."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    for ld in (0, 1, 95, (1 << 21) + 1, 1 << 50):
        d = _desc(blocks=3, rows=1, cols=96, ld=ld, stride=96)
        assert _call(L, op, [d]) == mb.MUON_ERR_HIP, mb.muon_last_error()
        # nor by the overlap rules: next to each other, and one element into each other
        (p, g, m), (_, g1, m1) = _three(), _three(1)
        for off, status in ((3 * 96, mb.MUON_ERR_HIP), (3 * 96 - 1, mb.MUON_ERR_ALIAS)):
            assert _call(L, op, [d, d], ptrs=[(p, g, m), (p + 2 * off, g1, m1)]) == status
        # blocks that share elements still do
        assert _call(L, op, [_desc(blocks=3, rows=1, cols=96, ld=ld, stride=95)]) == mb.MUON_ERR_ALIAS
    assert _call(L, op, [_desc(blocks=3, rows=2, cols=96, ld=95, stride=192)]) == mb.MUON_ERR_INVALID_ARGUMENT


def test_no_exception_leaves_a_c_entry(L, tmp_path):
    """Without memory for the error's text a call still ends with its status (host_plan/blocks_nomem.cpp)."""
    import shutil
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "blocks_nomem")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-rdynamic", "-I", os.path.dirname(HEADER), "-o", exe,
                        os.path.join(here, "host_plan", "blocks_nomem.cpp"), "-ldl"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe, mb.LIB_PATH], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "54 calls, 0 threw" in r.stdout, r.stdout + r.stderr[-2000:]


def test_stream_of_another_device_is_refused():
    """Kernels would run on the stream's device, on the other one's memory."""
    from types import SimpleNamespace
    one = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)
    assert mb._stream_on(one, torch.device("cuda", 1)) == 7 and mb._stream_on(9, torch.device("cuda", 1)) == 9
    with pytest.raises(ValueError, match="stream is on cuda:1, the stacks on cuda:0"):
        mb._stream_on(one, torch.device("cuda", 0))


# ------------------------------------------------------------- oracle pins

def _np_rng(seed):
    import numpy as np
    return np.random.default_rng(seed)


@pytest.mark.parametrize("rows,cols,coeffs,steps", [
    (1, 1, MUON, 3), (1, 9, MUON, 5), (6, 6, MUON, 2), (5, 17, MUON, 5), (17, 5, MUON, 5),
    (4, 11, (1.5, -0.5, 0.0), 5), (3, 8, MUON, 0), (4, 7, [(2.0, -1.5, 0.5), (1.5, -0.5, 0.0), MUON], 3)])
def test_vjp_oracle_against_autograd_and_differences(rows, cols, coeffs, steps):
    import numpy as np
    import oracle as orc
    rng = _np_rng(rows * 100 + cols)
    u, y = rng.standard_normal((2, rows, cols))
    got = orc.orthogonalise_vjp(u, y, coeffs, steps)
    # torch's reverse mode on the iteration written the other way round (from the right)
    x = torch.tensor(u, requires_grad=True)
    z = x / (torch.linalg.vector_norm(x) + 1e-7)
    tall = rows > cols
    for a, b, c in orc.schedule(coeffs, steps):
        g = z.T @ z if tall else z @ z.T
        q = a * torch.eye(len(g), dtype=z.dtype) + b * g + c * (g @ g)
        z = z @ q if tall else q @ z
    (z * torch.tensor(y)).sum().backward()
    ref = x.grad.numpy()
    # both are float64 sums of a few thousand terms of size up to 3.4445^5
    # times the entries: 2^-53 * 485 * 1e3 is below 1e-10 of the result's scale
    scale = max(np.abs(ref).max(), np.abs(y).max() / np.linalg.norm(u) * 1e-3)
    assert np.abs(got - ref).max() <= 1e-10 * scale
    # central differences along random directions: truncation h^2, rounding 2^-53 / h
    h = 1e-5
    for _ in range(3):
        d = rng.standard_normal((rows, cols))
        f = [(orc.orthogonalise(u + s * h * d, coeffs, steps) * y).sum() for s in (1, -1)]
        fd = (f[0] - f[1]) / (2 * h)
        assert abs(fd - (got * d).sum()) <= 1e-5 * (np.abs(got).sum() + np.abs(y).sum())


def test_vjp_oracle_invariants():
    import numpy as np
    import oracle as orc
    rng = _np_rng(3)
    u, y = rng.standard_normal((2, 6, 13))
    d = orc.orthogonalise_vjp(u, y, MUON, 4)
    # NS(s u) = NS(u) up to eps: the gradient is orthogonal to u
    assert abs((d * u).sum()) <= 1e-6 * np.linalg.norm(d) * np.linalg.norm(u)
    assert np.allclose(orc.orthogonalise_vjp(u.T, y.T, MUON, 4).T, d, rtol=0, atol=1e-14)
    assert np.allclose(orc.orthogonalise_vjp(u, 3 * y, MUON, 4), 3 * d, rtol=1e-12)
    # a zero matrix: X_0 = u / eps, P(0) = a^steps
    z = orc.orthogonalise_vjp(np.zeros((3, 4)), y[:3, :4], (2.0, -1.0, 0.5), 3)
    assert np.allclose(z, 8 * y[:3, :4] / 1e-7, rtol=1e-12)
