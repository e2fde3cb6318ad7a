"""The expert products and the head's loss without a GPU: exported names, refusals
on the host before any HIP call, and the oracle against differences."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle as orc
from muon_newton_schulz_02_amd import binding as mb
from muon_newton_schulz_02_amd import build as mbuild
import training_cases

INCLUDE = os.path.dirname(mb.HEADER)
BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mb.LIB_PATH):
        mbuild.build(verbose=False)
    return mb.lib()


@pytest.mark.parametrize("header,want", [
    ("muon_experts.h", ["muon_experts_product", "muon_experts_product_vjp", "muon_experts_workspace_bytes"]),
    ("muon_head.h", ["muon_head_loss", "muon_head_loss_vjp", "muon_head_workspace_bytes"]),
])
def test_exports(L, header, want):
    text = open(os.path.join(INCLUDE, header)).read()
    assert sorted(set(re.findall(r"^(?:muon_status|uint64_t) (muon_[a-z0-9_]+)\(", text, re.M))) == want
    out = subprocess.run(["nm", "-D", "--defined-only", mb.LIB_PATH], capture_output=True, text=True).stdout
    assert set(want) <= {line.split()[-1] for line in out.splitlines() if line.strip()}


def _at(i):
    return BASE + (i << 40)


def _experts(**kw):
    d = mb.ExpertsDesc()
    d.experts, d.rows, d.in_dim, d.out_dim = 4, 100, 64, 96
    d.ld_x = d.ld_w = d.ld_grad_x = d.ld_grad_w = 64
    d.ld_y, d.stride_w, d.stride_grad_w = 96, 64 * 96, 64 * 96
    d.dtype = d.grad_w_dtype = mb.DTYPE_BF16
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _product(L, d, ptr=None, ws=None, nbytes=0):
    p = [_at(i) for i in range(4)] if ptr is None else ptr
    return L.muon_experts_product(p[0], p[1], p[2], p[3], d, ws, nbytes, None)


def _product_vjp(L, d, ptr=None, ws=None, nbytes=0):
    p = [_at(i) for i in range(6)] if ptr is None else ptr
    return L.muon_experts_product_vjp(*p, d, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(reserved=1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(experts=-1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(rows=-1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(in_dim=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(out_dim=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(experts=2049), mb.MUON_ERR_UNSUPPORTED),
    (dict(rows=(1 << 24) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(in_dim=65537, ld_x=65537, ld_w=65537), mb.MUON_ERR_UNSUPPORTED),
    (dict(out_dim=65537, ld_y=65537), mb.MUON_ERR_UNSUPPORTED),
    (dict(dtype=2), mb.MUON_ERR_UNSUPPORTED),
    (dict(w_order=2), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_x=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_y=95), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_w=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(w_order=1, ld_w=95), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_x=(1 << 21) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(stride_w=-1), mb.MUON_ERR_INVALID_ARGUMENT),
])
def test_experts_descriptor_refusals(L, kw, status):
    assert _product(L, _experts(**kw)) == status
    assert mb.muon_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(ld_grad_x=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_grad_w=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(grad_w_dtype=2), mb.MUON_ERR_UNSUPPORTED),
    (dict(dtype=mb.DTYPE_F32), mb.MUON_ERR_UNSUPPORTED),       # bfloat16 gradient of binary32 weights
    (dict(accumulate=2), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(stride_grad_w=64 * 96 - 1), mb.MUON_ERR_ALIAS),
    (dict(stride_grad_w=0), mb.MUON_ERR_ALIAS),
    (dict(stride_grad_w=32, ld_grad_w=4 * 64), mb.MUON_ERR_ALIAS),
])
def test_experts_gradient_refusals(L, kw, status):
    assert _product_vjp(L, _experts(**kw)) == status
    assert mb.muon_last_error()


@pytest.mark.parametrize("i", range(4))
def test_experts_null_and_misaligned(L, i):
    p = [_at(k) for k in range(4)]
    p[i] = None
    assert _product(L, _experts(), p) == mb.MUON_ERR_INVALID_ARGUMENT
    p[i] = _at(i) + 1
    assert _product(L, _experts(), p) == mb.MUON_ERR_UNSUPPORTED


def test_experts_aliases_and_workspace(L):
    p = [_at(k) for k in range(4)]
    p[3] = p[0] + 2 * 64 * 99                      # y meets x's last row
    assert _product(L, _experts(), p) == mb.MUON_ERR_ALIAS
    p[3] = p[1] + 2 * (4 * 64 * 96 - 1)            # and w's last element
    assert _product(L, _experts(), p) == mb.MUON_ERR_ALIAS
    q = [_at(k) for k in range(6)]
    q[5] = q[4] + 2 * (99 * 64 + 63)               # grad_w meets grad_x
    assert _product_vjp(L, _experts(), q) == mb.MUON_ERR_ALIAS
    assert _product(L, _experts(), ws=_at(9) + 128, nbytes=1 << 20) == mb.MUON_ERR_UNSUPPORTED
    assert _product(L, _experts(), ws=_at(0), nbytes=1 << 20) == mb.MUON_ERR_ALIAS
    assert _product_vjp(L, _experts(), [_at(0), _at(1), _at(2), _at(3), None, None]) == mb.MUON_ERR_INVALID_ARGUMENT
    assert L.muon_experts_product(_at(0), _at(1), _at(2), _at(3), None, None, 0, None) == mb.MUON_ERR_INVALID_ARGUMENT


def test_experts_without_work(L):
    assert _product(L, _experts(experts=0), [None] * 4) == mb.MUON_OK
    assert _product(L, _experts(rows=0), [None, None, _at(2), None]) == mb.MUON_OK
    assert _product_vjp(L, _experts(experts=0)) == mb.MUON_OK
    assert L.muon_experts_workspace_bytes(4, _experts()) == 0 and "op" in mb.muon_last_error()


def _head(**kw):
    d = mb.HeadDesc()
    d.rows, d.dim, d.vocab = 50, 64, 1000
    d.ld_x = d.ld_w = d.ld_grad_x = d.ld_grad_w = 64
    d.ignore_index, d.softcap, d.dtype = -100, 15.0, mb.DTYPE_BF16
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _loss(L, d, ptr=None, ws=None, nbytes=0):
    p = [_at(i) for i in range(5)] if ptr is None else ptr
    return L.muon_head_loss(*p, d, ws, nbytes, None)


def _loss_vjp(L, d, ptr=None, ws=None, nbytes=0):
    p = [_at(i) for i in range(8)] if ptr is None else ptr
    return L.muon_head_loss_vjp(*p, d, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(reserved=1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(rows=-1), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(dim=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(vocab=0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(rows=(1 << 20) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(dim=65537, ld_x=65537, ld_w=65537), mb.MUON_ERR_UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1), mb.MUON_ERR_UNSUPPORTED),
    (dict(dtype=5), mb.MUON_ERR_UNSUPPORTED),
    (dict(softcap=-1.0), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(softcap=1e-4), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(softcap=float("inf")), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(softcap=float("nan")), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_x=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_w=63), mb.MUON_ERR_INVALID_ARGUMENT),
    (dict(ld_w=(1 << 21) + 1), mb.MUON_ERR_UNSUPPORTED),
])
def test_head_descriptor_refusals(L, kw, status):
    assert _loss(L, _head(**kw)) == status
    assert mb.muon_last_error()
    assert _loss_vjp(L, _head(**kw)) == status


def test_head_gradient_refusals(L):
    assert _loss_vjp(L, _head(ld_grad_x=63)) == mb.MUON_ERR_INVALID_ARGUMENT
    assert _loss_vjp(L, _head(ld_grad_w=63)) == mb.MUON_ERR_INVALID_ARGUMENT
    p = [_at(i) for i in range(8)]
    assert _loss_vjp(L, _head(), p[:6] + [None, None]) == mb.MUON_ERR_INVALID_ARGUMENT
    p[7] = p[6] + 2 * 49 * 64                      # grad_w meets grad_x
    assert _loss_vjp(L, _head(), p) == mb.MUON_ERR_ALIAS
    p[7] = p[1]                                    # grad_w is w
    assert _loss_vjp(L, _head(), p) == mb.MUON_ERR_ALIAS


@pytest.mark.parametrize("i", range(5))
def test_head_null_and_misaligned(L, i):
    p = [_at(k) for k in range(5)]
    p[i] = None
    assert _loss(L, _head(), p) == mb.MUON_ERR_INVALID_ARGUMENT
    p[i] = _at(i) + 1
    assert _loss(L, _head(), p) == mb.MUON_ERR_UNSUPPORTED


def test_head_aliases_workspace_and_nothing_to_do(L):
    p = [_at(k) for k in range(5)]
    p[4] = p[3] + 4 * 49
    assert _loss(L, _head(), p) == mb.MUON_ERR_ALIAS
    assert _loss(L, _head(), ws=_at(9) + 8, nbytes=1 << 20) == mb.MUON_ERR_UNSUPPORTED
    assert _loss(L, _head(rows=0), [None] * 5) == mb.MUON_OK
    assert L.muon_head_loss(*[_at(i) for i in range(5)], None, None, 0, None) == mb.MUON_ERR_INVALID_ARGUMENT
    assert L.muon_head_workspace_bytes(-1, _head()) == 0 and "op" in mb.muon_last_error()


def test_bindings_refuse_before_any_call():
    x, w = torch.zeros(3, 8), torch.zeros(2, 4, 8)
    off, y = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="not on a GPU"):
        mb.muon_experts_product(x, w, off, y)
    with pytest.raises(ValueError, match="not on a GPU"):
        mb.muon_head_loss(x, w[0], torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(3))


@pytest.mark.parametrize("call,missing", [
    (lambda t: mb.muon_experts_product(t), "w"),
    (lambda t: mb.muon_experts_product(t, t, None, t), "offsets"),
    (lambda t: mb.muon_experts_product(None, t, t, t), "x"),
    (lambda t: mb.muon_experts_product_vjp(t, t, t, None, t), "grad_y"),
    (lambda t: mb.muon_experts_product_vjp(t, t, None, t, t), "offsets"),
    (lambda t: mb.muon_head_loss(t), "w"),
    (lambda t: mb.muon_head_loss(t, t, t, None, t), "loss"),
    (lambda t: mb.muon_head_loss_vjp(t, t, t, t, None, t), "grad_loss"),
    (lambda t: mb.muon_head_loss_vjp(None, t, t, t, t, t), "x"),
])
def test_bindings_name_what_is_missing(call, missing):
    with pytest.raises(ValueError, match=f"^{missing} is missing"):
        call(torch.zeros(2, 2))


def test_oracle_against_differences():
    rng = np.random.default_rng(0)
    x, w = rng.normal(size=(5, 4)), rng.normal(size=(7, 4))
    t = np.array([1, -100, 6, 0, 9])               # ignored, and out of range
    g, h = rng.normal(size=5), rng.normal(size=5)

    def value(x, w):
        r = orc.training.head(x, w, t, softcap=2.0)
        keep = np.array([0, 2, 3])
        return (g * r["loss"])[keep].sum() + (h * r["lse"])[keep].sum()

    got = orc.training.head(x, w, t, softcap=2.0, grad_loss=g, grad_lse=h)
    assert np.isnan(got["loss"][4]) and got["loss"][1] == 0 and not got["grad_x"][[1, 4]].any()
    for name, at in (("grad_x", x), ("grad_w", w)):
        for i in np.ndindex(at.shape):
            e = np.zeros_like(at)
            e[i] = 1e-6
            pair = [(x + s * e, w) if name == "grad_x" else (x, w + s * e) for s in (1, -1)]
            diff = (value(*pair[0]) - value(*pair[1])) / 2e-6
            assert abs(diff - got[name][i]) < 1e-7     # steps of 1e-6: 1e-12 from curvature, 1e-10 from rounding
    off = [0, 2, 2, 4]
    we = rng.normal(size=(3, 6, 4))
    gy = rng.normal(size=(5, 6))
    y, _ = orc.training.experts(x, we, off)
    gx, _ = orc.training.experts(gy, we.transpose(0, 2, 1), off)
    gw, _ = orc.training.experts_grad_w(x, gy, off)
    assert not y[4].any() and not gw[1].any()
    # both sides of <y, gy> as a bilinear form
    assert np.isclose((y * gy)[:4].sum(), (gx * x)[:4].sum()) and np.isclose((y * gy)[:4].sum(), (gw * we).sum())


SHAPES = ("naive", "32", "128", "256", "narrow", "stream")
FORMS = ("NT", "NN", "TN")
EPILOGUES = ("store", "loss", "grad", "loss, cap", "grad, cap", "loss, large cap", "grad, large cap", "store, targets")
HIP_INC = "/opt/rocm/include"


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """The products of calls: lines of host_plan/training_plan.cpp to {name: [(form, epilogue, shape, f32, cut, queued)]}."""
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(HIP_INC, "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(mb.LIB_PATH), "csrc")
    exe = str(tmp_path_factory.mktemp("plan") / "training_plan")
    cmd = [gxx, "-std=c++17", "-O1", "-Wall", "-Wno-unused-result", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INC, "-I", INCLUDE,
           "-I", csrc, "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-o", exe,
           os.path.join(here, "host_plan", "training_plan.cpp"),
           *(os.path.join(csrc, f) for f in ("muon_experts.cpp", "muon_head.cpp", "products_plan.cpp"))]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=120,
                           env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0 and "FAIL" not in r.stdout and "OUTSIDE" not in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
        got = {}
        for line in r.stdout.splitlines():
            name, *v = line.split()
            form, epi, shape, f32, cut, queued = map(int, v)
            got.setdefault(name, []).append((FORMS[form], EPILOGUES[epi], SHAPES[shape], "f32" if f32 else "bf16", cut, queued))
        return got
    return run


def _head_lines(sizes, dtype, cap):
    return [f"head {r}x{d}x{v} {r} {d} {v} {int(dtype == 'f32')} {cap}" for r, d, v in sizes]


def test_every_kernel_of_the_head_has_a_test(plan):
    """The sizes of tests/test_gpu_head.py reach each kernel of the logits: every shape, soft cap and type, k in whole 16
    bytes and not; and the gradients' products on each shape, cut and not."""
    logits, products, stores = set(), set(), set()
    for dtype, caps in training_cases.HEAD_TILES_CAPS.items():
        for cap in caps:
            sizes = training_cases.HEAD_TILES + (training_cases.HEAD_LARGE if cap != 40.0 else [])
            for name, got in plan(_head_lines(sizes, dtype, cap)).items():
                whole = int(name.split("x")[1]) % 8 == 0
                logits |= {(e, s, t, whole) for f, e, s, t, _, _ in got if f == "NT"}
                products |= {(f, s, t, cut) for f, e, s, t, cut, _ in got if f != "NT"}
                stores |= {(e, t) for f, e, s, t, _, _ in got if f != "NT"}
    for dtype, kinds in (("bf16", ("", ", cap", ", large cap")), ("f32", ("", ", cap"))):
        for kind in kinds:
            for shape in ("128", "256"):
                for whole in (False, True):
                    assert {("loss" + kind, shape, dtype, whole), ("grad" + kind, shape, dtype, whole)} <= logits
    assert all(e == ("store, targets" if t == "bf16" else "store") for e, t in stores)
    assert {("NN", "256", "bf16", 0), ("NN", "256", "bf16", 1), ("TN", "256", "bf16", 0), ("NN", "128", "bf16", 1),
            ("TN", "128", "bf16", 0), ("TN", "narrow", "bf16", 0), ("NN", "256", "f32", 0), ("NN", "256", "f32", 1),
            ("TN", "256", "f32", 1), ("NN", "128", "f32", 1), ("TN", "128", "f32", 1)} <= products
    long = [got[3] for got in plan(_head_lines(training_cases.HEAD_LONG, "bf16", 0.0)).values()]
    assert [(f, s, cut) for f, _, s, _, cut, _ in long] == [("TN", "256", 0), ("TN", "128", 0), ("TN", "narrow", 0), ("TN", "narrow", 1)]
    small = set()
    for dtype in ("bf16", "f32"):
        for cap in (0.0, 15.0):
            for got in plan(_head_lines(training_cases.HEAD_SIZES, dtype, cap)).values():
                small |= {(e, s, t) for f, e, s, t, _, _ in got if f == "NT"}
    for dtype in ("bf16", "f32"):
        for kind in ("", ", cap"):
            assert {("loss" + kind, s, dtype) for s in ("naive", "32", "stream")} <= small
            assert {("grad" + kind, s, dtype) for s in ("naive", "32")} <= small


def test_few_rows_are_streamed_only_where_that_is_faster(plan):
    """The rule's measured sides: (experts, rows an expert, in, out, f32) and whether the product is streamed."""
    sides = [
        (64, 16, 1536, 2048, 0, False), (64, 1, 1536, 2048, 0, False), (8, 1, 1536, 6144, 0, True), (8, 4, 1536, 6144, 0, False),
        (32, 8, 768, 256, 0, True), (32, 3, 6144, 1536, 0, True), (1, 1, 1536, 6144, 0, True), (1, 16, 1536, 6144, 0, True),
        (64, 24, 1536, 2048, 0, False), (64, 1, 1536, 2048, 1, True), (64, 16, 1536, 2048, 1, False), (8, 8, 1536, 6144, 1, True),
        (32, 16, 768, 256, 1, True),
    ]
    for i, (experts, per, inn, out, f32, streamed) in enumerate(sides):
        got = plan([f"experts {i} {experts} {experts * per} {inn} {out} {f32} 0 {f32}"])[str(i)]
        assert (got[0][2] == "stream") == streamed, sides[i]
        assert got[0][4] == 0 or per > 16           # and needs no workspace
    counts, inn, out = training_cases.FEW_TO_ONE[0]
    for f32 in (0, 1):
        got = plan([f"experts few {len(counts)} {sum(counts) + 3} {inn} {out} {f32} 0 {f32}"])["few"]
        assert got[0][2] == "stream"


def test_no_exception_leaves_a_c_entry(L, tmp_path):
    """Without memory for the error's text a call still ends with its status (host_plan/training_nomem.cpp)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "training_nomem")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-I", INCLUDE, "-o", exe,
                        os.path.join(here, "host_plan", "training_nomem.cpp"), "-ldl"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe, mb.LIB_PATH], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "72 calls, 0 threw" in r.stdout, r.stdout + r.stderr
