"""Host-side checks of the group norm and gradient entry points, no GPU: the
library exports what their headers declare, bad arguments are refused before
any CUDA call, and every shape gets a plan that fits it."""
import ctypes
import os
import random
import re
import sys

import pytest
import torch

import row_wise_normalization_ln_gb300 as rn
from row_wise_normalization_ln_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rn.library()


@pytest.mark.parametrize("header", ["libnorm_group.h", "libnorm_grad.h"])
def test_library_exports_every_declared_symbol(lib, header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"^\s*norm_status\s+(\w+)\s*\(", src, flags=re.M)
    assert names
    for n in names:
        assert hasattr(lib, n), n


def fwd(lib, x=P, xb=512, xr=64, g=P, b=P, y=P, yb=512, yr=64, ws=P, nb=1 << 40, B=2, S=8, C=64, G=4, eps=1e-5, act=1,
        dt=rn.NORM_F32, plan=None):
    return lib.gn_fwd_planned(x, xb, xr, g, b, y, yb, yr, None, None, ws, nb, B, S, C, G, eps, act, dt, None, plan)


def bwd(lib, dy=P, x=P, xb=512, xr=64, g=P, b=P, m=P, r=P, dx=P, dxr=64, dg=P, db=P, ws=P, nb=1 << 40, B=2, S=8, C=64,
        G=4, act=1, dt=rn.NORM_F32, plan=None):
    return lib.gn_bwd_planned(dy, xb, xr, x, xb, xr, g, b, m, r, dx, xb, dxr, dg, db, ws, nb, B, S, C, G, act, dt, None,
                              plan)


BAD = [dict(B=-1), dict(S=-1), dict(C=0), dict(C=(1 << 24) + 64), dict(G=0), dict(G=65), dict(G=3), dict(act=9), dict(act=-1),
       dict(xr=63), dict(xb=511), dict(x=None), dict(g=None), dict(b=None), dict(B=1 << 30), dict(S=1 << 60),
       dict(xr=1 << 50), dict(x=ctypes.c_void_p(0x1002))]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_arguments_refused(lib, kw):
    assert fwd(lib, **kw) == rn.NORM_ERR_ARG
    assert bwd(lib, **kw) == rn.NORM_ERR_ARG


def test_more_bad_arguments(lib):
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(y=None), dict(yr=70, yb=640)):  # y over x with other pitches
        assert fwd(lib, **kw) == rn.NORM_ERR_ARG
    for kw in (dict(dy=None), dict(m=None), dict(r=None), dict(dx=None), dict(dg=None), dict(db=None)):
        assert bwd(lib, **kw) == rn.NORM_ERR_ARG
    assert fwd(lib, dt=7) == rn.NORM_ERR_DTYPE and bwd(lib, dt=-1) == rn.NORM_ERR_DTYPE


def test_empty_is_a_noop(lib):
    assert fwd(lib, B=0, x=None, y=None, g=None) == rn.NORM_OK
    assert fwd(lib, S=0, x=None, y=None, g=None) == rn.NORM_OK


def test_workspace_refused_before_any_cuda_call(lib):
    plan = rn.GnPlan.from_dict(dict(path=1, vec_elems=4, tile=16, threads=256, per_thread=1, cluster=1, chunks=2,
                                    out_chunks=1))
    n = ctypes.c_size_t()
    assert lib.gn_workspace_bytes(2, 8, 64, 4, rn.NORM_F32, 0, 0, ctypes.byref(plan), ctypes.byref(n)) == rn.NORM_OK
    assert n.value > 0
    for kw in (dict(ws=None), dict(nb=n.value - 1), dict(ws=ctypes.c_void_p(0x1008))):
        assert fwd(lib, plan=ctypes.byref(plan), **kw) == rn.NORM_ERR_ARG


def test_every_shape_gets_a_fitting_plan(lib):
    """The planner's plans pass the plan check (gn_workspace_bytes makes it)
    for one row to long ones, few to many samples, and any group width."""
    rng = random.Random(3)
    shapes = [(1, 1, 1, 1), (1, 1 << 40, 64, 8), (1 << 20, 1, 64, 8), (1, 1, 1 << 24, 1), (1, 7, 1 << 24, 1 << 24),
              (100, 100, 9999, 9999), (1, 1 << 31, 3, 1)]
    for _ in range(3000):
        D, G = rng.choice([1, 2, 3, 5, 7, 8, 10, 12, 40, 64, 100, 513, 1001, 4096]), rng.choice([1, 2, 3, 8, 25, 32, 64])
        shapes.append((rng.choice([1, 2, 5, 64, 1000]), int(10 ** rng.uniform(0, 6)), D * G, G))
    for B, S, C, G in shapes:
        for dt in (torch.float32, torch.bfloat16):
            for backward in (False, True):
                for vec in (4, 1) if dt == torch.float32 else (8, 2, 1):
                    if C % vec:
                        continue
                    p = rn.make_gn_plan(B, S, C, G, dt, backward, vec_elems=vec)
                    n, q = ctypes.c_size_t(), rn.GnPlan.from_dict(p)
                    assert lib.gn_workspace_bytes(B, S, C, G, rn._dtype_code(dt), int(backward), 0, ctypes.byref(q),
                                                  ctypes.byref(n)) == rn.NORM_OK
                    tiles = -(-(C // vec) // p["tile"])
                    ctas = B * tiles * (p["cluster"] if p["path"] == 0 else max(p["chunks"], p["out_chunks"]))
                    assert 1 <= ctas < 2 ** 31
                    if p["path"] == 0:  # every row is held by some thread
                        assert p["cluster"] * p["per_thread"] * (p["threads"] // p["tile"]) >= S


def test_chunks_longer_than_a_thread_counts_are_refused(lib):
    """A thread's count of the values it adds up (rows it visits times the
    access's channels) is 32 bits: one CTA of one row at a time over 2^30 rows
    in pairs would count 2^31."""
    n = ctypes.c_size_t()

    def need(S, vec, chunks, C=34, out_chunks=None):
        p = rn.GnPlan.from_dict(dict(path=1, vec_elems=vec, tile=17, threads=32, per_thread=1, cluster=1, chunks=chunks,
                                     out_chunks=out_chunks or chunks))
        return lib.gn_workspace_bytes(1, S, C, 1, rn.NORM_BF16, 0, 0, ctypes.byref(p), ctypes.byref(n))

    assert need(1 << 30, 2, 1) == rn.NORM_ERR_PLAN
    assert need(1 << 29, 8, 2, C=136) == rn.NORM_ERR_PLAN
    assert need(1 << 30, 2, 2) == need(1 << 29, 2, 1) == need(1 << 30, 1, 1) == rn.NORM_OK
    # what the planner makes of such lengths fits
    for S, C in ((1 << 31, 34), ((1 << 33) + 5, 8), ((1 << 35) + 1, 1)):
        for vec in (8, 2, 1):
            if C % vec == 0:
                p = rn.make_gn_plan(1, S, C, 1, torch.bfloat16, False, vec_elems=vec)
                assert -(-S // p["chunks"]) * vec <= 1 << 30


def test_make_plan_refuses_bad_shapes():
    for a in ((0, 8, 64, 4), (1, 0, 64, 4), (1, 8, 64, 3)):
        with pytest.raises((rn.NormError, StopIteration)):
            rn.make_gn_plan(*a, torch.float32)
    with pytest.raises(rn.NormError):
        rn.make_gn_plan(1, 8, 6, 3, torch.float32, vec_elems=4)


def test_binding_refuses():
    x = torch.zeros(2, 8, 64)
    g = torch.ones(64)
    with pytest.raises(ValueError):
        rn.gn_fwd(x, g, g, 4)
    with pytest.raises(ValueError):
        rn.gn_bwd(x, x, g, g, g, g, 4)
    with pytest.raises(ValueError):
        rn.grad_norm([x])
    with pytest.raises(ValueError):
        rn.grad_norm([])
    with pytest.raises(ValueError):
        rn.grad_clip([x], 1.0, out=[])


def test_pointers_off_their_elements_alignment_refused(lib):
    """Parameters, statistics, column gradients and the norm, like the
    tensors: an access at such an address would be an error on the GPU."""
    off = ctypes.c_void_p(0x1002)
    for kw in (dict(g=off), dict(b=off)):
        assert fwd(lib, **kw) == rn.NORM_ERR_ARG
    for kw in (dict(g=off), dict(b=off), dict(m=off), dict(r=off), dict(dg=off), dict(db=off)):
        assert bwd(lib, **kw) == rn.NORM_ERR_ARG
    for kw in (dict(g=ctypes.c_void_p(0x1001)), dict(b=ctypes.c_void_p(0x1001))):
        assert fwd(lib, dt=rn.NORM_BF16, **kw) == rn.NORM_ERR_ARG
    for m, r in ((off, None), (None, off)):
        assert lib.gn_fwd(P, 512, 64, P, P, ctypes.c_void_p(0x9000), 512, 64, m, r, P, 1 << 40, 2, 8, 64, 4, 1e-5, 0, 0,
                          None) == rn.NORM_ERR_ARG
    assert bwd(lib, B=0, dg=off) == rn.NORM_ERR_ARG
    for call in ("grad_norm", "grad_clip"):
        assert clip(lib, [(0x8000, 0x8000, 64, rn.NORM_F32)], norm=off, call=call) == rn.NORM_ERR_ARG


# ------------------------------------------------------------ gradients

class NormTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def clip(lib, entries, max_norm=1.0, norm=P, ws=P, nb=1 << 40, call="grad_clip"):
    ts = (NormTensor * max(1, len(entries)))(*[NormTensor(*e, 0) for e in entries])
    if call == "grad_norm":
        return lib.grad_norm(ctypes.addressof(ts), len(entries), norm, ws, nb, None)
    return lib.grad_clip(ctypes.addressof(ts), len(entries), max_norm, norm, ws, nb, None)


def test_gradient_arguments_refused(lib):
    ok = (0x1000, 0x1000, 64, rn.NORM_F32)
    for bad in ((None, 0x1000, 4, 0), (0x1002, 0x1000, 4, 0), (0x1000, 0x1000, -1, 0), (0x1000, 0x1000, 1 << 46, 0)):
        assert clip(lib, [ok, bad], call="grad_norm") == rn.NORM_ERR_ARG
        assert clip(lib, [ok, bad]) == rn.NORM_ERR_ARG
    assert clip(lib, [(0x1000, 0x1000, 4, 9)]) == rn.NORM_ERR_DTYPE
    long = (0x100000, 0x100000, 1 << 20, rn.NORM_F32)
    for kw in (dict(norm=None), dict(ws=None), dict(ws=ctypes.c_void_p(0x1004))):
        assert clip(lib, [long], **kw) == rn.NORM_ERR_ARG
        assert clip(lib, [long], call="grad_norm", **kw) == rn.NORM_ERR_ARG
    assert clip(lib, [ok], norm=None) == rn.NORM_ERR_ARG
    for m in (-1.0, float("nan"), float("inf")):
        assert clip(lib, [ok], max_norm=m) == rn.NORM_ERR_ARG
    assert clip(lib, [(0x1000, None, 4, 0)]) == rn.NORM_ERR_ARG
    assert lib.grad_norm(None, 1, P, P, 1 << 40, None) == rn.NORM_ERR_ARG
    assert lib.grad_norm(None, -1, P, P, 1 << 40, None) == rn.NORM_ERR_ARG


@pytest.mark.parametrize("entries", [
    [(0x1000, 0x1000, 64, 0), (0x1000, 0x1000, 64, 0)],      # the same tensor twice, in place
    [(0x1000, 0x1000, 64, 0), (0x10fc, 0x10fc, 64, 0)],      # neighbours that overlap by one value
    [(0x1000, 0x8000, 64, 0), (0x2000, 0x8000, 64, 0)],      # two outputs on one place
    [(0x1000, 0x1004, 64, 0)],                               # an output over its own input, shifted
    [(0x1000, 0x8000, 64, 0), (0x2000, 0x1080, 64, 0)],      # an output over another tensor's input
], ids=range(5))
def test_overlapping_outputs_refused(lib, entries):
    assert clip(lib, entries) == rn.NORM_ERR_ARG


@pytest.mark.parametrize("norm", [0x100000, 0x10fffc, 0x300000, 0x300ffc])
@pytest.mark.parametrize("count", [1, 70])
def test_norm_over_a_gradient_or_an_output_refused(lib, norm, count):
    """grad_clip writes the norm while gradients are still read and outputs
    written."""
    entries = [(0x100000, 0x300000, 1 << 14, rn.NORM_F32)] + [(0x500000 + 64 * i, 0x700000 + 64 * i, 16, rn.NORM_F32)
                                                             for i in range(count - 1)]
    assert clip(lib, entries, norm=ctypes.c_void_p(norm)) == rn.NORM_ERR_ARG
    inplace = [(d, d, n, t) for d, _, n, t in entries]
    if norm < 0x200000:
        assert clip(lib, inplace, norm=ctypes.c_void_p(norm)) == rn.NORM_ERR_ARG


def test_workspace_bytes(lib):
    n = ctypes.c_size_t()

    def need(sizes, sms=152):
        ts = (NormTensor * max(1, len(sizes)))(*[NormTensor(0x1000, None, v, rn.NORM_F32, 0) for v in sizes])
        return lib.grad_workspace_bytes(ctypes.addressof(ts), len(sizes), sms, ctypes.byref(n))

    assert need([]) == rn.NORM_OK and n.value == 0
    assert need([1024] * 24) == rn.NORM_OK and n.value == 0  # short: none
    assert need([1 << 20]) == rn.NORM_OK and n.value > 0
    one = n.value
    assert need([1] * 5000) == rn.NORM_OK and n.value > one
    assert need([-1]) == rn.NORM_ERR_ARG and need([1], 0) == rn.NORM_ERR_ARG
    assert lib.grad_workspace_bytes(None, 1, 152, ctypes.byref(n)) == rn.NORM_ERR_ARG
    assert lib.grad_workspace_bytes(None, 0, 152, None) == rn.NORM_ERR_ARG


# ------------------------------------------------------------ building the binding

def test_binding_of_another_torch_is_rebuilt(lib, monkeypatch, tmp_path):
    """_binding.so holds for the torch and the interpreter it was compiled
    against: after a change of either it is out of date, alone, and build()
    makes it again."""
    assert _build.up_to_date()
    for where, name, other in ((torch, "__version__", "1.0"), (torch, "__file__", "/elsewhere/torch/__init__.py"),
                               (sys.implementation, "cache_tag", "cpython-39")):
        with monkeypatch.context() as m:
            m.setattr(where, name, other)
            assert not _build.up_to_date()
    assert _build.up_to_date()
    made = []
    key = tmp_path / "binding.key"
    key.write_text("another")
    monkeypatch.setattr(_build, "NATIVE_KEY", str(key))
    monkeypatch.setattr(_build, "_compile_native", lambda: made.append("compiled") or "obj")
    monkeypatch.setattr(_build, "_link_native", lambda obj: made.append(obj))
    before = os.path.getmtime(_build.LIB)
    assert not _build.up_to_date()
    _build.build()
    assert made == ["compiled", "obj"] and os.path.getmtime(_build.LIB) == before and _build.up_to_date()
    _build.build()
    assert len(made) == 2


def test_binding_of_another_torch_is_not_loaded(lib, monkeypatch, tmp_path):
    """It may not fit, so a call says what to do instead of loading it."""
    key = tmp_path / "binding.key"
    key.write_text("another")
    monkeypatch.setattr(_build, "NATIVE_KEY", str(key))
    monkeypatch.setattr(rn, "_binding_module", None)
    with pytest.raises(rn.LibraryNotBuilt, match="build"):
        rn.grad_norm([torch.zeros(3)])


def test_row_norms_build_without_the_binding(lib, monkeypatch, tmp_path):
    """libnorm.so, and with it the row norms, needs nvcc alone: where the
    binding of the group norm and gradient calls does not compile (no Python or
    torch headers), build() says so and leaves none behind."""
    native, key = tmp_path / "_binding.so", tmp_path / "binding.key"
    native.write_text("stale")
    key.write_text("another")
    monkeypatch.setattr(_build, "NATIVE", str(native))
    monkeypatch.setattr(_build, "NATIVE_KEY", str(key))

    def fails():
        raise RuntimeError("Python.h: No such file or directory")

    monkeypatch.setattr(_build, "_compile_native", fails)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    assert not native.exists() and not key.exists() and not _build.up_to_date()
    assert lib.norm_abi_version() > 0
    built = []
    monkeypatch.setattr(_build, "_build_library", lambda *a: built.append(a))
    with pytest.warns(RuntimeWarning):
        _build.build(force=True)
    assert len(built) == 1
