"""Host-side checks of the head norms with rotation and of dropout + add + norm, no GPU: the library exports what their
headers declare, bad arguments are refused before any CUDA call, every shape gets a plan that covers it within the
limits, and the tests' generator gives the published answers."""
import ctypes
import os
import random
import re

import numpy as np
import pytest
import torch

import row_wise_normalization_ln_gb300 as rn
from row_wise_normalization_ln_gb300 import _build
from philox import keep_mask, philox4x32, threshold

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x1000
DT = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rn.library()


@pytest.mark.parametrize("header", ["libnorm_rope.h", "libnorm_dropout.h"])
def test_library_exports_every_declared_symbol(lib, header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"^\s*norm_status\s+(\w+)\s*\(", src, flags=re.M)
    assert len(names) >= 6
    for n in names:
        assert hasattr(lib, n), n


# ------------------------------------------------------------ the generator
def test_published_answers_of_the_generator():
    def words(counter, key, rounds):
        return [int(v) for v in philox4x32(np.array([counter], dtype=np.uint64), key, rounds)[0]]
    assert words([0, 0, 0, 0], (0, 0), 7) == [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]
    assert words([0, 0, 0, 0], (0, 0), 10) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert words([ones] * 4, (ones, ones), 10) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_mask_of_rows_is_a_part_of_the_whole():
    whole = keep_mask(7, 9, 0.3, 20, 37)
    assert (keep_mask(7, 9, 0.3, 20, 37, rows=(5, 11)) == whole[5:11]).all()
    # 740 words, each kept with probability 1 - 19661 / 65536: within 5 standard deviations
    assert abs(whole.mean() - (1 - threshold(0.3) / 65536)) < 5 * (0.3 * 0.7 / whole.size) ** 0.5


# ------------------------------------------------------------ dropout, add and norm
class Rng(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("device", ctypes.c_void_p)]


def fwd(lib, ln=1, x=P, r=P + 0x1000, g=P, b=P, p=0.1, rng=Rng(1, 2, None), h=P + 0x2000, y=P + 0x3000, mean=None, rstd=None, M=4,
        N=64, eps=1e-5, dt=rn.NORM_F32, plan=None):
    return lib.drop_fwd_planned(ln, x, r, g, b, p, None if rng is None else ctypes.addressof(rng), h, y, mean, rstd, M, N, eps, dt,
                                None, plan)


def bwd(lib, ln=1, dy=P, dh=P, h=P, g=P, mean=P, rstd=P, p=0.1, rng=Rng(1, 2, None), dx=P + 0x2000, dr=P + 0x3000, dg=P, db=P, ws=P,
        nb=1 << 40, M=4, N=64, eps=1e-5, dt=rn.NORM_F32, plan=None):
    return lib.drop_bwd_planned(ln, dy, dh, h, g, mean, rstd, p, None if rng is None else ctypes.addressof(rng), dx, dr, dg, db, ws,
                                nb, M, N, eps, dt, None, plan)


BOTH = [dict(M=-1), dict(N=0), dict(N=65537), dict(M=1 << 62), dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(p=0.999999),
        dict(rng=None), dict(rng=Rng(1, 2, 0x1004)), dict(g=None), dict(g=P + 2), dict(h=None)]
FWD = [dict(x=None), dict(r=None), dict(b=None), dict(y=None), dict(y=P + 0x2000), dict(eps=-1.0), dict(eps=float("nan")),
       dict(mean=P + 2), dict(rstd=P + 1), dict(x=P + 1)]
BWD = [dict(dy=None), dict(dr=None), dict(dx=None), dict(dx=P + 0x3000), dict(mean=None), dict(rstd=None), dict(dg=None),
       dict(db=None), dict(dh=P + 1)]


# (calls that are right up to the plan would go on to the device: a bad plan stops them on the host)
@pytest.mark.parametrize("kw", BOTH + FWD, ids=str)
def test_bad_forward_refused(lib, kw):
    assert fwd(lib, **kw) == rn.NORM_ERR_ARG


@pytest.mark.parametrize("kw", BOTH + BWD, ids=str)
def test_bad_backward_refused(lib, kw):
    assert bwd(lib, **kw) == rn.NORM_ERR_ARG


def test_other_refusals(lib):
    assert fwd(lib, dt=9) == rn.NORM_ERR_DTYPE and bwd(lib, dt=-1) == rn.NORM_ERR_DTYPE
    assert fwd(lib, M=0, x=None, h=None, y=None) == rn.NORM_OK
    # (the workspace a call needs depends on its plan, and the default one on the device)
    good = ctypes.byref(rn.NormPlan.from_dict(rn.make_drop_plan(4, 64, torch.float32, True, True)))
    for kw in (dict(ws=None), dict(ws=P + 8), dict(nb=100)):
        assert bwd(lib, plan=good, **kw) == rn.NORM_ERR_ARG, kw
    for plan in (dict(vec_elems=3), dict(threads=100), dict(threads=1024), dict(per_thread=3), dict(stages=1), dict(stages=5),
                 dict(grid=0), dict(grid=1 << 21), dict(cluster=3), dict(cluster=16), dict(mapping=7), dict(rounds=9), dict(group=48)):
        base = dict(rn.make_drop_plan(4, 4096, torch.float32, True), **plan)
        assert fwd(lib, N=4096, plan=ctypes.byref(rn.NormPlan.from_dict(base))) == rn.NORM_ERR_PLAN, plan
        base = dict(rn.make_drop_plan(4, 4096, torch.float32, True, True), **plan)
        assert bwd(lib, N=4096, plan=ctypes.byref(rn.NormPlan.from_dict(base))) == rn.NORM_ERR_PLAN, plan
    # rows of odd width take teams in whole phases
    p = rn.make_drop_plan(100, 5001, torch.bfloat16, True)
    assert p["vec_elems"] == 8 and p["grid"] % 8 == 0
    assert fwd(lib, N=5001, dt=rn.NORM_BF16, plan=ctypes.byref(rn.NormPlan.from_dict(dict(p, grid=12)))) == rn.NORM_ERR_PLAN
    # a plan of vectors does not fit pointers off the 16-byte grid
    assert fwd(lib, x=P + 8, N=5001, dt=rn.NORM_BF16, plan=ctypes.byref(rn.NormPlan.from_dict(p))) == rn.NORM_ERR_PLAN


def shapes():
    rng = random.Random(1)
    for N in [1, 2, 3, 7, 8, 9, 63, 64, 65, 127, 500, 511, 512, 513, 1000, 1023, 2047, 4095, 4096, 4097, 8191, 8192, 8193, 16384, 20001,
              32767, 32768, 40960, 65528, 65536]:
        yield rng.choice([1, 2, 100, 1000, 65536]), N
    for _ in range(300):
        yield int(2 ** rng.uniform(0, 24)), int(2 ** rng.uniform(0, 15.9))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("ln", [True, False])
@pytest.mark.parametrize("backward", [True, False])
def test_every_shape_gets_a_plan_that_covers_it(lib, dtype, ln, backward):
    es = dtype.itemsize
    for M, N in shapes():
        for aligned in (True, False):
            if not aligned and N > 32768:
                with pytest.raises(rn.NormError):
                    rn.make_drop_plan(M, N, dtype, ln, backward, aligned)
                continue
            p = rn.make_drop_plan(M, N, dtype, ln, backward, aligned)
            vec = p["vec_elems"]
            assert vec == (16 // es if aligned else 1), (M, N)
            lead = 0 if N % vec == 0 else max((r * N) % vec for r in range(vec))
            columns = (2 if vec == 1 else vec) * p["per_thread"]
            if p["mapping"] == 0:
                reach, team = p["group"] * columns, p["group"]
                assert p["cluster"] == 1 and p["group"] in (1, 2, 4, 8, 16, 32)
            else:
                team = p["group"] or p["threads"]
                reach = p["cluster"] * team * columns
                assert team % 32 == 0 and p["threads"] % team == 0 and (team == p["threads"] or p["cluster"] == 1)
            assert reach >= lead + N, (M, N, p)
            assert p["threads"] <= 512 and p["threads"] % 32 == 0 and 2 <= p["stages"] <= 4 and p["cluster"] in (1, 2, 4, 8)
            teams = p["grid"] // p["cluster"] * (p["threads"] // team)
            phases = 1
            while phases * N % vec:
                phases *= 2
            assert p["grid"] % p["cluster"] == 0 and teams % phases == 0 and 1 <= p["grid"] <= 1 << 20
            if backward:
                n = ctypes.c_size_t()
                plan = rn.NormPlan.from_dict(p)
                code = {4: rn.NORM_F32}.get(es, rn.NORM_BF16 if dtype == torch.bfloat16 else rn.NORM_F16)
                assert lib.drop_workspace_bytes(M, N, code, int(ln), 0, ctypes.byref(plan), ctypes.byref(n)) == rn.NORM_OK
                values = N * (2 if ln else 1)
                assert n.value == p["grid"] // p["cluster"] * (values + (-values) % 4) * 4
                whole = ctypes.c_size_t()
                assert lib.drop_workspace_bytes(M, N, code, int(ln), 152, None, ctypes.byref(whole)) == rn.NORM_OK
                assert whole.value >= n.value


# ------------------------------------------------------------ head norms with rotation
class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class Side(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int64), ("w", ctypes.c_void_p), ("x", Heads), ("dy", Heads), ("y", Heads), ("dw", ctypes.c_void_p)]


class Angles(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("table_pitch", ctypes.c_int64), ("P", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("position_bytes", ctypes.c_int32), ("R", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def rope(lib, backward=False, B=1, S=4, D=64, eps=1e-6, dt=rn.NORM_F32, ws=P, nb=1 << 40, heads=2, w=P, x=P, dy=P, y=P + 0x8000,
         dw=P, pitch=128, angles=None, plan=None, **a):
    ang = dict(cos=P, sin=P, table_pitch=32, P=16, positions=P, position_bytes=8, R=64, interleaved=0, reserved=0)
    ang.update(a)
    s = Side(heads, w, Heads(x, S * pitch, pitch, D), Heads(dy, S * pitch, pitch, D), Heads(y, S * pitch, pitch, D), dw)
    t = Angles(**ang)
    k = Side(0, None, Heads(), Heads(), Heads(), None)
    if backward:
        return lib.rms_bwd_rope_planned(ctypes.byref(s), ctypes.byref(k), ctypes.byref(t), ws, nb, B, S, D, eps, dt, None, plan)
    return lib.rms_fwd_rope_planned(ctypes.byref(s), ctypes.byref(k), ctypes.byref(t), B, S, D, eps, dt, None, plan)


ROPE = [dict(B=-1), dict(S=-1), dict(D=0), dict(D=513), dict(heads=-1), dict(heads=1 << 20), dict(eps=-1.0), dict(eps=float("inf")),
        dict(w=None), dict(x=None), dict(y=None), dict(x=P + 2), dict(R=3), dict(R=66), dict(R=-2), dict(cos=None), dict(sin=None),
        dict(table_pitch=31), dict(P=0), dict(positions=P + 4), dict(position_bytes=2), dict(reserved=1), dict(B=1 << 31),
        dict(pitch=1 << 41)]


@pytest.mark.parametrize("kw", ROPE, ids=str)
def test_bad_head_norms_refused(lib, kw):
    assert rope(lib, **kw) == rn.NORM_ERR_ARG
    assert rope(lib, True, **kw) == rn.NORM_ERR_ARG


def test_more_bad_head_norms(lib):
    good = ctypes.byref(rn.RopePlan.from_dict(rn.make_rope_plan(4, 2, 0, 64, 64, torch.float32, backward=True)))
    for kw in (dict(dy=None), dict(dw=None), dict(ws=None), dict(nb=10), dict(ws=P + 4)):
        assert rope(lib, True, plan=good, **kw) == rn.NORM_ERR_ARG
    assert rope(lib, dt=5) == rn.NORM_ERR_DTYPE
    assert rope(lib, S=0, x=None, y=None) == rn.NORM_OK
    assert rope(lib, heads=0, x=None, y=None) == rn.NORM_OK
    for kw in (dict(lanes=3), dict(lanes=64), dict(pairs=0), dict(heads=0), dict(warps=9), dict(vec_elems=3), dict(ctas=0), dict(few=2)):
        for backward in (False, True):
            p = rn.RopePlan.from_dict(dict(rn.make_rope_plan(4, 2, 0, 64, 64, torch.float32, backward=backward), **kw))
            assert rope(lib, backward, plan=ctypes.byref(p)) == rn.NORM_ERR_PLAN, kw


@pytest.mark.parametrize("dtype", DT)
def test_every_head_width_gets_a_plan(lib, dtype):
    rng = random.Random(2)
    for D in list(range(1, 513, 7)) + [64, 80, 96, 128, 256, 512]:
        R = 2 * rng.randint(0, D // 2)
        tokens, hq, hk = int(2 ** rng.uniform(0, 20)), rng.randint(1, 64), rng.randint(0, 16)
        for backward in (False, True):
            for vec in {1, 16 // dtype.itemsize if D % 8 == 0 and R % 16 == 0 else 1}:
                p = rn.make_rope_plan(tokens, hq, hk, D, R, dtype, backward=backward, vec_elems=vec)
                assert p["vec_elems"] == vec and p["lanes"] in (1, 2, 4, 8, 16, 32) and p["warps"] in (1, 2, 4, 8)
                assert p["lanes"] * p["pairs"] * 2 * vec >= D, (D, R, p)
                n = ctypes.c_size_t()
                plan = rn.RopePlan.from_dict(p)
                assert lib.rope_workspace_bytes(tokens, hq, hk, D, 152, ctypes.byref(plan), ctypes.byref(n)) == rn.NORM_OK


def test_tasks_of_a_plan_fit_their_counter(lib):
    """A warp of the forward without a loop counts its task in 31 bits: with the last CTA's idle warps, too."""
    T = (1 << 31) - 1
    base = dict(rn.make_rope_plan(T, 1, 0, 1, 0, torch.bfloat16, vec_elems=1), few=1, lanes=32, heads=1)
    for warps in (3, 5, 6, 7):  # (2^31 - 1 tasks in CTAs of these end beyond 2^31 - 1)
        p = ctypes.byref(rn.RopePlan.from_dict(dict(base, warps=warps)))
        assert rope(lib, B=1, S=T, D=1, R=0, heads=1, pitch=1, dt=rn.NORM_BF16, plan=p) == rn.NORM_ERR_PLAN, warps


@pytest.mark.parametrize("dtype", DT)
def test_workspaces_of_the_head_norms(lib, dtype):
    rng = random.Random(4)
    for _ in range(300):
        tokens, hq, hk, D = int(2 ** rng.uniform(0, 20)), rng.randint(1, 64), rng.randint(0, 16), rng.randint(1, 512)
        p = rn.make_rope_plan(tokens, hq, hk, D, 2 * rng.randint(0, D // 2), dtype, backward=True, vec_elems=1)
        n, whole = ctypes.c_size_t(), ctypes.c_size_t()
        assert lib.rope_workspace_bytes(tokens, hq, hk, D, 0, ctypes.byref(rn.RopePlan.from_dict(p)), ctypes.byref(n)) == rn.NORM_OK
        assert n.value == min(p["ctas"], tokens * (hq + hk)) * D * 4
        assert lib.rope_workspace_bytes(tokens, hq, hk, D, 152, None, ctypes.byref(whole)) == rn.NORM_OK
        assert whole.value >= n.value


@pytest.mark.parametrize("backward", [False, True])
def test_every_kernel_of_the_dropout_norms_is_planned(lib, backward):
    """Each instance (accesses a thread, rows a step, who shares a row) is some shape's."""
    for dtype in DT:
        got = set()
        for ln in (True, False):
            for M in (1, 100, 608, 609, 5000, 100000):
                for N in [8, 64, 128, 256, 500, 512, 1000, 1400, 2000, 2040, 4096, 5001, 8192, 20000]:
                    for aligned in (True, False):
                        p = rn.make_drop_plan(M, N, dtype, ln, backward, aligned)
                        got.add((p["vec_elems"] > 1, p["mapping"], p["per_thread"], p["rounds"]))
        wide = (True, 1, 2, 2) if backward and dtype.itemsize == 2 else (True, 1, 4, 1)
        assert got == {(False, 1, 8, 1), (True, 0, 2, 2), (True, 1, 1, 4), wide} | (set() if backward else {(True, 1, 1, 1)}), dtype
