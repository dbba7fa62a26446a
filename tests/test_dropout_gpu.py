"""Dropout + residual add + norm (ln_fwd_dropout_add, rms_fwd_dropout_add), their backwards and the plain add's
(ln_bwd_add, rms_bwd_add), through the Python binding, against the formulas in 64 bits and the generator's own
restatement (philox.py).

Tolerances, from the arithmetic (u = 2^-24, the fp32 rounding; eta = eps / 2 of the row type, one rounding of an output;
half the type's smallest subnormal below that):

h = residual + x scale (kept): the scale is rounded to fp32, the fused multiply-add once: 2 u |x scale| + u |h|, then
  eta |h|.
Norms are held to the h that the call returned. LayerNorm forward, mu the row's mean: with A a first mean, off by at most
  40 u mean|h| (16 values in each of a thread's two sums, their sum, 5 + 4 + 3 levels, the division), the differences
  h - A are within u |h - A|, their sum r and the sum q of their squares within 32 u of their terms' sums, and A + r / n and
  q - r^2 / n are the mean and M2 whatever A is: mean within t = 32 u mean|h - mu| + 4 u |mu|, rstd within
  64 u (1 + (40 u mean|h| rstd)^2); y = (h - mean) rstd gamma + beta: |xhat gamma| times rstd's bar, |gamma| rstd t,
  4 u (|xhat gamma| + |beta|), then eta |y|.
RMSNorm: rstd within 30 u (a thread's 32 squares, 12 levels, halved by the root, rsqrt): y within 36 u |y| + eta |y|.
Backward, A = |xhat| + |mean| rstd (LayerNorm), G = |dy gamma|:
  LayerNorm d: 64 u rstd (G + mean G + A mean(G A)) + 2 u |dh| + eta |d|
  RMSNorm d: 64 u rstd G + 200 u |h| rstd^3 mean(G |h|) + 2 u |dh| + eta |d|
  dx: scale times the part before the rounding, 2 u |d scale|, then eta |dx|.
Column sums: a chain of at most 64 rows, then of M / 64 such, then of at most 16 teams of a CTA, of 24 of at most 760
  partial rows by each of 32 warps and of those 32: (64 + M / 64 + 80 + c) u of the sum of the absolute terms, c = 8 for
  LayerNorm's terms (|dy| A) and 48 for RMSNorm's (|dy h| rstd)."""
import numpy as np
import pytest
import torch

import row_wise_normalization_ln_gb300 as rn
from philox import keep_mask, threshold

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
F = torch.float64
EPS = 1e-5
RNG = (0x123456789ABCDEF, 77)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from row_wise_normalization_ln_gb300 import _build
    _build.build()
    rn.library()


def make(M, N, dtype, seed, loc=0.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * scale + loc).to(dtype).cuda()


def params(N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.3 * torch.randn(N, generator=g)).to(dtype).cuda(), (0.3 * torch.randn(N, generator=g)).to(dtype).cuda())


def mask64(rng, p, M, N):
    scale = 65536 / (65536 - threshold(p))
    if threshold(p) == 0:
        return torch.ones(M, N, dtype=torch.bool, device="cuda"), 1.0
    return torch.from_numpy(keep_mask(*rng, p, M, N)).cuda(), scale


def eta(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 1e-45 if dtype == torch.float32 else torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def within(got, ref, tol, what):
    bad = ~((got.to(F) - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got.to(F) - ref).abs() / tol).nan_to_num(1e9).max()))


def check_h(h, x, r, p, rng):
    M, N = x.shape
    keep, scale = mask64(rng, p, M, N)
    term = torch.where(keep, x.to(F) * scale, 0.0)
    ref = r.to(F) + term
    within(h, ref, 2 * U * term.abs() + (U + eta(x.dtype) * (1 + 8 * U)) * ref.abs() + tiny(x.dtype), "h")
    # what is dropped leaves the residual as it was
    assert torch.equal(h[~keep], r[~keep])


def check_y(ln, h, y, gamma, beta, mean, rstd, eps=EPS):
    v, g = h.to(F), gamma.to(F)
    e = eta(h.dtype) * (1 + 64 * U)
    if not ln:
        rs = (v.square().mean(1, keepdim=True) + eps) ** -0.5
        ref = v * rs * g
        within(y, ref, (36 * U + e) * ref.abs() + tiny(h.dtype), "y")
        return
    mu = v.mean(1, keepdim=True)
    d = v - mu
    rs = (d.square().mean(1, keepdim=True) + eps) ** -0.5
    t_mean = 32 * U * d.abs().mean(1, keepdim=True) + 4 * U * mu.abs()
    t_rs = 64 * U * (1 + (40 * U * v.abs().mean(1, keepdim=True) * rs) ** 2)
    xg = (d * rs * g).abs()
    ref = d * rs * g + beta.to(F)
    within(y, ref, xg * t_rs + g.abs() * rs * t_mean + 4 * U * (xg + beta.to(F).abs()) + e * ref.abs() + tiny(h.dtype), "y")
    if mean is not None:
        within(mean, mu[:, 0], t_mean[:, 0] + 1e-45, "mean")
        within(rstd, rs[:, 0], (t_rs * rs)[:, 0], "rstd")


def fwd(ln, x, r, gamma, beta, p, rng, eps=EPS, **kw):
    if ln:
        return rn.ln_fwd_dropout_add(x, r, gamma, beta, p, rng, eps, **kw)
    return rn.rms_fwd_dropout_add(x, r, gamma, p, rng, eps, **kw) + (None, None)


def check_fwd(ln, x, r, gamma, beta, p, rng, **kw):
    h, y, mean, rstd = fwd(ln, x, r, gamma, beta, p, rng, **kw)
    x2, r2, h2, y2 = (t.reshape(-1, x.shape[-1]) for t in (x, r, h, y))
    check_h(h2, x2, r2, p, rng)
    check_y(ln, h2, y2, gamma, beta, mean, rstd)
    return h, y, mean, rstd


def bwd(ln, dropout, dy, dh, h, gamma, mean, rstd, p, rng, eps=EPS, **kw):
    if dropout:
        if ln:
            return rn.ln_bwd_dropout_add(dy, dh, h, gamma, mean, rstd, p, rng, **kw)
        dx, dr, dw = rn.rms_bwd_dropout_add(dy, dh, h, gamma, p, rng, eps, **kw)
        return dx, dr, dw, None
    if ln:
        d, dg, db = rn.ln_bwd_add(dy, dh, h, gamma, mean, rstd, **kw)
    else:
        (d, dg), db = rn.rms_bwd_add(dy, dh, h, gamma, eps, **kw), None
    return None, d, dg, db


def check_bwd(ln, got, dy, dh, h, gamma, mean, rstd, p, rng, eps=EPS):
    dx, dr, dg, db = got
    M, N = h.shape
    v, y, g = h.to(F), dy.to(F), gamma.to(F)
    e0 = dh.to(F) if dh is not None else torch.zeros_like(v)
    gr = y * g
    G = gr.abs()
    if ln:
        mu, rs = mean.to(F)[:, None], rstd.to(F)[:, None]
        xh = (v - mu) * rs
        A = xh.abs() + mu.abs() * rs
        d = e0 + rs * (gr - gr.mean(1, keepdim=True) - xh * (gr * xh).mean(1, keepdim=True))
        tol = 64 * U * rs * (G + G.mean(1, keepdim=True) + A * (G * A).mean(1, keepdim=True)) + 2 * U * e0.abs()
        term, per = y.abs() * A, 8
        cg = (y * xh).sum(0)
    else:
        rs = (v.square().mean(1, keepdim=True) + eps) ** -0.5
        d = e0 + rs * gr - v * rs ** 3 * (gr * v).mean(1, keepdim=True)
        tol = 64 * U * rs * G + 200 * U * v.abs() * rs ** 3 * (G * v.abs()).mean(1, keepdim=True) + 2 * U * e0.abs()
        term, per = (y * v).abs() * rs, 48
        cg = (y * v * rs).sum(0)
    e = eta(h.dtype) * (1 + 64 * U)
    within(dr, d, tol + (e + U) * d.abs() + tiny(h.dtype), "dresidual")
    if dx is not None:
        keep, scale = mask64(rng, p, M, N)
        ref = torch.where(keep, d * scale, 0.0)
        within(dx, ref, torch.where(keep, tol * scale + (2 * U + e) * ref.abs() + tiny(h.dtype), 0.0), "dx")
    depth = 64 + M / 64 + 80
    within(dg, cg, (depth + per) * U * term.sum(0) + 1e-45, "dgamma")
    assert dg.dtype == torch.float32 and dg.shape == (N,)
    if ln:
        within(db, y.sum(0), depth * U * y.abs().sum(0) + 1e-45, "dbeta")


def both(M, N, dtype, ln, p, seed=0, rng=RNG, fplan=None, bplan=None, loc=0.0):
    dt = DT[dtype]
    x, r = make(M, N, dt, seed), make(M, N, dt, seed + 1, loc, 2.0)
    gamma, beta = params(N, dt, seed + 2)
    h, _, mean, rstd = check_fwd(ln, x, r, gamma, beta, p, rng, plan=fplan)
    dy, dh = make(M, N, dt, seed + 3), make(M, N, dt, seed + 4)
    got = bwd(ln, True, dy, dh, h, gamma, mean, rstd, p, rng, plan=bplan)
    check_bwd(ln, got, dy, dh, h, gamma, mean, rstd, p, rng)
    if p == 0:
        assert torch.equal(got[0], got[1])
        plain = bwd(ln, False, dy, dh, h, gamma, mean, rstd, 0.0, None, plan=bplan)
        assert torch.equal(plain[1], got[1]) and torch.equal(plain[2], got[2])


WIDTHS = [1, 2, 7, 8, 16, 64, 100, 128, 200, 256, 257, 512, 513, 768, 1000, 1024, 1032, 2048, 2051, 4096, 5001, 8192, 8200]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("ln", [True, False])
def test_widths(N, dtype, ln):
    both(9, N, dtype, ln, 0.3, seed=N)


@pytest.mark.parametrize("N,dtype", [(16392, "bf16"), (32768, "f16"), (65536, "bf16"), (16388, "f32"), (65536, "f32"), (20001, "bf16"),
                                     (32767, "f32"), (9000, "f32"), (8191, "f16")])
@pytest.mark.parametrize("ln", [True, False])
def test_long_rows(N, dtype, ln):
    both(5, N, dtype, ln, 0.1, seed=N)


@pytest.mark.parametrize("M", [1, 2, 63, 152, 1000, 5003])
@pytest.mark.parametrize("N,dtype", [(64, "bf16"), (1024, "f32"), (1000, "bf16"), (33, "f16")])
@pytest.mark.parametrize("ln", [True, False])
def test_counts(M, N, dtype, ln):
    both(M, N, dtype, ln, 0.2, seed=M)


@pytest.mark.parametrize("M,N,dtype", [(700, 4096, "f32"), (1301, 4096, "bf16"), (900, 5001, "bf16"), (650, 5003, "f32"), (2000, 1000, "f16"),
                                       (3001, 1001, "bf16"), (4003, 301, "f16"), (5000, 96, "bf16"), (9001, 17, "f32"), (20001, 3, "bf16"),
                                       (10007, 130, "f32"), (640, 2051, "f32"), (333, 10001, "bf16"), (200, 16411, "f32")])
@pytest.mark.parametrize("ln", [True, False])
def test_many_rows(M, N, dtype, ln):
    """Several teams to a CTA, several rows to a team, rows that begin anywhere in a vector."""
    both(M, N, dtype, ln, 0.25, seed=M)


@pytest.mark.parametrize("N,dtype", [(1001, "bf16"), (1001, "f32"), (1000, "f16"), (5001, "bf16"), (31, "f32")])
@pytest.mark.parametrize("ln", [True, False])
def test_views_off_the_vectors(N, dtype, ln):
    """Rows of a larger buffer from any element on, alone or all of them; what lies around them stays."""
    dt, M, p = DT[dtype], 70, 0.25
    gamma, beta = params(N, dt, 1)
    x, r, dy, dh = (make(M, N, dt, i) for i in range(4))
    h, y, mean, rstd = fwd(ln, x, r, gamma, beta, p, RNG)
    grads = bwd(ln, True, dy, dh, h, gamma, mean, rstd, p, RNG)

    def view(t, off):
        buf = torch.full((t.numel() + 16,), 77.0, dtype=dt, device="cuda")
        v = buf[off:off + t.numel()].view(M, N)
        if t is not None:
            v.copy_(t)
        return buf, v

    for offs in ((1, 1, 1, 1, 1), (8, 8, 8, 8, 8), (3, 0, 0, 0, 0), (0, 0, 0, 0, 5), (1, 2, 3, 4, 5)):
        bufs, v = zip(*(view(t, o) for t, o in zip((x, r, dy, dh, h), offs)))
        out = [view(x, o) for o in offs[:2][::-1]]
        got = fwd(ln, v[0], v[1], gamma, beta, p, RNG, h_out=out[0][1], out=out[1][1])
        assert torch.equal(got[0], h)
        check_y(ln, got[0], got[1], gamma, beta, got[2], got[3])
        back = [view(x, o) for o in offs[3:]]
        got = bwd(ln, True, v[2], v[3], v[4], gamma, mean, rstd, p, RNG, dx=back[0][1], dresidual=back[1][1])
        check_bwd(ln, got, dy, dh, h, gamma, mean, rstd, p, RNG)
        assert torch.equal(got[0] == 0, grads[0] == 0)
        for (buf, t), o in list(zip(out, offs[:2][::-1])) + list(zip(back, offs[3:])):
            assert (buf[:o] == 77).all() and (buf[o + t.numel():] == 77).all()


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.05, 0.5, 0.99, 0.9999])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ln", [True, False])
def test_probabilities(p, dtype, ln):
    both(40, 512, dtype, ln, p)
    both(7, 509, dtype, ln, p)


def test_no_rng_where_nothing_is_dropped():
    x, r = make(5, 256, torch.bfloat16, 0), make(5, 256, torch.bfloat16, 1)
    gamma, beta = params(256, torch.bfloat16, 2)
    a = rn.ln_fwd_dropout_add(x, r, gamma, beta, 0.0, None, EPS)
    b = rn.ln_fwd_add(x, r, gamma, beta, EPS)
    assert torch.equal(a[0], b[0])  # h: the plain fused add's, bit for bit
    with pytest.raises(rn.NormError, match="status -1"):
        rn.ln_fwd_dropout_add(x, r, gamma, beta, 0.1, None, EPS)


def test_mask_is_the_same_everywhere():
    """One mask for every type, alignment, plan and place: x of ones on a residual of zeros shows it."""
    M, N, p = 37, 264, 0.25
    want = torch.from_numpy(keep_mask(*RNG, p, M, N)).cuda()
    assert 0.2 < 1 - want.float().mean() < 0.3
    for dtype in DT.values():
        for off in (0, 1):
            buf = torch.ones(M * N + off, dtype=dtype, device="cuda")
            x = buf[off:].view(M, N)
            h, _ = rn.rms_fwd_dropout_add(x, torch.zeros_like(x), torch.ones(N, dtype=dtype, device="cuda"), p, RNG)
            assert torch.equal(h != 0, want)
            one = torch.ones(M, N, dtype=dtype, device="cuda")
            dx, dr, _ = rn.rms_bwd_dropout_add(torch.zeros_like(one), x, one, one[0], p, RNG)
            assert torch.equal(dx != 0, want) and (dr == 1).all()
    other = rn.rms_fwd_dropout_add(one, torch.zeros_like(one), one[0], p, (RNG[0], RNG[1] + 1))[0]
    assert not torch.equal(other != 0, want)
    # seeds and offsets of 64 bits count in full
    for rng in ((RNG[0] ^ (1 << 63), RNG[1]), (RNG[0], RNG[1] ^ (1 << 62)), (-1, -1)):
        h, _ = rn.rms_fwd_dropout_add(one, torch.zeros_like(one), one[0], p, rng)
        assert torch.equal(h != 0, torch.from_numpy(keep_mask(*rng, p, M, N)).cuda())


def test_rng_from_the_device_and_in_graphs():
    M, N, p = 64, 1024, 0.1
    x, r = make(M, N, torch.bfloat16, 0), make(M, N, torch.bfloat16, 1)
    gamma, beta = params(N, torch.bfloat16, 2)
    rng = torch.tensor([5, 9], device="cuda")
    dy, dh = make(M, N, torch.bfloat16, 3), make(M, N, torch.bfloat16, 4)
    want = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, (5, 9), EPS)
    got = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, rng, EPS)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y, mean, rstd = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, rng, EPS)
        grads = rn.ln_bwd_dropout_add(dy, dh, h, gamma, mean, rstd, p, rng)
        rng[1] += 1
    for step in range(9, 12):
        graph.replay()
        torch.cuda.synchronize()
        want = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, (5, step), EPS)
        back = rn.ln_bwd_dropout_add(dy, dh, want[0], gamma, want[2], want[3], p, (5, step))
        assert all(torch.equal(a, b) for a, b in zip(want, (h, y, mean, rstd)))
        assert all(torch.equal(a, b) for a, b in zip(back, grads))


@pytest.mark.parametrize("dtype,N", [("bf16", 1024), ("f32", 1000), ("bf16", 1001), ("f32", 257)])
@pytest.mark.parametrize("ln", [True, False])
def test_in_place(dtype, N, ln):
    """Any output over any input, many rows per CTA."""
    dt = DT[dtype]
    M, p = 3000, 0.1
    x, r = make(M, N, dt, 0), make(M, N, dt, 1)
    gamma, beta = params(N, dt, 2)
    want = fwd(ln, x, r, gamma, beta, p, RNG)
    for h_at, y_at in (("x", "r"), ("r", "x"), ("r", None), (None, "x"), ("x", None), (None, "r")):
        t = {"x": x.clone(), "r": r.clone(), None: torch.empty_like(x)}
        got = fwd(ln, t["x"], t["r"], gamma, beta, p, RNG, h_out=t[h_at], out=t[y_at])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert got[0] is t[h_at] and got[1] is t[y_at]
    h, mean, rstd = want[0], want[2], want[3]
    dy, dh = make(M, N, dt, 3), make(M, N, dt, 4)
    want = bwd(ln, True, dy, dh, h, gamma, mean, rstd, p, RNG)
    for x_at, r_at in (("dy", "dh"), ("dh", "h"), ("h", "dy"), ("h", None), (None, "dh"), (None, "h")):
        t = {"dy": dy.clone(), "dh": dh.clone(), "h": h.clone(), None: torch.empty_like(h)}
        got = bwd(ln, True, t["dy"], t["dh"], t["h"], gamma, mean, rstd, p, RNG, dx=t[x_at], dresidual=t[r_at])
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("ln", [True, False])
def test_no_gradient_of_h(dtype, ln):
    dt = DT[dtype]
    for N in (512, 515):
        h = make(30, N, dt, 0)
        gamma, _ = params(N, dt, 1)
        mean, rstd = h.float().mean(1), (h.float().var(1, unbiased=False) + EPS).rsqrt()
        dy = make(30, N, dt, 2)
        for dropout in (True, False):
            got = bwd(ln, dropout, dy, None, h, gamma, mean, rstd, 0.25 if dropout else 0.0, RNG)
            check_bwd(ln, got, dy, None, h, gamma, mean, rstd, 0.25, RNG)


def test_dropped_values_are_not_looked_at():
    for N, dtype in ((512, torch.bfloat16), (512, torch.float32), (509, torch.float16)):
        x, r = make(20, N, dtype, 0), make(20, N, dtype, 1)
        gamma, beta = params(N, dtype, 2)
        p = 0.4
        keep = torch.from_numpy(keep_mask(*RNG, p, 20, N)).cuda()
        want = rn.rms_fwd_dropout_add(x, r, gamma, p, RNG)
        for v in (float("nan"), float("inf"), torch.finfo(dtype).min):
            got = rn.rms_fwd_dropout_add(torch.where(keep, x, torch.full_like(x, v)), r, gamma, p, RNG)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        y = torch.where(keep, x, torch.full_like(x, float("nan")))
        h, o, mean, rstd = rn.ln_fwd_dropout_add(y, r, gamma, beta, p, RNG, EPS)
        check_y(True, h, o, gamma, beta, mean, rstd)


def test_infinities_stay_in_their_row():
    x, r = make(6, 1024, torch.float32, 0), make(6, 1024, torch.float32, 1)
    gamma, beta = params(1024, torch.float32, 2)
    r[2, 5] = float("inf")
    h, y, mean, rstd = rn.ln_fwd_dropout_add(x, r, gamma, beta, 0.1, RNG, EPS)
    rest = [0, 1, 3, 4, 5]
    assert y[2].isnan().all() and y[rest].isfinite().all()
    d = rn.ln_bwd_dropout_add(x, x, h, gamma, mean, rstd, 0.1, RNG)
    assert d[1][rest].isfinite().all()


@pytest.mark.parametrize("loc", [1000.0, 3e4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_means_that_dwarf_the_spread(loc, dtype):
    both(33, 768, dtype, True, 0.0, loc=loc)
    both(3, 769, dtype, True, 0.1, loc=loc)


PLANS = []
for _N, _dt in ((512, "bf16"), (512, "f32"), (8192, "bf16"), (4096, "f32"), (515, "bf16"), (515, "f32")):
    for _bwd in (False, True):
        PLANS.append((_N, _dt, _bwd))


@pytest.mark.parametrize("N,dtype,backward", PLANS)
@pytest.mark.parametrize("ln", [True, False])
def test_every_plan(N, dtype, backward, ln):
    es = 4 if dtype == "f32" else 2
    tried = set()
    for vec in (1, 16 // es):
        nacc = -(-N // max(vec, 2)) + (vec > 1 and N % vec > 0)
        for per, rounds in ((1, 1), (1, 4), (2, 1), (2, 2), (4, 1), (8, 1)):
            for mapping, group, cluster, threads in [(0, 32, 1, 128), (0, 16, 1, 64)] + [(1, 0, c, t) for c in (1, 2, 8) for t in (32, 128, 320, 512)] + \
                    [(1, 32, 1, 128), (1, 64, 1, 256), (1, 128, 1, 512)]:
                for stages, grid in ((2, 8), (3, 304), (4, 16)):
                    plan = dict(mapping=mapping, vec_elems=vec, per_thread=per, group=group, threads=threads, cluster=cluster,
                                rounds=rounds, stages=stages, grid=grid)
                    reach = (group if group else cluster * threads) * per
                    if reach < nacc or reach > 8 * nacc:
                        continue
                    try:
                        both(13, N, dtype, ln, 0.15, **{"bplan" if backward else "fplan": plan})
                        tried.add((vec, per, rounds, mapping))
                    except rn.NormError as e:
                        assert e.status == rn.NORM_ERR_PLAN
    assert len(tried) >= (2 if N > 1000 or backward else 3), tried


def test_long_chains():
    """Many rows per thread: the chains are folded, on every kind of row."""
    for N, dtype in ((64, "bf16"), (1024, "f32"), (515, "bf16")):
        for ln in (True, False):
            p = rn.make_drop_plan(5000, N, DT[dtype], ln, True)
            both(5000, N, dtype, ln, 0.1, bplan=dict(p, grid=8))


def test_offsets_beyond_32_bits():
    """Rows whose elements, and groups of 8, lie beyond 2^32: only the last rows are looked at."""
    N = 8192
    M = (1 << 32) // N + 5
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-7:] = make(7, N, torch.bfloat16, 1)
    r = torch.zeros_like(x)
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    h, y = rn.rms_fwd_dropout_add(x, r, w, 0.1, RNG, h_out=r)
    keep = torch.from_numpy(keep_mask(*RNG, 0.1, M, N, rows=(M - 7, M))).cuda()
    scale = 65536 / (65536 - threshold(0.1))
    ref = torch.where(keep, x[-7:].to(F) * scale, 0.0)
    within(h[-7:], ref, (3 * U + eta(torch.bfloat16) * (1 + 8 * U)) * ref.abs() + tiny(torch.bfloat16), "h")
    del h, r
    dx, dr, _ = rn.rms_bwd_dropout_add(y, None, x, w, 0.1, RNG, dx=y)
    assert torch.equal(dx[-7:] != 0, keep & (dr[-7:] != 0))


def test_streams_threads_and_determinism():
    import threading
    M, N, p = 2000, 2048, 0.1
    x, r = make(M, N, torch.bfloat16, 0), make(M, N, torch.bfloat16, 1)
    gamma, beta = params(N, torch.bfloat16, 2)
    h, y, mean, rstd = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, RNG, EPS)
    want = (h, y, mean, rstd) + rn.ln_bwd_dropout_add(y, x, h, gamma, mean, rstd, p, RNG)
    torch.cuda.synchronize()
    got = [None] * 3

    def work(i):
        s = torch.cuda.Stream()
        f = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, RNG, EPS, stream=s)
        got[i] = f + rn.ln_bwd_dropout_add(f[1], x, f[0], gamma, f[2], f[3], p, RNG, stream=s)
        s.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_shapes_empty_and_copies():
    x, r = make(24, 128, torch.float16, 0).view(2, 3, 4, 128), make(24, 128, torch.float16, 1).view(2, 3, 4, 128)
    gamma, beta = params(128, torch.float16, 2)
    h, y, mean, rstd = check_fwd(True, x, r, gamma, beta, 0.1, RNG)
    assert h.shape == x.shape and mean.shape == (24,)
    t = x.transpose(0, 1)
    a = rn.ln_fwd_dropout_add(t, r.transpose(0, 1), gamma, beta, 0.1, RNG, EPS)
    b = rn.ln_fwd_dropout_add(t.contiguous(), r.transpose(0, 1).contiguous(), gamma, beta, 0.1, RNG, EPS)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    e = x[:0]
    h, y, mean, rstd = rn.ln_fwd_dropout_add(e, e, gamma, beta, 0.1, RNG, EPS)
    assert h.shape == e.shape and mean.numel() == 0
    out = rn.ln_bwd_dropout_add(e, e, e, gamma, mean, rstd, 0.1, RNG)
    assert (out[2] == 0).all() and (out[3] == 0).all()
    out = rn.rms_bwd_add(e, None, e, gamma)
    assert (out[1] == 0).all()


def test_gradients_against_differences():
    """d(sum(y dy) + sum(h dh)) along a direction of x, residual and parameters, by central differences of the 64-bit
    formula: the step's own error is of the order of its square, 1e-8."""
    M, N, p = 6, 48, 0.3
    x, r = make(M, N, torch.float32, 0), make(M, N, torch.float32, 1)
    gamma, beta = params(N, torch.float32, 2)
    dy, dh = make(M, N, torch.float32, 3), make(M, N, torch.float32, 4)
    keep, scale = mask64(RNG, p, M, N)
    for ln in (True, False):
        def loss(x, r, g, b):
            h = r + torch.where(keep, x * scale, 0.0)
            d = h - h.mean(1, keepdim=True) if ln else h
            y = d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5 * g + (b if ln else 0)
            return (y * dy.to(F)).sum() + (h * dh.to(F)).sum()

        h, _, mean, rstd = fwd(ln, x, r, gamma, beta, p, RNG)
        dx, dr, dg, db = bwd(ln, True, dy, dh, h, gamma, mean, rstd, p, RNG)
        vs = [make(*t.shape, F, 20 + i) if t.dim() == 2 else make(1, N, F, 20 + i)[0] for i, t in enumerate((x, r, gamma, beta))]
        at = [t.to(F) for t in (x, r, gamma, beta)]
        s = 1e-4
        num = (loss(*[a + s * v for a, v in zip(at, vs)]) - loss(*[a - s * v for a, v in zip(at, vs)])) / (2 * s)
        parts = [(g.to(F) * v) for g, v in zip((dx, dr, dg) + ((db,) if ln else ()), vs)]
        ana, size = sum(t.sum() for t in parts), sum(t.abs().sum() for t in parts)
        assert abs(num - ana) <= 1e-6 * size  # h is rounded (u of each value), the terms are within 64 u


def refused(match, kind=ValueError, **kw):
    x, r = make(4, 64, torch.bfloat16, 0), make(4, 64, torch.bfloat16, 1)
    gamma, beta = params(64, torch.bfloat16, 2)
    a = dict(x=x, residual=r, gamma=gamma, beta=beta, p=0.1, rng=RNG)
    a.update({n: (v(a) if callable(v) else v) for n, v in kw.items()})
    with pytest.raises(kind, match=match):
        rn.ln_fwd_dropout_add(**a)


def test_refusals():
    refused("needs CUDA", x=lambda a: a["x"].cpu())
    refused("float32, bfloat16", TypeError, x=lambda a: a["x"].double())
    refused("must be a torch.Tensor", TypeError, residual=3)
    refused("shape", residual=lambda a: a["residual"][:2])
    refused("dtype", residual=lambda a: a["residual"].float())
    refused("64 elements", gamma=lambda a: a["gamma"][:3])
    refused("dtype", beta=lambda a: a["beta"].float())
    refused("rng must be", TypeError, rng=3)
    refused("rng must be", TypeError, rng=(1, 2, 3))
    refused("rng must be", rng=lambda a: torch.tensor([1, 2]))
    refused("rng must be", rng=lambda a: torch.tensor([1, 2], device="cuda", dtype=torch.int32))
    refused("float", TypeError, rng=(1.5, 2))
    for p in (-0.1, 1.0, 1.5, float("nan"), 0.999999):
        refused("status -1", rn.NormError, p=p)
    refused("status -1", rn.NormError, h_out=lambda a: a["x"], out=lambda a: a["x"])
    refused("contiguous", out=lambda a: a["x"].t().contiguous().t())
    refused("status -1", rn.NormError, eps=float("inf"))
    wide = torch.zeros(1, 65537, device="cuda")
    with pytest.raises(rn.NormError):
        rn.rms_fwd_dropout_add(wide, wide, wide[0], 0.1, RNG)
    x, r = make(4, 64, torch.bfloat16, 0), make(4, 64, torch.bfloat16, 1)
    gamma, beta = params(64, torch.bfloat16, 2)
    h, y, mean, rstd = rn.ln_fwd_dropout_add(x, r, gamma, beta, 0.1, RNG)
    with pytest.raises(ValueError, match="mean"):
        rn.ln_bwd_dropout_add(y, None, h, gamma, mean[:2], rstd, 0.1, RNG)
    with pytest.raises(ValueError, match="dh must"):
        rn.ln_bwd_dropout_add(y, h[:2], h, gamma, mean, rstd, 0.1, RNG)
    with pytest.raises(rn.NormError):
        rn.ln_bwd_dropout_add(y, h, h, gamma, mean, rstd, 0.1, RNG, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(rn.NormError):
        rn.ln_bwd_dropout_add(y, h, h, gamma, mean, rstd, 0.1, RNG, dx=y, dresidual=y)
    with pytest.raises(rn.NormError, match="status -4"):
        rn.ln_fwd_dropout_add(x, r, gamma, beta, 0.1, RNG, plan=dict(rn.make_drop_plan(4, 64, x.dtype, True), per_thread=3))


@pytest.mark.parametrize("loc", [300.0, 3e4, -2e5])
@pytest.mark.parametrize("M,N", [(7, 96), (1000, 96), (5, 513), (33, 768), (9, 1024), (700, 1024), (33, 769), (6, 5001), (64, 4096), (300, 8192), (4, 16388)])
def test_outputs_keep_their_digits_under_a_large_mean(M, N, loc):
    """LayerNorm's y from h - A and mean - A, A near the mean: no rounding of the size of the mean itself. |h - A| <= S = 2 max|h - mu|
    + 40 u mean|h| for each warp's A; mean - A is within 40 u S (32 u of a sum of such differences, the merge's), h - A within u S, the
    fused multiply-add within 2 u of both: 44 u S rstd |gamma| beside rstd's own bar, and the output's roundings."""
    for off in (0, 1):  # vectors, elements
        x = torch.empty(M * N + off, device="cuda")[off:].view(M, N)
        x.copy_(make(M, N, torch.float32, 0))
        r = make(M, N, torch.float32, 1, loc, 2.0)
        gamma, beta = params(N, torch.float32, 2)
        for p in (0.0, 0.1):
            h, y, mean, rstd = rn.ln_fwd_dropout_add(x, r, gamma, beta, p, RNG, EPS)
            v, g, b = h.to(F), gamma.to(F), beta.to(F)
            d = v - v.mean(1, keepdim=True)
            rs = (d.square().mean(1, keepdim=True) + EPS) ** -0.5
            S = 2 * d.abs().amax(1, keepdim=True) + 40 * U * v.abs().mean(1, keepdim=True)
            t_rs = 64 * U * (1 + (40 * U * v.abs().mean(1, keepdim=True) * rs) ** 2)
            xg = (d * rs * g).abs()
            tol = xg * t_rs + 44 * U * S * rs * g.abs() + 4 * U * (xg + b.abs()) + U * (1 + 64 * U) * (d * rs * g + b).abs()
            within(y, d * rs * g + b, tol, "y")


def test_groups_beyond_32_bits():
    """The counter's upper word: elements from 2^35 on, 64 GB a tensor. Only the last rows, and those before the border, are looked at."""
    N = 8192
    M, border = (1 << 35) // N + 3, (1 << 35) // N
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of the device")
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-6:] = make(6, N, torch.bfloat16, 1)
    x[-6:] += (x[-6:] == 0)
    was = x[-6:].clone()
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    h, _ = rn.rms_fwd_dropout_add(x, x, w, 0.25, RNG, h_out=x, out=y)  # x is its own residual: x (1 + keep / P(keep))
    keep = torch.from_numpy(keep_mask(*RNG, 0.25, M, N, rows=(M - 6, M))).cuda()
    assert M - 6 < border < M
    ref = was.to(F) * (1 + keep * (65536 / (65536 - threshold(0.25))))
    within(h[-6:], ref, (3 * U + eta(torch.bfloat16) * (1 + 8 * U)) * ref.abs() + tiny(torch.bfloat16), "h")
    dx, dr, _ = rn.rms_bwd_dropout_add(h, h, h, w, 0.25, RNG, dx=y, dresidual=h)
    assert torch.equal(dx[-6:] != 0, keep & (dr[-6:] != 0)) and (dr[-6:] != 0).float().mean() > 0.9
    del x, y, h, dx, dr
    torch.cuda.empty_cache()
