"""Group norm with an activation, channels last (gn_fwd, gn_bwd), through the
Python binding, against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, the fp32 rounding; eta = eps / 2
of the output type, one rounding of the output):

mean: K + mu is rounded once, mu is a sum of differences from K, each exact
  to u, merged over at most ~20 levels: 32 u (|mean| + sigma + |K - mean|),
  with |K - mean| <= max|x - mean|.
rstd: relative 64 u plus what the rounding of mu adds to the variance, which
  is second order; the shifted squares of gn_fwd_sums lose at most
  u * rows-per-shift (32) * (K_t - mean)^2 / sigma^2 in the worst data; the
  data here has (K_t - mean)^2 <= 40 sigma^2, errors of the terms add as
  random: 64 u + 40 * 12 u < 600 u = 3.6e-5. Bar: 600 u.
y: z = xhat gamma + beta has an error of at most 600 u |xhat gamma| from rstd
  and 64 u (|mean| rstd |gamma| + |xhat gamma| + |beta|) from the rest (the
  forward adds back what the rounding of the mean leaves, but 64-bit inputs
  share only fp32 gamma, beta). |act'| <= 1.13 for silu and gelu; the activation itself adds
  at most 16 u (|z| + 1) (exp and the division are within a few ulp, the
  normal tail within 3 u). Then eta |y| for the output's rounding, and half the smallest
  subnormal of the type.
dx = rstd (g - m1 - xhat m2): per value 64 u rstd (|g| + |m1| + |xhat m2|) for
  the arithmetic and the slope (|act''| <= 0.8: z's error 64 u (|xhat gamma| +
  |beta| + |mean| rstd |gamma|) enters g times |dy gamma|), and for the sums
  m1, m2 their fp32 accumulation: 64 u times the mean of the absolute terms.
  Then eta |dx|.
dgamma, dbeta: 64 u times the sum of the absolute terms, plus the slope's and
  xhat's errors in each term: as for dx.
Sums over n values in blocks of 32 and trees have an error below (32 + 128) u
of the absolute sum in the worst case and about 13 u in practice; 64 u leaves
room and is far below any wrong formula (a dropped m2 is of order 1)."""
import math
import random

import pytest
import torch

import row_wise_normalization_ln_gb300 as rn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
F = torch.float64
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from row_wise_normalization_ln_gb300 import _build
    _build.build()
    rn.library()


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z


def slope64(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def make(B, S, C, dtype, seed, loc=0.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, C, generator=g) * scale * (0.5 + torch.rand(C, generator=g)) + loc
    dy = torch.randn(B, S, C, generator=g)
    gamma = 1 + 0.3 * torch.randn(C, generator=g)
    beta = 0.3 * torch.randn(C, generator=g)
    return [t.to(dtype).cuda() for t in (x, dy, gamma, beta)]


def spread(v, D):
    return v.repeat_interleave(D, dim=-1).unsqueeze(1)  # [B, G] -> [B, 1, C]


def out_tol(ref, dtype):
    fi = torch.finfo(dtype)
    return fi.eps / 2 * ref.abs() + fi.smallest_normal * fi.eps


def check_fwd(x, gamma, beta, G, act, y, mean, rstd, eps=EPS, extra=0.0):
    B, C = x.shape[0], x.shape[-1]
    D = C // G
    x = x.reshape(B, -1, C)
    x64, g64, b64 = x.to(F), gamma.to(F), beta.to(F)
    xg = x64.reshape(B, -1, G, D)
    mu = xg.mean((1, 3))
    dev = xg - mu.view(B, 1, G, 1)
    var = dev.square().mean((1, 3))
    eps = float(torch.tensor(eps, dtype=torch.float32))
    r = (var + eps).rsqrt()
    if mean is not None:
        far = dev.abs().amax((1, 3))
        assert ((mean.to(F) - mu).abs() <= 32 * U * (mu.abs() + var.sqrt() + far)).all()
    if rstd is not None:
        rel = ((rstd.to(F) - r).abs() / r).max().item()
        assert rel <= 600 * U, rel
    xh = dev.reshape(B, -1, C) * spread(r, D)
    z = xh * g64 + b64
    ref = act64(z, act)
    tol = 1.13 * U * (664 * (xh * g64).abs() + 64 * (b64.abs() + spread(mu.abs() * r, D) * g64.abs()))
    tol = tol + 16 * U * (z.abs() + 1) + out_tol(ref, y.dtype) + extra * U * g64.abs()
    bad = ~((y.reshape(B, -1, C).to(F) - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((y.reshape(B, -1, C).to(F) - ref).abs().max()))
    return mu, r


def check_bwd(dy, x, gamma, beta, mean, rstd, G, act, dx, dg, db):
    B, C = x.shape[0], x.shape[-1]
    D = C // G
    x, dy, dx = (t.reshape(B, -1, C) for t in (x, dy, dx))
    x64, dy64, g64, b64 = x.to(F), dy.to(F), gamma.to(F), beta.to(F)
    mu, r = spread(mean.to(F), D), spread(rstd.to(F), D)
    xh = (x64 - mu) * r
    z = xh * g64 + b64
    dz = dy64 * slope64(z, act)
    zerr = 64 * U * ((xh * g64).abs() + b64.abs() + mu.abs() * r * g64.abs() + 1)
    dzerr = dy64.abs() * (0.8 * zerr if act not in (None, "none") else 0) + 64 * U * dz.abs()
    g = dz * g64
    n = x.shape[1] * D

    def per_group(t):
        return spread(t.reshape(B, -1, G, D).sum((1, 3)) / n, D)

    m1, m2 = per_group(g), per_group(g * xh)
    xherr = 8 * U * (xh.abs() + mu.abs() * r)
    ge = dzerr * g64.abs() + 8 * U * g.abs()
    e1 = per_group(ge + 64 * U * g.abs())
    e2 = per_group(ge * xh.abs() + g.abs() * xherr + 64 * U * (g * xh).abs())
    ref = r * (g - m1 - xh * m2)
    tol = r * (ge + e1 + xh.abs() * e2 + xherr * m2.abs() + 16 * U * (g.abs() + m1.abs() + (xh * m2).abs()))
    err = (dx.to(F) - ref).abs()
    bad = ~(err <= tol + out_tol(ref, dx.dtype))
    assert not bad.any(), (int(bad.sum()), float(err.max()))
    for got, terms, te in ((db, dz, dzerr), (dg, dz * xh, dzerr * xh.abs() + dz.abs() * xherr)):
        t = (te + 64 * U * terms.abs()).sum((0, 1))
        bad = ~((got.to(F) - terms.sum((0, 1))).abs() <= t)
        assert not bad.any(), (int(bad.sum()), float((got.to(F) - terms.sum((0, 1))).abs().max()))


def check_both(B, S, C, G, dtype, act, seed=0, loc=0.0, scale=1.0, plans=(None, None)):
    x, dy, gamma, beta = make(B, S, C, dtype, seed, loc, scale)
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS, activation=act, plan=plans[0])
    check_fwd(x, gamma, beta, G, act, y, mean, rstd)
    dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, G, activation=act, plan=plans[1])
    check_bwd(dy, x, gamma, beta, mean, rstd, G, act, dx, dg, db)


SHAPES = [  # B, S, C, G: one value, one row, one channel a group, odd everything, straddling accesses, wide groups
    (1, 1, 1, 1), (1, 1, 64, 8), (3, 1, 40, 4), (2, 2, 8, 8), (1, 7, 5, 1), (2, 33, 30, 6), (3, 64, 32, 32),
    (1, 61, 320, 32), (2, 256, 320, 32), (1, 100, 1280, 32), (2, 37 * 41, 180, 30), (5, 129, 75, 25),
    (1, 4096, 320, 32), (1, 1023, 96, 1), (2, 17, 4096, 2), (1, 9, 8200, 8), (2, 300, 250, 25), (1, 70, 16, 2),
    (64, 4, 24, 3), (1, 20000, 64, 8), (1, 5000, 130, 13), (2, 16384, 128, 32), (1, 3, 5001, 1), (1, 2000, 1001, 7),
    (512, 3, 24, 3), (513, 3, 24, 3), (1300, 3, 40, 5), (20000, 2, 64, 8), (700, 1, 75, 25),  # many samples
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    B, S, C, G = shape
    check_both(B, S, C, G, DT[dtype], ["none", "silu", "gelu"][(S + C) % 3], seed=S)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("dtype", list(DT))
def test_activations(dtype, act):
    check_both(2, 300, 64, 8, DT[dtype], act, seed=3, scale=3.0)


def gn_plans(B, S, C, G, dtype, backward):
    """Explicit plans over every path, access width, cluster size and rows per
    thread that fit the shape."""
    D = C // G
    full = 16 // dtype.itemsize
    out = []
    for vec in (full, 2, 1):
        if C % vec or (vec == 2 and dtype.itemsize == 4):
            continue
        unit = D // math.gcd(D, vec)
        for cluster in (1, 2, 4, 8):
            rows = -(-S // cluster)
            for tile in {unit, min(2 * unit, C // vec), C // vec}:
                if tile > 256 or (D % vec and tile * vec > 512):
                    continue
                for v in (1, 2, 4) + (() if backward else (8,)):
                    par = -(-rows // v)
                    threads = -(-par * tile // 32) * 32
                    if threads <= 256:
                        out.append(dict(path=0, vec_elems=vec, tile=tile, threads=threads, per_thread=v,
                                        cluster=cluster, chunks=1, out_chunks=1))
                for threads in (128, 256):
                    if tile <= threads:
                        out.append(dict(path=1, vec_elems=vec, tile=tile, threads=threads, per_thread=1, cluster=1,
                                        chunks=2 * cluster - 1, out_chunks=9 - cluster))
            for tile in (8, 37):  # groups that straddle tiles
                out.append(dict(path=1, vec_elems=vec, tile=tile, threads=64, per_thread=1, cluster=1,
                                chunks=3 * cluster, out_chunks=5))
    return out


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(2, 77, 48, 6), (1, 130, 40, 4), (1, 50, 200, 2)], ids=str)
def test_every_plan(shape, dtype):
    B, S, C, G = shape
    dt = DT[dtype]
    x, dy, gamma, beta = make(B, S, C, dt, 11, loc=2.0)
    for plan in gn_plans(B, S, C, G, dt, False):
        y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS, activation="silu", plan=plan)
        try:
            check_fwd(x, gamma, beta, G, "silu", y, mean, rstd)
        except AssertionError as e:
            raise AssertionError(f"{plan}: {e}") from None
    for plan in gn_plans(B, S, C, G, dt, True):
        dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, G, activation="silu", plan=plan)
        try:
            check_bwd(dy, x, gamma, beta, mean, rstd, G, "silu", dx, dg, db)
        except AssertionError as e:
            raise AssertionError(f"{plan}: {e}") from None


@pytest.mark.parametrize("S", [40, 30000])
@pytest.mark.parametrize("loc,scale", [(1000.0, 0.01), (-3e4, 1.0), (0.0, 1e-4)])
def test_means_that_dwarf_the_spread(loc, scale, S):
    check_both(2, S, 64, 8, torch.float32, "none", seed=9, loc=loc, scale=scale)


@pytest.mark.parametrize("S,C,G", [(40, 64, 8), (2000, 64, 8), (4000, 64, 8), (40000, 64, 2)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_one_value_far_from_the_rest(S, C, G, where):
    """A value M far off in each group, the group's first too, from which the
    differences are taken: with n values, rstd is about sqrt(n) / M. The sums
    of a thread's up to 32 differences of size M round by about 60 u M, as
    random; averaged over the group's n / 32 threads and times rstd that is 10 u;
    64 u for six times it. Outputs formed from the differences themselves would
    be off by u M rstd = u sqrt(n) / 2 each, 560 u for the longest."""
    x, _, gamma, beta = make(2, S, C, torch.float32, 11)
    x[:, 0 if where == "first" else S - 1, ::C // G] = 1e4
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS)
    check_fwd(x, gamma, beta, G, "none", y, mean, rstd, extra=64)


@pytest.mark.parametrize("S", [64, 20000])
def test_constant_groups_give_beta(S):
    x = torch.full((2, S, 32), 7.25, device="cuda")
    gamma, beta = torch.rand(32, device="cuda") + 1, torch.randn(32, device="cuda")
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 4, EPS)
    assert torch.equal(y, beta.expand_as(y)) and (mean == 7.25).all()
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("S", [50, 20000])
def test_infinities_and_nan_stay_in_their_group(S):
    x, dy, gamma, beta = make(2, S, 64, torch.bfloat16, 4)
    clean, _, _ = rn.gn_fwd(x, gamma, beta, 8, EPS, activation="silu")
    x[0, S // 2, 9] = float("nan")   # group 1 of sample 0
    x[1, S - 1, 63] = float("inf")   # group 7 of sample 1
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 8, EPS, activation="silu")
    hit = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 7] = True
    assert torch.equal(~torch.isfinite(mean) | ~torch.isfinite(rstd), hit)
    per = y.view(2, S, 8, 8)
    assert torch.isnan(per[0, :, 1]).all() and torch.isnan(per[1, :, 7]).all()
    keep = ~hit.view(2, 1, 8, 1).expand(2, S, 8, 8)
    assert torch.equal(per[keep], clean.view(2, S, 8, 8)[keep])
    dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 8, activation="silu")
    d = dx.view(2, S, 8, 8)
    assert torch.isfinite(d[keep]).all() and torch.isnan(d[0, :, 1]).all() and torch.isnan(d[1, :, 7]).all()
    assert torch.isfinite(dg[16:56]).all() and torch.isfinite(db[16:56]).all()


def test_extreme_activation_arguments():
    """silu and gelu far out: y -> z or 0, slopes -> 1 or 0, no NaN."""
    x = torch.zeros(1, 4, 8, device="cuda")
    x[0, 0], x[0, 1] = 1.0, -1.0
    gamma = torch.full((8,), 200.0, device="cuda")
    beta = torch.zeros(8, device="cuda")
    for act in ("silu", "gelu"):
        y, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS, activation=act)
        check_fwd(x, gamma, beta, 1, act, y, mean, rstd)
        dx, dg, db = rn.gn_bwd(torch.ones_like(x), x, gamma, beta, mean, rstd, 1, activation=act)
        check_bwd(torch.ones_like(x), x, gamma, beta, mean, rstd, 1, act, dx, dg, db)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_over_their_range(act):
    """Arguments from -13 to 13 in steps of 1e-4, where the statistics leave
    them as they are (mean 0, rstd 1 up to roundings): outputs and slopes of
    every part of the approximations."""
    half = torch.linspace(1e-4, 13, 130000)
    x = torch.cat([half, -half]).view(1, -1, 1).cuda()
    sigma = float(x.double().square().mean().sqrt())
    gamma, beta = torch.full((1,), sigma, device="cuda"), torch.zeros(1, device="cuda")
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS, activation=act)
    check_fwd(x, gamma, beta, 1, act, y, mean, rstd)
    dx, dg, db = rn.gn_bwd(torch.ones_like(x), x, gamma, beta, mean, rstd, 1, activation=act)
    check_bwd(torch.ones_like(x), x, gamma, beta, mean, rstd, 1, act, dx, dg, db)


def test_gradient_against_differences():
    """dx, dgamma, dbeta against central differences of the 64-bit forward."""
    B, S, C, G = 2, 6, 12, 3
    for act in (None, "silu", "gelu"):
        x, dy, gamma, beta = make(B, S, C, torch.float32, 21)

        def loss(xv, gv, bv):
            xg = xv.reshape(B, S, G, C // G)
            m = xg.mean((1, 3), keepdim=True)
            r = ((xg - m).square().mean((1, 3), keepdim=True) + EPS).rsqrt()
            z = ((xg - m) * r).reshape(B, S, C) * gv + bv
            return (act64(z, act) * dy.to(F)).sum()

        p = [t.to(F) for t in (x, gamma, beta)]
        y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS, activation=act)
        got = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, G, activation=act)
        for k in range(3):
            want = torch.empty_like(p[k])
            for i in range(p[k].numel()):
                q = [t.clone() for t in p]
                q[k].view(-1)[i] += 1e-5
                up = loss(*q)
                q[k].view(-1)[i] -= 2e-5
                want.view(-1)[i] = (up - loss(*q)) / 2e-5
            # differences: h^2 = 1e-10 times third derivatives of order 100, fp32 gradients of order 10
            assert (got[k].to(F) - want).abs().max() <= 2e-5 * max(1.0, float(want.abs().max()))


# ------------------------------------------------------------ layouts

def strided(t, where, pad):
    """t [B, S, C] as a view of a wider buffer, canaries around it."""
    B, S, C = t.shape
    if where == "columns":
        buf = torch.full((B, S, C + 2 * pad), 77.0, dtype=t.dtype, device="cuda")
        v = buf[:, :, pad:pad + C]
    elif where == "rows":
        buf = torch.full((B, S + 2 * pad, C), 77.0, dtype=t.dtype, device="cuda")
        v = buf[:, pad:pad + S]
    else:
        buf = torch.full((B * S * C + 2 * pad,), 77.0, dtype=t.dtype, device="cuda")
        v = buf[pad:pad + B * S * C].view(B, S, C)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("S", [45, 9000])
@pytest.mark.parametrize("where,pad", [("columns", 8), ("columns", 3), ("columns", 2), ("rows", 5), ("flat", 1),
                                       ("flat", 2), ("flat", 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_alignment_and_guards(dtype, where, pad, S):
    dt = DT[dtype]
    x, dy, gamma, beta = make(2, S, 48, dt, 5)
    _, xv = strided(x, where, pad)
    _, dyv = strided(dy, where, pad)
    ybuf, yv = strided(torch.full_like(x, 77.0), where, pad)
    y, mean, rstd = rn.gn_fwd(xv, gamma, beta, 6, EPS, activation="silu", out=yv)
    assert y is yv
    check_fwd(x, gamma, beta, 6, "silu", yv, mean, rstd)
    dx, dg, db = rn.gn_bwd(dyv, xv, gamma, beta, mean, rstd, 6, activation="silu")
    check_bwd(dy, x, gamma, beta, mean, rstd, 6, "silu", dx, dg, db)
    rn.gn_bwd(dyv, xv, gamma, beta, mean, rstd, 6, activation="silu", dx=yv)
    check_bwd(dy, x, gamma, beta, mean, rstd, 6, "silu", yv, dg, db)
    yv.fill_(77.0)
    assert (ybuf == 77.0).all()  # nothing outside the view was written
    # inputs untouched
    assert torch.equal(xv, x) and torch.equal(dyv, dy)


def test_channels_last_memory_format_and_more_dims():
    x = torch.randn(2, 64, 9, 7, device="cuda").to(memory_format=torch.channels_last)
    gamma, beta = torch.rand(64, device="cuda") + 0.5, torch.randn(64, device="cuda")
    xv = x.permute(0, 2, 3, 1)
    y, mean, rstd = rn.gn_fwd(xv, gamma, beta, 8, EPS, activation="silu")
    assert y.shape == xv.shape and mean.shape == (2, 8)
    check_fwd(xv, gamma, beta, 8, "silu", y, mean, rstd)
    v = torch.randn(1, 3, 4, 5, 24, device="cuda").transpose(1, 2)  # no common pitch: copied
    g2 = torch.ones(24, device="cuda")
    y, mean, rstd = rn.gn_fwd(v, g2, 0 * g2, 4, EPS)
    check_fwd(v, g2, 0 * g2, 4, None, y, mean, rstd)
    two = torch.randn(6, 24, device="cuda")
    y, mean, rstd = rn.gn_fwd(two, g2, 0 * g2, 4, EPS)
    assert y.shape == (6, 24)
    check_fwd(two.unsqueeze(1), g2, 0 * g2, 4, None, y.unsqueeze(1), mean, rstd)


@pytest.mark.parametrize("S", [100, 30000])
def test_expanded_gradient_and_in_place(S):
    x, dy, gamma, beta = make(2, S, 40, torch.bfloat16, 6)
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 4, EPS, activation="gelu")
    one = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(2, S, 40)
    dx, dg, db = rn.gn_bwd(one, x, gamma, beta, mean, rstd, 4, activation="gelu")
    check_bwd(one, x, gamma, beta, mean, rstd, 4, "gelu", dx, dg, db)
    ref = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 4, activation="gelu")
    for target in ("dy", "x"):
        d2, x2 = dy.clone(), x.clone()
        got = rn.gn_bwd(d2, x2, gamma, beta, mean, rstd, 4, activation="gelu", dx=d2 if target == "dy" else x2)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    x2 = x.clone()
    assert rn.gn_fwd(x2, gamma, beta, 4, EPS, activation="gelu", out=x2)[0] is x2
    assert torch.equal(x2, y)


def test_more_than_2_31_values():
    """64-bit offsets: the last rows of the last sample of a large tensor."""
    B, S, C, G = 3, 1 << 22, 256, 8
    x = torch.empty(B, S, C, dtype=torch.bfloat16, device="cuda").normal_()
    gamma, beta = torch.ones(C, dtype=torch.bfloat16, device="cuda"), torch.zeros(C, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS)
    for b, s in ((0, 0), (B - 1, S - 1000)):
        xs = x[b, s:s + 1000].float()
        want = (xs - mean[b].repeat_interleave(C // G)) * rstd[b].repeat_interleave(C // G)
        assert (y[b, s:s + 1000].float() - want).abs().max() <= 2.0 ** -7 * 8
    dx, dg, db = rn.gn_bwd(y, x, gamma, beta, mean, rstd, G)
    # dy = xhat: dx vanishes but for roundings (dy is off xhat by up to 2^-8 |xhat|), dgamma = B S
    assert dx[B - 1, S - 1000:].float().abs().max() <= 2.0 ** -8 * 8
    assert ((dg / (B * S)) - 1).abs().max() <= 1e-2 and (db.abs() / (B * S)).max() <= 1e-2


# ------------------------------------------------------------ ways of calling

def test_no_statistics_and_empty_tensors():
    x, dy, gamma, beta = make(2, 50, 16, torch.float32, 1)
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 4, stats=False)
    assert mean is None and rstd is None and torch.equal(y, rn.gn_fwd(x, gamma, beta, 4)[0])
    for shape in ((0, 5, 16), (2, 0, 16)):
        e = torch.empty(shape, device="cuda")
        y, mean, rstd = rn.gn_fwd(e, gamma, beta, 4)
        assert y.shape == shape
        dg, db = torch.full((16,), 3.0, device="cuda"), torch.full((16,), 3.0, device="cuda")
        dx, dg, db = rn.gn_bwd(e, e, gamma, beta, mean, rstd, 4, dgamma=dg, dbeta=db)
        assert dx.shape == shape and not dg.any() and not db.any()


def test_deterministic():
    for B, S, C, G in ((2, 30000, 64, 8), (3, 100, 320, 32)):
        x, dy, gamma, beta = make(B, S, C, torch.bfloat16, 2)
        a = rn.gn_fwd(x, gamma, beta, G, activation="silu")
        ab = rn.gn_bwd(dy, x, gamma, beta, a[1], a[2], G, activation="silu")
        for _ in range(3):
            b = rn.gn_fwd(x, gamma, beta, G, activation="silu")
            bb = rn.gn_bwd(dy, x, gamma, beta, b[1], b[2], G, activation="silu")
            assert all(torch.equal(p, q) for p, q in zip(a + ab, b + bb))


def test_streams_and_graphs():
    """Calls on two streams at once (own workspaces), and forward and backward
    captured together and replayed on new inputs."""
    cases = [make(2, 20000, 64, torch.bfloat16, s) for s in (1, 2)]
    want = []
    for x, dy, gamma, beta in cases:
        y, m, r = rn.gn_fwd(x, gamma, beta, 8, activation="silu")
        want.append((y, m, r) + rn.gn_bwd(dy, x, gamma, beta, m, r, 8, activation="silu"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for rep in range(3):
        for k, ((x, dy, gamma, beta), s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                y, m, r = rn.gn_fwd(x, gamma, beta, 8, activation="silu")
                got[k] = (y, m, r) + rn.gn_bwd(dy, x, gamma, beta, m, r, 8, activation="silu")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    # the stream argument: the call runs there, not on the current stream
    x, dy, gamma, beta = cases[0]
    y = torch.empty_like(x)
    streams[0].wait_stream(torch.cuda.current_stream())
    rn.gn_fwd(x, gamma, beta, 8, activation="silu", out=y, stream=streams[0], stats=False,
              workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    streams[0].synchronize()
    assert torch.equal(y, want[0][0])
    x, dy, gamma, beta = (t.clone() for t in cases[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, m, r = rn.gn_fwd(x, gamma, beta, 8, activation="silu")
        res = (y, m, r) + rn.gn_bwd(dy, x, gamma, beta, m, r, 8, activation="silu")
    for k in (1, 0):
        for t, src in zip((x, dy, gamma, beta), cases[k]):
            t.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want[k]))


def test_large_tensors():
    """Tensors beyond L2, forward and backward, in place too."""
    for B, S, C, G, dt, act in ((1, 130001, 256, 32, torch.bfloat16, "silu"), (3, 70003, 320, 32, torch.float16, "gelu"),
                                (2, 40009, 384, 2, torch.float32, None)):
        x, dy, gamma, beta = make(B, S, C, dt, 8, loc=1.0)
        y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS, activation=act)
        dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, G, activation=act)
        for b in range(B):  # (sample by sample: the 64-bit copies stay small)
            check_fwd(x[b:b + 1], gamma, beta, G, act, y[b:b + 1], mean[b:b + 1], rstd[b:b + 1])
        if B == 1:
            check_bwd(dy, x, gamma, beta, mean, rstd, G, act, dx, dg, db)
        else:
            parts = [rn.gn_bwd(dy[b:b + 1], x[b:b + 1], gamma, beta, mean[b:b + 1], rstd[b:b + 1], G, activation=act)
                     for b in range(B)]
            for b in range(B):
                check_bwd(dy[b:b + 1], x[b:b + 1], gamma, beta, mean[b:b + 1], rstd[b:b + 1], G, act, dx[b:b + 1],
                          parts[b][1], parts[b][2])
            # the columns of all samples: each sample's within its bound, one more fp32 addition each
            for got, k in ((dg, 1), (db, 2)):
                each = torch.stack([p[k] for p in parts]).to(F)
                assert ((got.to(F) - each.sum(0)).abs() <= 64 * U * (S ** 0.5) * (each.abs().sum(0) + 8)).all()
        y2 = rn.gn_fwd(x.clone(), gamma, beta, G, EPS, activation=act)[0]
        x2 = x.clone()
        rn.gn_fwd(x2, gamma, beta, G, EPS, activation=act, out=x2)
        assert torch.equal(x2, y) and torch.equal(y2, y)
        d2 = dy.clone()
        rn.gn_bwd(d2, x, gamma, beta, mean, rstd, G, activation=act, dx=d2)
        assert torch.equal(d2, dx)


def test_random_shapes():
    rng = random.Random(7)
    for i in range(60):
        D = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 20, 33, 40, 64])
        G = rng.choice([1, 2, 4, 8, 25, 32])
        B = rng.choice([1, 1, 2, 3, 9])
        S = max(1, int(math.exp(rng.uniform(0, math.log(3e6 / (B * D * G))))))
        dtype = rng.choice(list(DT.values()))
        try:
            check_both(B, S, D * G, G, dtype, rng.choice([None, "silu", "gelu"]), seed=i, loc=rng.choice([0.0, 5.0]))
        except AssertionError as e:
            raise AssertionError(f"{(B, S, D * G, G, dtype)}: {e}") from None


def test_plans_that_do_not_fit_are_refused():
    x, dy, gamma, beta = make(1, 1000, 64, torch.bfloat16, 0)
    good = rn.make_gn_plan(1, 1000, 64, 8, torch.bfloat16)
    for kw in (dict(path=7), dict(vec_elems=4), dict(threads=0), dict(threads=288), dict(tile=0), dict(tile=10 ** 6),
               dict(cluster=3), dict(cluster=16), dict(path=0, per_thread=1, cluster=1, threads=32, tile=1),
               dict(path=1, cluster=2), dict(path=1, cluster=1, chunks=0), dict(path=1, cluster=1, out_chunks=0)):
        with pytest.raises(rn.NormError):
            rn.gn_fwd(x, gamma, beta, 8, plan={**good, **kw})
    odd = torch.zeros(1000 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 1000, 64)
    with pytest.raises(rn.NormError):  # 16-byte accesses on a tensor that is not 16-byte aligned
        rn.gn_fwd(odd, gamma, beta, 8, plan=good)


@pytest.mark.parametrize("B,S,C,G", [(2, 30, 64, 8), (2, 3000, 64, 8), (2, 9000, 70, 5), (2, 70000, 64, 8),
                                     (2, 9000, 35, 5), (700, 3, 24, 3)])
def test_in_place_chain_equals_copies(B, S, C, G):
    """Every call reads what the one before wrote, queued back to back and
    replayed from a graph: the bits of calls with buffers of their own, each
    finished before the next."""
    x, dy, gamma, beta = make(B, S, C, torch.bfloat16, 13)
    want = x
    for _ in range(6):
        want = rn.gn_fwd(want, gamma, beta, G, activation="silu")[0]
        torch.cuda.synchronize()
    mean, rstd = rn.gn_fwd(x, gamma, beta, G)[1:]
    wdy = dy
    for _ in range(4):
        wdy, wdg, wdb = rn.gn_bwd(wdy, x, gamma, beta, mean, rstd, G, activation="gelu")
        torch.cuda.synchronize()

    def chain(a, b):
        for _ in range(6):
            rn.gn_fwd(a, gamma, beta, G, activation="silu", out=a, stats=False)
        for _ in range(4):
            rn.gn_bwd(b, x, gamma, beta, mean, rstd, G, activation="gelu", dx=b, dgamma=dg, dbeta=db)

    dg, db = torch.empty_like(wdg), torch.empty_like(wdb)
    a, b = x.clone(), dy.clone()
    chain(a, b)
    assert torch.equal(a, want) and torch.equal(b, wdy) and torch.equal(dg, wdg) and torch.equal(db, wdb)
    a.copy_(x)
    b.copy_(dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(a, b)
    for _ in range(2):
        a.copy_(x)
        b.copy_(dy)
        dg.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, wdy) and torch.equal(dg, wdg) and torch.equal(db, wdb)


def test_calls_from_two_threads():
    import threading
    cases = [make(2, 5000 + 40 * k, 64, torch.bfloat16, k) for k in range(2)]
    want = [rn.gn_fwd(x, gamma, beta, 8, activation="gelu") for x, _, gamma, beta in cases]
    norms = [rn.grad_norm([x, dy]) for x, dy, _, _ in cases]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        x, dy, gamma, beta = cases[k]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = rn.gn_fwd(x, gamma, beta, 8, activation="gelu")
                n = rn.grad_norm([x, dy])
                torch.cuda.current_stream().synchronize()
                if not (all(torch.equal(a, b) for a, b in zip(got, want[k])) and torch.equal(n, norms[k])):
                    bad.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("dtype,B,S,C,G", [
    ("bf16", 2, 9000, 64, 8), ("bf16", 2, 9000, 70, 5), ("bf16", 2, 9000, 35, 5), ("f32", 2, 9000, 64, 8),
    ("f32", 2, 9000, 35, 5), ("bf16", 2, 100, 64, 8), ("f32", 1, 40000, 30, 6)])
def test_chain_that_rewrites_parameters_and_statistics(dtype, B, S, C, G):
    """Everything a call reads is written by the call queued before it, into
    the same buffers round after round, with no gap between the launches: x,
    dy, gamma and beta by group norm calls of their own, the statistics by the
    forward. Bits as from calls that are each finished before the next; on
    every access width, queued back to back and replayed from a graph."""
    dt, rounds = DT[dtype], 5
    sets = [make(B, S, C, dt, 31 + k) for k in range(rounds)]
    one, zero = torch.ones(C, dtype=dt, device="cuda"), torch.zeros(C, dtype=dt, device="cuda")

    def renew(dst, src):  # dst = group norm of src: a short and a long kernel of the library as the writer
        rn.gn_fwd(src.view(-1, *src.shape[-2:]) if src.dim() > 1 else src.view(1, 1, C), one, zero, 1,
                  out=dst if dst.dim() > 1 else dst.view(1, 1, C), stats=False)

    buf = [torch.empty_like(t) for t in sets[0]]
    stats = [torch.empty(B, G, device="cuda") for _ in range(2)]
    outs = [(torch.empty_like(buf[0]), torch.empty_like(buf[0]), torch.empty(C, device="cuda"), torch.empty(C, device="cuda"),
             torch.empty(B, G, device="cuda"), torch.empty(B, G, device="cuda")) for _ in range(rounds)]

    def chain(pause):
        for (x, dy, gamma, beta), (y, dx, dg, db, m, r) in zip(sets, outs):
            bx, bdy, bg, bb = buf
            for step in (lambda: renew(bx, x), lambda: renew(bg, gamma), lambda: renew(bb, beta),
                         lambda: rn.gn_fwd(bx, bg, bb, G, activation="silu", out=y, mean=stats[0], rstd=stats[1]),
                         lambda: renew(bdy, dy),
                         lambda: rn.gn_bwd(bdy, bx, bg, bb, stats[0], stats[1], G, activation="silu", dx=dx, dgamma=dg,
                                           dbeta=db),
                         # the parameters change straight before a backward, the statistics straight before another
                         lambda: renew(bg, beta), lambda: renew(bb, gamma),
                         lambda: rn.gn_bwd(bdy, bx, bg, bb, stats[0], stats[1], G, activation="silu", dx=dx, dgamma=dg,
                                           dbeta=db),
                         lambda: rn.gn_fwd(dx, bg, bb, G, activation="silu", out=y, mean=m, rstd=r),
                         lambda: rn.gn_bwd(bdy, dx, bg, bb, m, r, G, activation="gelu", dx=dx, dgamma=dg, dbeta=db)):
                step()
                if pause:
                    torch.cuda.synchronize()

    chain(True)
    want = [tuple(t.clone() for t in o) for o in outs]
    assert all(torch.isfinite(t).all() for o in want for t in o)

    def check():
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a, b)
                a.fill_(3.0)

    for _ in range(3):
        chain(False)
        check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(False)
    for _ in range(3):
        g.replay()
        check()


@pytest.mark.parametrize("dtype,B,S,C,G", [("f32", 16384, 1100, 8, 1), ("bf16", 3000, 1030, 6, 2), ("f32", 1500, 3001, 12, 3),
                                           ("f32", 4096, 1100, 8, 1), ("f32", 4097, 1100, 8, 1),
                                           ("f32", (1 << 21) + 3, 1, 4, 1), ("bf16", 5000, 1030, 6, 2)])
def test_column_sums_of_many_samples(dtype, B, S, C, G):
    """Thousands of samples with more positions than one CTA holds, and millions
    of one: as many partial rows of the column gradients, all of one sign. Every
    addition of a sum of positive terms rounds by at most u of the sum so far,
    so the sum is off by u times the additions a term goes through: a thread's
    32 rows and its blocks (2), the row slots of a CTA (40), and either the
    partial rows folded by 8 warps (16) and their warps (8), the folded rows (8)
    and their warps (32), or the partial rows in blocks of 32, at most 16
    of them, and their warps (8): 138 at most. Chains of thousands of equal
    terms are off by ten times that."""
    dt = DT[dtype]
    x, _, gamma, beta = make(1, S, C, dt, 17)
    x = torch.cat([torch.randn(B // 500 + 1, S, C, device="cuda").to(dt)] * 500)[:B].contiguous()
    v = (0.7 + 0.1 * torch.rand(C, generator=torch.Generator().manual_seed(3))).to(dt).cuda()
    dy = v.expand(B, S, C).contiguous()
    _, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS)
    dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, G)
    want = v.to(F) * B * S
    rel = ((db.to(F) - want) / want).abs().max().item()
    assert rel <= 138 * U, rel / U
    s = torch.zeros(C, dtype=F, device="cuda")
    total = torch.zeros(C, dtype=F, device="cuda")
    for k in range(0, B, 1000):
        xh = (x[k:k + 1000].to(F) - spread(mean[k:k + 1000].to(F), C // G)) * spread(rstd[k:k + 1000].to(F), C // G)
        s += xh.sum((0, 1)) * v
        total += xh.abs().sum((0, 1)) * v
    assert ((dg.to(F) - s).abs() <= 146 * U * total).all()  # (and 8 u for xh and the products)
    for k in (0, B - 3):
        check_bwd(dy[k:k + 3], x[k:k + 3], gamma, beta, mean[k:k + 3], rstd[k:k + 3], G, None, dx[k:k + 3],
                  *rn.gn_bwd(dy[k:k + 3], x[k:k + 3], gamma, beta, mean[k:k + 3], rstd[k:k + 3], G)[1:])


def test_statistics_of_empty_samples_are_nan():
    """The mean and the variance of no values are NaN, as the formula gives
    them; the caller's own tensors are left as they were."""
    gamma, beta = torch.ones(16, device="cuda"), torch.zeros(16, device="cuda")
    e = torch.empty(2, 0, 16, device="cuda")
    for _ in range(4):
        old = [torch.full((2, 4), 7.0, device="cuda") for _ in range(4)]
        del old  # (new tensors of this size find these values in memory)
        y, mean, rstd = rn.gn_fwd(e, gamma, beta, 4)
        assert y.shape == e.shape and mean.shape == rstd.shape == (2, 4)
        assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    mine = [torch.full((2, 4), 7.0, device="cuda") for _ in range(2)]
    _, mean, rstd = rn.gn_fwd(e, gamma, beta, 4, mean=mine[0], rstd=mine[1])
    assert mean is mine[0] and rstd is mine[1] and (mean == 7).all() and (rstd == 7).all()


def test_out_of_memory_has_torchs_type():
    """An allocation that the allocator refuses raises torch.OutOfMemoryError, as from the
    row norms, and the next call works."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # (so that x lies in a block of its own, with no free space beside it)
    x = torch.zeros(1, 1 << 20, 64, device="cuda")  # 256 MB
    gamma, beta = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    small = x[:, :1000]
    rn.gn_fwd(small, gamma, beta, 8)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    try:
        # (the process's own limit, checked before the driver is asked)
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) /
                                                   torch.cuda.get_device_properties(0).total_memory)
        for call in (lambda: rn.ln_fwd(x[0], gamma, beta), lambda: rn.gn_fwd(x, gamma, beta, 8),
                     lambda: rn.gn_bwd(x, x, gamma, beta, *(torch.zeros(1, 8, device="cuda"),) * 2, 8)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
        y, mean, rstd = rn.gn_fwd(small, gamma, beta, 8)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert (y == 0).all() and (mean == 0).all()
    assert (rn.gn_fwd(x, gamma, beta, 8)[0] == 0).all()


# ------------------------------------------------------------ how exact the statistics and the activations are

@pytest.mark.parametrize("loc", [0.0, 1.0])
@pytest.mark.parametrize("dtype,B,S,C,G", [
    ("f32", 2, 30000, 64, 8), ("f32", 1, 65536, 128, 4), ("f32", 3, 9001, 35, 5), ("f32", 2, 20000, 30, 6),
    ("bf16", 2, 30000, 64, 8), ("f16", 2, 9000, 70, 5), ("f32", 2, 512, 320, 32), ("bf16", 2, 256, 1280, 32),
    # a hundred rows a thread and more
    ("bf16", 1, 262144, 256, 32), ("f16", 40, 20000, 64, 8), ("f32", 40, 20000, 64, 8), ("bf16", 8, 60000, 35, 5)])
def test_statistics_to_a_few_roundings(dtype, B, S, C, G, loc):
    """Mean and rstd of ordinary data in every layout of the sums, held closer
    than the bound for the worst data. In units of u: a thread's chain of at
    most 64 squares loses some 3.4 of the sum on average, 1.7 of rstd; the
    merges are some 20 additions whose errors are random and average over the
    group's threads, below 1; count, eps, root and division round once each: 2.5.
    Together 6. The mean: chains of up to 64 differences from K, whose partial
    sums reach 64 |K - mean|, are off by some 2 u |K - mean| + 2 u sigma in one
    thread's share of the mean, as random, and less over all of a group's
    threads; the merged sum is a pair, and the mean is rounded once. With chains
    four times as long and the merged sum in one fp32 number, rstd was off by
    13 u and the mean by 10 u sigma on 1 x 262144 x 256: neither passes."""
    x, _, gamma, beta = make(B, S, C, DT[dtype], 41, loc=loc)
    _, mean, rstd = rn.gn_fwd(x, gamma, beta, G, EPS)
    xg = x.to(F).reshape(B, S, G, C // G)
    mu = xg.mean((1, 3))
    var = (xg - mu.view(B, 1, G, 1)).square().mean((1, 3))
    r = (var + float(torch.tensor(EPS))).rsqrt()
    rel = ((rstd.to(F) - r) / r).abs().max().item()
    assert rel <= 6 * U, rel / U
    off = (mean.to(F) - mu).abs()
    bar = U * (mu.abs() + 2 * var.sqrt() + 2 * (xg[:, 0, :, 0] - mu).abs())
    assert (off <= bar).all(), (off / bar).max().item()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_to_their_own_arithmetic(act):
    """Outputs for arguments from -13 to 13 in steps of 1e-4, relative to the
    output itself: in the negative tails too, where y is far below any
    absolute bound. z is taken from the returned statistics: x - mean, rstd
    gamma and the product round once each and what the rounding of the mean
    left is added back, so z is off by zerr = 3 u |z| + u |mean| rstd gamma, y by
    |act'| zerr + 0.4 zerr^2 (|act''| <= 0.8).
    silu, z / (1 + e): e = 2^t with |t| ln 2 = |z| off by 2 u relative and the
    hardware's 2^t by 4 u: (2 |z| + 4) u of e, e / (1 + e) of which is
    passed on; the sum 1, the reciprocal 2, the product 1.
    gelu, max(z, 0) - m tail, m = |z|: with t = 1 / (1 + p m) off by 4 u, the
    polynomial Q(t) passes on 2.7 times that and its own roundings are at most
    15.7 u (the sum of |coefficient| t^i times the roundings each goes through, over
    Q, is below that on the whole range); exp(-m^2 / 2): 1.5 m^2 + 4; two
    products 2; the fit itself 18 (1.06e-6). Together (52 + 1.5 m^2) u of
    m tail, and one rounding of y."""
    half = torch.linspace(1e-4, 13, 130000)
    x = torch.cat([half, -half]).view(1, -1, 1).cuda()
    sigma = float(x.double().square().mean().sqrt())
    gamma, beta = torch.full((1,), sigma, device="cuda"), torch.zeros(1, device="cuda")
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS, activation=act)
    mean, s = float(mean), float(rstd) * float(gamma)
    z = (x.to(F) - mean) * s
    assert z.min() < -12.9 and z.max() > 12.9
    zerr = U * (3 * z.abs() + abs(mean) * s)
    tol = slope64(z, act).abs() * zerr + 0.4 * zerr.square()
    if act == "silu":
        ref = z * torch.sigmoid(z)
        own = (torch.sigmoid(-z) * (2 * z.abs() + 4) + 4) * U * ref.abs()
    else:
        tail = 0.5 * torch.erfc(z.abs() / math.sqrt(2))
        ref = z.clamp(min=0) - z.abs() * tail
        own = (52 + 1.5 * z.square()) * U * z.abs() * tail + U * ref.abs()
    # (below fp32's smallest normal numbers the tail keeps 2^-149 steps)
    tol = tol + own + 16 * 2.0 ** -149
    err = (y.to(F) - ref).abs()
    worst = (err / tol).max().item()
    assert worst <= 1, (worst, float(z.flatten()[(err / tol).argmax()]))


@pytest.mark.parametrize("dtype,B,S,C", [("f32", 1, 100003, 1), ("f32", 3, 20001, 1), ("bf16", 2, 30000, 2), ("f32", 2, 30000, 4),
                                         ("bf16", 1, 60000, 8), ("f16", 9, 5001, 3), ("f32", 2, 1000, 1), ("f32", 1, 900000, 1)])
def test_column_sums_of_few_channels(dtype, B, S, C):
    """Few channels leave few sums with many threads each. A chain of L
    additions of terms alike in size, of either sign, is off by u / sqrt 3
    sqrt(L / 2) of the root of its terms' squares where every addition's
    rounding is taken as even over half a step (at most; 0.73 of that over a
    binade), and a tree by u / sqrt 3 a level. The sums go through chains of
    32 rows a thread (2.3 u), their blocks (8 at most here: 1.2), a tree and
    a chain of 8 over the CTA's row slots (5 levels and 1.2: 1.8), blocks of 16
    partial rows (1.6), the blocks (6: 1) and 8 warps (1.2): together, as
    independent, 3.9 u of the root of the squares. Held over 40 sums of 40 seeds
    as their root mean square, whose own spread is a ninth: 1.3 times that
    bound would be off by three of those, the bound itself leaves the 0.73.
    One chain over 256 row slots alone is 6.5 u."""
    dt = DT[dtype]
    rel = []
    for seed in range(-(-40 // C)):
        x, dy, gamma, beta = make(B, S, C, dt, 1000 + seed)
        _, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS)
        _, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 1)
        xh = (x.to(F) - spread(mean.to(F), C)) * spread(rstd.to(F), C)
        for got, terms in ((dg, dy.to(F) * xh), (db, dy.to(F))):
            rel.append((got.to(F) - terms.sum((0, 1))) / terms.square().sum((0, 1)).sqrt())
    rel = torch.stack(rel).view(-1, 2, C)
    for k in range(2):
        rms = rel[:, k].square().mean().sqrt().item()
        assert rms <= 3.9 * U, (k, rms / U)


def test_most_samples():
    """As many samples as the limits allow, of one value each: y is beta, dx
    vanishes but for two roundings of rstd gamma dy, dgamma is 0, and dbeta's
    additions are at most 32 partial rows, 8 warps, 8 folded rows and 32 warps, and
    the blocks of rows, whose errors are kept: 80 u of a sum of one sign, and
    8 more for the pair's last digits."""
    B, v = (1 << 31) - 2, 0.7
    x = torch.empty(B, 1, dtype=torch.bfloat16, device="cuda").normal_()
    gamma, beta = torch.full((1,), 1.5, dtype=torch.bfloat16, device="cuda"), torch.full((1,), 0.25, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS)
    assert (y == 0.25).all() and torch.equal(mean[-1000:], x[-1000:].float())
    assert (rstd == rstd[0]).all() and abs(float(rstd[0]) * EPS ** 0.5 - 1) <= 4 * U
    dy = y.fill_(v)
    dx, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 1)
    assert dx.abs().max() <= 4 * U * float(rstd[0]) * 1.5 * v * 1.01 and float(dg) == 0.0
    want = float(torch.tensor(v).bfloat16()) * B
    assert abs(float(db) - want) <= 88 * U * want


@pytest.mark.parametrize("B,S,C", [(3, 50, 8), (3000, 3, 8), (9000, 1030, 6), (40, 5000, 8)])
def test_infinite_gradients_stay_in_their_channels(B, S, C):
    """An infinity in dy is an infinite dbeta of its channel, however the
    partial rows are added; the other channels' sums are as without it."""
    x, dy, gamma, beta = make(1, S, C, torch.float32, 51)
    x, dy = (torch.randn(B, S, C, device="cuda") for _ in range(2))
    _, mean, rstd = rn.gn_fwd(x, gamma, beta, 1, EPS)
    dy[B // 2, S // 2, 2] = 0.0
    _, cg, cb = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 1)
    for v in (math.inf, -math.inf):
        dy[B // 2, S // 2, 2] = v
        _, dg, db = rn.gn_bwd(dy, x, gamma, beta, mean, rstd, 1)
        assert float(db[2]) == v and torch.isinf(dg[2])
        keep = torch.arange(C, device="cuda") != 2
        assert torch.equal(db[keep], cb[keep]) and torch.equal(dg[keep], cg[keep])
