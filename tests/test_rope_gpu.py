"""RMSNorm of query and key heads with the rotary rotation (rms_fwd_rope,
rms_bwd_rope), through the Python binding, against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, the fp32 rounding; eta = eps / 2
of the output type, one rounding of the output; half the type's smallest
subnormal below that):

r = 1 / sqrt(mean x^2 + eps): a lane adds at most 32 squares one after the
  other, 5 butterfly levels follow, then one product, one sum and rsqrt (2
  ulp): below 32 + 5 + 2 + 2 and halved by the root, plus 4 u: 30 u.
y: z = x r w has 2 u more, the rotation z_a c - z_b s 2 u of both terms:
  40 u (|z_a c| + |z_b s|), then eta |y|.
dx = r g - x r^3 m, g = dz w, m = mean(g x): dz has 2 u of its two terms
  (their absolute sum: Z), so with G = |w| Z: 40 u r G for the first part; m's
  own sum adds 40 u of mean(G |x|), r^3 90 u: 160 u |x| r^3 mean(G |x|); eta |dx|.
dw = sum dz x r: each term within 40 u of Z |x| r, and a chain of additions of
  at most 64 heads, then of n / 64 chains at most, 256 lanes' shares, and 32
  rows' worth of partial sums: (40 + 64 + n / 64 + 256 + 64) u sum Z |x| r."""
import itertools

import pytest
import torch

import row_wise_normalization_ln_gb300 as rn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
F = torch.float64
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from row_wise_normalization_ln_gb300 import _build
    _build.build()
    rn.library()


def tables(P, R, seed=0):
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=F) / max(R, 1))
    angle = torch.arange(P, dtype=F)[:, None] * freq
    return angle.cos().float().cuda(), angle.sin().float().cuda()


def make(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def pairs(R, interleaved):
    """Per rotating value: its mate, its angle, and the sign of the mate's part."""
    j = torch.arange(R, device="cuda")
    if interleaved:
        return j ^ 1, j // 2, torch.where(j % 2 == 0, -1.0, 1.0).to(F)
    return (j + R // 2) % R, j % max(R // 2, 1), torch.where(j < R // 2, -1.0, 1.0).to(F)


def rotate64(z, cos, sin, interleaved, back=False, absolute=False):
    """z [..., heads, D]; cos, sin [..., R / 2] of the tokens, 64 bits."""
    R = 2 * cos.shape[-1]
    mate, at, sign = pairs(R, interleaved)
    c, s = cos[..., None, :][..., at], sin[..., None, :][..., at] * sign * (-1 if back else 1)
    if absolute:
        z, c, s = z.abs(), c.abs(), s.abs()
    out = z.clone()
    out[..., :R] = z[..., :R] * c + z[..., mate] * s
    return out


def at_positions(cos, sin, pos):
    p = pos.clamp(0, cos.shape[0] - 1)
    return cos.to(F)[p], sin.to(F)[p]


def eta(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def check_fwd(y, x, w, cos, sin, pos, interleaved, eps=EPS):
    v, w64 = x.to(F), w.to(F)
    r = (v.square().mean(-1, keepdim=True) + eps) ** -0.5
    c, s = at_positions(cos, sin, pos)
    z = v * r * w64
    ref = rotate64(z, c, s, interleaved)
    tol = 40 * U * rotate64(z, c, s, interleaved, absolute=True) + eta(x.dtype) * ref.abs() * (1 + 64 * U) + tiny(x.dtype) + 1e-45
    pad = (pos < 0)[..., None, None]
    ref = torch.where(pad, 0.0, ref)
    bad = (y.to(F) - ref).abs() > torch.where(pad, 0.0, tol)
    assert y.shape == x.shape and y.dtype == x.dtype
    assert not bad.any(), (int(bad.sum()), float((y.to(F) - ref).abs().max()))


def check_bwd(dx, dw, dy, x, w, cos, sin, pos, interleaved, eps=EPS):
    v, w64, d = x.to(F), w.to(F), dy.to(F)
    D = x.shape[-1]
    r = (v.square().mean(-1, keepdim=True) + eps) ** -0.5
    c, s = at_positions(cos, sin, pos)
    live = (pos >= 0)[..., None, None].to(F)
    dz = rotate64(d, c, s, interleaved, back=True) * live
    Z = rotate64(d, c, s, interleaved, back=True, absolute=True) * live
    g, G = dz * w64, w64.abs() * Z
    ref = r * g - v * r ** 3 * (g * v).mean(-1, keepdim=True)
    tol = 40 * U * r * G + 160 * U * v.abs() * r ** 3 * (G * v.abs()).mean(-1, keepdim=True) + \
        eta(x.dtype) * ref.abs() * (1 + 64 * U) + (tiny(x.dtype) + 1e-45) * live
    bad = (dx.to(F) - ref).abs() > tol
    assert dx.shape == x.shape and dx.dtype == x.dtype
    assert not bad.any(), (int(bad.sum()), float((dx.to(F) - ref).abs().max()))
    lead = tuple(range(x.dim() - 1))
    n = x.numel() // D
    rw = (dz * v * r).sum(lead)
    tw = (40 + 64 + n / 64 + 256 + 64) * U * (Z * v.abs() * r).sum(lead) + 1e-45
    assert dw.dtype == torch.float32 and dw.shape == (D,)
    bad = (dw.to(F) - rw).abs() > tw
    assert not bad.any(), (int(bad.sum()), float(((dw.to(F) - rw).abs() / tw).max()))


def both(q, k, wq, wk, cos, sin, pos, interleaved, dq, dk, given=True, plan=None, bplan=None):
    """Forward and backward through the binding, checked; `pos` as the calls see it."""
    p = pos if given else None
    yq, yk = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, p, EPS, interleaved=interleaved, plan=plan)
    check_fwd(yq, q, wq, cos, sin, pos, interleaved)
    gq, gk, gwq, gwk = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, p, EPS, interleaved=interleaved, plan=bplan)
    check_bwd(gq, gwq, dq, q, wq, cos, sin, pos, interleaved)
    if k is not None:
        check_fwd(yk, k, wk, cos, sin, pos, interleaved)
        check_bwd(gk, gwk, dk, k, wk, cos, sin, pos, interleaved)
    else:
        assert yk is None and gk is None and gwk is None


def case(T, Hq, Hk, D, R, dtype, seed=0, P=97, pad=True):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(P, (T,), generator=g)
    if pad and T > 1:
        pos[torch.rand(T, generator=g) < 0.2] = -1
    cos, sin = tables(P, R)
    q, k = make((T, Hq, D), dtype, seed + 1, 2.0), make((T, Hk, D), dtype, seed + 2, 0.3)
    dq, dk = make((T, Hq, D), dtype, seed + 3), make((T, Hk, D), dtype, seed + 4)
    wq, wk = make((D,), dtype, seed + 5) + 1, make((D,), dtype, seed + 6) + 1
    return q, k, wq, wk, cos, sin, pos.cuda(), dq, dk


SHAPES = [  # D, R: whole and part rotations, odd counts of accesses, widths of every access and lane count
    (128, 128), (64, 64), (96, 24), (80, 32), (80, 20), (256, 64), (512, 512), (512, 128), (72, 72), (100, 50), (40, 0),
    (50, 50), (7, 4), (7, 6), (1, 0), (2, 2), (511, 510), (320, 160), (24, 16), (136, 16), (8, 8), (130, 26),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", SHAPES)
def test_widths(D, R, interleaved, dtype):
    q, k, wq, wk, cos, sin, pos, dq, dk = case(13, 5, 2, D, R, DT[dtype], seed=D + R)
    both(q, k, wq, wk, cos, sin, pos, interleaved, dq, dk)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 4), (2, 64, 8), (3, 7, 1), (257, 9, 3), (1000, 33, 17), (4097, 3, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_counts(T, Hq, Hk, dtype):
    q, k, wq, wk, cos, sin, pos, dq, dk = case(T, Hq, Hk, 64, 64, DT[dtype], seed=T)
    both(q, k, wq, wk, cos, sin, pos, False, dq, dk)


@pytest.mark.parametrize("interleaved", [False, True])
def test_no_positions_counts_along_each_sequence(interleaved):
    B, S = 3, 19
    q, k, wq, wk, cos, sin, _, dq, dk = case(B * S, 4, 2, 64, 32, torch.bfloat16)
    q, k, dq, dk = (t.view(B, S, -1, 64) for t in (q, k, dq, dk))
    pos = torch.arange(S, device="cuda").expand(B, S)
    both(q, k, wq, wk, cos, sin, pos, interleaved, dq, dk, given=False)


@pytest.mark.parametrize("dtype", list(DT))
def test_packed_and_transposed_layouts(dtype):
    dt = DT[dtype]
    B, S, Hq, Hk, D = 2, 21, 6, 2, 64
    q, k, wq, wk, cos, sin, pos, dq, dk = case(B * S, Hq, Hk, D, 64, dt)
    # heads of a packed projection, and their gradients into a packed one
    qkv = make((B * S, (Hq + 2 * Hk) * D), dt, 9)
    q = qkv[:, :Hq * D].view(-1, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(-1, Hk, D)
    both(q, k, wq, wk, cos, sin, pos, False, dq, dk)
    packed = torch.full_like(qkv, 7.0)
    oq, ok = packed[:, :Hq * D].view(-1, Hq, D), packed[:, Hq * D:(Hq + Hk) * D].view(-1, Hk, D)
    gq, gk, gwq, gwk = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, dq_out=oq, dk_out=ok)
    assert gq is oq and gk is ok
    check_bwd(oq, gwq, dq, q, wq, cos, sin, pos, False)
    check_bwd(ok, gwk, dk, k, wk, cos, sin, pos, False)
    assert (packed[:, (Hq + Hk) * D:] == 7).all()  # the values' gradient is left alone
    # [B, heads, S, D] in memory
    qt, kt = make((B, Hq, S, D), dt, 10).transpose(1, 2), make((B, Hk, S, D), dt, 11).transpose(1, 2)
    dqt, dkt = make((B, Hq, S, D), dt, 12).transpose(1, 2), make((B, Hk, S, D), dt, 13).transpose(1, 2)
    both(qt, kt, wq, wk, cos, sin, pos.view(B, S), False, dqt, dkt)
    # the keys of this step into their rows of a cache, the others left alone
    cache = torch.full((B, S + 5, Hk, D), 3.0, dtype=dt, device="cuda")
    row = cache[:, 4:4 + S]
    _, out = rn.rms_fwd_rope(qt, kt, wq, wk, cos, sin, pos.view(B, S), EPS, k_out=row)
    assert out is row
    check_fwd(row, kt, wk, cos, sin, pos.view(B, S), False)
    assert (cache[:, :4] == 3).all() and (cache[:, 4 + S:] == 3).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_offsets_and_odd_pitches(offset, dtype):
    dt = DT[dtype]
    T, H, D, R = 11, 3, 64, 32
    _, k, wq, wk, cos, sin, pos, dq, dk = case(T, H, 2, D, R, dt)
    buf = make((T, H * D + 5 + offset), dt, 3)
    q = buf.as_strided((T, H, D), (H * D + 5 + offset, D, 1), offset)
    both(q, k, wq, wk, cos, sin, pos, False, dq, dk)
    # a weight and tables off their 16-byte boundaries
    w2 = torch.cat((wq[:1], wq))[1:]
    big_c, big_s = (torch.cat((t, t), 1)[:, 1:1 + R // 2] for t in (cos.roll(1, 1), sin.roll(1, 1)))
    assert torch.equal(big_c, cos) and not big_c.is_contiguous()
    both(k, None, w2, None, big_c, big_s, pos, True, dk, None)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    q, k, wq, wk, cos, sin, pos, dq, dk = case(37, 8, 4, 128, 64, torch.bfloat16)
    want = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved)
    q2, k2 = q.clone(), k.clone()
    got = rn.rms_fwd_rope(q2, k2, wq, wk, cos, sin, pos, EPS, interleaved=interleaved, q_out=q2, k_out=k2)
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    want = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved)
    for over in ("dy", "x"):
        t = [v.clone() for v in (dq, dk, q, k)]
        o = t[:2] if over == "dy" else t[2:]
        got = rn.rms_bwd_rope(*t, wq, wk, cos, sin, pos, EPS, interleaved=interleaved, dq_out=o[0], dk_out=o[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_int32_positions_and_int64_agree():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(29, 4, 2, 64, 64, torch.float16)
    a = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS)
    b = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos.int(), EPS)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    far = pos.clone()
    far[3] = 1 << 40  # beyond the tables, and beyond 32 bits
    y, _ = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, far, EPS)
    assert y[3].isnan().all() and not y[:3].isnan().any() and not y[4:].isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_beyond_the_tables(dtype):
    q, k, wq, wk, cos, sin, pos, dq, dk = case(9, 3, 1, 64, 32, DT[dtype], pad=False)
    pos = pos.clone()
    pos[4] = cos.shape[0]
    yq, yk = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS)
    rest = [i for i in range(9) if i != 4]
    assert yq[4].isnan().all() and yk[4].isnan().all() and not yq[rest].isnan().any()
    gq, gk, gwq, gwk = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    assert gq[4].isnan().all() and gwq.isnan().all() and gwk.isnan().all() and not gq[rest].isnan().any()


def test_padding_holds_anything():
    """What a padding token's heads hold reaches no output."""
    q, k, wq, wk, cos, sin, pos, dq, dk = case(40, 4, 2, 64, 64, torch.bfloat16, seed=3)
    assert (pos < 0).any()
    want = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS) + rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    for v in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        for t in (q, k, dq, dk):
            t[pos < 0] = v
        got = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS) + rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_infinities_stay_in_their_head():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(6, 4, 2, 128, 64, torch.bfloat16, pad=False)
    q[2, 1, 100] = float("inf")  # a value that does not rotate
    y, _ = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS)
    # r = 0: every value is 0 but the infinite one, which is 0 * inf
    assert y[2, 1, 100].isnan() and int(y.isnan().sum()) == 1 and (y[2, 1, :100] == 0).all()
    q[2, 1, 100] = float("nan")
    y, _ = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS)
    assert y[2, 1].isnan().all() and int(y.isnan().sum()) == 128


def test_zero_rows_and_eps():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(5, 2, 1, 64, 64, torch.float32, pad=False)
    q.zero_()
    both(q, k, wq, wk, cos, sin, pos, False, dq, dk)


def test_empty_calls():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(4, 2, 1, 64, 32, torch.bfloat16, pad=False)
    e = slice(0, 0)
    y = rn.rms_fwd_rope(q[e], k[e], wq, wk, cos, sin, pos[e], EPS)
    assert y[0].shape == (0, 2, 64) and y[1].shape == (0, 1, 64)
    r = rn.rms_bwd_rope(dq[e], dk[e], q[e], k[e], wq, wk, cos, sin, pos[e], EPS)
    assert (r[2] == 0).all() and (r[3] == 0).all() and r[2].shape == (64,)
    # queries without heads, keys alone have some
    r = rn.rms_bwd_rope(dq[:, e], dk, q[:, e], k, wq, wk, cos, sin, pos, EPS)
    assert (r[2] == 0).all()
    check_bwd(r[1], r[3], dk, k, wk, cos, sin, pos, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_plan(dtype):
    """Narrow accesses, every lane count, chunk and CTA size give the same as the default, to rounding of the sums."""
    dt = DT[dtype]
    q, k, wq, wk, cos, sin, pos, dq, dk = case(50, 6, 3, 64, 32, dt)
    tried = 0
    for vec, heads, warps in itertools.product((4, 1) if dt == torch.float32 else (8, 4, 2, 1), (1, 2, 5), (1, 4, 8)):
        for backward in (False, True):
            p = rn.make_rope_plan(50, 6, 3, 64, 32, dt, backward=backward, vec_elems=vec)
            for lanes in {p["lanes"], 32}:
                p = dict(p, heads=heads, warps=warps, lanes=lanes, ctas=7)
                if backward:
                    both(q, k, wq, wk, cos, sin, pos, False, dq, dk, bplan=p)
                else:
                    for few in (0, 1):
                        both(q, k, wq, wk, cos, sin, pos, False, dq, dk, plan=dict(p, few=few))
                tried += 1
    assert tried > 30


def test_long_chains():
    """Many heads per CTA: the chains' sums are folded."""
    q, k, wq, wk, cos, sin, pos, dq, dk = case(6000, 8, 1, 64, 64, torch.float32)
    p = rn.make_rope_plan(6000, 8, 1, 64, 64, torch.float32, backward=True)
    both(q, k, wq, wk, cos, sin, pos, False, dq, dk, bplan=dict(p, ctas=2, warps=1))


def test_deterministic_on_streams_and_in_graphs():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(700, 8, 2, 128, 128, torch.bfloat16)
    want = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS) + rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, stream=side) + \
        rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, q_out=outs[0], k_out=outs[1])
        rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, dq_out=outs[2], dk_out=outs[3], dwq=outs[4], dwk=outs[5])
    for _ in range(3):
        for t in outs:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # other positions, the same graph
    pos.copy_((pos + 1).clamp(max=cos.shape[0] - 1))
    graph.replay()
    check_fwd(outs[0], q, wq, cos, sin, pos, False)
    check_bwd(outs[2], outs[4], dq, q, wq, cos, sin, pos, False)


def test_gradients_against_differences():
    """d(sum(y * dy)) along a direction, by central differences of the 64-bit
    formula: the step's own error is of the order of its square, 1e-8."""
    q, k, wq, wk, cos, sin, pos, dq, dk = case(7, 3, 1, 32, 16, torch.float32)

    def loss(x, w):
        r = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
        c, s = at_positions(cos, sin, pos)
        return (rotate64(x * r * w, c, s, False) * dq.to(F) * (pos >= 0)[:, None, None]).sum()

    gq, _, gwq, _ = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
    vx, vw = make(q.shape, F, 20), make(wq.shape, F, 21)
    h = 1e-4
    num = (loss(q.to(F) + h * vx, wq.to(F) + h * vw) - loss(q.to(F) - h * vx, wq.to(F) - h * vw)) / (2 * h)
    ana = (gq.to(F) * vx).sum() + (gwq.to(F) * vw).sum()
    scale = (gq.to(F) * vx).abs().sum() + (gwq.to(F) * vw).abs().sum()
    assert abs(num - ana) <= 1e-6 * scale  # 16 u of every term, and the step's error


def test_far_offsets():
    """Tokens whose elements lie beyond 2^31: only the last ones are looked at."""
    T, H, D = (1 << 31) // (8 * 128) + 40, 8, 128
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-33:] = make((33, H, D), torch.bfloat16, 5)
    cos, sin = tables(64, D)
    w = make((D,), torch.bfloat16, 6) + 1
    pos = torch.randint(64, (T,), device="cuda")
    y, _ = rn.rms_fwd_rope(q, None, w, None, cos, sin, pos, EPS)
    check_fwd(y[-33:], q[-33:], w, cos, sin, pos[-33:], False)
    assert int((y[:1000] != 0).sum()) == 0


def refused(match, kind=ValueError, **kw):
    q, k, wq, wk, cos, sin, pos, dq, dk = case(4, 2, 1, 64, 32, torch.bfloat16)
    a = dict(q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, positions=pos)
    a.update({n: (v(a) if callable(v) else v) for n, v in kw.items()})
    with pytest.raises(kind, match=match):
        rn.rms_fwd_rope(**a)


def test_refusals():
    refused("needs CUDA", q=lambda a: a["q"].cpu())
    refused("float32, bfloat16", TypeError, q=lambda a: a["q"].double())
    refused("must be a torch.Tensor", TypeError, cos=3)
    refused(r"\[tokens, heads, D\]", q=lambda a: a["q"][0])
    refused("dtype", k=lambda a: a["k"].float())
    refused("tokens", k=lambda a: a["k"][:3])
    refused("64 elements", wq=lambda a: a["wq"][:10])
    refused("dtype", wk=lambda a: a["wk"].float())
    refused("fp32 tables", cos=lambda a: a["cos"].bfloat16())
    refused("fp32 tables", sin=lambda a: a["sin"][:5])
    refused("room for", cos=lambda a: a["cos"].repeat(1, 3), sin=lambda a: a["sin"].repeat(1, 3))
    refused("no positions", cos=lambda a: a["cos"][:0], sin=lambda a: a["sin"][:0])
    refused("one value per token", positions=lambda a: a["positions"][:2])
    refused("int64 or int32", positions=lambda a: a["positions"].float())
    refused("wk is given", k=None)
    refused("shape", q_out=lambda a: a["q"][:2])
    refused("do not share memory", q_out=lambda a: a["q"][:1].expand(4, 2, 64))
    refused("status -1", rn.NormError, eps=-1.0)
    refused("status -1", rn.NormError, q_out=lambda a: a["q"].as_strided((4, 2, 64), (64, 256, 1)))
    q, k, wq, wk, cos, sin, pos, dq, dk = case(4, 2, 1, 64, 32, torch.bfloat16)
    with pytest.raises(ValueError, match="dq must have"):
        rn.rms_bwd_rope(dq[:2], dk, q, k, wq, wk, cos, sin, pos)
    with pytest.raises(rn.NormError):
        rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(rn.NormError, match="status -4"):
        rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, plan=dict(rn.make_rope_plan(4, 2, 1, 64, 32, torch.bfloat16), lanes=2))
    big = torch.zeros(1, 1, 513, device="cuda")
    with pytest.raises(rn.NormError):
        rn.rms_fwd_rope(big, None, big[0, 0], None, cos, sin)


# ------------------------------------------------------------ tokens without values, weights without bounds
def finite(*ts):
    return all(t is None or bool(t.isfinite().all()) for t in ts)


@pytest.mark.parametrize("eps", [0.0, 1e-50, 1e-6, 100.0])
@pytest.mark.parametrize("T,D,R,interleaved", [(1, 128, 128, False), (3, 128, 64, True), (5, 128, 128, False), (37, 80, 32, True), (50, 7, 4, False)])
@pytest.mark.parametrize("dtype", list(DT))
def test_every_eps(dtype, T, D, R, interleaved, eps):
    """Padding and token counts that leave lane groups idle, where nothing but the values keeps the root from 0."""
    q, k, wq, wk, cos, sin, pos, dq, dk = case(T, 5, 2, D, R, DT[dtype], seed=T)
    if T > 2:
        pos[1] = -1
    plan, bplan = (rn.make_rope_plan(T, 5, 2, D, R, DT[dtype], interleaved, backward=b) for b in (False, True))
    for few in (0, 1):
        y = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, eps, interleaved=interleaved, plan=dict(plan, few=few))
        assert finite(*y)
        check_fwd(y[0], q, wq, cos, sin, pos, interleaved, eps)
        check_fwd(y[1], k, wk, cos, sin, pos, interleaved, eps)
    for ctas in (2, bplan["ctas"]):
        g = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, eps, interleaved=interleaved, plan=dict(bplan, ctas=ctas))
        assert finite(*g)
        check_bwd(g[0], g[2], dq, q, wq, cos, sin, pos, interleaved, eps)
        check_bwd(g[1], g[3], dk, k, wk, cos, sin, pos, interleaved, eps)


@pytest.mark.parametrize("v", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_padding_is_zero_beside_any_weight_and_table(interleaved, dtype, v):
    """Padding reads no angle and no weight: its outputs are zeros and it adds nothing to dw."""
    for D, R in ((128, 64), (50, 20)):
        q, k, wq, wk, cos, sin, pos, dq, dk = case(11, 3, 2, D, R, DT[dtype], seed=5)
        pos[pos == 0] = 1  # row 0 belongs to nobody
        pos[2] = -1
        pad = pos < 0
        want = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved)
        cos[0], sin[0] = v, v
        got = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        wq[3], wq[D - 1], wk[0] = v, v, v
        plan = rn.make_rope_plan(11, 3, 2, D, R, DT[dtype], interleaved)
        for few in (0, 1):
            y = rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved, plan=dict(plan, few=few))
            assert (y[0][pad] == 0).all() and (y[1][pad] == 0).all()
        got = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, interleaved=interleaved)
        assert (got[0][pad] == 0).all() and (got[1][pad] == 0).all()
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])  # (dw has no weight in it)


@pytest.mark.parametrize("v", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
def test_weights_reach_their_own_column(interleaved, dtype, v):
    """A weight that is not finite reaches its column, and its partner's where that one rotates, alone."""
    for D, R, at in ((128, 64, 70), (128, 64, 100), (128, 64, 3), (96, 24, 95), (50, 20, 21), (50, 20, 49)):
        q, _, wq, _, cos, sin, pos, _, _ = case(9, 3, 1, D, R, DT[dtype], seed=at, pad=False)
        cos, sin = cos.clamp(min=0.1), sin.clamp(min=0.1)  # no angle hides a partner
        plain = wq.clone()
        wq[at] = v
        hit = {at} if at >= R else {at, int(pairs(R, interleaved)[0][at])}
        rest = [i for i in range(D) if i not in hit]
        widest = rn.make_rope_plan(9, 3, 0, D, R, DT[dtype], interleaved)["vec_elems"]
        for vec in [w for w in ((4, 1) if dtype == "f32" else (8, 4, 2, 1)) if w <= widest]:
            for few in (0, 1):
                plan = dict(rn.make_rope_plan(9, 3, 0, D, R, DT[dtype], interleaved, vec_elems=vec), few=few)
                want, _ = rn.rms_fwd_rope(q, None, plain, None, cos, sin, pos, EPS, interleaved=interleaved, plan=plan)
                y, _ = rn.rms_fwd_rope(q, None, wq, None, cos, sin, pos, EPS, interleaved=interleaved, plan=plan)
                assert torch.equal(y[..., rest], want[..., rest]), (D, R, at, vec, few)
                assert not y[..., sorted(hit)].isfinite().any()


def test_positions_of_another_shape():
    """Sequences' positions come as [B, S] (or flat): another shape with as many values is another order."""
    B, S = 3, 5
    q, _, wq, _, cos, sin, pos, dq, _ = case(B * S, 2, 1, 64, 32, torch.bfloat16)
    q, dq = q.view(B, S, 2, 64), dq.view(B, S, 2, 64)
    want = rn.rms_fwd_rope(q, None, wq, None, cos, sin, pos, EPS)[0]
    for good in (pos.view(B, S), pos.view(B, S, 1), pos.view(1, B, S), pos.view(1, -1), pos.view(B, S).t().contiguous().t()):
        assert torch.equal(rn.rms_fwd_rope(q, None, wq, None, cos, sin, good, EPS)[0], want)
    for bad in (pos.view(S, B), pos.view(B, S).t(), pos.view(S, 1, B)):
        with pytest.raises(ValueError, match="one value per token"):
            rn.rms_fwd_rope(q, None, wq, None, cos, sin, bad, EPS)
        with pytest.raises(ValueError, match="one value per token"):
            rn.rms_bwd_rope(dq, None, q, None, wq, None, cos, sin, bad, EPS)
    # one sequence, and one token a sequence: the dimension of one counts for nothing
    one = rn.rms_fwd_rope(q.reshape(1, B * S, 2, 64), None, wq, None, cos, sin, pos.view(-1, 1), EPS)[0]
    assert torch.equal(one.view(B, S, 2, 64), want)
    # tokens without sequences: any shape, in its order
    flat = rn.rms_fwd_rope(q.reshape(B * S, 2, 64), None, wq, None, cos, sin, pos.view(B, S), EPS)[0]
    assert torch.equal(flat.view(B, S, 2, 64), want)


def test_outputs_that_share_memory_are_refused():
    q, k, wq, wk, cos, sin, pos, dq, dk = case(4, 2, 1, 64, 32, torch.bfloat16)
    buf = torch.zeros(4 * 2 * 64, dtype=torch.bfloat16, device="cuda")
    for strides in ((64, 64, 1), (128, 32, 1), (32, 128, 1), (127, 64, 1), (64, 192, 1)):
        out = buf.as_strided((4, 2, 64), strides)
        with pytest.raises(ValueError, match="do not share memory"):
            rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, q_out=out)
        with pytest.raises(ValueError, match="do not share memory"):
            rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, dq_out=out)
    for strides in ((128, 64, 1), (64, 256, 1)):  # tokens of heads, heads of tokens
        out = buf.as_strided((4, 2, 64), strides)
        assert torch.equal(rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS, q_out=out)[0], rn.rms_fwd_rope(q, k, wq, wk, cos, sin, pos, EPS)[0])


def test_workspace_of_exactly_its_size():
    for dtype, T, hq, hk, D in ((torch.float32, 700, 5, 2, 80), (torch.bfloat16, 3, 1, 1, 64), (torch.bfloat16, 5000, 16, 4, 128)):
        q, k, wq, wk, cos, sin, pos, dq, dk = case(T, hq, hk, D, D // 8 * 4, dtype)
        want = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS)
        n = min(rn.make_rope_plan(T, hq, hk, D, D // 8 * 4, dtype, backward=True,
                                  num_sms=torch.cuda.get_device_properties(0).multi_processor_count)["ctas"], T * (hq + hk)) * D * 4
        buf = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
        got = rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, workspace=buf[:n])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (buf[n:] == 77).all()
        with pytest.raises(rn.NormError, match="status -1"):
            rn.rms_bwd_rope(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, workspace=buf[:n - 16])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("interleaved", [False, True])
def test_what_ran_before_changes_no_bit(interleaved, dtype):
    """Lanes without a token hold what an earlier kernel left; the sign of a resting -0 shows whether it counts."""
    T, H, D, R = 5, 4, 128, 64
    q, _, wq, _, cos, sin, pos, _, _ = case(T, H, 1, D, R, DT[dtype], pad=False)
    wq = wq.abs() + 0.5
    q[..., R:] = q[..., R:].abs() + 0.5
    q[..., R::3] = -0.0
    before = make((4096, H, D), DT[dtype], 1)
    plan = dict(rn.make_rope_plan(T, H, 0, D, R, DT[dtype], interleaved), few=0)
    far = torch.zeros(4096, dtype=torch.int64, device="cuda")
    bits = []
    for v in (0.0, float("inf")):
        rn.rms_fwd_rope(before.fill_(v), None, wq, None, cos, sin, far, EPS, interleaved=interleaved, plan=dict(plan, ctas=1216, heads=4))
        y, _ = rn.rms_fwd_rope(q, None, wq, None, cos, sin, pos, EPS, interleaved=interleaved, plan=plan)
        assert y.isfinite().all()
        bits.append(y.view(torch.int32 if DT[dtype] == torch.float32 else torch.int16))
    assert torch.equal(*bits)
