"""The global gradient norm and clipping (grad_norm, grad_clip) against 64-bit
arithmetic.

Tolerances: the norm's squares are added in fp32 over at most 64 values in
two chains or more (short lists: over a warp, in chains of 5 and 8 and a
tree of 5 levels), then in
fp64 or as pairs of fp32 numbers with every error kept: relative error of the
sum at most 33 u (u = 2^-24), of the norm 17 u, plus its own rounding: 18 u. A clipped value is
v * coef with coef rounded once from fp64 (its error: u, and the norm's does
not enter, the coefficient comes from the fp64 sum: 17 u) and the product
rounded once in fp32 and once to the type: 20 u |v coef| + eta |v coef| + half
the type's smallest subnormal."""
import math

import pytest
import torch

import row_wise_normalization_ln_gb300 as rn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F = torch.float64
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from row_wise_normalization_ln_gb300 import _build
    _build.build()
    rn.library()


def norm64(ts):
    return math.sqrt(math.fsum(float(t.to(F).square().sum()) for t in ts))


def check_norm(ts, got):
    want = norm64(ts)
    assert abs(float(got) - want) <= 18 * U * want, (float(got), want)


def check_clip(ins, outs, max_norm, got_norm):
    check_norm(ins, got_norm)
    coef = min(1.0, max_norm / (norm64(ins) + 1e-6))
    for t, o in zip(ins, outs):
        want = t.to(F) * coef
        fi = torch.finfo(t.dtype)
        tol = (20 * U + fi.eps / 2) * want.abs() + fi.smallest_normal * fi.eps / 2
        assert o.dtype == t.dtype and ((o.to(F) - want).abs() <= tol).all()


def tensors(shapes, dtypes, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


SETS = {
    "one value": [(1,)],
    "scalar": [()],
    "small": [(3,), (7, 5), (1, 1, 1), (1023,), (8,), (64,)],
    "units": [(1024,), (1025,), (2047,), (2048,), (2049,), (4096 * 8,), (4096 * 8 + 1,)],
    "with empty ones": [(0,), (5,), (0, 4), (0,), (1000,), (0,)],
    "only empty": [(0,), (0, 3)],
    "many": [(i % 37 + 1,) for i in range(1500)],
    "mixed sizes": [(4096, 512), (1,), (513,), (1024, 1024), (3, 3, 3), (65536,), (77, 1001)],
    "one large": [(5000, 5001)],
}


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.float16], DTYPES], ids=str)
@pytest.mark.parametrize("name", list(SETS))
def test_sets(name, dtypes):
    ts = tensors(SETS[name], dtypes, 5)
    check_norm(ts, rn.grad_norm(ts))
    keep = [t.clone() for t in ts]
    total = norm64(ts)
    for max_norm in (0.5 * total, 2 * total + 1, 0.0):
        outs = [torch.empty_like(t) for t in ts]
        got, norm = rn.grad_clip(ts, max_norm, out=outs)
        assert got is outs and all(torch.equal(a, b) for a, b in zip(ts, keep))
        check_clip(keep, outs, max_norm, norm)
        mine = [t.clone() for t in ts]
        got, norm = rn.grad_clip(mine, max_norm)
        assert got is mine and all(torch.equal(a, b) for a, b in zip(mine, outs))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("off_in,off_out", [(0, 0), (1, 1), (3, 3), (1, 0), (2, 7), (7, 7)])
def test_offsets_and_guards(dtype, off_in, off_out):
    """Views at any element of a buffer, inputs and outputs at the same or
    another offset within 16 bytes; nothing else is written."""
    for n in (1, 2, 7, 8, 9, 4095, 50001):
        a = torch.zeros(n + 64, dtype=dtype, device="cuda")
        v = a[16 + off_in:16 + off_in + n]
        v.copy_(torch.randn(n, device="cuda").to(dtype))
        b = torch.full((n + 64,), 5.0, dtype=dtype, device="cuda")
        o = b[16 + off_out:16 + off_out + n]
        _, norm = rn.grad_clip([v], 0.5, out=[o])
        check_clip([v], [o], 0.5, norm)
        o.fill_(5.0)
        assert (b == 5.0).all()
        v2 = v.clone()
        rn.grad_clip([v], 0.5)
        check_clip([v2], [v], 0.5, norm)
        v.zero_()
        assert not a.any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_every_pair_of_phases(dtype):
    """Inputs and outputs at every pair of offsets within 16 bytes, lengths
    around one and two accesses, one and several units: every value clipped,
    nothing beside it written."""
    per = 16 // dtype.itemsize
    lengths = [1, per - 1, per, per + 1, 2 * per - 1, 2 * per + 1, 3 * per, 256 * per - 1, 256 * per + per + 1, 2000 * per + 3]
    g = torch.Generator(device="cuda").manual_seed(5)
    ins, outs, pads = [], [], []
    for a in range(per):
        for b in range(per):
            for n in lengths:
                ins.append(torch.randn(n + 2 * per, generator=g, device="cuda").to(dtype)[a:a + n])
                pads.append(torch.full((n + 3 * per,), 7.0, device="cuda", dtype=dtype))
                outs.append(pads[-1][per + b:per + b + n])
    _, norm = rn.grad_clip(ins, 1.0, out=outs)
    check_clip(ins, outs, 1.0, norm)
    at = 0
    for a in range(per):
        for b in range(per):
            for n in lengths:
                assert (pads[at][:per + b] == 7).all() and (pads[at][per + b + n:] == 7).all()
                at += 1


def test_flat_buffer_of_neighbours():
    """Neighbouring views of one buffer, clipped in place: each once."""
    flat = torch.randn(30000, device="cuda").bfloat16()
    keep = flat.clone()
    cuts = [0, 1, 4, 5000, 5001, 12345, 29999, 30000]
    ts = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    _, norm = rn.grad_clip(ts, 3.0)
    check_clip([keep], [flat], 3.0, norm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("size", [1e25, 1e19, 3e17, 1e17, 1e-12, 1e-13, 1e-19, 1e-25, 1e-37])
def test_squares_beyond_fp32(dtype, size):
    """Values whose squares overflow or vanish in fp32."""
    ts = tensors([(1000,), (33, 77), (5,)], [dtype], 3, size)
    check_norm(ts, rn.grad_norm(ts))
    ts.append(torch.zeros(5000, dtype=dtype, device="cuda"))
    check_norm(ts, rn.grad_norm(ts))
    ts.append(tensors([(3000,)], [dtype], 4, 1.0)[0])
    check_norm(ts, rn.grad_norm(ts))


@pytest.mark.parametrize("size", [1e25, 1e19, 3e17, 1e17, 1e-12, 1e-13, 1e-19, 1e-25, 1e-37])
@pytest.mark.parametrize("numel", [300001, 40 * (1 << 20) + 3])
def test_long_lists_beyond_fp32(numel, size):
    """The same over many CTAs and, for the longer list, many steps of each:
    sums that leave fp32's range although every step's is within it."""
    ts = tensors([(numel,)], [torch.float32], 3, size)
    ts[0] = ts[0][1:]
    check_norm(ts, rn.grad_norm(ts))
    ts.append(tensors([(70001,)], [torch.bfloat16], 4, 1.0)[0][3:])
    check_norm(ts, rn.grad_norm(ts))


def test_fp16_range():
    ts = [torch.full((3001,), 65504.0, dtype=torch.float16, device="cuda"),
          torch.full((5,), 6e-8, dtype=torch.float16, device="cuda")]
    check_norm(ts, rn.grad_norm(ts))
    check_norm(ts[1:], rn.grad_norm(ts[1:]))


@pytest.mark.parametrize("at", [0, 4097, 30000])
def test_infinities_and_nan(at):
    for v in (float("inf"), float("-inf"), float("nan")):
        t = torch.randn(30001, device="cuda")
        t[at] = v
        other = torch.randn(100, device="cuda").half()
        n = rn.grad_norm([other, t])
        assert torch.isnan(n) if math.isnan(v) else torch.isposinf(n)
        outs = [torch.empty_like(other), torch.empty_like(t)]
        _, n = rn.grad_clip([other, t], 1.0, out=outs)
        if math.isnan(v):  # coefficient NaN
            assert all(torch.isnan(o).all() for o in outs)
        else:              # coefficient 0: finite values to 0, the infinite one to NaN
            assert not outs[0].any()
            bad = torch.isnan(outs[1])
            assert bad[at] and int(bad.sum()) == 1 and not outs[1][~bad].any()


def test_all_zero():
    ts = [torch.zeros(70000, dtype=d, device="cuda") for d in DTYPES]
    _, n = rn.grad_clip(ts, 1.0)
    assert float(n) == 0.0 and not any(t.any() for t in ts)


def test_dense_orders_and_a_tensor_listed_twice():
    t = torch.randn(4, 6, 8, 10, device="cuda").to(memory_format=torch.channels_last)
    m = torch.randn(30, 40, device="cuda").t()
    check_norm([t, m], rn.grad_norm([t, m]))
    check_norm([t, t], rn.grad_norm([t, t]))
    keep = [t.clone(), m.clone()]
    _, n = rn.grad_clip([t, m], 1.0)
    check_clip(keep, [t, m], 1.0, n)


def test_deterministic_and_any_history_of_the_workspace():
    ts = tensors([(1000, 1000), (77,), (123456,)], DTYPES, 8)
    n = rn.grad_norm(ts)
    for fill in (0, 255):
        ws = torch.full((1 << 16,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(rn.grad_norm(ts, workspace=ws), n)
        assert torch.equal(rn.grad_clip(ts, 1.0, out=[torch.empty_like(t) for t in ts], workspace=ws)[1], n)
    out = torch.zeros(1, device="cuda")
    assert rn.grad_norm(ts, norm=out) is out and torch.equal(out[0], n)


def test_streams_and_graphs():
    sets = [tensors([(2000, 1000), (3,), (1001,)], DTYPES, s) for s in (1, 2)]
    want = [rn.grad_clip(ts, 1.0, out=[torch.empty_like(t) for t in ts]) for ts in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for ts, s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append(rn.grad_clip(ts, 1.0, out=[torch.empty_like(t) for t in ts]))
        torch.cuda.synchronize()
        for (a, n), (b, m) in zip(got, want):
            assert torch.equal(n, m) and all(torch.equal(p, q) for p, q in zip(a, b))
    mine = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, norm = rn.grad_clip(mine, 1.0)
    for k in (1, 0):
        for t, src in zip(mine, sets[k]):
            t.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want[k][1]) and all(torch.equal(p, q) for p, q in zip(mine, want[k][0]))


def test_more_than_2_31_values():
    t = torch.empty((1 << 31) + 12345, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    t[-1] = 1024.0
    n = rn.grad_norm([t])
    want = math.sqrt((t.numel() - 1) * 0.25 + 1024.0 ** 2)
    assert abs(float(n) - want) <= 18 * U * want
    rn.grad_clip([t], float(want) / 4)
    assert float(t[-1]) == 256.0 and (t[:1000] == 0.125).all() and (t[-1000:-1] == 0.125).all()


def test_clipping_a_training_step():
    """A step as it is used: group norm forward and backward, a row norm's
    backward, then all their gradients clipped together."""
    g = torch.Generator(device="cuda").manual_seed(0)
    B, S, C, G = 2, 300, 64, 8
    x = torch.randn(B, S, C, generator=g, device="cuda").bfloat16()
    dy = torch.randn(B, S, C, generator=g, device="cuda").bfloat16()
    gamma, beta = torch.ones(C, device="cuda").bfloat16(), torch.zeros(C, device="cuda").bfloat16()
    y, mean, rstd = rn.gn_fwd(x, gamma, beta, G, activation="silu")
    h, m2, r2 = rn.ln_fwd(y, gamma, beta)
    dh, dg2, db2 = rn.ln_bwd(dy, y, gamma, m2, r2)
    dx, dg1, db1 = rn.gn_bwd(dh, x, gamma, beta, mean, rstd, G, activation="silu")
    grads = [dg1, db1, dg2, db2, dx]
    keep = [t.clone() for t in grads]
    _, norm = rn.grad_clip(grads, 1.0)
    check_clip(keep, grads, 1.0, norm)
    # and the gradients themselves, against 64-bit autograd of the same two norms
    xr = x.double().requires_grad_()
    ps = [p.double().requires_grad_() for p in (gamma, beta, gamma, beta)]
    yr = torch.nn.functional.silu(torch.nn.functional.group_norm(xr.transpose(1, 2), G, ps[0], ps[1]).transpose(1, 2))
    hr = torch.nn.functional.layer_norm(yr, (C,), ps[2], ps[3])
    hr.backward(dy.double())
    for got, want in zip(keep, (ps[0].grad, ps[1].grad, ps[2].grad, ps[3].grad, xr.grad)):
        # y, h's statistics and dh pass through bf16: relative 2^-8 each, errors of many values add as random
        assert (got.double() - want).norm() <= 4 * 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("size", [1e28, 1e29, 1e30, 1e31, 1e34, 1e35])
@pytest.mark.parametrize("shape", [[(1000,), (33, 77)], [(300001,), (50,)]], ids=["short", "long"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_clipping_by_norms_far_out(dtype, shape, size):
    """Norms from 5e29 to 6e37: clipped where the norm is above max_norm, and
    left as they are where it is below, whatever max_norm is."""
    ts = tensors(shape, [dtype], 3, size)
    total = norm64(ts)
    for max_norm in (1.0, 0.5 * total, 0.999 * total, 1.001 * total, 20 * total, 3.4e38):
        max_norm = min(max_norm, 3.4e38)
        outs = [torch.empty_like(t) for t in ts]
        _, norm = rn.grad_clip(ts, max_norm, out=outs)
        check_clip(ts, outs, max_norm, norm)
        mine = [t.clone() for t in ts]
        rn.grad_clip(mine, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
        if max_norm > 1.0005 * total:
            assert all(torch.equal(a, b) for a, b in zip(outs, ts))


def test_lists_from_iterators():
    """Gradients that come from a generator or a dict's values, as a program
    collects them from its parameters: used once, and the list of them is what
    grad_clip hands back."""
    ts = tensors([(1000,), (7, 5), (20001,)], DTYPES, 8)
    n = rn.grad_norm(ts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for make in (lambda v: (t for t in v), lambda v: dict(enumerate(v)).values(), tuple, list):
            assert torch.equal(rn.grad_norm(make(ts), stream=stream), n)
            mine, outs = [t.clone() for t in ts], [torch.empty_like(t) for t in ts]
            torch.cuda.synchronize()
            got, norm = rn.grad_clip(make(mine), 0.5, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(norm, n) and all(a is b for a, b in zip(list(got), mine, strict=True))
            check_clip(ts, mine, 0.5, norm)
            got, norm = rn.grad_clip(make(ts), 0.5, out=make(outs), stream=stream)
            torch.cuda.synchronize()
            assert all(a is b for a, b in zip(list(got), outs, strict=True))
            assert all(torch.equal(a, b) for a, b in zip(outs, mine))
    for empty in ([], (t for t in ()), {}.values()):
        for stream in (None, side):
            with pytest.raises(ValueError):
                rn.grad_norm(empty, stream=stream)
