"""The row operators of a transformer block run together, as a program would run them: norm, head norms with rotation,
attention (torch's), dropout + add + norm twice, and all gradients back to the input and the weights; the same chain in
graphs and on streams.

Tolerance of the chain against float64: each of about twelve stages (norms, products, attention, rotations, their
gradients) sums at most 512 terms in float32, which adds at most 512 u, u = 2^-24, of the norm of its terms, and the
stages' terms have norms near their results' (random values, no cancellation): 12 * 512 u < 4e-4 of a result's norm."""
import math

import pytest
import torch
import torch.nn.functional as F

import row_wise_normalization_ln_gb300 as rn
from philox import keep_mask, threshold

pytestmark = pytest.mark.gpu

B, S, HQ, HK, D, R, C = 2, 33, 6, 2, 24, 16, 96
T, P, EPS = B * S, 0.2, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from row_wise_normalization_ln_gb300 import _build
    _build.build()
    rn.library()


def weights():
    g = torch.Generator().manual_seed(3)

    def n(*shape, scale=1.0, loc=0.0):
        return (torch.randn(*shape, generator=g) * scale + loc).cuda()
    w = dict(w1=n(C, scale=0.2, loc=1), qkv=n(C, (HQ + 2 * HK) * D, scale=C ** -0.5), wq=n(D, scale=0.2, loc=1),
             wk=n(D, scale=0.2, loc=1), wo=n(HQ * D, C, scale=(HQ * D) ** -0.5), g2=n(C, scale=0.2, loc=1), b2=n(C, scale=0.2),
             wa=n(C, 2 * C, scale=C ** -0.5), wb=n(2 * C, C, scale=(2 * C) ** -0.5), w3=n(C, scale=0.2, loc=1))
    angle = torch.arange(64)[:, None] / 10000 ** (torch.arange(R // 2) / (R // 2))
    fixed = dict(cos=angle.cos().cuda(), sin=angle.sin().cuda(), c1=n(T, C), c2=n(T, C))
    return n(T, C), w, fixed


def attention(q, k, v):
    q, k, v = (t.reshape(B, S, -1, D).transpose(1, 2) for t in (q, k, v))
    k, v = (t.repeat_interleave(HQ // HK, 1) for t in (k, v))
    s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=s.device).triu(1), float("-inf"))
    return (s.softmax(-1) @ v).transpose(1, 2).reshape(T, HQ * D)


def mlp(z, wa, wb):
    return F.gelu(z @ wa) @ wb


def reference(x, w, f, seed, offsets):
    """Everything in float64, by autograd."""
    x, w = x.double().requires_grad_(), {n: t.double().requires_grad_() for n, t in w.items()}
    f = {n: t.double() for n, t in f.items()}

    def rms(v, g):
        return v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * g

    def rotate(v):
        cos, sin = (t[:S].repeat(B, 1)[:, None, :] for t in (f["cos"], f["sin"]))
        a, b, rest = v[..., :R // 2], v[..., R // 2:R], v[..., R:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    def drop(v, offset):
        keep = torch.from_numpy(keep_mask(seed, offset, P, T, C)).cuda()
        return v * keep * (65536 / (65536 - threshold(P)))

    qkv = rms(x, w["w1"]) @ w["qkv"]
    q, k, v = qkv.split([HQ * D, HK * D, HK * D], 1)
    q, k = rotate(rms(q.reshape(T, HQ, D), w["wq"])), rotate(rms(k.reshape(T, HK, D), w["wk"]))
    h1 = x + drop(attention(q, k, v) @ w["wo"], offsets[0])
    z = F.layer_norm(h1, (C,), w["g2"], w["b2"], EPS)
    h2 = h1 + drop(mlp(z, w["wa"], w["wb"]), offsets[1])
    y = rms(h2, w["w3"])
    ((y * f["c1"]).sum() + (h2 * f["c2"]).sum()).backward()
    return y.detach(), h2.detach(), dict({n: t.grad for n, t in w.items()}, x=x.grad)


def test_a_block_and_its_gradients():
    x, w, f = weights()
    seed, offsets = 11, (3, 4)
    # forward
    y1 = rn.rms_fwd(x, w["w1"], EPS)
    qkv = y1 @ w["qkv"]
    q, k = qkv[:, :HQ * D].view(B, S, HQ, D), qkv[:, HQ * D:(HQ + HK) * D].view(B, S, HK, D)
    qr, kr = rn.rms_fwd_rope(q, k, w["wq"], w["wk"], f["cos"], f["sin"], eps=EPS)
    leaves = [t.detach().requires_grad_() for t in (qr, kr, qkv[:, (HQ + HK) * D:], w["wo"])]
    o = attention(*leaves[:3]) @ leaves[3]
    h1, z, mean, rstd = rn.ln_fwd_dropout_add(o.detach(), x, w["g2"], w["b2"], P, (seed, offsets[0]), EPS)
    inner = [t.detach().requires_grad_() for t in (z, w["wa"], w["wb"])]
    m = mlp(*inner)
    h2, y = rn.rms_fwd_dropout_add(m.detach(), h1, w["w3"], P, (seed, offsets[1]), EPS)
    # backward
    grad = {}
    dm, dh1, grad["w3"] = rn.rms_bwd_dropout_add(f["c1"], f["c2"], h2, w["w3"], P, (seed, offsets[1]), EPS)
    dz, grad["wa"], grad["wb"] = torch.autograd.grad(m, inner, dm)
    do, dx, grad["g2"], grad["b2"] = rn.ln_bwd_dropout_add(dz, dh1, h1, w["g2"], mean, rstd, P, (seed, offsets[0]))
    dqr, dkr, dv, grad["wo"] = torch.autograd.grad(o, leaves, do)
    dqkv = torch.empty_like(qkv)
    dqkv[:, (HQ + HK) * D:] = dv
    into = dict(dq_out=dqkv[:, :HQ * D].view(B, S, HQ, D), dk_out=dqkv[:, HQ * D:(HQ + HK) * D].view(B, S, HK, D))
    _, _, grad["wq"], grad["wk"] = rn.rms_bwd_rope(dqr, dkr, q, k, w["wq"], w["wk"], f["cos"], f["sin"], eps=EPS, **into)
    grad["qkv"] = y1.t() @ dqkv
    # the first norm's input is the residual stream: its gradient and the stream's in one call
    grad["x"], grad["w1"] = rn.rms_bwd_add(dqkv @ w["qkv"].t(), dx, x, w["w1"], EPS)

    want_y, want_h, want = reference(x, w, f, seed, offsets)
    assert (y - want_y).norm() <= 4e-4 * want_y.norm() and (h2 - want_h).norm() <= 4e-4 * want_h.norm()
    assert grad.keys() == want.keys()
    for n, t in grad.items():
        assert (t - want[n]).norm() <= 4e-4 * want[n].norm(), (n, float((t - want[n]).norm() / want[n].norm()))


def chain(s):
    """The row operators alone, one after the other, on a dict of tensors."""
    q, k = s["qkv"][:, :HQ * D].view(T, HQ, D), s["qkv"][:, HQ * D:(HQ + HK) * D].view(T, HK, D)
    qr, kr = rn.rms_fwd_rope(q, k, s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS)
    h, y, mean, rstd = rn.ln_fwd_dropout_add(s["x"], s["r"], s["g"], s["b"], P, s["rng"], EPS)
    h2, y2 = rn.rms_fwd_dropout_add(y, h, s["g"], P, s["rng"], EPS)
    dm, dh, dw = rn.rms_bwd_dropout_add(y2, h2, h2, s["g"], P, s["rng"], EPS, workspace=s["ws"])
    dx, dr, dg, db = rn.ln_bwd_dropout_add(dm, dh, h, s["g"], mean, rstd, P, s["rng"], workspace=s["ws"])
    d, dw2 = rn.rms_bwd_add(dx, dr, s["r"], s["g"], EPS, workspace=s["ws"])
    dq, dk, dwq, dwk = rn.rms_bwd_rope(qr, kr, q, k, s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS, workspace=s["ws"])
    s["rng"][1] += 1
    return [qr, kr, h, y, h2, y2, dm, dh, dw, dx, dr, dg, db, d, dw2, dq, dk, dwq, dwk]


def state(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()
    angle = torch.rand(64, R // 2, generator=g).cuda() * 6
    pos = (torch.arange(T) % 64).cuda()
    pos[-5:] = -1  # padding
    return dict(qkv=n(T, (HQ + 2 * HK) * D), wq=n(D), wk=n(D), cos=angle.cos(), sin=angle.sin(), pos=pos, x=n(T, C), r=n(T, C), g=n(C),
                b=n(C), rng=torch.tensor([seed, 9], device="cuda"), ws=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))


def test_the_chain_replayed_and_on_two_streams():
    """A captured chain gives the eager one's bits with each step's mask, alone and beside another on a second stream."""
    a, b = state(1), state(2)
    want = {}
    for n, s in (("a", a), ("b", b)):
        want[n] = [[t.clone() for t in chain(s)] for _ in range(3)]
        s["rng"][1] = 9
    torch.cuda.synchronize()
    graphs = {}
    for n, s in (("a", a), ("b", b)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = chain(s)
        graphs[n] = (graph, out)
    streams = {"a": torch.cuda.Stream(), "b": torch.cuda.Stream()}
    torch.cuda.synchronize()
    for step in range(3):
        for n in ("a", "b"):
            with torch.cuda.stream(streams[n]):
                graphs[n][0].replay()
        torch.cuda.synchronize()
        for n in ("a", "b"):
            assert all(torch.equal(u, v) for u, v in zip(graphs[n][1], want[n][step])), (n, step)
    assert not torch.equal(want["a"][0][2], want["a"][1][2])  # another mask each step


def test_the_chain_on_another_stream():
    a = state(5)
    want = [t.clone() for t in chain(a)]
    a["rng"][1] = 9
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain(a)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
